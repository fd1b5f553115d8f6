"""Serving steps around the paged cache, from their definitions in float64: rotary tables,
per-head norm with rotation, the ragged append, the read-back of tokens, and attention of
several new tokens per sequence.

Test infrastructure: the CUDA library is checked against this module; nothing in the library
imports it.  A sequence holds n_sink + t_quant + t_res tokens (t_res < 0 while its sink
fills); see oracle.paged for the pool.
"""
from __future__ import annotations

import numpy as np

from . import attention as oatt
from . import cache as ocache
from . import fp, paged
from .formats import BF16, F16, KEYS, VALUES

PLAIN, LINEAR, BANDS, RAMP = range(4)


def frequencies(R, base, scaling=PLAIN, factor=1.0, original_len=0.0, low=0.0, high=0.0):
    """f_i of the R / 2 pairs."""
    out = []
    for i in range(R // 2):
        w = float(base) ** (-2.0 * i / R)
        if scaling == LINEAR:
            f = w / factor
        elif scaling == BANDS:
            g = min(max((original_len * w / (2 * np.pi) - low) / (high - low), 0.0), 1.0)
            f = (1 - g) * w / factor + g * w
        elif scaling == RAMP:
            def x(b):
                return R * np.log(original_len / (2 * np.pi * b)) / (2 * np.log(base))
            a, z = max(np.floor(x(high)), 0.0), min(np.ceil(x(low)), R - 1.0)
            g = min(max((i - a) / max(z - a, 0.001), 0.0), 1.0)
            f = (1 - g) * w + g * w / factor
        else:
            f = w
        out.append(f)
    return np.array(out)


def rope_table(freq, pos0, n_pos, amplitude=1.0):
    """[n_pos, 2 len(freq)]: cosines then sines, unrounded."""
    ang = (pos0 + np.arange(n_pos, dtype=np.float64))[:, None] * freq[None]
    return amplitude * np.concatenate([np.cos(ang), np.sin(ang)], 1)


def _pairs(x, R, inter):
    return (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])


def _join(x, a, b, R, inter):
    y = np.array(x, np.float64)
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = a, b
    else:
        y[..., :R // 2], y[..., R // 2:R] = a, b
    return y


def rotate(x, row, inter):
    """x [..., D] turned by its table row [..., R] (float64)."""
    R = row.shape[-1]
    c, s = row[..., :R // 2], row[..., R // 2:]
    a, b = _pairs(np.asarray(x, np.float64), R, inter)
    return _join(x, a * c - b * s, b * c + a * s, R, inter)


def rotate32(x, row, inter):
    """The same with every product and sum rounded to fp32 (the order the library states)."""
    R = row.shape[-1]
    c, s = row[..., :R // 2], row[..., R // 2:]
    a, b = _pairs(np.asarray(x, np.float64), R, inter)
    return _join(x, fp.sub32(fp.mul32(a, c), fp.mul32(b, s)), fp.add32(fp.mul32(b, c), fp.mul32(a, s)), R, inter)


def round_src(x, dtype):
    return fp.f16(x) if dtype == F16 else fp.bf16(x) if dtype == BF16 else fp.f32(x)


def norm_rope(x, weight, eps, offset, row, inter):
    """One set of head rows x [T, H, D] with table rows [T, R] (None: no rotation)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + np.asarray(weight, np.float64))
    return x if row is None else rotate(x, row[:, None, :], inter)


def append(pc: paged.PagedCache, s, t_quant, t_res, k_new, v_new):
    """Append k_new, v_new [n, H, D] (already turned and rounded to the source type) to
    sequence s; returns its lengths after it."""
    f = pc.fmt
    cap, g, ns = f.residual_cap, f.group_tokens, f.n_sink
    n = len(k_new)
    to_sink = min(n, max(0, -t_res))
    for name, x in (("sink_k", k_new), ("sink_v", v_new)):
        for i in range(to_sink):
            pc.raw[name][s][:, ns + t_res + i] = ocache.raw_encode(x[i], f.src_dtype)
    if n == 0:
        return t_quant, t_res
    old = max(t_res, 0)
    rows = {}
    for name, x in (("res_k", k_new), ("res_v", v_new)):
        held = ocache.raw_decode(pc.raw[name][s][:, :old], f.src_dtype).swapaxes(0, 1)
        rows[name] = np.concatenate([held, x[to_sink:]], 0)
    total = len(rows["res_k"])
    groups = total // g if total >= cap else 0
    for j in range(groups):
        blk = int(pc.block_table[s, t_quant // g + j])
        for name, which in (("res_k", KEYS), ("res_v", VALUES)):
            paged.quantize_group(pc, which, rows[name][j * g:(j + 1) * g].swapaxes(0, 1), blk, g)
    if total > 0:
        for name in rows:
            left = rows[name][groups * g:]
            pc.raw[name][s][:, :len(left)] = ocache.raw_encode(left, f.src_dtype).swapaxes(0, 1)
    if groups:
        return t_quant + groups * g, total - groups * g
    return t_quant, t_res + n


def tokens(pc: paged.PagedCache, s, t_quant, t_res):
    """K, V [H, L, D] of sequence s in position order."""
    f = pc.fmt
    c = paged.sequence_cache(pc, s, t_quant)
    ns = f.n_sink + min(0, t_res)
    out = []
    for h in range(pc.H):
        kv = []
        for which, x in ((KEYS, "k"), (VALUES, "v")):
            parts = [ocache.raw_decode(c["sink_" + x][0, h, :ns], f.src_dtype)] if f.n_sink else []
            parts.append(ocache.dequantize(f, c, which, 0, t_quant, 0, h))
            if t_res > 0:
                parts.append(ocache.raw_decode(c["res_" + x][0, h, :t_res], f.src_dtype))
            kv.append(np.concatenate(parts, 0))
        out.append(kv)
    return np.stack([k for k, _ in out]), np.stack([v for _, v in out])


def attention(pc: paged.PagedCache, s, t_quant, t_res, q, scale, causal=True):
    """q [n, Hq, D], the last n tokens of sequence s -> out [n, Hq, D], lse [n, Hq]."""
    q = np.asarray(q, np.float64)
    n, Hq, D = q.shape
    K, V = tokens(pc, s, t_quant, t_res)
    L, G = K.shape[1], Hq // pc.H
    out, lse = np.zeros_like(q), np.full((n, Hq), -np.inf)
    for i in range(n):
        seen = max(0, L - n + i + 1) if causal else L
        if seen == 0:
            continue
        for h in range(pc.H):
            hs = slice(h * G, (h + 1) * G)
            out[i, hs], lse[i, hs] = oatt.attention_lse(q[i, hs], K[h, :seen], V[h, :seen], scale)
    return out, lse
