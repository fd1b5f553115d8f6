"""ctypes binding of libkvq.so (include/kvq.h).

Argument marshalling only: every entry point forwards to the C ABI with the same
name; device memory and streams come from PyTorch.  There is no fallback: when the
shared library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

# enums of include/kvq.h
KVQ_OK, KVQ_ERR_INVALID, KVQ_ERR_UNSUPPORTED, KVQ_ERR_CUDA, KVQ_ERR_WORKSPACE = range(5)
KVQ_DEV_NONFINITE, KVQ_DEV_RANGE, KVQ_DEV_TIMEOUT, KVQ_DEV_BOUNDS = 1, 2, 4, 8
F32, F16, BF16 = 0, 1, 2
NONE, SYM8, ASYM, NUQ, MIXED, KQV = range(6)
TENSOR, TOKEN, CHANNEL = range(3)
KEYS, VALUES = 0, 1

ARRAYS = [
    "k_codes", "k_scale", "k_zero", "k_order",
    "k_out_rowptr", "k_out_col", "k_out_val",
    "v_codes", "v_scale", "v_zero",
    "v_out_col", "v_out_val",
    "k_lut", "v_lut",
    "sink_k", "sink_v", "res_k", "res_v",
    "v_sketch",
]
RAW_ARRAYS = ("sink_k", "sink_v", "res_k", "res_v")

TORCH_DTYPE = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
KVQ_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


class kvq_format(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "head_dim", "group_tokens", "src_dtype",
        "k_scheme", "k_bits", "k_axis", "k_outliers",
        "v_scheme", "v_bits", "v_axis", "v_outliers",
        "mixed_hi", "mixed_mid", "n_sink", "residual_cap", "rope")] + [("rope_base", ctypes.c_float),
                                                                ("k_rotate", ctypes.c_int32)]


class kvq_cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("capacity", ctypes.c_int64)] + [(n, ctypes.c_void_p) for n in ARRAYS]


class kvq_paged_cache(ctypes.Structure):
    _fields_ = [("pool", kvq_cache), ("num_seqs", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("sink_k", ctypes.c_void_p), ("sink_v", ctypes.c_void_p),
                ("res_k", ctypes.c_void_p), ("res_v", ctypes.c_void_p)]


ROPE_PLAIN, ROPE_LINEAR, ROPE_BANDS, ROPE_RAMP = range(4)


class kvq_rope_spec(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_len", "low", "high", "amplitude")]


class kvq_rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class kvq_head_rows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("x_stride_t", "x_stride_h", "y_stride_t", "y_stride_h")] + [
        ("heads", ctypes.c_int32), ("weight", ctypes.c_void_p)]


class KvqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """The loaded libkvq.so (raises when it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not built; run python -m quantized_decode_attention_quantize_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        FP, CP = ctypes.POINTER(kvq_format), ctypes.POINTER(kvq_cache)
        PP = ctypes.POINTER(kvq_paged_cache)
        sig = {
            "kvq_version": (I32, []),
            "kvq_status_string": (ctypes.c_char_p, [I32]),
            "kvq_format_check": (I32, [FP]),
            "kvq_cache_array_bytes": (SZ, [FP, I32, I32, I64, I32]),
            "kvq_kqv_codebook": (I32, [I32, I32, ctypes.POINTER(ctypes.c_float)]),
            "kvq_quantize_keys": (I32, [FP, CP, P, I64, I64, I64, I64, I64, P, P]),
            "kvq_quantize_values": (I32, [FP, CP, P, I64, I64, I64, I64, I64, P, P]),
            "kvq_quantize_kv": (I32, [FP, CP, P, P, I64, I64, I64, I64, I64, P, P]),
            "kvq_dequantize": (I32, [FP, CP, I32, I64, I64, P, I32, P, P]),
            "kvq_key_salience": (I32, [FP, P, I64, I64, I64, P, I64, I64, I64, I32, I32, I32, I32,
                                       P, P, I64, I64, P, P]),
            "kvq_decode_workspace_bytes": (SZ, [FP, I32, I32, I32, I64, I32, I32]),
            "kvq_decode_attention": (I32, [FP, CP, P, I32, I32, I64, I32, ctypes.c_float, P, I32,
                                           P, SZ, I32, P, P]),
            "kvq_append_decode_attention": (I32, [FP, CP, P, P, I64, I64, I64, I64, I64, P, I32, I32, I64, I32,
                                                  ctypes.c_float, P, I32, P, SZ, I32, P, P]),
            "kvq_decode_partial_slots": (I32, [FP, I32, I32, I32, I64, I32, I32]),
            "kvq_decode_partial": (I32, [FP, CP, P, I32, I32, I64, I32, ctypes.c_float, P, SZ, I32,
                                         P, P]),
            "kvq_decode_combine": (I32, [FP, I32, I32, I32, I64, I32, I32, P, SZ, P, I32, P]),
            "kvq_decode_combine_lse": (I32, [FP, I32, I32, I32, I64, I32, I32, P, SZ, P, P, P]),
            "kvq_merge_states": (I32, [I32, I64, I32, P, P, P, I32, P, P]),
            "kvq_decode_attention_noalloc": (I32, [FP, CP, P, I32, I32, I64, I32, ctypes.c_float,
                                                   P, I32, I32, P, P]),
            "kvq_quantize_kv_paged": (I32, [FP, PP, P, P, I64, I64, I64, P, I64, P, P]),
            "kvq_decode_paged_workspace_bytes": (SZ, [FP, I32, I32, I32, I64, I32]),
            "kvq_decode_attention_paged": (I32, [FP, PP, P, P, I64, I32, P, I32, I32, ctypes.c_float, P,
                                                 I32, P, SZ, P, P]),
            "kvq_rope_table": (I32, [ctypes.POINTER(kvq_rope_spec), I64, I64, P, P]),
            "kvq_norm_rope": (I32, [I32, I32, I64, P, P,
                                    ctypes.c_float, ctypes.c_float, ctypes.POINTER(kvq_rope), P, P, P]),
            "kvq_append_paged": (I32, [FP, PP, P, I64, I64, P, P, P, I64, I64, P, I64, I64,
                                       ctypes.POINTER(kvq_rope), P, P, P, P, P]),
            "kvq_read_paged": (I32, [FP, PP, P, I64, I64, P, P, P, P, P, I32, P, P]),
            "kvq_attention_paged_workspace_bytes": (SZ, [FP, I32, I32, I32, I64, I64, I64, I32]),
            "kvq_attention_paged": (I32, [FP, PP, P, I64, I64, P, P, I64, I32, P, I32, I32, ctypes.c_float, I32, P,
                                          I32, P, P, SZ, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(st):
    return lib().kvq_status_string(int(st)).decode()


def _check(fn, st):
    if st != KVQ_OK:
        raise KvqError(fn, st)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_format(d: dict) -> kvq_format:
    f = kvq_format()
    for name, _ in kvq_format._fields_:
        setattr(f, name, d.get(name, 0) if name == "k_rotate" else d[name])
    return f


def format_check(fmt: kvq_format) -> int:
    return lib().kvq_format_check(ctypes.byref(fmt))


def cache_array_bytes(fmt: kvq_format, B, H, C, array_id) -> int:
    return lib().kvq_cache_array_bytes(ctypes.byref(fmt), B, H, C, array_id)


def kqv_codebook(bits: int, head_dim: int):
    """kvq_kqv_codebook: the 2^bits fp32 Lloyd-Max centroids (a list of floats)."""
    out = (ctypes.c_float * (1 << bits))()
    _check("kvq_kqv_codebook", lib().kvq_kqv_codebook(bits, head_dim, out))
    return list(out)


def _given(fmt, name, t, need, device):
    """Checks a caller's tensor for the array `name` of `need` bytes: kernels get its bare address."""
    if t is None or not t.is_contiguous() or t.numel() * t.element_size() != need:
        raise ValueError(f"{name}: a contiguous tensor of {need} bytes is needed")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the cache's other arrays on {device}")
    if t.is_floating_point():
        own = (TORCH_DTYPE[fmt.src_dtype],) if name in RAW_ARRAYS else () if "code" in name else (torch.float16, torch.float32)
        if t.dtype not in own:
            raise ValueError(f"{name}: {t.dtype} is not the array's type")
    if t.data_ptr() % 16:
        raise ValueError(f"{name}: must start on a 16-byte boundary")


class Cache:
    """Device arrays of a packed cache (torch uint8 tensors), owned by this object.
    k_lut / v_lut: the codebooks (NUQ: stored as fp16, KQV: fp32); sketch: the KQV sketch
    matrix [D][D] (stored as fp32).  arrays: name -> the caller's tensor, used in place of new
    ones (all that the format needs; checked as PagedCache's)."""

    def __init__(self, fmt: kvq_format, B: int, H: int, C: int, device="cuda", k_lut=None,
                 v_lut=None, sketch=None, arrays=None):
        self.fmt, self.B, self.H, self.C = fmt, B, H, C
        self.tensors = {}
        self.struct = kvq_cache(batch=B, kv_heads=H, capacity=C)
        if arrays is not None:   # the caller's tensors
            for name, t in arrays.items():
                if name not in ARRAYS:
                    raise ValueError(f"{name}: not an array of a cache")
                _given(fmt, name, t, cache_array_bytes(fmt, B, H, C, ARRAYS.index(name)), next(iter(arrays.values())).device)
                setattr(self.struct, name, t.data_ptr())
            self.tensors.update(arrays)
            return
        for i, name in enumerate(ARRAYS):
            n = cache_array_bytes(fmt, B, H, C, i)
            if n:
                t = torch.zeros(n, dtype=torch.uint8, device=device)
                self.tensors[name] = t
                setattr(self.struct, name, t.data_ptr())
        for name, lut, scheme in (("k_lut", k_lut, fmt.k_scheme), ("v_lut", v_lut, fmt.v_scheme)):
            if name in self.tensors and lut is not None:
                dt = torch.float32 if scheme == KQV else torch.float16
                self.tensors[name].copy_(torch.tensor(lut, dtype=dt).reshape(-1).view(torch.uint8))
        if "v_sketch" in self.tensors and sketch is not None:
            self.tensors["v_sketch"].copy_(torch.as_tensor(sketch, dtype=torch.float32).reshape(-1).view(torch.uint8))

    def array(self, name):
        return self.tensors[name]

    def ref(self):
        return ctypes.byref(self.struct)


def quantize_keys(fmt, cache: Cache, src: torch.Tensor, t0: int, n: int, status=None, stream=None):
    """src [B, H, n, D] (strided over the first three dims, channels contiguous)."""
    st = lib().kvq_quantize_keys(ctypes.byref(fmt), cache.ref(), _ptr(src), src.stride(0),
                                 src.stride(1), src.stride(2), t0, n, _ptr(status), _stream(stream))
    _check("kvq_quantize_keys", st)


def quantize_values(fmt, cache: Cache, src: torch.Tensor, t0: int, n: int, status=None,
                    stream=None):
    st = lib().kvq_quantize_values(ctypes.byref(fmt), cache.ref(), _ptr(src), src.stride(0),
                                   src.stride(1), src.stride(2), t0, n, _ptr(status),
                                   _stream(stream))
    _check("kvq_quantize_values", st)


def quantize_kv(fmt, cache: Cache, k_src: torch.Tensor, v_src: torch.Tensor, t0: int, n: int,
                status=None, stream=None):
    """Keys and values of one append (same strides), one launch where the kernels allow."""
    if k_src.stride() != v_src.stride():
        raise ValueError("k_src and v_src must have the same strides")
    st = lib().kvq_quantize_kv(ctypes.byref(fmt), cache.ref(), _ptr(k_src), _ptr(v_src),
                               k_src.stride(0), k_src.stride(1), k_src.stride(2), t0, n,
                               _ptr(status), _stream(stream))
    _check("kvq_quantize_kv", st)


def dequantize(fmt, cache: Cache, which: int, t0: int, n: int, out_dtype=F32, out=None,
               status=None, stream=None):
    if out is None:
        out = torch.empty((cache.B, cache.H, n, fmt.head_dim), dtype=TORCH_DTYPE[out_dtype],
                          device="cuda")
    st = lib().kvq_dequantize(ctypes.byref(fmt), cache.ref(), which, t0, n, _ptr(out), out_dtype,
                              _ptr(status), _stream(stream))
    _check("kvq_dequantize", st)
    return out


def key_salience(fmt, q: torch.Tensor, k: torch.Tensor, order_out: torch.Tensor,
                 order_stride_b: int, order_stride_h: int, salience_out=None, status=None,
                 stream=None):
    """q [B, Hq, R, D], k [B, Hkv, R, D]; order_out is a uint8 tensor whose element
    (b, h, slot) sits at b * order_stride_b + h * order_stride_h + slot."""
    B, Hq, R, D = q.shape
    Hkv = k.shape[1]
    st = lib().kvq_key_salience(ctypes.byref(fmt), _ptr(q), q.stride(0), q.stride(1), q.stride(2),
                                _ptr(k), k.stride(0), k.stride(1), k.stride(2), B, Hq, Hkv, R,
                                _ptr(salience_out), _ptr(order_out), order_stride_b,
                                order_stride_h, _ptr(status), _stream(stream))
    _check("kvq_key_salience", st)


def decode_workspace_bytes(fmt, B, Hq, Hkv, t_quant, t_res, num_splits=0) -> int:
    return lib().kvq_decode_workspace_bytes(ctypes.byref(fmt), B, Hq, Hkv, t_quant, t_res,
                                            num_splits)


def decode_attention(fmt, cache: Cache, q: torch.Tensor, t_quant: int, t_res: int, scale: float,
                     out_dtype=F32, out=None, workspace=None, num_splits=0, status=None,
                     stream=None):
    """q [B, Hq, D] contiguous -> out [B, Hq, D]."""
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=TORCH_DTYPE[out_dtype], device=q.device)
    need = decode_workspace_bytes(fmt, B, Hq, cache.H, t_quant, t_res, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib().kvq_decode_attention(ctypes.byref(fmt), cache.ref(), _ptr(q), KVQ_DTYPE[q.dtype],
                                    Hq, t_quant, t_res, scale, _ptr(out), out_dtype,
                                    _ptr(workspace), workspace.numel(), num_splits, _ptr(status),
                                    _stream(stream))
    _check("kvq_decode_attention", st)
    return out


def append_decode_attention(fmt, cache: Cache, k_src: torch.Tensor, v_src: torch.Tensor, t0: int, n: int,
                            q: torch.Tensor, t_quant: int, t_res: int, scale: float, out_dtype=F32, out=None,
                            workspace=None, num_splits=0, status=None, stream=None):
    """kvq_append_decode_attention: quantize_kv(k_src, v_src, t0, n) then decode_attention(q)."""
    if k_src.stride() != v_src.stride():
        raise ValueError("k_src and v_src must have the same strides")
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=TORCH_DTYPE[out_dtype], device=q.device)
    need = decode_workspace_bytes(fmt, B, Hq, cache.H, t_quant, t_res, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib().kvq_append_decode_attention(ctypes.byref(fmt), cache.ref(), _ptr(k_src), _ptr(v_src),
                                           k_src.stride(0), k_src.stride(1), k_src.stride(2), t0, n,
                                           _ptr(q), KVQ_DTYPE[q.dtype], Hq, t_quant, t_res, scale, _ptr(out),
                                           out_dtype, _ptr(workspace), workspace.numel(), num_splits,
                                           _ptr(status), _stream(stream))
    _check("kvq_append_decode_attention", st)
    return out


def decode_partial_slots(fmt, B, Hq, Hkv, t_quant, t_res, num_splits=0) -> int:
    return lib().kvq_decode_partial_slots(ctypes.byref(fmt), B, Hq, Hkv, t_quant, t_res, num_splits)


def decode_partial(fmt, cache: Cache, q: torch.Tensor, t_quant: int, t_res: int, scale: float,
                   workspace: torch.Tensor, num_splits=0, status=None, stream=None):
    B, Hq, D = q.shape
    st = lib().kvq_decode_partial(ctypes.byref(fmt), cache.ref(), _ptr(q), KVQ_DTYPE[q.dtype], Hq,
                                  t_quant, t_res, scale, _ptr(workspace), workspace.numel(),
                                  num_splits, _ptr(status), _stream(stream))
    _check("kvq_decode_partial", st)


def decode_combine(fmt, B, Hq, Hkv, t_quant, t_res, workspace: torch.Tensor, out: torch.Tensor,
                   num_splits=0, stream=None):
    st = lib().kvq_decode_combine(ctypes.byref(fmt), B, Hq, Hkv, t_quant, t_res, num_splits,
                                  _ptr(workspace), workspace.numel(), _ptr(out),
                                  KVQ_DTYPE[out.dtype], _stream(stream))
    _check("kvq_decode_combine", st)
    return out


def decode_combine_lse(fmt, B, Hq, Hkv, t_quant, t_res, workspace: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, num_splits=0, stream=None):
    """kvq_decode_combine_lse: out [B, Hq, D] fp32 and lse [B, Hq] fp32 of one part."""
    st = lib().kvq_decode_combine_lse(ctypes.byref(fmt), B, Hq, Hkv, t_quant, t_res, num_splits,
                                      _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
                                      _stream(stream))
    _check("kvq_decode_combine_lse", st)
    return out, lse


def merge_states(outs: torch.Tensor, lses: torch.Tensor, out_dtype=F32, out=None, lse_out=None,
                 stream=None):
    """kvq_merge_states: outs [n, rows..., D] fp32, lses [n, rows...] fp32 -> out [rows..., D]."""
    n, D = outs.shape[0], outs.shape[-1]
    rows = lses[0].numel()
    if out is None:
        out = torch.empty(outs.shape[1:], dtype=TORCH_DTYPE[out_dtype], device=outs.device)
    st = lib().kvq_merge_states(n, rows, D, _ptr(outs), _ptr(lses), _ptr(out), KVQ_DTYPE[out.dtype],
                                _ptr(lse_out), _stream(stream))
    _check("kvq_merge_states", st)
    return out


NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_attention_noalloc(fmt, cache: Cache, q: torch.Tensor, t_quant: int, t_res: int,
                             scale: float, out_dtype=F32, out=None, num_splits=0, status=None,
                             stream=None):
    """kvq_decode_attention_noalloc: no workspace argument (the library's own scratch)."""
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=TORCH_DTYPE[out_dtype], device=q.device)
    st = lib().kvq_decode_attention_noalloc(ctypes.byref(fmt), cache.ref(), _ptr(q),
                                            KVQ_DTYPE[q.dtype], Hq, t_quant, t_res, scale,
                                            _ptr(out), out_dtype, num_splits, _ptr(status),
                                            _stream(stream))
    _check("kvq_decode_attention_noalloc", st)
    return out


class PagedCache:
    """A paged cache: a pool of num_blocks blocks (one token group of every KV head each,
    the layout of a Cache with batch = num_blocks and capacity = group_tokens), per-sequence
    sink / residual arrays and a device block table [num_seqs][max_blocks] (int32, -1)."""

    def __init__(self, fmt: kvq_format, kv_heads: int, num_blocks: int, num_seqs: int, max_blocks: int,
                 device="cuda", arrays=None):
        """arrays: name -> contiguous tensor of the array's bytes, 16-byte aligned, in its own type or one of
        integers, all on the device of block_table (int32 [num_seqs][max_blocks]); used in place
        of new zeroed ones, they stay the caller's."""
        self.fmt, self.H, self.num_blocks = fmt, kv_heads, num_blocks
        self.num_seqs, self.max_blocks = num_seqs, max_blocks
        if arrays is None:
            self.pool = Cache(fmt, num_blocks, kv_heads, fmt.group_tokens, device=device)
            raw = Cache(fmt, num_seqs, kv_heads, fmt.group_tokens, device=device)
            self.raw = {n: raw.tensors[n] for n in RAW_ARRAYS if n in raw.tensors}
            self.block_table = torch.full((num_seqs, max_blocks), -1, dtype=torch.int32, device=device)
        else:
            self.block_table = arrays.get("block_table")
            if self.block_table is None or self.block_table.dtype != torch.int32 or \
                    tuple(self.block_table.shape) != (num_seqs, max_blocks) or not self.block_table.is_contiguous():
                raise ValueError("block_table must be a contiguous int32 [num_seqs][max_blocks]")
            self.pool = Cache(fmt, num_blocks, kv_heads, fmt.group_tokens, arrays=self._part(arrays, False, num_blocks))
            self.raw = self._part(arrays, True, num_seqs)
        self.device = self.block_table.device
        self.struct = kvq_paged_cache(pool=self.pool.struct, num_seqs=num_seqs, max_blocks=max_blocks,
                                      block_table=self.block_table.data_ptr())
        for n, t in self.raw.items():
            setattr(self.struct, n, t.data_ptr())

    def _part(self, arrays, per_seq, slabs):
        """The given pool (or per-sequence raw) arrays that the format needs, checked."""
        got = {}
        for i, n in enumerate(ARRAYS):
            if (n in RAW_ARRAYS) != per_seq:
                continue
            need = cache_array_bytes(self.fmt, slabs, self.H, self.fmt.group_tokens, i)
            if not need:
                continue
            t = arrays.get(n)
            _given(self.fmt, n, t, need, self.block_table.device)
            got[n] = t
        return got

    def array(self, name):
        return self.raw[name] if name in self.raw else self.pool.tensors[name]

    def ref(self):
        return ctypes.byref(self.struct)


def quantize_kv_paged(fmt, cache: PagedCache, k_src: torch.Tensor, v_src: torch.Tensor, blocks: torch.Tensor,
                      n: int, status=None, stream=None):
    """kvq_quantize_kv_paged: k_src, v_src [num_seqs, H, n, D]; blocks int32 [num_seqs] (device)."""
    _need(cache.device.type == "cuda", "the cache must be on a CUDA device")
    if k_src.stride() != v_src.stride():
        raise ValueError("k_src and v_src must have the same strides")
    st = lib().kvq_quantize_kv_paged(ctypes.byref(fmt), cache.ref(), _ptr(k_src), _ptr(v_src), k_src.stride(0),
                                     k_src.stride(1), k_src.stride(2), _ptr(blocks), n, _ptr(status),
                                     _stream(stream))
    _check("kvq_quantize_kv_paged", st)


def decode_paged_workspace_bytes(fmt, num_seqs, Hq, Hkv, max_t_quant, max_t_res) -> int:
    return lib().kvq_decode_paged_workspace_bytes(ctypes.byref(fmt), num_seqs, Hq, Hkv, max_t_quant, max_t_res)


def decode_attention_paged(fmt, cache: PagedCache, t_quant: torch.Tensor, t_res: torch.Tensor, max_t_quant: int,
                           max_t_res: int, q: torch.Tensor, scale: float, out_dtype=F32, out=None, workspace=None,
                           status=None, stream=None):
    """kvq_decode_attention_paged: t_quant, t_res int32 [num_seqs] (device); q [num_seqs, Hq, D]."""
    _need(cache.device.type == "cuda", "the cache must be on a CUDA device")
    S, Hq, D = q.shape
    if out is None:
        out = torch.empty((S, Hq, D), dtype=TORCH_DTYPE[out_dtype], device=q.device)
    need = decode_paged_workspace_bytes(fmt, S, Hq, cache.H, max_t_quant, max_t_res)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib().kvq_decode_attention_paged(ctypes.byref(fmt), cache.ref(), _ptr(t_quant), _ptr(t_res), max_t_quant,
                                          max_t_res, _ptr(q), KVQ_DTYPE[q.dtype], Hq, scale, _ptr(out), out_dtype,
                                          _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check("kvq_decode_attention_paged", st)
    return out


# ---- serving steps around the paged cache ---------------------------------------------------
# A decode step makes several of these calls, each of a few microseconds on the device: the checks
# below avoid building messages and stream objects for calls that pass.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_INT32 = torch.int32


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on(device, stream, body):
    """body(raw stream) with `device` current, on `stream` or the device's current one (new
    tensors belong to that stream)."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    if stream is None and device.index == torch.cuda.current_device():
        return body(_raw_stream(device.index))
    _need(stream is None or stream.device == device, "the stream is on another device than the tensors")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return body(_raw_stream(device.index))


def _ints(t, n, device, what):
    if t.dtype is _INT32 and t.dim() == 1 and t.numel() == n and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    raise ValueError(f"{what}: a contiguous int32 tensor of {n} values on the same device is needed")


def _status_ptr(status, device):
    return None if status is None else _ints(status, 1, device, "status")


def make_rope_spec(rot_dim: int, base=10000.0, scaling=ROPE_PLAIN, factor=1.0, original_len=0.0, low=0.0, high=0.0,
                   amplitude=1.0) -> kvq_rope_spec:
    return kvq_rope_spec(rot_dim=rot_dim, scaling=scaling, base=base, factor=factor, original_len=original_len,
                         low=low, high=high, amplitude=amplitude)


def rope_table(spec: kvq_rope_spec, n_pos: int, pos0=0, out=None, device="cuda", stream=None):
    """kvq_rope_table: fp32 [n_pos, rot_dim], cosines then sines of each position."""
    if out is not None:
        device = out.device
        _need(out.dtype == torch.float32 and tuple(out.shape) == (n_pos, spec.rot_dim) and out.is_contiguous(),
              "out: a contiguous fp32 [n_pos, rot_dim] tensor is needed")
    else:
        _need(n_pos >= 0, "n_pos must not be negative")
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())

    def body(s):
        t = torch.empty((n_pos, spec.rot_dim), dtype=torch.float32, device=device) if out is None else out
        _check("kvq_rope_table", lib().kvq_rope_table(spec, pos0, n_pos, t.data_ptr(), s))
        return t
    return _on(device, stream, body)


class Rope:
    """A rotation by the rows of `table` (fp32 [n_pos, rot_dim], see rope_table)."""

    def __init__(self, table: torch.Tensor, interleaved=False):
        _need(table.dtype == torch.float32 and table.dim() == 2 and table.is_contiguous(),
              "table: a contiguous fp32 [n_pos, rot_dim] tensor is needed")
        self.table = table
        self.struct = kvq_rope(table=table.data_ptr(), n_pos=table.shape[0], rot_dim=table.shape[1],
                               interleaved=int(interleaved))


def _rope_ptr(rope, device):
    if rope is None:
        return None
    if rope.table.device != device:
        raise ValueError("the rotary table is on another device")
    return rope.struct


_HEAD_ROWS = struct.Struct("@PPqqqqiP")   # kvq_head_rows
assert _HEAD_ROWS.size == ctypes.sizeof(kvq_head_rows)


def _row_strides(x):
    """Strides of rows x [T, H, D]; where a dimension has no extent, those of a contiguous tensor."""
    t, h, c = x.stride()
    T, H, D = x.shape
    if H > 1 and T > 1:
        return t, h, c
    return (t if T > 1 else H * D), (h if H > 1 and T else D), (c if T else 1)


def _head_rows(x, y, weight, what):
    xt, xh, xc = _row_strides(x)
    yt, yh, yc = _row_strides(y) if y.dim() == 3 else (0, 0, 0)
    if xc != 1 or yc != 1 or y.shape != x.shape or y.dtype != x.dtype or y.device != x.device:
        raise ValueError(f"{what}: channels must be contiguous, the output of the same shape, dtype and device")
    w = 0
    if weight is not None:
        if weight.dtype != x.dtype or weight.dim() != 1 or weight.numel() != x.shape[2] or \
                not weight.is_contiguous() or weight.device != x.device:
            raise ValueError(f"{what}: a weight of [head_dim] in the rows' dtype is needed")
        w = weight.data_ptr()
    return _HEAD_ROWS.pack(x.data_ptr(), y.data_ptr(), xt, xh, yt, yh, x.shape[1], w)


def norm_rope(q: torch.Tensor, k=None, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, rope=None,
              positions=None, q_out=None, k_out=None, status=None, stream=None):
    """kvq_norm_rope: q [T, Hq, D] and k [T, Hk, D] (strided over tokens and heads) -> both
    normed per head (with a weight) and turned at `positions` (int32 [T]).  q_out = q and
    k_out = k work in place; new contiguous tensors otherwise."""
    if q.dtype not in KVQ_DTYPE or q.dim() != 3:
        raise ValueError("q: [tokens, heads, head_dim] in fp32, fp16 or bf16 is needed")
    T, _, D = q.shape
    d = q.device
    if k is None:
        _need(k_weight is None and k_out is None, "k_weight and k_out go with k")
    elif k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype != q.dtype or k.device != d:
        raise ValueError("k: the tokens, head_dim, dtype and device of q are needed")

    def body(s):
        qo = torch.empty(q.shape, dtype=q.dtype, device=d) if q_out is None else q_out
        ko, rows_k = None, None
        if k is not None:
            ko = torch.empty(k.shape, dtype=k.dtype, device=d) if k_out is None else k_out
            rows_k = _head_rows(k, ko, k_weight, "k")
        _check("kvq_norm_rope", lib().kvq_norm_rope(
            D, KVQ_DTYPE[q.dtype], T, _head_rows(q, qo, q_weight, "q"), rows_k, eps, weight_offset, _rope_ptr(rope, d),
            None if positions is None else _ints(positions, T, d, "positions"), _status_ptr(status, d), s))
        return qo, ko
    return _on(d, stream, body)


def _batch(cache, cu, t_quant, t_res):
    d, n = cache.device, cache.num_seqs
    return (_ints(cu, n + 1, d, "cu"), _ints(t_quant, n, d, "t_quant"), _ints(t_res, n, d, "t_res"))


def append_paged(fmt, cache: PagedCache, cu_new: torch.Tensor, max_new: int, t_quant: torch.Tensor,
                 t_res: torch.Tensor, k_src: torch.Tensor, v_src: torch.Tensor, t_quant_out: torch.Tensor,
                 t_res_out: torch.Tensor, rope=None, positions=None, status=None, stream=None):
    """kvq_append_paged: k_src, v_src [rows, Hkv, D] (strided over rows and heads), the rows
    [cu_new[s], cu_new[s + 1]) following what sequence s holds; the lengths after it go to
    t_quant_out / t_res_out."""
    dt, d = TORCH_DTYPE[fmt.src_dtype], cache.device
    rows = k_src.shape[0]
    shape = (rows, cache.H, fmt.head_dim)
    kt, kh, kc = _row_strides(k_src) if k_src.dim() == 3 else (0, 0, 0)
    vt, vh, vc = _row_strides(v_src) if v_src.dim() == 3 else (0, 0, 0)
    if k_src.shape != shape or v_src.shape != shape or k_src.dtype != dt or v_src.dtype != dt or kc != 1 or vc != 1 or \
            k_src.device != d or v_src.device != d:
        raise ValueError("k_src, v_src: [rows, kv_heads, head_dim] in the format's source dtype is needed")
    cu, tq, tr = _batch(cache, cu_new, t_quant, t_res)
    tq_o, tr_o = _ints(t_quant_out, cache.num_seqs, d, "t_quant_out"), _ints(t_res_out, cache.num_seqs, d, "t_res_out")
    pos = None if positions is None else _ints(positions, rows, d, "positions")

    def body(s):
        _check("kvq_append_paged", lib().kvq_append_paged(
            fmt, cache.struct, cu, rows, max_new, tq, tr, k_src.data_ptr(), kt, kh, v_src.data_ptr(), vt, vh,
            _rope_ptr(rope, d), pos, tq_o, tr_o, _status_ptr(status, d), s))
    _on(d, stream, body)


def read_paged(fmt, cache: PagedCache, cu: torch.Tensor, max_rows: int, first: torch.Tensor, t_quant: torch.Tensor,
               t_res: torch.Tensor, n_rows: int, out_dtype=None, k_out=None, v_out=None, status=None, stream=None,
               keys=True, values=True):
    """kvq_read_paged: the tokens at positions first[s], ... of every sequence as rows
    [cu[s], cu[s + 1]) -> k, v [n_rows, Hkv, D] (out_dtype: the source dtype by default); a side that is not
    wanted (keys / values = False) is None."""
    d = cache.device
    out_dtype = fmt.src_dtype if out_dtype is None else out_dtype
    shape, dt = (n_rows, cache.H, fmt.head_dim), TORCH_DTYPE[out_dtype]
    cu, tq, tr = _batch(cache, cu, t_quant, t_res)
    p0 = _ints(first, cache.num_seqs, d, "first")
    for x, wanted in ((k_out, keys), (v_out, values)):
        if x is not None and (not wanted or x.shape != shape or x.dtype != dt or x.device != d or not x.is_contiguous()):
            raise ValueError("k_out / v_out: contiguous [n_rows, kv_heads, head_dim] in out_dtype is needed, for a side that is read")
    _need(keys or values, "keys or values are needed")

    def body(s):
        k = torch.empty(shape, dtype=dt, device=d) if keys and k_out is None else k_out
        v = torch.empty(shape, dtype=dt, device=d) if values and v_out is None else v_out
        _check("kvq_read_paged", lib().kvq_read_paged(
            fmt, cache.struct, cu, n_rows, max_rows, p0, tq, tr, None if k is None else k.data_ptr(),
            None if v is None else v.data_ptr(), out_dtype, _status_ptr(status, d), s))
        return k, v
    return _on(d, stream, body)


def attention_paged_workspace_bytes(fmt, num_seqs, Hq, Hkv, n_rows, max_new, max_t_quant, max_t_res) -> int:
    return lib().kvq_attention_paged_workspace_bytes(fmt, num_seqs, Hq, Hkv, n_rows, max_new, max_t_quant, max_t_res)


def attention_paged(fmt, cache: PagedCache, cu_q: torch.Tensor, max_new: int, t_quant: torch.Tensor,
                    t_res: torch.Tensor, max_t_quant: int, max_t_res: int, q: torch.Tensor, scale: float, causal=True,
                    out_dtype=None, out=None, lse=None, workspace=None, status=None, stream=None):
    """kvq_attention_paged: q [rows, Hq, D] contiguous, the last cu_q[s + 1] - cu_q[s] tokens of
    every sequence -> out [rows, Hq, D] (out_dtype: q's by default); lse: fp32 [rows, Hq]."""
    d = cache.device
    if q.dtype not in KVQ_DTYPE or q.dim() != 3 or q.shape[2] != fmt.head_dim or not q.is_contiguous() or q.device != d:
        raise ValueError("q: a contiguous [rows, q_heads, head_dim] in fp32, fp16 or bf16 is needed")
    rows, Hq, _ = q.shape
    out_dtype = KVQ_DTYPE[q.dtype] if out_dtype is None else out_dtype
    dt = TORCH_DTYPE[out_dtype]
    if out is not None and (out.shape != q.shape or out.dtype != dt or out.device != d or not out.is_contiguous()):
        raise ValueError("out: a contiguous tensor of q's shape in out_dtype is needed")
    if lse is not None and (lse.shape != (rows, Hq) or lse.dtype != torch.float32 or lse.device != d or
                            not lse.is_contiguous()):
        raise ValueError("lse: a contiguous fp32 [rows, q_heads] tensor is needed")
    if workspace is not None and (not workspace.is_contiguous() or workspace.device != d):
        raise ValueError("workspace: a contiguous tensor on q's device")
    cu, tq, tr = _batch(cache, cu_q, t_quant, t_res)

    def body(s):
        o = torch.empty(q.shape, dtype=dt, device=d) if out is None else out
        w = workspace
        if w is None:
            need = attention_paged_workspace_bytes(fmt, cache.num_seqs, Hq, cache.H, rows, max_new, max_t_quant, max_t_res)
            w = torch.empty(max(need, 16), dtype=torch.uint8, device=d)
        _check("kvq_attention_paged", lib().kvq_attention_paged(
            fmt, cache.struct, cu, rows, max_new, tq, tr, max_t_quant, max_t_res, q.data_ptr(), KVQ_DTYPE[q.dtype],
            Hq, scale, int(causal), o.data_ptr(), out_dtype, None if lse is None else lse.data_ptr(), w.data_ptr(),
            w.numel() * w.element_size(), _status_ptr(status, d), s))
        return o
    return _on(d, stream, body)
