"""Pins of oracle.serving from identities the definitions imply."""
import numpy as np
import pytest

import synth
from oracle import paged, serving
from oracle.formats import BF16, Format


@pytest.mark.parametrize("scaling", range(4))
def test_scaling_limits(scaling):
    kw = dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0 if scaling == serving.BANDS else 32.0)
    plain = serving.frequencies(128, 10000.0)
    f = serving.frequencies(128, 10000.0, scaling, **kw)
    if scaling == serving.PLAIN:
        np.testing.assert_array_equal(f, plain)
    elif scaling == serving.LINEAR:
        np.testing.assert_allclose(f, plain / 8, rtol=1e-15)
    else:   # fast pairs keep their frequency, slow ones are divided, the rest lie between
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8, rel=1e-14)
        assert np.all(f <= plain * (1 + 1e-14)) and np.all(f >= plain / 8 * (1 - 1e-14))
        assert np.all(np.diff(f) < 0)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_norms_and_relative_positions(inter):
    rng = np.random.default_rng(1)
    t = serving.rope_table(serving.frequencies(32, 10000.0), 0, 100)
    q, k = rng.standard_normal((2, 64))
    qa, ka = serving.rotate(q, t[17], inter), serving.rotate(k, t[5], inter)
    qb, kb = serving.rotate(q, t[82], inter), serving.rotate(k, t[70], inter)
    assert np.linalg.norm(qa) == pytest.approx(np.linalg.norm(q))
    assert qa @ ka == pytest.approx(qb @ kb)
    np.testing.assert_array_equal(qa[32:], q[32:])
    np.testing.assert_allclose(serving.rotate32(np.float32(q), np.float32(t[17]), inter), qa, atol=1e-5)


def test_append_in_one_call_or_many_holds_the_same_tokens():
    f = Format(**synth._fmt(src_dtype=BF16, n_sink=3, residual_cap=128))
    rng = np.random.default_rng(2)
    n, H = 400, 2
    k, v = (synth.to_bf16_values(rng.standard_normal((n, H, 128)).astype(np.float32)).astype(np.float64) for _ in "kv")
    got = []
    for steps in ([n], [1, 1, 1, 125, 3, 200, 69], [100] * 4):
        pc = paged.PagedCache(f, H, 4, 1, 4)
        pc.block_table[0] = [2, 0, 3, 1]
        tq, tr, at = 0, -3, 0
        for m in steps:
            tq, tr = serving.append(pc, 0, tq, tr, k[at:at + m], v[at:at + m])
            at += m
        assert (tq, tr) == (384, 13) and f.n_sink + tq + tr == n
        got.append(serving.tokens(pc, 0, tq, tr))
    for a, b in got[1:]:
        np.testing.assert_array_equal(a, got[0][0])
        np.testing.assert_array_equal(b, got[0][1])
    # raw tokens are themselves, packed ones within a step of themselves
    K = got[0][0].swapaxes(0, 1)
    np.testing.assert_array_equal(K[:3], k[:3])
    np.testing.assert_array_equal(K[387:], k[387:])
    assert np.max(np.abs(K[3:387] - k[3:387])) < 0.5


def test_attention_of_a_chunk_is_its_rows_one_by_one():
    f = Format(**synth._fmt(src_dtype=BF16, n_sink=1, residual_cap=128))
    rng = np.random.default_rng(3)
    x = synth.to_bf16_values(rng.standard_normal((2, 150, 1, 128)).astype(np.float32)).astype(np.float64)
    pc = paged.PagedCache(f, 1, 2, 1, 2)
    pc.block_table[0] = [1, 0]
    tq, tr = serving.append(pc, 0, 0, -1, x[0], x[1])
    q = rng.standard_normal((5, 2, 128))
    out, _ = serving.attention(pc, 0, tq, tr, q, 0.1)
    one, _ = serving.attention(pc, 0, tq, tr, q[4:], 0.1)
    np.testing.assert_allclose(out[4:], one, rtol=1e-13)
    ref = paged.decode_attention(pc, q[4:], [tq], [tr], 0.1)
    np.testing.assert_allclose(out[4:], ref, rtol=1e-12)
    none, lse = serving.attention(pc, 0, 0, -1, q, 0.1)
    assert np.all(none == 0) and np.all(lse == -np.inf)
