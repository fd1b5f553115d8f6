"""The serving steps at the ends of their number ranges: packed and raw magnitudes beyond fp16,
scales near its end, rows that are not finite, and what the status word says of them.

Bars as in test_gpu_serving, u = 2^-11 being half a step of fp16, with one term more.  Attention of at
most 64 query rows per KV head and sequence sums p s c in fp16 products and p z apart, so the rounding of
p s counts against s c = v - z and not against v: the sums of p |v| become sums of p (|v| + |z|), z the token's
zero-point.  Its key products round q s against c - 8, at most 8 s = (k_15 - k_0) 8 / 15 per channel, k_0 and k_15
the ends of the channel's range: below the largest |q| |k| of the group's tokens where the ends are reached."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import serving
from oracle.formats import BF16, F16, F32
from quantized_decode_attention_quantize_b200 import kvq
from tests.gpu_util import dev
from tests.test_gpu_serving import POOL, U, WHT, Paged, check_norm, cu_of, fmt, ints, normal, np64, rope_of, status0

pytestmark = pytest.mark.gpu
RANGE, NONFINITE, BOUNDS = kvq.KVQ_DEV_RANGE, kvq.KVQ_DEV_NONFINITE, kvq.KVQ_DEV_BOUNDS
TOP = 65504.0


def filled(fd, k, v, H=2, blocks=5):
    """One sequence without a sink that holds the rows k, v [L, H, 128] (exact in the source type)."""
    p = Paged(fd, H, 1, blocks, seed=3)
    out = ints([0]), ints([0])
    kvq.append_paged(p.fmt, p.gpu, ints([0, len(k)]), len(k), ints([0]), ints([0]), dev(k, p.dt), dev(v, p.dt), *out,
                     status=p.status)
    tq, tr = serving.append(p.ora, 0, 0, 0, k.astype(np.float64), v.astype(np.float64))
    p.tq, p.tr = [tq], [tr]
    assert out[0].tolist() == p.tq and out[1].tolist() == p.tr
    return p


def check_rows(p, q, scale, out, lse, K, V):
    """Causal rows of the one sequence over K, V [H, L, 128]."""
    u, n, L, G = 2.0 ** -11, len(q), K.shape[1], q.shape[1] // K.shape[0]
    out, lse = np64(out), np64(lse)
    z = np.abs(V.min(-1))
    for i in range(n):
        seen = L - n + i + 1
        for h in range(q.shape[1]):
            k, v, row = K[h // G, :seen], V[h // G, :seen], q[i, h].astype(np.float64)
            qb, kb = (row, k) if not p.fd["k_rotate"] else (row @ WHT, k @ WHT)
            # the group's other tokens share its scales, seen or not
            every = K[h // G] if not p.fd["k_rotate"] else K[h // G] @ WHT
            d = (2 * u + u * u) * scale * np.max(np.abs(every) @ np.abs(qb))
            x = scale * kb @ qb
            rl = x.max() + np.log(np.exp(x - x.max()).sum())
            w = np.exp(x - rl)
            want = w @ v
            bar = ((1 + 2 * u) * (1 + 2.0 ** -16) * np.exp(2 * d) - 1) * (w @ (np.abs(v) + z[h // G, :seen, None])) + 1e-7
            err = np.abs(out[i, h] - want)
            assert np.all(err <= bar), (i, h, float(np.max(err / bar)))
            assert abs(lse[i, h] - rl) <= d + 2.0 ** -16 * (1 + abs(rl)), (i, h)


# ---- packed magnitudes beyond fp16 ------------------------------------------------------------
@pytest.mark.parametrize("n", [4, 30, 200])      # 16 rows per KV head, 120, and 800
@pytest.mark.parametrize("what", ["value", "key", "both", "fp16 value", "fp16 key"])
def test_packed_magnitudes_beyond_fp16(n, what):
    dt = F16 if what.startswith("fp16") else BF16
    rng = np.random.default_rng(80)
    k, v = normal(rng, (384, 2, 128), dt), normal(rng, (384, 2, 128), dt)
    at = 382                                       # the last but one: few rows see it
    if what in ("value", "both"):
        v[at, :, 7] = synth.to_bf16_values(np.float32(150000))
    if what in ("key", "both"):
        k[at, :, 9] = synth.to_bf16_values(np.float32(900000))
    if what == "fp16 value":
        v[at, :, 7], v[at, :, 90] = TOP, -TOP       # 3 s + z = 65536
    if what == "fp16 key":
        k[at, :, 9], k[at - 1, :, 9] = TOP, -TOP    # 15 s + z = 65536
    p = filled(fmt(n_sink=0, src_dtype=dt), k, v)
    assert int(p.status) == 0                      # every scale and zero-point fits
    K, V = serving.tokens(p.ora, 0, p.tq[0], p.tr[0])
    assert max(K.max(), V.max()) > TOP
    if n > 16:                                     # tiles of fp16 keys and values: the largest number stands in
        K, V = np.minimum(K, TOP), np.minimum(V, TOP)
    q, scale, out, lse = p.attend([n], 4, scale=2.0 ** -18)
    assert int(p.status) == RANGE
    assert torch.isfinite(out).all()
    check_rows(p, q, scale, out, lse, K, V)


@pytest.mark.parametrize("n", [4, 30, 200])
@pytest.mark.parametrize("names", [("k_scale",), ("k_zero",), ("v_scale",), ("v_zero",), ("k_scale", "v_zero")])
def test_packed_metadata_that_did_not_fit_counts_as_zero(n, names):
    # an append of larger magnitudes yet (which raised KVQ_DEV_RANGE) leaves Inf in the metadata
    rng = np.random.default_rng(81)
    p = filled(fmt(n_sink=0), normal(rng, (384, 2, 128), BF16), normal(rng, (384, 2, 128), BF16))
    K, V = serving.tokens(p.ora, 0, p.tq[0], p.tr[0])
    for name in names:
        sign = -1 if name.endswith("zero") else 1
        p.gpu.pool.tensors[name].view(torch.float16).view(-1, 2, 128)[int(p.table[0, 2]), :, 126] = sign * float("inf")
        if name[0] == "k":
            K[:, 256:, 126] = 0
        else:
            V[:, 256 + 126] = 0
    q, scale, out, lse = p.attend([n], 4)
    assert int(p.status) == RANGE
    check_rows(p, q, scale, out, lse, K, V)


# ---- key scales near fp16's end ------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 4, 30, 200])
@pytest.mark.parametrize("kw", [dict(), dict(src_dtype=F16), dict(src_dtype=F16, k_rotate=1)])
@pytest.mark.parametrize("c", range(8))
def test_key_scales_near_the_end_of_fp16(n, kw, c):
    # a channel from -62000 to 62000 has scale 8267; every number stays inside fp16
    fd = fmt(**dict(dict(n_sink=0), **kw))
    dt = fd["src_dtype"]
    rng = np.random.default_rng(82)
    k, v = normal(rng, (384, 2, 128), dt), normal(rng, (384, 2, 128), dt)
    if fd["k_rotate"]:
        e = np.zeros(128)
        e[c] = 62000
        row = synth.to_dtype_values((e @ WHT).astype(np.float32), dt)
        k[380], k[381] = row, -row
    else:
        k[380, :, c], k[381, :, c] = synth.to_dtype_values(np.float32(62000), dt), synth.to_dtype_values(np.float32(-62000), dt)
    p = filled(fd, k, v)
    assert int(p.status) == 0
    K, V = serving.tokens(p.ora, 0, p.tq[0], p.tr[0])
    q = normal(rng, (n, 8, 128), BF16)
    if fd["k_rotate"]:
        e[c] = 7.96875
        q = synth.to_bf16_values((0.01 * q + e @ WHT).astype(np.float32))
    else:
        q[:, :, c] = 7.96875                       # just below a power of two, the row's largest
    q, scale, out, lse = p.attend([n], 4, scale=2.0 ** -16, q=q)
    assert int(p.status) == 0
    check_rows(p, q, scale, out, lse, K, V)


@pytest.mark.parametrize("n", [1, 4, 16])
@pytest.mark.parametrize("top", [100000.0, 300000.0, 600000.0, 940000.0])
@pytest.mark.parametrize("kw", [dict(), dict(src_dtype=F32)])
def test_key_scales_up_to_the_end_of_fp16(n, top, kw):
    # all eight channels of an octet, some with small scales beside them; at most 64 rows take packed keys as they are
    fd = fmt(n_sink=0, **kw)
    dt = fd["src_dtype"]
    rng = np.random.default_rng(86)
    k, v = normal(rng, (384, 2, 128), dt), normal(rng, (384, 2, 128), dt)
    k[300, :, 8:16] = synth.to_dtype_values(np.float32(top), dt)
    k[:, :, 16:64] *= np.float32(2.0 ** -12)
    p = filled(fd, k, v)
    assert int(p.status) == 0
    K, V = serving.tokens(p.ora, 0, p.tq[0], p.tr[0])
    q = normal(rng, (n, 8, 128), BF16)
    q[:, ::2, 8:16] = 7.96875
    q, scale, out, lse = p.attend([n], 4, scale=2.0 ** -20, q=q)
    assert int(p.status) == RANGE
    check_rows(p, q, scale, out, lse, K, V)


# ---- raw rows of a transforming format ------------------------------------------------------------
@pytest.mark.parametrize("n", [4, 30, 100])
@pytest.mark.parametrize("where", ["window", "sink"])
def test_raw_keys_that_leave_fp16_in_the_transformed_basis(n, where):
    # a constant row has sqrt(128) times its magnitude in one channel of the transform
    rng = np.random.default_rng(83)
    ns = 0 if where == "window" else 120
    k, v = normal(rng, (110, 2, 128), F16), normal(rng, (110, 2, 128), F16)
    p = Paged(fmt(n_sink=ns, src_dtype=F16, k_rotate=1), 2, 1, 3, seed=3)
    tr0 = -ns
    for rows in ("clean", "large"):
        if rows == "large":
            k[109] = 60000
        out = ints([0]), ints([0])
        kvq.append_paged(p.fmt, p.gpu, ints([0, 110]), 110, ints([0]), ints([tr0]), dev(k, F16), dev(v, F16), *out)
        p.tq, p.tr = [0], out[1].tolist()
        if rows == "clean":
            q, scale, clean, _ = p.attend([n], 4, scale=2.0 ** -16)
            assert int(p.status) == 0
        else:
            _, _, out, lse = p.attend([n], 4, scale=2.0 ** -16, q=q)
    assert int(p.status) == RANGE
    assert torch.equal(out[:n - 1], clean[:n - 1])
    T = np.clip(k.astype(np.float64) @ WHT, -TOP, TOP) @ WHT
    check_rows(p, q, scale, out, lse, T.swapaxes(0, 1), v.astype(np.float64).swapaxes(0, 1))


# ---- the append's codes ------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("bad", [-100000.0, 2000000.0, float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rotate", [0, 1])
def test_appended_groups_equal_the_quantizers_whatever_they_hold(dt, bad, rotate):
    # one key channel and one value token that do not fit (or are no numbers): the other channels and
    # tokens must not notice, and a group appended holds what kvq_quantize_kv_paged packs
    if dt == F16 and np.isfinite(bad):
        bad = float(np.sign(bad)) * TOP            # all that the type has; it fits
    rng = np.random.default_rng(84)
    k, v = normal(rng, (128, 2, 128), dt), normal(rng, (128, 2, 128), dt)
    clean = k.copy(), v.copy()
    k[40, :, 9] = v[41, :, 70] = bad
    pools = []
    for ks, vs in ((k, v), clean):
        p = Paged(fmt(n_sink=0, src_dtype=dt, k_rotate=rotate), 2, 1, 2, seed=4, spare=2)
        out = ints([0]), ints([0])
        kvq.append_paged(p.fmt, p.gpu, ints([0, 128]), 128, ints([0]), ints([0]), dev(ks, dt), dev(vs, dt), *out,
                         status=p.status)
        assert out[0].tolist() == [128] and out[1].tolist() == [0]
        blk, other = int(p.table[0, 0]), int(p.table[0, 1])
        st = status0()
        kvq.quantize_kv_paged(p.fmt, p.gpu, dev(ks, dt).transpose(0, 1)[None], dev(vs, dt).transpose(0, 1)[None],
                              ints([other]), 128, status=st)
        assert int(st) == int(p.status)
        pools.append([p.gpu.pool.tensors[n].view(p.gpu.num_blocks, 2, -1)[[blk, other]].cpu().numpy() for n in POOL])
    fits = dt == F16 and np.isfinite(bad)
    assert (int(p.status) == 0) and (fits or not np.array_equal(pools[0][0], pools[1][0]))
    for name, got, same in zip(POOL, *pools):
        np.testing.assert_array_equal(got[0], got[1], err_msg=name)
        if rotate and name[0] == "k":
            continue                               # the transform spreads a row's element over its channels
        a, b = got[0], same[0]                     # [head, bytes]: keys by channel, values by token
        if name == "k_codes":
            keep = np.ones((128, 64), bool)
            keep[:, 4] = False                     # channels 8 and 9 share a byte
            a, b = (x.reshape(2, 128, 64)[:, keep] for x in (a, b))
            hi = [x[0].reshape(2, 128, 64)[:, :, 4] & 15 for x in (got, same)]
            np.testing.assert_array_equal(*hi)
        elif name == "v_codes":
            a, b = (np.delete(x.reshape(2, 64, 64), 20, 1) for x in (a, b))   # tokens 40 and 41 share words
        else:
            a, b = (np.delete(x.view(np.float16), 9 if name[0] == "k" else 41, 1) for x in (a, b))
        np.testing.assert_array_equal(a, b, err_msg=name)


# ---- one side read back -------------------------------------------------------------------------------
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("long", [False, True])
def test_read_of_one_side_raises_what_both_raise(side, long):
    p = Paged(fmt(), 2, 3, 3, seed=14)
    p.append([200, 150, 10])
    n = 140 if long else 100

    def read(tq, first):
        cu, first, tq, tr = ints([0, n, 2 * n, 2 * n + 5]), ints(first), ints(tq), ints(p.tr)
        out = torch.full((3 * n, 2, 128), 3.0, device="cuda", dtype=torch.bfloat16)
        p.status.zero_()
        args = [out.data_ptr(), None] if side == "k" else [None, out.data_ptr()]
        st = kvq.lib().kvq_read_paged(ctypes.byref(p.fmt), p.gpu.ref(), kvq._ptr(cu), 3 * n, n, kvq._ptr(first),
                                      kvq._ptr(tq), kvq._ptr(tr), *args, BF16, kvq._ptr(p.status), None)
        torch.cuda.synchronize()
        assert st == kvq.KVQ_OK
        return out, int(p.status)

    want = [serving.tokens(p.ora, s, p.tq[s], p.tr[s])[side == "v"] for s in range(3)]

    def rows(s, lo, m):
        return serving.round_src(want[s][:, lo:lo + m].swapaxes(0, 1), BF16)

    out, st = read(p.tq, [3, 4, 2])
    assert st == 0
    for s, (lo, m) in enumerate(((3, n), (4, n), (2, 5))):
        np.testing.assert_array_equal(np64(out[s * n:s * n + m]), rows(s, lo, m))
    assert torch.all(out[2 * n + 5:] == 3.0)
    for tq, first in ((p.tq, [3, 200, 2]), ([p.tq[0], -5, p.tq[2]], [3, 4, 2])):   # tokens it does not hold; a bad length
        out, st = read(tq, first)
        assert st == BOUNDS
        np.testing.assert_array_equal(np64(out[:n]), rows(0, 3, n))
        assert torch.all(out[n:2 * n] == 3.0)
        np.testing.assert_array_equal(np64(out[2 * n:2 * n + 5]), rows(2, 2, 5))
    # the wrapper reads one side of the same rows
    args = (p.fmt, p.gpu, ints([0, n, 2 * n, 2 * n + 5]), n, ints([3, 4, 2]), ints(p.tq), ints(p.tr), 2 * n + 5)
    got = kvq.read_paged(*args, keys=side == "k", values=side == "v")
    both = kvq.read_paged(*args)
    i = "kv".index(side)
    assert got[1 - i] is None and torch.equal(got[i], both[i])


# ---- keys turned beyond their type ----------------------------------------------------------------------
@pytest.mark.parametrize("dt,x", [(F16, 60000.0), (BF16, 3e38), (F32, 3e38)])
@pytest.mark.parametrize("n", [1, 100, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_keys_turned_beyond_their_type_are_flagged(dt, x, n, inter):
    # cos + sin reaches sqrt 2: a pair of large channels leaves the source type
    rng = np.random.default_rng(85)
    k, v = normal(rng, (n, 2, 128), dt), normal(rng, (n, 2, 128), dt)
    pair = (0, 1) if inter else (0, 64)
    k[n - 1, 1, list(pair)] = synth.to_dtype_values(np.full(2, x, np.float32), dt)
    p = Paged(fmt(n_sink=0, src_dtype=dt), 2, 1, 3, seed=5)
    table = torch.ones(n, 128, device="cuda") * np.float32(np.sqrt(0.5))
    out = ints([0]), ints([0])
    call = lambda k, rope: kvq.append_paged(p.fmt, p.gpu, ints([0, n]), n, ints([0]), ints([0]), dev(k, dt), dev(v, dt), *out,
                                            rope=rope, status=p.status)
    rope = kvq.Rope(table, inter)
    call(k, rope)
    assert int(p.status) == RANGE
    # unturned it fits the type; a number that is none is still called that, turned or not
    p.status.zero_()
    if n < 128:
        call(k, None)
        assert int(p.status) == 0
    for bad in (float("nan"), float("inf")):
        k[n - 1, 1, pair[1]] = bad
        for r in (rope, None):
            p.status.zero_()
            call(k, r)
            assert int(p.status) & NONFINITE and (n == 256 or int(p.status) == NONFINITE)


# ---- norm of subnormal rows ---------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [48, 128, 256])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-30])
def test_norm_of_subnormal_rows(D, dt, eps):
    # whole numbers of the type's smallest steps (2^-149, bf16 2^-133), exact in every type
    rng = np.random.default_rng(D + dt)
    x = rng.integers(-3, 4, (5, 3, D)).astype(np.float32) * np.float32(2.0 ** -149 if dt == F32 else 2.0 ** -133)
    x[2] *= np.float32(64)
    x[3] *= np.float32(2.0 ** 60)
    x[:, :, 0] = x[:, :, 0] + (x[:, :, 0] == 0) * np.abs(x[:, :, 1:]).max(-1)   # no row is all zero
    w = normal(rng, (D,), dt)
    st = status0()
    q, _ = kvq.norm_rope(dev(x, dt), q_weight=dev(w, dt), eps=eps, status=st)
    check_norm(q, x, w, np.float64(np.float32(eps)), 0.0, None, False, dt)
    assert int(st) == 0
