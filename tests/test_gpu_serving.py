"""GPU parity of the serving steps around the paged cache (kvq_rope_table, kvq_norm_rope,
kvq_append_paged, kvq_read_paged, kvq_attention_paged) against oracle.serving.

Bars.  u(t) = eps(t) / 2 is the unit roundoff of a type.
 - rope_table: one rounding to fp32 and the errors of a double cosine and of the angle's
   product, below 2^-40 for these positions: |err| <= amplitude (u32 + 2^-40).
 - norm_rope: in fp32, the mean square of D <= 256 terms (tree and FMA sums, error below
   16 u32 relative), the root, quotient and two products (each within 2 u32), then at most
   three roundings in the rotation of a pair with |(x1, x2)| <= sqrt 2 max: elementwise
   32 u32 times the pair's norm, plus one rounding to the type (fp16 values below 2^-14: to a
   multiple of 2^-24).
 - append, read: the packed bytes, metadata and raw rows equal the oracle's; rows read back
   equal the oracle's fp32 x^ rounded to the type (keys of rotating formats: the
   transform's fp32 evaluation is fixed, so equal as well).
 - attention: queries, probabilities, keys and values are rounded to fp16 once each (u =
   2^-11; bf16 queries and raw bf16 / fp16 rows are exact in fp16 after scaling, rounded
   ones count all the same).  A score moves by at most d = (2u + u^2) scale sum |q||k^|, so
   a softmax weight by a factor within e^(+-2d), and elementwise
   |err| <= ((1 + 2u) (1 + 2^-16) e^(2d) - 1) sum_j p_j |v_j| + u(out) |out|
   (2^-16: fp32 sums and exponentials).  lse: |err| <= d + 2^-16 (1 + |lse|).
   Roundings of either sign average out; that they do is held by the relative L2 error:
   4 sqrt(u^2 / 3 (2 s^2 + 2)) + u(out), where s^2 is the largest row mean of
   scale^2 sum_c q_c^2 k^_c^2 (a rounding error is within u / sqrt 3 root mean square)."""
import numpy as np
import pytest
import torch

import synth
from oracle import cache as ocache
from oracle import paged as opaged
from oracle import serving
from oracle.formats import BF16, F16, F32, Format
from quantized_decode_attention_quantize_b200 import kvq
from tests.gpu_util import TORCH, dev

pytestmark = pytest.mark.gpu
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
POOL = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero")
WHT = np.array([[(-1.0) ** bin(i & j).count("1") for j in range(128)] for i in range(128)]) / np.sqrt(128)
RAW = ("sink_k", "sink_v", "res_k", "res_v")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def status0():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


def cu_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int)


def heavy(rng, shape, dt, cols=3):
    x = rng.standard_t(4, shape).astype(np.float32)
    x[..., rng.choice(shape[-1], cols, replace=False)] *= 10
    return synth.to_dtype_values(x, dt)


def normal(rng, shape, dt):
    return synth.to_dtype_values(rng.standard_normal(shape).astype(np.float32), dt)


# ---- rotary tables -------------------------------------------------------------------------
@pytest.mark.parametrize("scaling", range(4))
@pytest.mark.parametrize("R,pos0,n", [(16, 0, 1), (128, 0, 1000), (64, 131000, 77), (256, 7, 129), (48, 2 ** 31 - 40, 40)])
def test_rope_table(scaling, R, pos0, n):
    low, high = (1.0, 4.0) if scaling == kvq.ROPE_BANDS else (1.0, 32.0)
    kw = dict(factor=8.0, original_len=8192.0, low=low, high=high)
    amp = 1.25 if scaling == kvq.ROPE_RAMP else 1.0
    t = kvq.rope_table(kvq.make_rope_spec(R, base=500000.0, scaling=scaling, amplitude=amp, **kw), n, pos0=pos0)
    ref = serving.rope_table(serving.frequencies(R, 500000.0, scaling, **kw), pos0, n, amp)
    # positions near 2^31 turn by an angle of 2^31: its double product is off by up to 2^31 2^-53
    # and the host's power by a few units of 2^-53 relative
    far = (pos0 + n) * 2.0 ** -50
    assert np.max(np.abs(np64(t) - ref)) <= amp * (U[F32] + 2.0 ** -40 + far)


# ---- norm and rotation -----------------------------------------------------------------------
def check_norm(got, x, w, eps, off, row, inter, dt):
    ref = serving.norm_rope(x, w, eps, off, row, inter)
    u = serving.norm_rope(x, w, eps, off, None, False)
    bar = np.abs(u)
    if row is not None:
        a, b = serving._pairs(u, row.shape[-1], inter)
        p = np.hypot(a, b)
        bar = serving._join(bar, p, p, row.shape[-1], inter)
    err = np.abs(np64(got) - ref)
    bar = 32 * U[F32] * bar
    # the type's rounding of the computed value y, |y| <= |ref| + bar: half a step is at most u |y| for
    # a normal y and half the smallest step for a subnormal one (fp16: 2^-24 / 2)
    if dt != F32:
        bar = bar + np.maximum(U[dt] * (np.abs(ref) + bar), 2.0 ** -25 if dt == F16 else 0.0)
    assert np.all(err <= bar + 1e-30), float(np.max(err / (bar + 1e-30)))


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 64, True), (64, 64, False), (64, 16, False),
                                       (256, 256, True), (96, 48, False), (80, 80, True), (16, 16, False),
                                       (128, 0, False)])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 4, 1), (37, 5, 3)])
def test_norm_rope(D, R, inter, dt, T, Hq, Hk):
    rng = np.random.default_rng(D + R + dt + T)
    qkv = normal(rng, (T, Hq + 2 * Hk, D), dt)
    w = [normal(rng, (D,), dt) * 0.25 + 1 for _ in range(2)]
    w = [synth.to_dtype_values(x, dt) for x in w]
    pos = rng.integers(0, 500, T)
    table = serving.rope_table(serving.frequencies(R, 10000.0), 0, 500).astype(np.float32) if R else None
    g = dev(qkv, dt)
    rope = kvq.Rope(torch.from_numpy(table).cuda(), inter) if R else None
    st = status0()
    q, k = kvq.norm_rope(g[:, :Hq], g[:, Hq:Hq + Hk], dev(w[0], dt), dev(w[1], dt), eps=1e-5, rope=rope,
                         positions=ints(pos), status=st)
    row = table[pos].astype(np.float64) if R else None
    check_norm(q, qkv[:, :Hq], w[0], 1e-5, 0.0, row, inter, dt)
    check_norm(k, qkv[:, Hq:Hq + Hk], w[1], 1e-5, 0.0, row, inter, dt)
    # rotation alone equals the stepwise fp32 evaluation exactly; positions default to the index
    if R:
        q, _ = kvq.norm_rope(g[:, :Hq], rope=rope)
        row = table[np.arange(T)].astype(np.float64)
        want = serving.round_src(serving.rotate32(qkv[:, :Hq], row[:, None], inter), dt)
        np.testing.assert_array_equal(np64(q), want)
    # in place, weight offset, one side only; the v heads between are left alone
    h = g.clone()
    kvq.norm_rope(h[:, :Hq], h[:, Hq:Hq + Hk], k_weight=dev(w[1], dt), weight_offset=1.0, eps=1e-5,
                  q_out=h[:, :Hq], k_out=h[:, Hq:Hq + Hk])
    assert torch.equal(h[:, :Hq], g[:, :Hq]) and torch.equal(h[:, Hq + Hk:], g[:, Hq + Hk:])
    check_norm(h[:, Hq:Hq + Hk], qkv[:, Hq:Hq + Hk], w[1], 1e-5, 1.0, None, False, dt)
    assert int(st) == 0


def test_norm_rope_flags_positions_and_values():
    rng = np.random.default_rng(5)
    x = normal(rng, (6, 2, 64), BF16)
    rope = kvq.Rope(kvq.rope_table(kvq.make_rope_spec(64), 10))
    st = status0()
    g = dev(x, BF16)
    q, _ = kvq.norm_rope(g, rope=rope, positions=ints([0, -1, 3, 10, 9, 1 << 30]), status=st)
    assert int(st) == kvq.KVQ_DEV_BOUNDS
    for t in (0, 1, 3, 5):    # position 0 turns by nothing, the others are left unturned
        assert torch.equal(q[t], g[t])
    assert not torch.equal(q[4], g[4])
    st.zero_()
    g[2, 1, 3] = float("inf")
    g[4, 0, 5] = float("nan")
    clean, _ = kvq.norm_rope(dev(x, BF16), rope=rope)
    q, _ = kvq.norm_rope(g, rope=rope, status=st)
    assert int(st) == kvq.KVQ_DEV_NONFINITE
    assert torch.equal(q[[0, 1, 3, 5]], clean[[0, 1, 3, 5]]) and torch.equal(q[2, 0], clean[2, 0])
    # zero rows stay zero under the norm; no tokens is no work
    z = torch.zeros(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    assert not kvq.norm_rope(z, q_weight=w, eps=1e-6, rope=rope)[0].any()
    assert kvq.norm_rope(z[:0], q_weight=w)[0].shape == (0, 1, 64)


@pytest.mark.parametrize("D", [48, 128, 256])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_norm_of_rows_whose_squares_leave_fp32(D, dt, eps):
    rng = np.random.default_rng(D + dt)
    x = normal(rng, (6, 4, D), dt)
    x *= np.exp2(np.array([100, -80, 0, 64, -64, 120], np.float32))[:, None, None]   # within one warp, too
    x[:, 1] *= np.float32(2.0 ** -20)
    w = normal(rng, (D,), dt)
    st = status0()
    q, _ = kvq.norm_rope(dev(x, dt), q_weight=dev(w, dt), eps=eps, status=st)
    check_norm(q, x, w, np.float64(np.float32(eps)), 0.0, None, False, dt)
    assert int(st) == 0


# ---- cache pairs -------------------------------------------------------------------------------
class Paged:
    """The library's and the oracle's paged cache side by side."""

    def __init__(self, fd, H, S, max_blocks, seed, spare=2):
        self.fd, self.H, self.S = fd, H, S
        self.dt = fd["src_dtype"]
        self.rng = np.random.default_rng(seed)
        nb = S * max_blocks + spare
        self.fmt, self.of = kvq.make_format(fd), Format(**fd)
        self.gpu = kvq.PagedCache(self.fmt, H, nb, S, max_blocks)
        self.ora = opaged.PagedCache(self.of, H, nb, S, max_blocks)
        self.table = self.rng.permutation(nb)[:S * max_blocks].reshape(S, max_blocks).astype(np.int32)
        self.gpu.block_table.copy_(torch.from_numpy(self.table))
        self.ora.block_table[...] = self.table
        self.tq, self.tr = [0] * S, [-fd["n_sink"]] * S
        self.status = status0()

    def append(self, counts, rope=None, positions=None, max_new=None, pad=0, expect=0, skip=()):
        """Append counts[s] new tokens; `skip`: sequences that have to stay as they were."""
        n, H, rng, dt = sum(counts), self.H, self.rng, self.dt
        k, v = heavy(rng, (n + pad, H, 128), dt), normal(rng, (n + pad, H, 128), dt)
        cu = cu_of(counts)
        # k rows lie in a wider buffer, v rows token by token with heads outermost
        kt = dev(np.concatenate([k, k], 1), dt)[:, :H]
        vt = dev(v, dt).transpose(0, 1).contiguous().transpose(0, 1)
        tq_o, tr_o = ints(self.tq) * 0 - 7, ints(self.tr) * 0 - 7
        self.status.zero_()
        kvq.append_paged(self.fmt, self.gpu, ints(cu), max(counts) if max_new is None else max_new, ints(self.tq),
                         ints(self.tr), kt, vt, tq_o, tr_o, rope=rope,
                         positions=None if positions is None else ints(positions), status=self.status)
        table = None if rope is None else np64(rope.table)
        for s in range(self.S):
            if s in skip:
                continue
            ks = k[cu[s]:cu[s + 1]].astype(np.float64)
            if rope is not None and len(ks):
                first = self.fd["n_sink"] + self.tq[s] + self.tr[s]
                pos = np.arange(first, first + len(ks)) if positions is None else positions[cu[s]:cu[s + 1]]
                inter = bool(rope.struct.interleaved)
                ks = serving.round_src(serving.rotate32(ks, table[pos][:, None], inter), dt)
            self.tq[s], self.tr[s] = serving.append(self.ora, s, self.tq[s], self.tr[s], ks, v[cu[s]:cu[s + 1]])
        assert tq_o.tolist() == self.tq and tr_o.tolist() == self.tr
        assert int(self.status) == expect

    def check(self):
        """Every byte of the pool and of the raw arrays."""
        for name in POOL:
            got = self.gpu.pool.tensors[name].cpu().numpy()
            want = np.ascontiguousarray(self.ora.pool[name]).reshape(-1).view(np.uint8)
            assert np.array_equal(got, want), name
        for name in RAW:
            if name in self.gpu.raw:
                got = self.gpu.raw[name].cpu().numpy()
                want = np.ascontiguousarray(self.ora.raw[name]).reshape(-1).view(np.uint8)
                assert np.array_equal(got, want), name

    def fill(self, lengths):
        """Sequences of these lengths in one append (no comparison)."""
        self.append([x for x in lengths])

    def attend(self, counts, G, q_dt=BF16, out_dt=F32, causal=True, scale=None, with_lse=True, q=None, **kw):
        cu, Hq = cu_of(counts), G * self.H
        if q is None:
            q = normal(self.rng, (cu[-1], Hq, 128), q_dt)
        scale = 1 / np.sqrt(128) if scale is None else scale
        lse = torch.full((len(q), Hq), 7.0, device="cuda") if with_lse else None
        self.status.zero_()
        out = kvq.attention_paged(self.fmt, self.gpu, ints(cu), max(1, max(counts)) if len(q) else 0, ints(self.tq),
                                  ints(self.tr), max(self.tq), max(0, max(self.tr)), dev(q, q_dt), scale,
                                  causal=causal, out_dtype=out_dt, lse=lse, status=self.status, **kw)
        return q, scale, out, lse

    def check_attention(self, q, scale, out, lse, counts, causal, out_dt, seqs=None):
        u, cu, G = 2.0 ** -11, cu_of(counts), out.shape[1] // self.H
        out, lse = np64(out), None if lse is None else np64(lse)
        for s in range(self.S) if seqs is None else seqs:
            n = counts[s]
            if n == 0:
                continue
            qs = q[cu[s]:cu[s + 1]].astype(np.float64)
            ref, rl = serving.attention(self.ora, s, self.tq[s], self.tr[s], qs, scale, causal)
            K, V = serving.tokens(self.ora, s, self.tq[s], self.tr[s])
            L, worst, num, den = K.shape[1], 0.0, 0.0, 0.0
            for i in range(n):
                seen = max(0, L - n + i + 1) if causal else L
                got = out[cu[s] + i]
                if seen == 0:
                    assert not got.any() and (lse is None or np.all(lse[cu[s] + i] == -np.inf))
                    continue
                for hq in range(out.shape[1]):
                    k, v = K[hq // G, :seen], V[hq // G, :seen]
                    # the operands as they are rounded: in the transformed basis for rotating formats
                    # (the same products, but other magnitudes: the error bound is not invariant)
                    qb, kb = (qs[i, hq], k) if not self.fd["k_rotate"] else (qs[i, hq] @ WHT, k @ WHT)
                    d = (2 * u + u * u) * scale * np.max(np.abs(kb) @ np.abs(qb))
                    p = np.exp(scale * k @ qs[i, hq] - rl[i, hq])
                    bar = ((1 + 2 * u) * (1 + 2.0 ** -16) * np.exp(2 * d) - 1) * (p @ np.abs(v))
                    bar = bar + (U[out_dt] if out_dt != F32 else 0) * (np.abs(ref[i, hq]) + bar) + 1e-7
                    err = np.abs(got[hq] - ref[i, hq])
                    assert np.all(err <= bar), (s, i, hq, float(np.max(err / bar)))
                    if lse is not None:
                        assert abs(lse[cu[s] + i, hq] - rl[i, hq]) <= d + 2.0 ** -16 * (1 + abs(rl[i, hq]))
                    worst = max(worst, scale ** 2 * float(p @ (kb * kb) @ (qb ** 2)))
                    num, den = num + float(err @ err), den + float(ref[i, hq] @ ref[i, hq])
            if den:
                bar = 4 * np.sqrt(u * u / 3 * (2 * worst + 2)) + (U[out_dt] if out_dt != F32 else 0)
                assert np.sqrt(num / den) <= bar, (s, np.sqrt(num / den), bar)


def fmt(**kw):
    return synth._fmt(**dict(dict(src_dtype=BF16, n_sink=1, residual_cap=128), **kw))


def rope_of(R=128, inter=False, n=3000):
    return kvq.Rope(kvq.rope_table(kvq.make_rope_spec(R, base=10000.0), n), inter)


# ---- append and read -----------------------------------------------------------------------------
@pytest.mark.parametrize("kw", [dict(), dict(src_dtype=F16, n_sink=0), dict(src_dtype=F32, n_sink=5),
                                dict(residual_cap=256), dict(k_rotate=1), dict(residual_cap=384, n_sink=130)])
@pytest.mark.parametrize("turn", [None, (128, False), (64, True), (32, False)])
def test_append_matches_oracle_byte_for_byte(kw, turn):
    p = Paged(fmt(**kw), 2, 5, 6, seed=11)
    rope = None if turn is None else rope_of(*turn)
    for counts in ([0, 1, 3, 130, 300], [1, 1, 1, 1, 1], [128, 127, 0, 126, 5], [255, 0, 129, 1, 128], [2, 140, 1, 64, 0]):
        p.append(counts, rope)
        p.check()
    # read back: all of it, then a ragged window of it
    for trial in range(2):
        held = [p.fd["n_sink"] + a + b for a, b in zip(p.tq, p.tr)]
        first = [0] * 5 if trial == 0 else [h // 3 for h in held]
        counts = held if trial == 0 else [h // 2 for h in held]
        for out_dt in (F32, BF16, F16):
            k, v = kvq.read_paged(p.fmt, p.gpu, ints(cu_of(counts)), max(counts), ints(first), ints(p.tq), ints(p.tr),
                                  sum(counts), out_dtype=out_dt, status=p.status)
            at = 0
            for s in range(5):
                K, V = serving.tokens(p.ora, s, p.tq[s], p.tr[s])
                for got, want in ((k, K), (v, V)):
                    want = serving.round_src(want[:, first[s]:first[s] + counts[s]].swapaxes(0, 1), out_dt)
                    np.testing.assert_array_equal(np64(got[at:at + counts[s]]), want)
                at += counts[s]
    assert int(p.status) == 0


def test_append_takes_positions():
    p = Paged(fmt(), 2, 2, 3, seed=12)
    p.append([40, 100], rope_of(), positions=p.rng.integers(0, 3000, 140))
    p.append([200, 3], rope_of(), positions=p.rng.integers(0, 3000, 203))
    p.check()


def test_append_leaves_padding_and_bad_sequences_alone():
    p = Paged(fmt(), 2, 4, 3, seed=13)
    p.append([100, 100, 50, 60], rope_of())
    # sequence 1 misses its block, sequence 2 points outside the pool: both stay as they were
    good = p.table.copy()
    p.gpu.block_table[1, 0] = -1
    p.gpu.block_table[2, 0] = 10 ** 6
    p.append([100, 100, 100, 0], pad=9, expect=kvq.KVQ_DEV_BOUNDS, skip=(1, 2))
    p.check()
    p.gpu.block_table.copy_(torch.from_numpy(good))
    # more than max_new tokens
    p.append([3, 30, 4, 5], max_new=29, expect=kvq.KVQ_DEV_BOUNDS, skip=(1,))
    # 49 + 400 rows are three groups, all the table has room for; a fourth finds none
    p.append([3, 4, 400, 5])
    p.append([0, 0, 100, 5], expect=kvq.KVQ_DEV_BOUNDS, skip=(2,))
    p.check()
    # a position outside the table leaves the key unturned
    p.append([1, 0, 0, 0], rope=rope_of(n=200), positions=np.array([0]))
    k = dev(heavy(p.rng, (1, 2, 128), BF16), BF16)
    outs = ints(p.tq) * 0, ints(p.tr) * 0
    kvq.append_paged(p.fmt, p.gpu, ints([0, 1, 1, 1, 1]), 1, ints(p.tq), ints(p.tr), k, k, *outs, rope=rope_of(n=4),
                     positions=ints([4]), status=p.status)
    assert int(p.status) == kvq.KVQ_DEV_BOUNDS
    got, _ = kvq.read_paged(p.fmt, p.gpu, ints([0, 1, 1, 1, 1]), 1, ints([1 + p.tq[0] + p.tr[0], 0, 0, 0]), *outs, 1)
    assert torch.equal(got, k)


def test_read_leaves_what_it_cannot_read():
    p = Paged(fmt(), 2, 3, 3, seed=14)
    p.append([200, 150, 10])
    p.gpu.block_table[1, 0] = -1
    outs = [torch.full((330, 2, 128), 3.0, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    kvq.read_paged(p.fmt, p.gpu, ints([0, 150, 300, 320]), 200, ints([50, 0, 0]), ints(p.tq), ints(p.tr), 330,
                   k_out=outs[0], v_out=outs[1], status=p.status)
    assert int(p.status) == kvq.KVQ_DEV_BOUNDS
    for which, x in enumerate(outs):
        K = serving.tokens(p.ora, 0, p.tq[0], p.tr[0])[which][:, 50:200].swapaxes(0, 1)
        np.testing.assert_array_equal(np64(x[:150]), serving.round_src(K, BF16))
        K = serving.tokens(p.ora, 1, p.tq[1], p.tr[1])[which].swapaxes(0, 1)
        np.testing.assert_array_equal(np64(x[150:151]), serving.round_src(K[:1], BF16))   # the sink row
        assert torch.all(x[151:279] == 3.0)                                               # its missing page
        np.testing.assert_array_equal(np64(x[279:300]), serving.round_src(K[129:], BF16))
        assert torch.all(x[300:] == 3.0)      # more rows than sequence 2 holds; padding


# ---- attention -----------------------------------------------------------------------------------
@pytest.mark.parametrize("G,kw,q_dt,out_dt", [(4, dict(), BF16, F32), (1, dict(src_dtype=F16, n_sink=0), F16, F16),
                                              (3, dict(n_sink=4), BF16, BF16), (2, dict(src_dtype=F32), F32, F32),
                                              (4, dict(k_rotate=1), BF16, F32), (8, dict(residual_cap=256), BF16, F32),
                                              (16, dict(n_sink=150), F16, BF16)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_ragged(G, kw, q_dt, out_dt, causal):
    p = Paged(fmt(**kw), 2, 8, 8, seed=20 + G)
    lengths = [1, 2, 129, 128, 400, 257, 700, 31]
    p.fill(lengths)
    counts = [1, 2, 5, 0, 77, 257, 1, 30]
    q, scale, out, lse = p.attend(counts, G, q_dt, out_dt, causal)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, causal, out_dt)


@pytest.mark.parametrize("n,L,G", [(1, 1, 4), (1, 5000, 4), (4, 4000, 4), (64, 2000, 2), (300, 300, 4), (33, 1300, 7),
                                   (3, 4600, 16), (16, 2500, 4), (17, 2500, 4), (5, 700, 3)])
def test_attention_one_sequence(n, L, G):
    p = Paged(fmt(), 2, 1, 40, seed=40)
    p.fill([L])
    q, scale, out, lse = p.attend([n], G)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, [n], True, F32)


@pytest.mark.parametrize("kw,causal", [(dict(), True), (dict(n_sink=200, k_rotate=1), True), (dict(src_dtype=F16), False)])
def test_attention_long_chunks_with_and_without_expanded_pages(kw, causal):
    # chunks of several row blocks: with the workspace asked for the pages are expanded first, with the
    # smallest one they are not; block remainders of 1 .. 128 and of 129 .. 256 rows, windows that the
    # first rows of a chunk do not see
    p = Paged(fmt(**kw), 2, 3, 14, seed=49)
    p.fill([900, 1500, 330])
    counts = [257, 400, 330]
    full = kvq.attention_paged_workspace_bytes(p.fmt, 3, 8, 2, sum(counts), max(counts), max(p.tq), max(p.tr))
    least = kvq.attention_paged_workspace_bytes(p.fmt, 60000, 8, 2, sum(counts), max(counts), max(p.tq), max(p.tr))
    assert full - least == 3 * 2 * 65536 * (-(-max(p.tq) // 128) + -(-(p.fd["n_sink"] + max(p.tr)) // 128))
    q, scale, out, lse = p.attend(counts, 4, causal=causal)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, causal, F32)
    ws = torch.empty(least, dtype=torch.uint8, device="cuda")
    _, _, out, lse = p.attend(counts, 4, causal=causal, q=q, workspace=ws)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, causal, F32)


def test_attention_many_short_sequences():
    p = Paged(fmt(), 1, 40, 2, seed=41)
    lengths = [int(x) for x in p.rng.integers(1, 200, 40)]
    p.fill(lengths)
    counts = [min(x, int(c)) for x, c in zip(lengths, p.rng.integers(0, 6, 40))]
    q, scale, out, lse = p.attend(counts, 4, out_dt=BF16)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, True, BF16)


@pytest.mark.parametrize("G,kw,q_dt,out_dt", [(4, dict(n_sink=0), BF16, F32), (1, dict(src_dtype=F16), F16, F16),
                                              (4, dict(k_rotate=1, n_sink=140), BF16, BF16),
                                              (3, dict(src_dtype=F32), F32, F32)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_drafts(G, kw, q_dt, out_dt, causal):
    # a few tokens per sequence: blocks of 16 rows, some full, some not, some sequences without any
    p = Paged(fmt(**kw), 2, 6, 14, seed=60 + G)
    p.fill([1700, 3, 129, 600, 260, 128])
    counts = [5, 3, 0, 4, 1, 2]
    q, scale, out, lse = p.attend(counts, G, q_dt, out_dt, causal)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, causal, out_dt)


def test_attention_rows_without_tokens_and_steep_scores():
    # more query rows than tokens: the first rows see nothing
    p = Paged(fmt(n_sink=3), 2, 3, 3, seed=42)
    p.fill([2, 150, 1])
    counts = [5, 3, 40]
    q, scale, out, lse = p.attend(counts, 4)
    p.check_attention(q, scale, out, lse, counts, True, F32)
    # one score towers over the rest (the softmax is a single token), and tiny / huge queries
    q = normal(p.rng, (48, 8, 128), BF16)
    q[3] = synth.to_bf16_values(q[3] * np.float32(30))
    q[5] = synth.to_bf16_values(q[5] * np.float32(1e-30))
    q[6] = 0
    q[7] = synth.to_bf16_values(q[7] * np.float32(2.0 ** 100))
    _, scale, out, lse = p.attend(counts, 4, scale=2.0 ** -100, q=q)
    p.check_attention(q, scale, out, lse, counts, True, F32)


@pytest.mark.parametrize("counts", [[2, 1, 3], [40, 100, 1], [300, 130, 70]])
def test_attention_over_nothing(counts):
    # sequences without a single token, without a sink, at each of the kernels
    p = Paged(fmt(n_sink=0), 2, 3, 2, seed=64)
    p.fill([0, 130, 0])
    q, scale, out, lse = p.attend(counts, 4)
    assert int(p.status) == 0
    p.check_attention(q, scale, out, lse, counts, True, F32)


@pytest.mark.parametrize("n", [4, 30, 200])
def test_attention_ignores_unseen_values_that_did_not_fit(n):
    # a packed value token with an infinite scale, later than the queries' first rows see
    p = Paged(fmt(n_sink=0), 2, 1, 3, seed=65)
    p.fill([256])
    q, scale, clean, _ = p.attend([n], 4)
    for name in ("v_scale", "v_zero"):
        p.gpu.pool.tensors[name].view(torch.float16).view(-1, 2, 128)[int(p.table[0, 1]), :, 126] = float("inf")
    _, _, out, _ = p.attend([n], 4, q=q)
    assert torch.equal(out[:n - 2], clean[:n - 2])


def test_attention_agrees_with_decode():
    p = Paged(fmt(), 2, 4, 8, seed=43)
    p.fill([700, 129, 1, 330])
    q, scale, out, _ = p.attend([1] * 4, 4)
    dec = kvq.decode_attention_paged(p.fmt, p.gpu, ints(p.tq), ints(p.tr), max(p.tq), max(p.tr), dev(q, BF16), scale)
    # both within 1e-3 relative L2 of the oracle, the bar of the decode's own tests
    assert float((out - dec).norm() / dec.norm()) <= 2e-3


def test_attention_masked_places_may_hold_anything():
    # a NaN / Inf / huge window row that a query does not see changes nothing for it
    p = Paged(fmt(), 2, 1, 3, seed=44)
    p.fill([60])
    q, scale, clean, _ = p.attend([20], 4)
    res = {n: p.gpu.raw[n].view(torch.bfloat16).view(2, 128, 128) for n in ("res_k", "res_v")}
    res["res_k"][:, 58, 3] = float("inf")
    res["res_v"][:, 58, 5] = float("nan")
    res["res_v"][:, 58, 6] = 1e30
    for n in res:
        res[n][:, 59:] = float("nan")          # behind the sequence: not even flagged
    _, _, out, _ = p.attend([20], 4, q=q)
    assert torch.equal(out[:19], clean[:19])
    assert int(p.status) == kvq.KVQ_DEV_NONFINITE | kvq.KVQ_DEV_RANGE
    # whatever the pages hold behind a partial group, and the blocks nobody owns
    p = Paged(fmt(), 2, 1, 3, seed=45)
    p.fill([1 + 200])                          # one packed group of 128, a window of 72
    q, scale, clean, _ = p.attend([3], 4)
    for b in set(range(p.gpu.num_blocks)) - {int(p.table[0, 0])}:
        for n in POOL:
            p.gpu.pool.tensors[n].view(p.gpu.num_blocks, -1)[b] = 255
    _, _, out, _ = p.attend([3], 4, q=q)
    assert torch.equal(out, clean) and int(p.status) == 0
    # packed lengths that end inside a group: codes and metadata behind the end are not read into it
    part = Paged(fmt(), 2, 1, 3, seed=46)
    part.fill([1 + 128])
    k = dev(normal(part.rng, (1, 2, 40, 128), BF16), BF16)
    view = kvq.PagedCache(part.fmt, 2, part.gpu.num_blocks, 1, 3, arrays=dict(part.gpu.pool.tensors, **part.gpu.raw,
                                                                           block_table=part.gpu.block_table))
    blk = int(part.table[0, 1])
    kvq.quantize_kv_paged(part.fmt, view, k, k, ints([blk]), 40)
    opaged.quantize_group(part.ora, 0, np64(k)[0], blk, 40)
    opaged.quantize_group(part.ora, 1, np64(k)[0], blk, 40)
    for n, per in (("v_scale", 2), ("v_zero", 2)):
        part.gpu.pool.tensors[n].view(torch.float16).view(-1, 2, 128)[blk, :, 40:] = float("nan")
    part.gpu.pool.tensors["v_codes"].view(-1, 2, 64, 64)[blk, :, 20:] = 255
    part.tq, part.tr = [168], [0]
    q, scale, out, lse = part.attend([50], 4)
    assert int(part.status) == 0
    part.check_attention(q, scale, out, lse, [50], True, F32)


def test_attention_bounds_are_flagged_not_followed():
    p = Paged(fmt(), 2, 3, 6, seed=47)
    p.fill([500, 300, 40])
    counts = [3, 4, 5]
    q, scale, clean, _ = p.attend(counts, 4)
    good = p.table.copy()
    p.gpu.block_table[1, 0] = 1 << 30          # read from block 0, flagged; the others unaffected
    _, _, out, _ = p.attend(counts, 4, q=q)
    assert int(p.status) == kvq.KVQ_DEV_BOUNDS
    assert torch.equal(out[:3], clean[:3]) and torch.equal(out[7:], clean[7:])
    p.gpu.block_table.copy_(torch.from_numpy(good))
    # a length above the bound it was launched with: its rows are left as they were
    out = torch.full_like(clean, 3.0)
    p.status.zero_()
    kvq.attention_paged(p.fmt, p.gpu, ints(cu_of(counts)), 5, ints(p.tq), ints(p.tr), 256, max(p.tr), dev(q, BF16),
                        scale, out_dtype=F32, out=out, status=p.status)
    assert int(p.status) == kvq.KVQ_DEV_BOUNDS
    assert torch.all(out[:3] == 3.0)
    # the others: with sequence 0 gone the work is cut at other tiles, so the sums round otherwise
    # (not bit for bit the same), within the bars that hold for any cut
    p.check_attention(q, scale, out, None, counts, True, F32, seqs=(1, 2))
    # rows behind the last sequence and rows of an empty one
    out = torch.full((20, 8, 128), 3.0, device="cuda")
    q2 = torch.cat([dev(q, BF16), dev(q, BF16)])[:20]
    kvq.attention_paged(p.fmt, p.gpu, ints(cu_of(counts)), 5, ints(p.tq), ints(p.tr), max(p.tq), max(p.tr), q2, scale,
                        out_dtype=F32, out=out)
    assert torch.equal(out[:12], clean) and torch.all(out[12:] == 3.0)


def test_attention_long_tail_of_small_weights():
    # 2^14 tokens of equal weight 2^-12 below one: the tail holds most of the mass
    p = Paged(fmt(n_sink=0), 1, 1, 140, seed=48)
    L = 128 * 128
    k = np.zeros((L, 1, 128), np.float32)
    k[:, 0, 0] = -12 * np.log(2.0)
    k[5, 0, 0] = 0
    k = synth.to_bf16_values(k)
    v = normal(p.rng, (L, 1, 128), BF16)
    v[..., 1] = 1.0
    outs = ints([0]), ints([0])
    kvq.append_paged(p.fmt, p.gpu, ints([0, L]), L, ints([0]), ints([0]), dev(k, BF16), dev(v, BF16), *outs)
    p.tq, p.tr = serving.append(p.ora, 0, 0, 0, k.astype(np.float64), v.astype(np.float64))
    p.tq, p.tr = [p.tq], [p.tr]
    assert outs[0].tolist() == p.tq
    q = np.zeros((2, 1, 128), np.float32)
    q[:, 0, 0] = 1.0
    _, scale, out, lse = p.attend([2], 1, scale=1.0, q=q)
    p.check_attention(q, scale, out, lse, [2], True, F32)


# ---- the steps together, streams, graphs ------------------------------------------------------------
def step(p, h, cu, counts, tq, tr, qkv, rope, w, bufs, Hq, stream=None):
    """One serving step: norm and rotate q and k in place, append, attend."""
    H = p.H
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    kvq.norm_rope(q, k, w, w, rope=rope, positions=bufs["pos"], q_out=bufs["q"], k_out=k, stream=stream)
    kvq.append_paged(p.fmt, p.gpu, cu, counts, tq, tr, k, v, bufs["tq"], bufs["tr"], stream=stream)
    kvq.attention_paged(p.fmt, p.gpu, cu, counts, bufs["tq"], bufs["tr"], 6 * 128, 128, bufs["q"], 1 / np.sqrt(128),
                        out=bufs["out"], workspace=bufs["ws"], stream=stream)


def test_steps_together_eager_on_a_stream_and_in_a_graph():
    S, H, G = 3, 2, 4
    Hq = G * H
    rope = rope_of()
    rng = np.random.default_rng(50)
    w = dev(synth.to_bf16_values(1 + 0.1 * rng.standard_normal(128).astype(np.float32)), BF16)
    results = []
    for mode in ("eager", "stream", "graph"):
        p = Paged(fmt(), H, S, 6, seed=51)
        rng = np.random.default_rng(52)
        tq, tr = ints(p.tq), ints(p.tr)
        outs = []
        for counts, reps in (([130, 7, 127], 1), ([1, 1, 1], 4), ([5, 0, 200], 1)):
            n = sum(counts)
            bufs = dict(pos=ints([0] * n), q=torch.empty(n, Hq, 128, device="cuda", dtype=torch.bfloat16),
                        out=torch.empty(n, Hq, 128, device="cuda", dtype=torch.bfloat16), tq=tq.clone(), tr=tr.clone())
            need = kvq.attention_paged_workspace_bytes(p.fmt, S, Hq, H, n, max(counts), 6 * 128, 128)
            bufs["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
            qkv = torch.empty(n, Hq + 2 * H, 128, device="cuda", dtype=torch.bfloat16)
            cu = ints(cu_of(counts))
            graph = None
            for _ in range(reps):
                qkv.copy_(dev(normal(rng, tuple(qkv.shape), BF16), BF16))
                held = (1 + tq + tr).tolist()
                bufs["pos"].copy_(ints([h + i for h, c in zip(held, counts) for i in range(c)]))
                args = (p, None, cu, max(counts), tq, tr, qkv, rope, w, bufs, Hq)
                if mode == "eager":
                    step(*args)
                elif mode == "stream":
                    other = torch.cuda.Stream()
                    other.wait_stream(torch.cuda.current_stream())
                    step(*args, stream=other)
                    torch.cuda.current_stream().wait_stream(other)
                else:
                    if graph is None:
                        graph = torch.cuda.CUDAGraph()
                        torch.cuda.synchronize()
                        with torch.cuda.graph(graph):
                            step(*args)
                    graph.replay()
                outs.append(bufs["out"].clone())
                tq.copy_(bufs["tq"])
                tr.copy_(bufs["tr"])
        torch.cuda.synchronize()
        results.append((torch.cat(outs), {n: t.clone() for n, t in {**p.gpu.pool.tensors, **p.gpu.raw}.items()},
                        tq.tolist(), tr.tolist()))
    for r in results[1:]:
        assert torch.equal(r[0], results[0][0]) and r[2:] == results[0][2:]
        for n in r[1]:
            assert torch.equal(r[1][n], results[0][1][n]), n
    assert torch.isfinite(results[0][0].float()).all()


def test_attention_repeats_itself_bit_for_bit():
    p = Paged(fmt(), 2, 4, 30, seed=53)
    p.fill([3500, 129, 1000, 330])
    counts = [4, 1, 30, 3]
    q, scale, out, lse = p.attend(counts, 4)
    for _ in range(3):
        _, _, again, lse2 = p.attend(counts, 4, q=q)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_pools_past_32_bits_of_offset():
    # 40 000 blocks of 8 heads: 2.6 GB of key codes; the sequences' blocks lie anywhere among them
    p = Paged(fmt(), 8, 2, 5, seed=70, spare=40000)
    assert p.gpu.pool.tensors["k_codes"].numel() > 2 ** 31 and p.table.max() > 33000
    p.append([500, 300], rope_of())
    for counts in ([2, 1], [150, 40], [500, 300]):
        q, scale, out, lse = p.attend(counts, 2)
        assert int(p.status) == 0
        for s in range(2):
            ref, _ = serving.attention(p.ora, s, p.tq[s], p.tr[s],
                                       q[cu_of(counts)[s + 1] - 1:cu_of(counts)[s + 1]].astype(np.float64), scale)
            got = np64(out[cu_of(counts)[s + 1] - 1])
            # 2e-3: twice the relative L2 bar of the decode's own tests for fp32 output
            assert np.linalg.norm(got - ref[0]) <= 2e-3 * np.linalg.norm(ref)
    k, v = kvq.read_paged(p.fmt, p.gpu, ints([0, 500, 800]), 500, ints([0, 0]), ints(p.tq), ints(p.tr), 800)
    for s, (lo, hi) in enumerate(((0, 500), (500, 800))):
        K, V = serving.tokens(p.ora, s, p.tq[s], p.tr[s])
        np.testing.assert_array_equal(np64(k[lo:hi]), serving.round_src(K.swapaxes(0, 1), BF16))
        np.testing.assert_array_equal(np64(v[lo:hi]), serving.round_src(V.swapaxes(0, 1), BF16))


def test_many_sequences():
    # 700 sequences: the partition, the searches and the flat grids over more than one pass of a warp
    S = 700
    p = Paged(fmt(), 1, S, 2, seed=71)
    rng = np.random.default_rng(72)
    lengths = rng.integers(0, 230, S)
    lengths[rng.integers(0, S, 150)] = 0
    p.append([int(x) for x in lengths], rope_of(32, True))
    p.check()
    for most in (3, 70):
        counts = [int(min(x, c)) for x, c in zip(lengths, rng.integers(0, most + 1, S))]
        q, scale, out, lse = p.attend(counts, 2, out_dt=BF16)
        assert int(p.status) == 0
        p.check_attention(q, scale, out, lse, counts, True, BF16, seqs=list(range(0, S, 9)) + [S - 1])
