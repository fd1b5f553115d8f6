"""Host checks of the serving entry points (no GPU): what they refuse, before anything is
launched."""
import ctypes

import pytest
import torch

import synth
from quantized_decode_attention_quantize_b200 import kvq

A = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(24)]
# made-up device addresses: only where no launch could follow a check that has regressed
fake_pointers = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses; CPU only")
INV, UNS, WS = kvq.KVQ_ERR_INVALID, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE


def fmt(**kw):
    return kvq.make_format(synth._fmt(**dict(dict(src_dtype=synth.BF16, n_sink=1, residual_cap=128), **kw)))


def cache(f, H=2, S=3, blocks=4, cols=2):
    pc = kvq.kvq_paged_cache(pool=kvq.kvq_cache(batch=blocks, kv_heads=H, capacity=128), num_seqs=S, max_blocks=cols,
                             block_table=0x7000000)
    for i, n in enumerate(kvq.ARRAYS):
        setattr(pc.pool, n, 0x8000000 + 0x100000 * i)
    for i, n in enumerate(("sink_k", "sink_v", "res_k", "res_v")):
        setattr(pc, n, 0xA000000 + 0x100000 * i)
    return pc


@fake_pointers
@pytest.mark.parametrize("kw,pos0,n", [
    (dict(rot_dim=24), 0, 4), (dict(rot_dim=0), 0, 4), (dict(rot_dim=272), 0, 4), (dict(base=1.0), 0, 4),
    (dict(base=float("nan")), 0, 4), (dict(scaling=4), 0, 4), (dict(scaling=1, factor=0.0), 0, 4), (dict(scaling=1, factor=1e-310), 0, 4),
    (dict(scaling=2, factor=2.0), 0, 4), (dict(scaling=2, factor=2.0, original_len=8.0, low=4.0, high=1.0), 0, 4),
    (dict(amplitude=0.0), 0, 4), (dict(amplitude=float("inf")), 0, 4), (dict(), -1, 4), (dict(), 0, -1),
    (dict(), 2 ** 31 - 1, 2)])
def test_rope_table_refuses(kw, pos0, n):
    spec = kvq.make_rope_spec(**dict(dict(rot_dim=64), **kw))
    assert kvq.lib().kvq_rope_table(spec, pos0, n, A[0], None) == INV


@fake_pointers
def test_rope_table_pointers():
    spec = kvq.make_rope_spec(64)
    assert kvq.lib().kvq_rope_table(spec, 0, 4, None, None) == INV
    assert kvq.lib().kvq_rope_table(spec, 0, 4, ctypes.c_void_p(0x100004), None) == INV
    assert kvq.lib().kvq_rope_table(None, 0, 4, A[0], None) == INV
    assert kvq.lib().kvq_rope_table(spec, 0, 0, None, None) == kvq.KVQ_OK


@fake_pointers
def test_norm_rope_refuses():
    def rows(**kw):
        d = dict(x=0x100000, y=0x200000, x_stride_t=256, x_stride_h=128, y_stride_t=256, y_stride_h=128, heads=2,
                 weight=None)
        return kvq.kvq_head_rows(**dict(d, **kw))

    def rope(**kw):
        return kvq.kvq_rope(**dict(dict(table=0x300000, n_pos=8, rot_dim=64, interleaved=0), **kw))

    def call(D=128, dt=kvq.BF16, n=4, q=rows(), k=None, eps=1e-6, off=0.0, r=None, pos=None, st=None):
        q, k = (None if x is None else ctypes.byref(x) for x in (q, k))
        return kvq.lib().kvq_norm_rope(D, dt, n, q, k, eps, off, r, pos, st, None)

    for kw in (dict(D=120), dict(D=0), dict(D=272), dict(dt=5), dict(n=-1), dict(q=None), dict(q=rows(heads=0)),
               dict(q=rows(x=0x100008)), dict(q=rows(x=None)), dict(q=rows(x_stride_h=100)),
               dict(q=rows(y_stride_h=64)), dict(q=rows(y=0x100000, x_stride_t=512)), dict(q=rows(y_stride_t=64)),
               dict(q=rows(weight=0x400004)), dict(q=rows(weight=0x400000), eps=-1.0),
               dict(q=rows(weight=0x400000), off=float("nan")), dict(k=rows(heads=-1)), dict(r=rope(rot_dim=24)),
               dict(r=rope(rot_dim=144)), dict(r=rope(n_pos=0)), dict(r=rope(interleaved=2)), dict(r=rope(table=None)),
               dict(r=rope(), pos=ctypes.c_void_p(0x500002)), dict(st=ctypes.c_void_p(0x500001))):
        assert call(**kw) == INV, kw
    assert call(n=1 << 30, q=rows(heads=4)) == UNS
    assert call(n=0) == kvq.KVQ_OK


@fake_pointers
def test_append_refuses():
    f = fmt()

    def call(f=f, pc=None, cu=A[0], n=8, m=8, tq=A[1], tr=A[2], k=A[3], ks=(256, 128), v=A[4], vs=(256, 128), r=None,
             pos=None, tqo=A[5], tro=A[6], st=None):
        return kvq.lib().kvq_append_paged(f, cache(f) if pc is None else pc, cu, n, m, tq, tr, k, *ks, v, *vs, r, pos,
                                          tqo, tro, st, None)

    odd = ctypes.c_void_p(0x100002)
    for kw in (dict(cu=None), dict(cu=odd), dict(n=-1), dict(m=9), dict(m=-1), dict(tq=None), dict(tr=odd),
               dict(k=None), dict(k=ctypes.c_void_p(0x100008)), dict(ks=(256, 100)), dict(ks=(-256, 128)),
               dict(vs=(3, 128)), dict(tqo=None), dict(tqo=A[6]), dict(tqo=A[1]), dict(tro=A[2]), dict(tro=A[1]),
               dict(pos=odd), dict(st=odd), dict(r=kvq.kvq_rope(0x300000, 8, 144, 0))):
        assert call(**kw) == INV, kw
    pc = cache(f)
    pc.res_k = None
    assert call(pc=pc) == INV
    pc = cache(f)
    pc.sink_v = 0xA000008
    assert call(pc=pc) == INV
    for kw in (dict(residual_cap=64), dict(residual_cap=200), dict(residual_cap=0), dict(k_bits=8), dict(v_bits=4),
               dict(head_dim=64), dict(rope=1)):
        assert call(f=fmt(**kw)) == UNS, kw


@fake_pointers
def test_read_refuses():
    f = fmt()

    def call(f=f, cu=A[0], n=8, m=8, first=A[1], tq=A[2], tr=A[3], k=A[4], v=A[5], dt=kvq.BF16):
        return kvq.lib().kvq_read_paged(f, cache(f), cu, n, m, first, tq, tr, k, v, dt, None, None)

    for kw in (dict(cu=None), dict(n=-1), dict(m=9), dict(first=None), dict(tq=None), dict(tr=None),
               dict(k=None, v=None), dict(k=ctypes.c_void_p(0x100008)), dict(dt=3)):
        assert call(**kw) == INV, kw
    assert call(f=fmt(k_bits=2)) == UNS
    assert call(n=0, m=0) == kvq.KVQ_OK


@fake_pointers
def test_attention_refuses():
    f = fmt()

    def call(f=f, cu=A[0], n=8, m=8, tq=A[1], tr=A[2], mq=256, mr=128, q=A[3], qdt=kvq.BF16, Hq=8, scale=0.1, causal=1,
             out=A[4], odt=kvq.BF16, lse=None, ws=A[5], wsb=1 << 30, st=None):
        return kvq.lib().kvq_attention_paged(f, cache(f), cu, n, m, tq, tr, mq, mr, q, qdt, Hq, scale, causal, out,
                                             odt, lse, ws, wsb, st, None)

    for kw in (dict(cu=None), dict(n=-1), dict(m=9), dict(tq=None), dict(mq=-1), dict(mq=257), dict(mr=129),
               dict(mr=-1), dict(q=None), dict(q=ctypes.c_void_p(0x100008)), dict(qdt=3), dict(Hq=7), dict(Hq=0),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(out=None),
               dict(odt=-1), dict(lse=ctypes.c_void_p(0x100002)), dict(ws=None), dict(ws=ctypes.c_void_p(0x100008)),
               dict(st=ctypes.c_void_p(0x100002))):
        assert call(**kw) == INV, kw
    assert call(Hq=34) == UNS and call(f=fmt(v_bits=4)) == UNS
    assert call(wsb=4) == WS
    assert call(n=0, m=0) == kvq.KVQ_OK


def test_workspace_sizes():
    f = fmt()
    assert kvq.attention_paged_workspace_bytes(f, 3, 8, 2, 8, 8, 256, 128) > 0
    for args in ((0, 8, 2, 8, 8, 256, 128), (3, 7, 2, 8, 8, 256, 128), (3, 8, 2, 8, 9, 256, 128),
                 (3, 34, 2, 8, 8, 256, 128), (3, 8, 2, 8, 8, 256, 129), (3, 8, 2, -1, 0, 256, 128)):
        assert kvq.attention_paged_workspace_bytes(f, *args) == 0
    assert kvq.attention_paged_workspace_bytes(fmt(k_bits=8), 3, 8, 2, 8, 8, 256, 128) == 0


def test_wrappers_refuse_what_the_c_side_cannot_see():
    f = fmt()
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kvq.norm_rope(x)                                            # not on a CUDA device
    with pytest.raises(ValueError):
        kvq.norm_rope(x.double())
    with pytest.raises(ValueError):
        kvq.norm_rope(x, x[:3])
    with pytest.raises(ValueError):
        kvq.norm_rope(x, k_weight=x[0, 0])
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(64, 4).t())
    with pytest.raises(ValueError):
        kvq.rope_table(kvq.make_rope_spec(64), 4, out=torch.zeros(4, 32))
    with pytest.raises(ValueError):
        kvq.rope_table(kvq.make_rope_spec(64), 4, device="cpu")
    c = kvq.PagedCache(f, 2, 4, 3, 2, device="cpu")
    i = [torch.zeros(n, dtype=torch.int32) for n in (4, 3, 3, 3, 3)]
    call = dict(cu_new=i[0], max_new=1, t_quant=i[1], t_res=i[2], k_src=x, v_src=x, t_quant_out=i[3], t_res_out=i[4])
    for bad in (dict(k_src=x.half()), dict(v_src=x[:, :1]), dict(cu_new=i[0][:3]), dict(t_res=i[2].long()),
                dict(positions=i[1]), dict(k_src=x.transpose(1, 2).contiguous().transpose(1, 2)), dict()):
        with pytest.raises(ValueError):
            kvq.append_paged(f, c, **dict(call, **bad))
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    for bad in (dict(q=q[..., :64]), dict(q=q.transpose(0, 1)), dict(out=q.float()), dict(lse=torch.zeros(4, 2)),
                dict(workspace=torch.zeros(8)), dict()):
        with pytest.raises(ValueError):
            kvq.attention_paged(f, c, i[0], 1, i[1], i[2], 0, 0, **dict(dict(q=q, scale=0.1), **bad))
    with pytest.raises(ValueError):
        kvq.read_paged(f, c, i[0], 1, i[1], i[2], i[3], 4, k_out=q)
    arrays = dict(c.pool.tensors, **c.raw, block_table=c.block_table)
    assert kvq.PagedCache(f, 2, 4, 3, 2, arrays=arrays).array("k_codes") is arrays["k_codes"]
    with pytest.raises(ValueError):
        kvq.PagedCache(f, 2, 4, 3, 2, arrays=dict(arrays, k_codes=arrays["k_codes"][:-1]))
    with pytest.raises(ValueError):
        kvq.PagedCache(f, 2, 4, 3, 2, arrays=dict(arrays, block_table=c.block_table.long()))
