"""Strides of dimensions without extent: those of a single token, a single head or no rows at all say
nothing, whatever the tensor carries there."""
import numpy as np
import pytest
import torch

from oracle.formats import BF16, F16
from quantized_decode_attention_quantize_b200 import kvq
from tests.gpu_util import TORCH
from tests.test_gpu_serving import Paged, fmt, ints, rope_of

pytestmark = pytest.mark.gpu


def single(x, t_stride=None, h_stride=None):
    """x [T, H, D] with other strides for its dimensions of size one."""
    s = list(x.stride())
    s[0] = s[0] if t_stride is None else t_stride
    s[1] = s[1] if h_stride is None else h_stride
    return x.as_strided(x.shape, s)


@pytest.mark.parametrize("T,H,kw", [(1, 4, dict(t_stride=3)), (1, 4, dict(t_stride=0)), (5, 1, dict(h_stride=7)),
                                    (1, 1, dict(t_stride=1, h_stride=1))])
def test_norm_rope_ignores_strides_of_single_tokens_and_heads(T, H, kw):
    x = torch.randn(T, H, 64, device="cuda").bfloat16()
    rope = rope_of(64)
    want, _ = kvq.norm_rope(x, rope=rope)
    got, _ = kvq.norm_rope(single(x, **kw), rope=rope)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    kvq.norm_rope(x, single(x, **kw), rope=rope, k_out=single(out, **kw))
    assert torch.equal(out, want)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_no_rows_at_all(dt):
    empty = torch.tensor(np.zeros((0, 2, 128), np.float32), device="cuda").to(TORCH[dt])
    assert empty.stride() == (0, 0, 0)
    q, k = kvq.norm_rope(empty, empty, rope=rope_of())
    assert q.shape == k.shape == (0, 2, 128)
    p = Paged(fmt(src_dtype=dt), 2, 3, 3, seed=90)
    p.append([0, 0, 0])
    assert p.tq == [0, 0, 0] and p.tr == [-1, -1, -1]
    p.append([3, 0, 200])
    p.append([0, 0, 0], rope_of())
    p.check()
    k, v = kvq.read_paged(p.fmt, p.gpu, ints([0] * 4), 0, ints([0] * 3), ints(p.tq), ints(p.tr), 0)
    assert k.shape == v.shape == (0, 2, 128)
    q = torch.tensor(np.zeros((0, 8, 128), np.float32), device="cuda").bfloat16()
    out = kvq.attention_paged(p.fmt, p.gpu, ints([0] * 4), 0, ints(p.tq), ints(p.tr), 128, 100, q, 0.1)
    assert out.shape == (0, 8, 128)


def test_append_of_one_row_and_of_one_head_ignores_their_strides():
    for H, rows in ((2, 1), (1, 5), (1, 1)):
        caches = []
        for odd in (False, True):
            p = Paged(fmt(n_sink=0), H, 1, 2, seed=91)
            k, v = (torch.arange(rows * H * 128, device="cuda").view(rows, H, 128).bfloat16() * s for s in (1, -1))
            if odd:
                k = single(k, 5 if rows == 1 else None, 3 if H == 1 else None)
                v = single(v, 0 if rows == 1 else None, 0 if H == 1 else None)
            kvq.append_paged(p.fmt, p.gpu, ints([0, rows]), rows, ints([0]), ints([0]), k, v, ints([0]), ints([0]), status=p.status)
            assert int(p.status) == 0
            caches.append(p.gpu.raw)
        for n in caches[0]:
            assert torch.equal(caches[0][n], caches[1][n])
