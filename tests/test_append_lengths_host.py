"""What kvq_append_paged refuses of the arrays that receive the lengths (no GPU)."""
import ctypes

import pytest
import torch

from quantized_decode_attention_quantize_b200 import kvq
from tests.test_serving_host import A, INV, cache, fmt

# made-up device addresses: only where no launch could follow a check that has regressed
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses; CPU only")


@pytest.mark.parametrize("which", range(2))
@pytest.mark.parametrize("other", range(3))
@pytest.mark.parametrize("by", [-8, -4, 4, 8])
def test_lengths_that_share_a_place_are_refused(which, other, by):
    # three sequences: arrays of 12 bytes; the CTAs of one sequence still read what another's has written
    f = fmt()
    lens = [A[1], A[2], A[5 + (1 - which)]]
    outs = [A[5], A[6]]
    outs[which] = ctypes.c_void_p(lens[other].value + by)
    st = kvq.lib().kvq_append_paged(f, cache(f), A[0], 8, 8, A[1], A[2], A[3], 256, 128, A[4], 256, 128, None, None, *outs,
                                    None, None)
    assert st == INV
