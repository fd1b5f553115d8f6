"""Workspace sizes of the chunk attention (no GPU): what is enough for a bound on the new tokens is enough
for fewer, so that a server may size it once."""
import pytest

import synth
from quantized_decode_attention_quantize_b200 import kvq


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 16])
def test_a_workspace_for_many_tokens_serves_fewer(G):
    f = kvq.make_format(synth._fmt(src_dtype=synth.BF16, n_sink=1, residual_cap=128))
    # many sequences: no expanded pages on top
    sizes = [kvq.attention_paged_workspace_bytes(f, 60000, 2 * G, 2, 1000, n, 256, 128) for n in range(0, 300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[1] > 0
