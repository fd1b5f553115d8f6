"""What the read-back of one side refuses (no GPU)."""
import pytest
import torch

import synth
from quantized_decode_attention_quantize_b200 import kvq


def test_read_needs_a_side_and_no_output_for_the_other():
    f = kvq.make_format(synth._fmt(src_dtype=synth.BF16, n_sink=1, residual_cap=128))
    c = kvq.PagedCache(f, 2, 4, 3, 2, device="cpu")
    i = [torch.zeros(n, dtype=torch.int32) for n in (4, 3, 3, 3)]
    out = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for kw, what in ((dict(keys=False, values=False), "keys or values"), (dict(keys=False, k_out=out), "k_out / v_out"),
                     (dict(values=False, v_out=out), "k_out / v_out"), (dict(values=False, k_out=out), "CUDA")):
        with pytest.raises(ValueError, match=what):
            kvq.read_paged(f, c, i[0], 1, i[1], i[2], i[3], 4, **kw)
