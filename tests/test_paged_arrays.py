"""What a cache over the caller's arrays refuses (no GPU): arrays of another size, place, alignment or
type than the format asks for would be read by kernels through bare addresses."""
import pytest
import torch

import synth
from quantized_decode_attention_quantize_b200 import kvq

FMT = kvq.make_format(synth._fmt(src_dtype=synth.BF16, n_sink=1, residual_cap=128))
NAMES = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "sink_k", "sink_v", "res_k", "res_v")


def given(device="cpu"):
    c = kvq.PagedCache(FMT, 2, 4, 3, 2, device="cpu")
    a = dict(c.pool.tensors, **c.raw, block_table=c.block_table)
    return {n: t if device == "cpu" else torch.empty_like(t, device=device) for n, t in a.items() if n in NAMES + ("block_table",)}


def paged(arrays):
    return kvq.PagedCache(FMT, 2, 4, 3, 2, arrays=arrays)


def test_arrays_of_the_right_kind_are_taken():
    a = given()
    assert paged(a).array("k_codes") is a["k_codes"] and paged(a).struct.pool.k_codes == a["k_codes"].data_ptr()
    # the array's own type, or integers as plain bytes; names that the format has no use for are left out
    typed = dict(a, k_scale=a["k_scale"].view(torch.float16), sink_k=a["sink_k"].view(torch.bfloat16),
                 res_v=a["res_v"].view(torch.int16), v_codes=a["v_codes"].view(torch.int32), k_lut=torch.zeros(3))
    assert paged(typed).array("res_v") is typed["res_v"]


@pytest.mark.parametrize("name", NAMES)
def test_arrays_on_another_device_are_refused(name):
    # the meta device stands for another GPU: its tensors have a size and no address of this device
    a = given()
    with pytest.raises(ValueError, match=name):
        paged(dict(a, **{name: torch.empty_like(a[name], device="meta")}))
    a = given("meta")
    with pytest.raises(ValueError):
        paged(dict(a, **{name: torch.zeros(a[name].shape, dtype=a[name].dtype)}))


@pytest.mark.parametrize("name", NAMES)
def test_arrays_of_another_size_alignment_or_type_are_refused(name):
    a = given()
    n = a[name].numel()
    odd = torch.zeros(n + 64, dtype=torch.uint8)
    at = -odd.data_ptr() % 16 + 8
    wrong = torch.float16 if name in ("sink_k", "sink_v", "res_k", "res_v") else torch.bfloat16
    for t in (a[name][:-1], torch.zeros(n + 1, dtype=torch.uint8), torch.zeros(2 * n, dtype=torch.uint8)[::2],
              odd[at:at + n], a[name].view(wrong), a[name].view(torch.float64)):
        with pytest.raises(ValueError, match=name):
            paged(dict(a, **{name: t}))
    del a[name]
    with pytest.raises(ValueError, match=name):
        paged(a)


def test_a_cache_over_arrays_checks_them_too():
    a = {n: t for n, t in given().items() if n[0] in "kv"}
    assert kvq.Cache(FMT, 4, 2, 128, arrays=a).array("v_zero") is a["v_zero"]
    for bad in (dict(k_codes=a["k_codes"][:-1]), dict(k_codes=torch.empty_like(a["k_codes"], device="meta")),
                dict(k_code=a["k_codes"])):
        with pytest.raises(ValueError):
            kvq.Cache(FMT, 4, 2, 128, arrays=dict(a, **bad))


def test_calls_over_a_cache_outside_the_gpu_are_refused():
    c = paged(given())
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(3, 2, 4, 128, dtype=torch.bfloat16)
    for call in (lambda: kvq.decode_attention_paged(FMT, c, i, i, 0, 0, q, 0.1),
                 lambda: kvq.quantize_kv_paged(FMT, c, k, k, i, 4)):
        with pytest.raises(ValueError):
            call()
