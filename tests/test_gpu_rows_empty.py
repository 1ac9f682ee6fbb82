"""Rows without elements: every row operator accepts [tokens, 0] operands and
writes nothing.  MI355X only (marker gpu)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("form", ["bf16", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("layout", ["dense", "apart"])
def test_silu_without_elements(tokens, form, layout):
    """A dense [5, 0] tensor's rows are 1 element apart, and a slice of none of
    a wider tensor's columns as far as the wider rows."""
    import fp4_post_weight_amd as focus
    e = torch.empty((tokens, 0 if layout == "dense" else 12), dtype=torch.bfloat16, device=DEV)[:, :0]
    assert e.stride(0) % 8 != 0
    call = {"bf16": focus.silu_mul, "nvfp4": focus.silu_mul_nvfp4, "mxfp8": focus.silu_mul_mxfp8}[form]
    got = call(e, e)
    if form == "bf16":
        assert got.shape == (tokens, 0)
        return
    assert got.codes.shape == (tokens, 0) and got.scales.shape == (tokens, 0) and got.deq is None
    # the caller's token scales are left as they were
    s2 = torch.full((tokens,), 7.0, device=DEV)
    call(e, e, out=focus.Quantized(got.codes, got.scales, None, s2))
    assert (s2 == 7.0).all()


@pytest.mark.parametrize("tokens", [1, 5])
def test_norm_and_mxfp8_without_elements(tokens):
    import fp4_post_weight_amd as focus
    x = torch.empty((tokens, 0), dtype=torch.bfloat16, device=DEV)
    w = torch.empty((0,), dtype=torch.bfloat16, device=DEV)
    y, h = focus.rmsnorm(x, w, residual=x)
    assert y.shape == (tokens, 0) and h.shape == (tokens, 0)
    for call in (focus.rmsnorm_nvfp4, focus.rmsnorm_mxfp8):
        assert call(x, w)[0].codes.shape == (tokens, 0)
    assert focus.quantize_mxfp8(x).codes.shape == (tokens, 0)
