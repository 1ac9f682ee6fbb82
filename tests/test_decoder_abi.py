"""The decoder-layer operators' C ABI rejects bad arguments on the host before
any HIP call, and their references agree with the quantizer's (CPU only: no
call here reaches a kernel launch)."""
import os

import numpy as np
import pytest
import torch

import decoder_ref as ref
import synth
from fp4_post_weight_amd import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_RANGE = 0, 1, 2, 3, 4, 5
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfocus_nvfp4.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def test_rmsnorm_validation(lib):
    f = lib.focus_rmsnorm
    inf, nan = float("inf"), float("nan")
    #        x     res   w     eps   T  H   res_out y   stream
    assert f(None, None, FAKE, 1e-5, 4, 64, None, FAKE, None) == ERR_NULL
    assert f(FAKE, None, None, 1e-5, 4, 64, None, FAKE, None) == ERR_NULL
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, None, None) == ERR_NULL
    assert f(FAKE, None, FAKE, 1e-5, 4, 60, None, FAKE, None) == ERR_SHAPE
    assert f(FAKE, None, FAKE, 1e-5, -1, 64, None, FAKE, None) == ERR_SHAPE
    assert f(FAKE, None, FAKE, 1e-5, (1 << 31) + 1, 64, None, FAKE, None) == ERR_RANGE
    assert f(FAKE, None, FAKE, 1e-5, 1, (1 << 31) + 8, None, FAKE, None) == ERR_RANGE
    for eps in (0.0, -1e-5, inf, nan):
        assert f(FAKE, None, FAKE, eps, 4, 64, None, FAKE, None) == ERR_RANGE
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, FAKE, FAKE, None) == ERR_RANGE  # residual_out without residual
    assert f(FAKE + 8, None, FAKE, 1e-5, 4, 64, None, FAKE, None) == ERR_ALIGN
    assert f(FAKE, FAKE + 2, FAKE, 1e-5, 4, 64, None, FAKE, None) == ERR_ALIGN
    assert f(FAKE, None, FAKE + 4, 1e-5, 4, 64, None, FAKE, None) == ERR_ALIGN
    assert f(FAKE, FAKE, FAKE, 1e-5, 4, 64, FAKE + 8, FAKE, None) == ERR_ALIGN
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE + 8, None) == ERR_ALIGN
    assert f(None, None, None, 1e-5, 0, 64, None, None, None) == OK
    assert f(None, None, None, 1e-5, 4, 0, None, None, None) == OK


def test_quantized_norm_validation(lib):
    f = lib.focus_rmsnorm_nvfp4
    #        x     res   w     eps   T  H   rout  codes scales s2  deq   stream
    assert f(FAKE, None, FAKE, 1e-5, 4, 72, None, FAKE, FAKE, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, None, FAKE, FAKE, None, None) == ERR_NULL
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE, None, FAKE, None, None) == ERR_NULL
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE, FAKE, None, None, None) == ERR_NULL
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE + 4, FAKE, FAKE, None, None) == ERR_ALIGN
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE, FAKE, FAKE + 2, None, None) == ERR_ALIGN
    assert f(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE, FAKE, FAKE, FAKE + 8, None) == ERR_ALIGN
    g = lib.focus_rmsnorm_mxfp8
    assert g(FAKE, None, FAKE, 1e-5, 4, 48, None, FAKE, FAKE, None, None) == ERR_SHAPE
    assert g(FAKE, None, FAKE, 1e-5, 4, 64, None, None, FAKE, None, None) == ERR_NULL
    assert g(FAKE, None, FAKE, 1e-5, 4, 64, None, FAKE, FAKE, FAKE + 2, None) == ERR_ALIGN
    assert g(FAKE, None, FAKE, float("nan"), 4, 64, None, FAKE, FAKE, None, None) == ERR_RANGE


def test_silu_validation(lib):
    f = lib.focus_silu_mul
    #        gate  gs   up   us  T  H   y     stream
    assert f(None, 64, FAKE, 64, 4, 64, FAKE, None) == ERR_NULL
    assert f(FAKE, 64, None, 64, 4, 64, FAKE, None) == ERR_NULL
    assert f(FAKE, 64, FAKE, 64, 4, 64, None, None) == ERR_NULL
    assert f(FAKE, 64, FAKE, 64, 4, 60, FAKE, None) == ERR_SHAPE
    assert f(FAKE, 56, FAKE, 64, 4, 64, FAKE, None) == ERR_SHAPE   # rows overlap
    assert f(FAKE, 64, FAKE, 68, 4, 64, FAKE, None) == ERR_SHAPE   # not a multiple of 8
    assert f(FAKE, 1 << 59, FAKE, 64, 4, 64, FAKE, None) == ERR_SHAPE
    assert f(FAKE + 8, 64, FAKE, 64, 4, 64, FAKE, None) == ERR_ALIGN
    assert f(FAKE, 64, FAKE + 8, 64, 4, 64, FAKE, None) == ERR_ALIGN
    assert f(FAKE, 64, FAKE, 64, (1 << 31) + 1, 64, FAKE, None) == ERR_RANGE
    assert f(None, 64, None, 64, 0, 64, None, None) == OK
    n = lib.focus_silu_mul_nvfp4
    assert n(FAKE, 64, FAKE, 64, 4, 56, FAKE, FAKE, FAKE, None, None) == ERR_SHAPE
    assert n(FAKE, 64, FAKE, 64, 4, 64, FAKE, FAKE, None, None, None) == ERR_NULL
    m = lib.focus_silu_mul_mxfp8
    assert m(FAKE, 64, FAKE, 64, 4, 48, FAKE, FAKE, None, None) == ERR_SHAPE
    assert m(FAKE, 64, FAKE, 64, 4, 64, FAKE + 4, FAKE, None, None) == ERR_ALIGN


def test_quantize_mxfp8_validation(lib):
    f = lib.focus_quantize_mxfp8
    assert f(None, 4, 64, FAKE, FAKE, None, None) == ERR_NULL
    assert f(FAKE, 4, 64, FAKE, None, None, None) == ERR_NULL
    assert f(FAKE, 4, 48, FAKE, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE + 4, 4, 64, FAKE, FAKE, None, None) == ERR_ALIGN
    assert f(FAKE, 4, 64, FAKE, FAKE, FAKE + 4, None) == ERR_ALIGN
    assert f(None, 0, 64, None, None, None, None) == OK


def test_mxfp4_linear_validation(lib):
    f = lib.focus_mxfp4_linear
    #        xc    xs    M  wc    ws    N  K   y    dt stream
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, 48, FAKE, 0, None) == ERR_SHAPE
    assert f(FAKE, FAKE, -1, FAKE, FAKE, 8, 64, FAKE, 0, None) == ERR_SHAPE
    assert f(FAKE, FAKE, (1 << 31) + 1, FAKE, FAKE, 8, 64, FAKE, 0, None) == ERR_RANGE
    assert f(FAKE, FAKE, 4, FAKE, FAKE, (1 << 26) + 1, 64, FAKE, 0, None) == ERR_RANGE
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, 64, FAKE, 2, None) == ERR_RANGE
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, (1 << 22) + 32, FAKE, 0, None) == ERR_RANGE
    for k in range(4):
        p = [FAKE] * 4
        p[k] = None
        assert f(p[0], p[1], 4, p[2], p[3], 8, 64, FAKE, 0, None) == ERR_NULL
        if k in (0, 2):  # codes
            p[k] = FAKE + 8
            assert f(p[0], p[1], 4, p[2], p[3], 8, 64, FAKE, 0, None) == ERR_ALIGN
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, 64, None, 0, None) == ERR_NULL
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, 64, FAKE + 2, 0, None) == ERR_ALIGN
    assert f(FAKE, FAKE, 4, FAKE, FAKE, 8, 64, FAKE + 1, 1, None) == ERR_ALIGN
    assert f(None, None, 0, None, None, 8, 64, None, 0, None) == OK
    assert f(None, None, 4, None, None, 0, 64, None, 0, None) == OK


def test_w4a16_linear_validation(lib):
    f = lib.focus_w4a16_linear
    #        x    M  fmt wc    ws    s2    N  K   y    dt stream
    assert f(FAKE, 4, 2, FAKE, FAKE, FAKE, 8, 64, FAKE, 0, None) == ERR_RANGE
    assert f(FAKE, 4, 0, FAKE, FAKE, FAKE, 8, 40, FAKE, 0, None) == ERR_SHAPE
    assert f(FAKE, 4, 1, FAKE, FAKE, None, 8, 48, FAKE, 0, None) == ERR_SHAPE
    assert f(FAKE, 4, 0, FAKE, FAKE, None, 8, 48, FAKE, 0, None) == ERR_NULL   # NVFP4 needs s2
    assert f(None, 4, 1, FAKE, FAKE, None, 8, 64, FAKE, 0, None) == ERR_NULL
    assert f(FAKE, 4, 1, FAKE, None, None, 8, 64, FAKE, 0, None) == ERR_NULL
    assert f(FAKE, 4, 0, FAKE, FAKE, FAKE + 2, 8, 64, FAKE, 0, None) == ERR_ALIGN
    assert f(FAKE + 8, 4, 0, FAKE, FAKE, FAKE, 8, 64, FAKE, 0, None) == ERR_ALIGN
    assert f(FAKE, 4, 0, FAKE + 8, FAKE, FAKE, 8, 64, FAKE, 0, None) == ERR_ALIGN
    assert f(FAKE, 4, 0, FAKE, FAKE, FAKE, 8, 64, FAKE, 3, None) == ERR_RANGE
    assert f(None, 0, 0, None, None, None, 8, 64, None, 1, None) == OK


def test_bindings_refuse_cpu_tensors():
    import fp4_post_weight_amd as focus
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    u8 = torch.zeros((4, 64), dtype=torch.uint8)
    q = focus.Quantized(u8, u8[:, :2], None, None)
    for call in (lambda: focus.rmsnorm(x, x[0]), lambda: focus.rmsnorm_nvfp4(x, x[0]),
                 lambda: focus.rmsnorm_mxfp8(x, x[0]), lambda: focus.silu_mul(x, x),
                 lambda: focus.silu_mul_nvfp4(x, x), lambda: focus.silu_mul_mxfp8(x, x),
                 lambda: focus.quantize_mxfp8(x), lambda: focus.mxfp4_linear(q, q),
                 lambda: focus.w4a16_linear(x, q)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        focus.rmsnorm(x.float(), x[0])


def test_reference_nvfp4_is_the_quantizers(orc):
    """On BF16 rows the reference gives what the oracle's per-token quantizer
    gives, zero rows and zero blocks included."""
    x = synth.make_activations((24, 512))
    x[3] = 0
    x[4] = -0.0
    x[5, 16:48] = 0
    x[6] *= 2.0 ** -90
    codes, scales, s2, deq = ref.nvfp4(x.float().numpy())
    c, s, t, d = orc.quantize_act_per_token(synth.bits(x), dequant=True)
    assert np.array_equal(codes, c) and np.array_equal(scales, s) and np.array_equal(s2, t)
    assert np.array_equal(torch.from_numpy(deq).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16), d)


def test_reference_e2m1_rounds_to_nearest_even():
    mids = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for m, code in mids.items():
        assert ref.e2m1_code(np.array([m, -m])).tolist() == [code, code | 8]
        up = np.nextafter(m, 9.0)
        down = np.nextafter(m, 0.0)
        lo, hi = ref.e2m1_code(np.array([down, up]))
        assert hi == lo + 1 and ref.E2M1[lo] < m < ref.E2M1[hi]
    assert ref.e2m1_code(np.array([7.0, 0.0, -0.0])).tolist() == [7, 0, 8]
