"""E8M0 scale bytes at the ends of their range in the linear layers with
MXFP4 weights, bit for bit: byte 0 is 2^-127, a binary32 and BF16 subnormal,
and with it the weights themselves; byte 254 is 2^127.  MI355X only (marker
gpu)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")

# On a device of 256 compute units: the decode kernel, tiles of whole steps,
# tiles of steps begun, 256 x 256.
SHAPES = [(3, 70, 1056), (61, 700, 1024), (100, 4000, 768), (70, 300, 1120), (300, 4000, 672), (2100, 8400, 512)]


def _weights(focus, g, N, K, low):
    """Codes and scale bytes, alternating along k between the two ends' last
    bytes; at the upper end only codes whose value stays in BF16's range."""
    byte = np.tile(np.array([0, 1] if low else [253, 254], dtype=np.uint8), K // 32)[:K // 32]
    ws = np.broadcast_to(byte, (N, K // 32)).copy()
    c = g.integers(0, 8, (N, K), dtype=np.uint8)
    if not low:
        c = np.minimum(c, np.repeat(np.where(byte == 254, 3, 5).astype(np.uint8), 32)[None])  # 1.5 * 2^127, 3 * 2^126
    c |= g.integers(0, 2, (N, K), dtype=np.uint8) << 3
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    return focus.Quantized(torch.from_numpy(codes).to(DEV), torch.from_numpy(ws).to(DEV), None, None), \
        ref.weight_values(codes, ws, "mxfp4")


def _check(y, xv, wv, dtype):
    """Products are multiples of one power of two and their sums below 2^24 of
    it: exact in binary32, rounded once to BF16."""
    want = xv @ wv.T
    got = y.cpu()
    if dtype == torch.bfloat16:
        assert torch.equal(got, torch.from_numpy(want).to(torch.bfloat16))
    else:
        assert np.array_equal(got.double().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("low", [True, False], ids=["low", "high"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mx(M, N, K, low, dtype):
    import fp4_post_weight_amd as focus
    g = np.random.default_rng(K)
    w, wv = _weights(focus, g, N, K, low)
    xc = g.choice(np.array([0x30, 0x38, 0x3C, 0x40, 0xB0, 0xB8, 0xBC, 0xC0], dtype=np.uint8), (M, K))  # +-0.5 .. 2
    xs = np.broadcast_to(g.choice(np.array([253, 254] if low else [0, 1], dtype=np.uint8), (M, 1)), (M, K // 32)).copy()
    x = focus.Quantized(torch.from_numpy(xc).to(DEV), torch.from_numpy(xs).to(DEV), None, None)
    _check(focus.mxfp4_linear(x, w, out_dtype=dtype), ref.mxfp8_values(xc, xs), wv, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("low", [True, False], ids=["low", "high"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_w4a16(M, N, K, low, dtype):
    """At the upper end the activations of odd rows are BF16 subnormals."""
    import fp4_post_weight_amd as focus
    g = np.random.default_rng(K)
    w, wv = _weights(focus, g, N, K, low)
    size = np.where(np.arange(M)[:, None] % 2 == 0, *((2.0 ** 120, 2.0 ** 118) if low else (2.0 ** -120, 2.0 ** -132)))
    x = torch.from_numpy(g.integers(-6, 7, (M, K)) * 0.5 * size).to(torch.bfloat16)
    _check(focus.w4a16_linear(x.to(DEV), w, out_dtype=dtype), x.double().numpy(), wv, dtype)
