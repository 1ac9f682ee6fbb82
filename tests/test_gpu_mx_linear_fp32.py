"""FP32 results of the MXFP8 x MXFP4 linear layer carry a binary32 sum of
exact products.  MI355X only (marker gpu)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def _operand(focus, codes, scales):
    return focus.Quantized(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), None, None)


# On a device of 256 compute units: the decode kernel with 1, 2 and 4 column
# tiles and two token tiles, tiles of whole steps and of steps begun from 32 x 32
# up, and 256 x 256.
SHAPES = [(1, 40, 512), (3, 5000, 544), (16, 9000, 1056), (33, 129, 1056), (61, 4000, 512), (20, 9000, 512),
          (100, 4100, 768), (100, 14003, 512), (250, 14000, 512), (500, 14000, 256), (70, 300, 1120), (300, 4000, 672),
          (2100, 9100, 640), (1100, 9000, 416)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_products_beside_large_ones(M, N, K):
    """In every 8 values of k two products of magnitude up to 2688 cancel, and
    six of at most 2^-5 remain: multiples of 2^-10 whose sums stay below
    K * 2^-5, so that every partial sum fits 24 bits and the result is exact in
    any order."""
    import fp4_post_weight_amd as focus
    g = np.random.default_rng(M + N + K)
    x = np.empty((M, K), dtype=np.uint8)
    w = g.integers(0, 16, (N, K), dtype=np.uint8)
    x[:] = g.choice(np.array([0x00, 0x01, 0x02, 0x81, 0x82], dtype=np.uint8), (M, K))  # 0, +-2^-9, +-2^-8
    at = g.integers(0, 4, K // 8) * 2 + 8 * np.arange(K // 8)
    big = g.choice(np.array([0x7E, 0xFE, 0x40, 0x78], dtype=np.uint8), (M, K // 8))  # 448, -448, 2, 256
    x[:, at], x[:, at + 1] = big, big ^ 0x80
    w[:, at + 1] = w[:, at]
    codes = w[:, 0::2] | (w[:, 1::2] << 4)
    xs, ws = np.full((M, K // 32), 127, dtype=np.uint8), np.full((N, K // 32), 127, dtype=np.uint8)
    want = ref.E4M3[x] @ ref.E2M1[w].T
    y = focus.mxfp4_linear(_operand(focus, x, xs), _operand(focus, codes, ws), out_dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), want)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (20, 70, 96), (70, 300, 160), (100, 4100, 256), (500, 14000, 256)])
def test_error_is_of_the_sum_alone(M, N, K):
    """Codes over the whole of E4M3, scales over 2^12: K additions and at most
    17 more per 128 k (products of groups and the running sum), each off by
    less than 2^-23 of the sum of the magnitudes."""
    import fp4_post_weight_amd as focus
    g = np.random.default_rng(K)
    x = g.integers(0, 256, (M, K), dtype=np.uint8)
    x[(x & 0x7F) == 0x7F] = 0x05
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    xs = g.integers(121, 133, (M, K // 32), dtype=np.uint8)
    ws = g.integers(121, 133, (N, K // 32), dtype=np.uint8)
    xv, wv = ref.mxfp8_values(x, xs), ref.weight_values(codes, ws, "mxfp4")
    y = focus.mxfp4_linear(_operand(focus, x, xs), _operand(focus, codes, ws), out_dtype=torch.float32)
    off = np.abs(y.cpu().double().numpy() - xv @ wv.T)
    bound = (1.25 * K + 4) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv.T))
    assert (off <= bound).all(), float((off / np.maximum(bound, 1e-300)).max())
