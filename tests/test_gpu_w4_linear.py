"""The linear layers with 4-bit weights and MXFP8 or BF16 activations on the
GPU.  Against sums in binary64, within the bounds of the binary32 sum (and of
the block-scaled product's truncation), and bit for bit on operands whose
every partial sum is exact.  MI355X only (marker gpu)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
FORMATS = ["mx", "nvfp4", "mxfp4"]  # MXFP8 x MXFP4; BF16 x NVFP4; BF16 x MXFP4


@pytest.fixture(scope="module")
def focus():
    import fp4_post_weight_amd as f
    f._lib.lib()
    return f


class Case:
    """Operands of a layer, on the host (numpy) and on the GPU."""

    def __init__(self, focus, fmt, M, N, K, seed, exact=False):
        g = np.random.default_rng(seed)
        self.fmt, self.M, self.N, self.K = fmt, M, N, K
        wc = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
        spread = 1 if exact else 6
        if fmt == "nvfp4":
            if exact:
                ws = g.choice(np.array([0x30, 0x38, 0x40], dtype=np.uint8), (N, K // 16))
                s2 = np.float32(0.5)
            else:
                ws = g.integers(0x01, 0x7F, (N, K // 16), dtype=np.uint8)  # subnormals to the maximum
                s2 = np.float32(1.7e-4)
        else:
            ws = g.integers(127 - spread, 128 + spread, (N, K // 32), dtype=np.uint8)
            s2 = np.float32(1.0)
        self.wc, self.ws, self.s2 = wc, ws, s2
        self.wv = ref.weight_values(wc, ws, "nvfp4" if fmt == "nvfp4" else "mxfp4") * np.float64(s2)
        if fmt == "mx":
            if exact:  # +-{0.5, 1, 1.5, 2, 3}: no group spans 2^9
                self.xc = g.choice(np.array([0x30, 0x38, 0x3C, 0x40, 0x44, 0xB0, 0xB8, 0xBC, 0xC0, 0xC4], dtype=np.uint8), (M, K))
            else:
                self.xc = g.integers(0, 256, (M, K), dtype=np.uint8)
                self.xc[(self.xc & 0x7F) == 0x7F] = 0x05  # no NaN; a subnormal instead
            self.xs = g.integers(127 - spread, 128 + spread, (M, K // 32), dtype=np.uint8)
            self.xv = ref.mxfp8_values(self.xc, self.xs)
            self.x = focus.Quantized(torch.from_numpy(self.xc).to(DEV), torch.from_numpy(self.xs).to(DEV), None, None)
        else:
            if exact:
                x = torch.from_numpy(g.integers(-6, 7, (M, K)) * 0.5).to(torch.bfloat16)
            else:
                x = torch.from_numpy(g.standard_normal((M, K)) * np.exp(g.standard_normal((M, 1)))).to(torch.bfloat16)
            self.xv = x.double().numpy()
            self.x = x.to(DEV)
        self.w = focus.Quantized(torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV), None,
                                 torch.tensor([s2], device=DEV) if fmt == "nvfp4" else None)
        self.want = self.xv @ self.wv.T
        self.call = focus.mxfp4_linear if fmt == "mx" else focus.w4a16_linear

    def bound(self):
        """K additions and at most 17 more per 128 k (products of groups and
        the running sum) of relative 2^-23 (an addition that truncates), the
        multiplication by s2; plus the block-scaled product's truncation."""
        mag = np.abs(self.xv) @ np.abs(self.wv.T)
        b = (self.K * 1.25 + 4) * 2.0 ** -23 * mag
        return b + ref.mx_truncation(self.xc, self.xs, self.wc, self.ws) if self.fmt == "mx" else b

    def check(self, y, dtype):
        got = y.cpu().double().numpy()
        b = self.bound()
        if dtype == torch.bfloat16:
            b = b + (np.abs(self.want) + b) * 2.0 ** -8
        off = np.abs(got - self.want)
        assert (off <= b).all(), (self.fmt, self.M, self.N, self.K, float((off / np.maximum(b, 1e-300)).max()))


# (M, N, K): one value up; column, token and k edges of the tiles; K in parts of a
# step; scale rows at odd bytes (K/32 odd)
SHAPES = [(1, 1, 32), (1, 16, 512), (1, 17, 544), (2, 33, 96), (3, 130, 2080), (15, 64, 1056), (16, 48, 4096),
          (17, 65, 480), (31, 40, 1536), (33, 96, 672), (64, 128, 2048), (65, 257, 1120), (100, 100, 512),
          (129, 80, 576), (1, 500, 8224), (70, 2100, 160)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(focus, fmt, M, N, K, dtype):
    c = Case(focus, fmt, M, N, K, seed=M * 1009 + N * 31 + K)
    c.check(c.call(c.x, c.w, out_dtype=dtype), dtype)


@pytest.mark.parametrize("M,N,K", [(1, 40, 16), (5, 33, 48), (20, 70, 528), (3, 50, 1040), (40, 64, 2064), (150, 200, 1072)])
def test_nvfp4_odd_blocks(focus, M, N, K):
    """K % 32 == 16: rows of codes at multiples of 8 bytes."""
    c = Case(focus, "nvfp4", M, N, K, seed=K)
    c.check(c.call(c.x, c.w, out_dtype=torch.float32), torch.float32)


@pytest.mark.parametrize("fmt", FORMATS)
# On a device of 256 compute units each line but the last takes another kernel
# of some format: one and two token tiles per wavefront with 1, 2 and 4 column
# tiles, eight wavefronts, then tiles from 32 x 32 to 256 x 256 tokens x columns.
# K: whole steps, a step begun, several steps (every LDS stage in use).
@pytest.mark.parametrize("M,N,K", [(1, 96, 4096), (16, 200, 1024), (3, 5000, 544), (16, 9000, 1056), (2, 300, 8224),
                                   (1, 5000, 8704), (33, 129, 2592), (64, 4090, 640), (64, 64, 8192),
                                   (70, 300, 2592), (20, 9000, 1120), (100, 4000, 1312), (130, 4000, 2592),
                                   (200, 5000, 1312), (300, 4000, 672), (300, 9000, 672), (520, 9000, 416),
                                   (1100, 9000, 416), (260, 260, 736)])
def test_linear_exact(focus, fmt, M, N, K):
    """Operands in a narrow range: every product and partial sum is a multiple
    of one power of two and below 2^24 of it, so any order gives the exact
    sum."""
    c = Case(focus, fmt, M, N, K, seed=K + M, exact=True)
    y = c.call(c.x, c.w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), c.want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(1, 72), (3, 72), (20, 72), (70, 72), (140, 72), (130, 4000), (1100, 9000)])
def test_bad_rows_stay_their_own(focus, fmt, M, N):
    """NaN activations reach their own output rows only, and the rows after the
    last are not written."""
    K = 1088
    c = Case(focus, fmt, M, N, K, seed=4, exact=True)
    buf = torch.full((M + 2, N), 7.0, device=DEV)
    clean = c.call(c.x, c.w, out_dtype=torch.float32).clone()
    bad = M // 2
    if fmt == "mx":
        codes = c.x.codes.clone()
        codes[bad, 40] = 0x7F
        x = focus.Quantized(codes, c.x.scales, None, None)
    else:
        x = c.x.clone()
        x[bad, 40] = float("nan")
    y = c.call(x, c.w, out_dtype=torch.float32, out=buf[:M])
    if fmt == "mx":  # a NaN scale does the same
        scales = c.x.scales.clone()
        scales[bad, 1] = 255
        z = c.call(focus.Quantized(c.x.codes, scales, None, None), c.w, out_dtype=torch.float32)
        assert torch.isnan(z[bad]).all() and torch.isfinite(z).sum() == (M - 1) * N
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i != bad]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[bad]).all()
    assert (buf[M:] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_scale_extremes(focus, fmt):
    """Scale bytes near both ends of what a binary32 result can hold (NVFP4: of
    the format)."""
    M, N, K = 5, 48, 1024
    c = Case(focus, fmt, M, N, K, seed=11)
    if fmt == "nvfp4":
        lo, hi = 0x01, 0x7E
        ws = np.where(np.arange(N)[:, None] % 2 == 0, lo, hi).repeat(K // 16, 1).astype(np.uint8)
    else:
        ws = np.where(np.arange(N)[:, None] % 2 == 0, 30, 220).repeat(K // 32, 1).astype(np.uint8)
    c.ws = ws
    c.w = focus.Quantized(c.w.codes, torch.from_numpy(ws).to(DEV), None, c.w.s2)
    c.wv = ref.weight_values(c.wc, ws, "nvfp4" if fmt == "nvfp4" else "mxfp4") * np.float64(c.s2)
    c.want = c.xv @ c.wv.T
    c.check(c.call(c.x, c.w, out_dtype=torch.float32), torch.float32)


@pytest.mark.parametrize("fmt", FORMATS)
def test_row_slices_as_operands(focus, fmt):
    """Weights and tokens taken as row ranges of larger stored tensors, so that
    scale rows start at odd addresses."""
    M, N, K = 6, 50, 2080  # K/32 = 65, K/16 = 130
    c = Case(focus, fmt, M + 3, N + 5, K, seed=21)
    w = focus.Quantized(c.w.codes[5:], c.w.scales[5:], None, c.w.s2)
    x = focus.Quantized(c.x.codes[3:], c.x.scales[3:], None, None) if fmt == "mx" else c.x[3:]
    y = c.call(x, w, out_dtype=torch.float32)
    off = np.abs(y.cpu().double().numpy() - c.want[3:, 5:])
    assert (off <= c.bound()[3:, 5:]).all()


def test_empty_and_refusals(focus):
    c = Case(focus, "mx", 4, 8, 64, seed=1)
    d = Case(focus, "nvfp4", 4, 8, 64, seed=1)
    y = focus.mxfp4_linear(focus.Quantized(c.x.codes[:0], c.x.scales[:0], None, None), c.w)
    assert y.shape == (0, 8)
    assert focus.w4a16_linear(d.x, focus.Quantized(d.w.codes[:0], d.w.scales[:0], None, d.w.s2)).shape == (4, 0)
    z = focus.w4a16_linear(d.x[:, :0].contiguous(), focus.Quantized(d.w.codes[:, :0].contiguous(),
                                                                    d.w.scales[:, :0].contiguous(), None, d.w.s2))
    assert z.shape == (4, 8) and (z == 0).all()
    out = torch.full((4, 8), 7.0, device=DEV)
    bad = [
        lambda: focus.mxfp4_linear(c.x, c.w, out_dtype=torch.float16),
        lambda: focus.mxfp4_linear(c.x, c.w, out_dtype=torch.float32, out=out[:2]),
        lambda: focus.mxfp4_linear(c.x, c.w, out_dtype=torch.bfloat16, out=out),
        lambda: focus.mxfp4_linear(c.x, focus.Quantized(c.w.codes[:, :16], c.w.scales, None, None), out_dtype=torch.float32, out=out),
        lambda: focus.mxfp4_linear(c.x, focus.Quantized(c.w.codes, d.w.scales, None, None), out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x.float(), d.w, out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x, focus.Quantized(d.w.codes, d.w.scales, None, None), out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x, focus.Quantized(d.w.codes, d.w.scales, None, torch.ones(2, device=DEV)), out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x[:, :32], d.w, out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x[0], d.w, out_dtype=torch.float32, out=out),
        lambda: focus.w4a16_linear(d.x.cpu(), d.w, out_dtype=torch.float32, out=out),
    ]
    for i, call in enumerate(bad):
        print("refusal", i, flush=True)
        with pytest.raises((ValueError, TypeError, focus.FocusError)):
            call()
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_another_stream_and_graph(focus, fmt):
    cases = [Case(focus, fmt, M, N, K, seed=M) for M, N, K in ((1, 200, 2080), (40, 300, 1024), (200, 520, 1504), (600, 4200, 288))]

    def run():
        return [c.call(c.x, c.w, out_dtype=torch.float32) for c in cases]

    eager = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mine = run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(eager, mine):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = run()
    for _ in range(3):
        for t in caught:
            t.fill_(float("nan"))
        run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, caught):
            assert torch.equal(a, b)


# More 256 x 256 tiles than compute units: workgroups take several in turn.
# Column edges inside a store, a last chunk of scale bytes that overlaps the one
# before, one chunk only, and lengths that are whole steps for BF16
# activations alone (832) or for none (736).
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2100, 9100, 640), (2100, 9103, 832), (4400, 5000, 512), (4360, 4376, 1664), (3000, 6000, 736)])
def test_many_tiles(focus, fmt, M, N, K):
    c = Case(focus, fmt, M, N, K, seed=K, exact=True)
    buf = torch.full((M + 1, N), 7.0, device=DEV)
    y = c.call(c.x, c.w, out_dtype=torch.float32, out=buf[:M])
    assert np.array_equal(y.cpu().double().numpy(), c.want)
    assert (buf[M] == 7.0).all()
    h = c.call(c.x, c.w, out_dtype=torch.bfloat16)
    assert torch.equal(h.cpu(), torch.from_numpy(c.want).to(torch.bfloat16))
    # a result that starts 4 bytes off a multiple of 16
    off = torch.full((M * N + 8,), 7.0, device=DEV)
    z = c.call(c.x, c.w, out_dtype=torch.float32, out=off[1:1 + M * N].view(M, N))
    assert torch.equal(z, y)
    assert off[0] == 7.0 and (off[1 + M * N:] == 7.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = c.call(c.x, c.w, out_dtype=torch.bfloat16)
    for _ in range(3):
        caught.fill_(float("nan"))
        c.call(c.x, c.w, out_dtype=torch.float32)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(caught, h)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tiles_spread(focus, fmt):
    """Scales and values over their range, and a bad row."""
    M, N, K = 2100, 8500, 640
    c = Case(focus, fmt, M, N, K, seed=77)
    rows = np.r_[0:M:67, M - 20:M]  # the bounds of these
    c.xv, c.want = c.xv[rows], c.want[rows]
    if fmt == "mx":
        c.xc, c.xs = c.xc[rows], c.xs[rows]
    for dtype in (torch.float32, torch.bfloat16):
        c.check(c.call(c.x, c.w, out_dtype=dtype)[torch.from_numpy(rows).to(DEV)], dtype)
    y = c.call(c.x, c.w, out_dtype=torch.float32)
    bad = 1801
    if fmt == "mx":
        scales = c.x.scales.clone()
        scales[bad, K // 32 - 1] = 255
        x = focus.Quantized(c.x.codes, scales, None, None)
    else:
        x = c.x.clone()
        x[bad, K - 1] = float("nan")
    z = c.call(x, c.w, out_dtype=torch.float32)
    assert torch.isnan(z[bad]).all()
    z[bad] = y[bad]
    assert torch.equal(z, y)


# Lengths of whole steps.  On a device of 256 compute units each line takes
# another tile of some format, in one step, in fewer steps than LDS stages and in
# more; token and column edges inside the tiles.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(9, 40, 512), (33, 129, 2560), (61, 4000, 1536), (20, 9000, 1536), (61, 6000, 1024),
                                   (100, 4100, 768), (70, 300, 256), (61, 14000, 768), (20, 14000, 1280),
                                   (8, 9000, 4608), (100, 14003, 512), (250, 14000, 1024), (500, 14000, 768),
                                   (130, 4001, 4352), (30, 4000, 1280), (10, 18100, 2048), (17, 2050, 1024)])
def test_whole_steps(focus, fmt, M, N, K):
    c = Case(focus, fmt, M, N, K, seed=M + K, exact=True)
    buf = torch.full((M + 1, N), 7.0, device=DEV)
    y = c.call(c.x, c.w, out_dtype=torch.float32, out=buf[:M])
    assert np.array_equal(y.cpu().double().numpy(), c.want)
    assert (buf[M] == 7.0).all()
    h = c.call(c.x, c.w, out_dtype=torch.bfloat16)
    assert torch.equal(h.cpu(), torch.from_numpy(c.want).to(torch.bfloat16))
    bad = M - 2
    if fmt == "mx":
        codes = c.x.codes.clone()
        codes[bad, K - 1] = 0x7F
        x = focus.Quantized(codes, c.x.scales, None, None)
    else:
        x = c.x.clone()
        x[bad, K - 1] = float("nan")
    z = c.call(x, c.w, out_dtype=torch.float32)
    assert torch.isnan(z[bad]).all()
    z[bad] = y[bad]
    assert torch.equal(z, y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(12, 300, 1024), (61, 700, 1024), (200, 4000, 512), (2100, 8400, 512)])
def test_scales_at_odd_addresses(focus, fmt, M, N, K):
    c = Case(focus, fmt, M, N, K, seed=M, exact=True)

    def odd(t):
        buf = torch.empty(t.numel() + 1, dtype=torch.uint8, device=DEV)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    w = focus.Quantized(c.w.codes, odd(c.w.scales), None, c.w.s2)
    x = focus.Quantized(c.x.codes, odd(c.x.scales), None, None) if fmt == "mx" else c.x
    y = c.call(x, w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), c.want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(61, 6144, 512), (100, 5000, 768), (250, 14000, 256)])
def test_whole_steps_spread(focus, fmt, M, N, K):
    """Scales and values over their range, on some of the columns."""
    c = Case(focus, fmt, M, N, K, seed=5)
    cols = np.r_[0:N:29, N - 16:N]
    c.wv, c.wc, c.ws, c.want = c.wv[cols], c.wc[cols], c.ws[cols], c.want[:, cols]
    for dtype in (torch.float32, torch.bfloat16):
        c.check(c.call(c.x, c.w, out_dtype=dtype)[:, torch.from_numpy(cols).to(DEV)], dtype)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_at_once(focus, fmt):
    """No call keeps anything another could use: the same calls on two streams,
    in turn and unsynchronized."""
    cases = [Case(focus, fmt, M, N, K, seed=M) for M, N, K in ((1, 2000, 2048), (61, 6144, 1024), (300, 5000, 768), (2100, 8500, 512))]
    want = [c.call(c.x, c.w, out_dtype=torch.float32) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for s, out in zip(streams, got):
            with torch.cuda.stream(s):
                out += [c.call(c.x, c.w, out_dtype=torch.float32) for c in cases]
    torch.cuda.synchronize()
    for out in got:
        for i, y in enumerate(out):
            assert torch.equal(y, want[i % len(cases)])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(3, 50), (12, 9000), (100, 4000), (2100, 9100)])
def test_no_k(focus, fmt, M, N):
    e = torch.empty
    u8 = dict(dtype=torch.uint8, device=DEV)
    w = focus.Quantized(e((N, 0), **u8), e((N, 0), **u8), None, torch.ones(1, device=DEV) if fmt == "nvfp4" else None)
    if fmt == "mx":
        y = focus.mxfp4_linear(focus.Quantized(e((M, 0), **u8), e((M, 0), **u8), None, None), w)
    else:
        y = focus.w4a16_linear(e((M, 0), dtype=torch.bfloat16, device=DEV), w)
    assert y.shape == (M, N) and (y == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [2, 40, 520])
def test_offsets_past_32_bits(focus, fmt, M):
    """4.6 GB of codes and, at 520 tokens, 4.7 GB of results: the last columns
    equal those of the same layer cut to them (exact sums, any tile)."""
    N, K, cut = 2_250_000, 4096, 300
    g = torch.Generator(device=DEV).manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    block = 16 if fmt == "nvfp4" else 32
    scales = torch.randint(0x37 if block == 16 else 126, 0x39 if block == 16 else 128, (N, K // block), dtype=torch.uint8,
                           device=DEV, generator=g)
    if block == 16:
        scales = (scales & 0x38) | 0x30  # 0.5 and 1
    s2 = torch.ones(1, device=DEV) if fmt == "nvfp4" else None
    if fmt == "mx":
        pool = torch.tensor([0x30, 0x38, 0x40, 0xB0, 0xB8, 0xC0], dtype=torch.uint8, device=DEV)
        x = focus.Quantized(pool[torch.randint(0, 6, (M, K), device=DEV, generator=g)],
                            torch.full((M, K // 32), 127, dtype=torch.uint8, device=DEV), None, None)
        call = focus.mxfp4_linear
    else:
        x = torch.randint(-4, 5, (M, K), device=DEV, generator=g).to(torch.bfloat16)
        call = focus.w4a16_linear
    y = call(x, focus.Quantized(codes, scales, None, s2), out_dtype=torch.bfloat16)
    for part in (slice(0, cut), slice(N - cut, N)):
        w = focus.Quantized(codes[part].clone(), scales[part].clone(), None, s2)
        assert torch.equal(y[:, part], call(x, w, out_dtype=torch.bfloat16))
    assert torch.isfinite(y[M - 1]).all()
