"""NVFP4 weights whose rows end in half a pair of scale blocks (K % 32 == 16),
so that rows of codes start at multiples of 8 bytes only, at many tokens: exact
results, and a cost near that of a length without the last block.  MI355X only
(marker gpu)."""
import numpy as np
import pytest
import torch

from test_gpu_w4_linear import Case, focus  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


# On a device of 256 compute units: tiles of 32 x 64, 64 x 128 and 256 x 256
# tokens x columns (fewer tokens take the decode kernel); K below one step, one
# block past whole steps, and one block short of them.
@pytest.mark.parametrize("M,N,K", [(70, 72, 16), (65, 500, 48), (70, 4000, 272), (128, 9000, 1040), (130, 4001, 1008),
                                   (200, 5000, 528), (500, 9000, 144), (300, 12000, 496), (1000, 4096, 1040),
                                   (1100, 9000, 464), (2100, 9103, 80), (61, 14000, 1040), (20, 20000, 528)])
def test_exact(focus, M, N, K):  # noqa: F811
    c = Case(focus, "nvfp4", M, N, K, seed=K + M, exact=True)
    buf = torch.full((M + 1, N), 7.0, device=DEV)
    y = focus.w4a16_linear(c.x, c.w, out_dtype=torch.float32, out=buf[:M])
    assert np.array_equal(y.cpu().double().numpy(), c.want)
    assert (buf[M] == 7.0).all()
    h = focus.w4a16_linear(c.x, c.w, out_dtype=torch.bfloat16)
    assert torch.equal(h.cpu(), torch.from_numpy(c.want).to(torch.bfloat16))
    bad = M - 2
    x = c.x.clone()
    x[bad, K - 1] = float("nan")
    z = focus.w4a16_linear(x, c.w, out_dtype=torch.float32)
    assert torch.isnan(z[bad]).all()
    z[bad] = y[bad]
    assert torch.equal(z, y)


def test_weights_taken_from_larger_ones(focus):  # noqa: F811
    """Row ranges of stored tensors: codes 16 bytes past a multiple of 32 and
    scale rows 2 past a multiple of 4; and nothing behind the last row is read as a
    weight (its codes and scales are set to others without effect)."""
    M, N, K = 300, 700, 1040
    c = Case(focus, "nvfp4", M, N + 4, K, seed=3, exact=True)
    w = focus.Quantized(c.w.codes[2:N + 2], c.w.scales[2:N + 2], None, c.w.s2)
    y = focus.w4a16_linear(c.x, w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), c.want[:, 2:N + 2])
    c.w.codes[N + 2:] = 0x77
    c.w.scales[N + 2:] = 0x7E
    assert torch.equal(focus.w4a16_linear(c.x, w, out_dtype=torch.float32), y)


def test_spread(focus):  # noqa: F811
    """Scales over their range, some of the columns, both result types."""
    M, N, K = 260, 5000, 1072
    c = Case(focus, "nvfp4", M, N, K, seed=6)
    cols = np.r_[0:N:29, N - 16:N]
    c.wv, c.want = c.wv[cols], c.want[:, cols]
    for dtype in (torch.float32, torch.bfloat16):
        c.check(focus.w4a16_linear(c.x, c.w, out_dtype=dtype)[:, torch.from_numpy(cols).to(DEV)], dtype)


def test_graph(focus):  # noqa: F811
    cases = [Case(focus, "nvfp4", M, N, K, seed=M, exact=True) for M, N, K in ((70, 4000, 272), (500, 9000, 144), (1100, 9000, 464))]

    def run():
        return [focus.w4a16_linear(c.x, c.w, out_dtype=torch.float32) for c in cases]

    eager = run()
    torch.cuda.synchronize()
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


def test_cost_of_the_last_block(focus):  # noqa: F811
    """One block more than a length of whole steps: the same class of time
    (the least of several runs, 8 calls each; reading W again for every 32
    tokens took five times as long)."""
    M, N = 4096, 4096

    def least(K):
        g = torch.Generator(device=DEV).manual_seed(K)
        w = focus.Quantized(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g),
                            torch.full((N, K // 16), 0x38, dtype=torch.uint8, device=DEV), None, torch.ones(1, device=DEV))
        x = torch.randn((M, K), device=DEV, generator=g).to(torch.bfloat16)
        out = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        best = float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(8):
                focus.w4a16_linear(x, w, out=out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    whole, odd = least(4096), least(4112)
    print("us", whole * 1e3 / 8, odd * 1e3 / 8, flush=True)
    assert odd < 2.5 * whole
