"""A decoder layer's feed-forward part through the library's calls as a model
makes them: quantize the weights, norm with the residual's addition, gate and
up, the gated activation, down -- in NVFP4, in MXFP8 x MXFP4 and weight-only
-- against the same chain of the references, and as one captured graph.
MI355X only (marker gpu)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


@pytest.fixture(scope="module")
def focus():
    import fp4_post_weight_amd as f
    f._lib.lib()
    return f


def _model(hidden, inner, tokens, seed):
    g = torch.Generator().manual_seed(seed)
    def w(n, k):
        return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16)
    return {"gate": w(inner, hidden), "up": w(inner, hidden), "down": w(hidden, inner),
            "norm": (1 + 0.2 * torch.randn(hidden, generator=g)).to(torch.bfloat16),
            "x": torch.randn(tokens, hidden, generator=g).to(torch.bfloat16),
            "res": (3 * torch.randn(tokens, hidden, generator=g)).to(torch.bfloat16)}


def _quantized(focus, m, kind):
    q = {}
    for n in ("gate", "up", "down"):
        w = m[n].to(DEV)
        q[n] = focus.quantize_mx(w, dequant=False) if kind in ("mx", "w4a16 mxfp4") else focus.quantize(w, dequant=False)
    return q


def _forward(focus, kind, q, x, res, wn):
    if kind == "mx":
        n, h = focus.rmsnorm_mxfp8(x, wn, EPS, residual=res)
        a = focus.silu_mul_mxfp8(focus.mxfp4_linear(n, q["gate"]), focus.mxfp4_linear(n, q["up"]))
        return n, a, focus.mxfp4_linear(a, q["down"], out_dtype=torch.float32), h
    if kind == "nvfp4":
        n, h = focus.rmsnorm_nvfp4(x, wn, EPS, residual=res)
        g, u = focus.nvfp4_linear_grouped(n, [q["gate"], q["up"]])
        a = focus.silu_mul_nvfp4(g, u)
        return n, a, focus.nvfp4_linear(a, q["down"], out_dtype=torch.float32), h
    n, h = focus.rmsnorm(x, wn, EPS, residual=res)
    a = focus.silu_mul(focus.w4a16_linear(n, q["gate"]), focus.w4a16_linear(n, q["up"]))
    return n, a, focus.w4a16_linear(a, q["down"], out_dtype=torch.float32), h


def _values(kind, v):
    """binary64 values of an activation as the linear layer reads it."""
    if kind == "mx":
        return ref.mxfp8_values(v.codes.cpu().numpy(), v.scales.cpu().numpy())
    if kind == "nvfp4":
        return ref.weight_values(v.codes.cpu().numpy(), v.scales.cpu().numpy(), "nvfp4") * \
            v.s2.cpu().double().numpy()[:, None]
    return v.cpu().double().numpy()


KINDS = ["nvfp4", "mx", "w4a16 nvfp4", "w4a16 mxfp4"]


@pytest.mark.parametrize("tokens", [1, 13, 150])
@pytest.mark.parametrize("kind", KINDS)
def test_feed_forward(focus, kind, tokens):
    m = _model(256, 704, tokens, seed=tokens)
    q = _quantized(focus, m, kind)
    x, res, wn = m["x"].to(DEV), m["res"].to(DEV), m["norm"].to(DEV)
    n, a, y, h = _forward(focus, kind, q, x, res, wn)
    # each step against its reference on the step's own input
    hh = ref.norm_h(m["x"], m["res"])
    yn = ref.norm_y(hh, m["norm"], EPS)
    assert np.array_equal(h.cpu().float().numpy(), hh)
    if kind == "mx":
        assert np.array_equal(n.codes.cpu().numpy(), ref.mxfp8(yn)[0])
    elif kind == "nvfp4":
        assert np.array_equal(n.codes.cpu().numpy(), ref.nvfp4(yn)[0])
    else:
        assert np.array_equal(n.cpu().float().numpy(), ref.bf16_round(yn))
    fmt = "mxfp4" if kind in ("mx", "w4a16 mxfp4") else "nvfp4"
    w = {k: ref.weight_values(v.codes.cpu().numpy(), v.scales.cpu().numpy(), fmt) *
         (v.s2.cpu().double().numpy() if v.s2 is not None else 1.0) for k, v in q.items()}
    want = _values(kind, a) @ w["down"].T
    mag = np.abs(_values(kind, a)) @ np.abs(w["down"].T)
    # binary32 sums, and for MXFP8 the truncation of products to 2^-13 of
    # the power of two of their group's largest (ref.mx_truncation)
    tol = (704 * 1.25 + 4) * 2.0 ** -23 * mag
    if kind == "mx":
        tol = tol + ref.mx_truncation(a.codes.cpu().numpy(), a.scales.cpu().numpy(), q["down"].codes.cpu().numpy(),
                                      q["down"].scales.cpu().numpy())
    assert (np.abs(y.cpu().double().numpy() - want) <= tol).all()
    # the whole chain near the unquantized layer: 4-bit weights (and
    # activations) carry a relative error of the order of a tenth each
    xn = yn.astype(np.float64)
    g, u = xn @ m["gate"].double().numpy().T, xn @ m["up"].double().numpy().T
    full = (g / (1 + np.exp(-g)) * u) @ m["down"].double().numpy().T
    rel = np.linalg.norm(y.cpu().double().numpy() - full) / np.linalg.norm(full)
    assert rel < 0.5


@pytest.mark.parametrize("kind", KINDS)
def test_feed_forward_graph(focus, kind):
    m = _model(512, 1024, 4, seed=3)
    q = _quantized(focus, m, kind)
    x, res, wn = m["x"].to(DEV), m["res"].to(DEV), m["norm"].to(DEV)
    eager = _forward(focus, kind, q, x, res, wn)[2].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _forward(focus, kind, q, x, res, wn)[2]
    for _ in range(3):
        y.fill_(float("nan"))
        _forward(focus, kind, q, x, res, wn)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
    # new inputs in the same buffers
    x.copy_(torch.randn(4, 512, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, _forward(focus, kind, q, x, res, wn)[2])
