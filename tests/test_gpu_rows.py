"""The norm, the gated activation and the MXFP8 quantizer on the GPU against
their references (tests/decoder_ref.py): codes, scale bytes, token scales and
stored residuals bit for bit, BF16 results to the half step of their rounding
from a binary64 evaluation of the formula.  MI355X only (marker gpu)."""
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


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy()


def _bf16_bits(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).view(torch.int16).numpy()


def _input(t, h, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, generator=g) * scale * torch.exp(torch.randn(t, 1, generator=g))
    x[:, torch.randint(0, h, (max(1, h // 200),), generator=g)] *= 20.0
    return x.to(torch.bfloat16)


def _weight(h, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.3 * torch.randn(h, generator=g)).to(torch.bfloat16)


def _check_nvfp4(q, y, deq):
    codes, scales, s2, d = ref.nvfp4(y)
    assert np.array_equal(q.s2.cpu().numpy(), s2)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    if deq:
        assert np.array_equal(_bits(q.deq), _bf16_bits(d))
    else:
        assert q.deq is None


def _check_mxfp8(q, y, deq):
    codes, scales, d = ref.mxfp8(y)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    if deq:
        assert np.array_equal(_bits(q.deq), _bf16_bits(d))
    else:
        assert q.deq is None
    assert q.s2 is None


def _check_bf16(got, y, exact):
    """`y`: the binary32 contract, met bit for bit; `exact`: binary64 formula,
    from which four binary32 roundings (2^-24 each) and one BF16 rounding
    (2^-8, or half the least subnormal 2^-133) may lead away."""
    assert np.array_equal(_bits(got), _bf16_bits(y))
    tol = np.abs(exact) * (2.0 ** -8 + 5 * 2.0 ** -24) + 2.0 ** -133
    assert (np.abs(got.cpu().double().numpy() - exact) <= tol).all()


# one vector; part of a wavefront's row; the edges of each row form; a length
# between them; rows beyond registers
NORM_H = [32, 480, 512, 544, 2048, 2080, 4096, 5120, 8192, 8224, 16384, 28672, 32768, 32800, 40992]


@pytest.mark.parametrize("residual", [False, True], ids=["x", "x+r"])
@pytest.mark.parametrize("h", NORM_H)
def test_norm(focus, h, residual):
    t = 5 if h > 8192 else 9
    x, w = _input(t, h, h), _weight(h, h + 1)
    r = _input(t, h, h + 2, 3.0) if residual else None
    x[1] = 0
    if residual:
        r[1] = 0
    if h > 64:
        x[2, 32:64] = 0
        if residual:
            r[2, 32:64] = 0
    hh = ref.norm_h(x, r)
    y = ref.norm_y(hh, w, EPS)
    h64 = hh.astype(np.float64)
    eps = np.float64(np.float32(EPS))
    exact = h64 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + eps) * w.double().numpy()
    xd, wd = x.to(DEV), w.to(DEV)
    rd = None if r is None else r.to(DEV)
    got, res = focus.rmsnorm(xd, wd, EPS, residual=rd)
    _check_bf16(got, y, exact)
    for out in (res,):
        assert (out is None) == (r is None)
        if out is not None:
            assert np.array_equal(_bits(out), _bf16_bits(hh))
    for deq in (False, True):
        q, res = focus.rmsnorm_nvfp4(xd, wd, EPS, residual=rd, dequant=deq)
        _check_nvfp4(q, y, deq)
        assert res is None or np.array_equal(_bits(res), _bf16_bits(hh))
        q, res = focus.rmsnorm_mxfp8(xd, wd, EPS, residual=rd, dequant=deq)
        _check_mxfp8(q, y, deq)
        assert res is None or np.array_equal(_bits(res), _bf16_bits(hh))
    assert np.array_equal(_bits(xd), _bits(x))  # inputs are left as they were
    assert r is None or np.array_equal(_bits(rd), _bits(r))


@pytest.mark.parametrize("h", [8, 24, 16, 48])
def test_norm_narrow(focus, h):
    """Rows shorter than a scale block of the wider formats."""
    x, w = _input(70, h, h), _weight(h, h + 1)
    y = ref.norm_y(ref.norm_h(x, None), w, EPS)
    got, _ = focus.rmsnorm(x.to(DEV), w.to(DEV), EPS)
    assert np.array_equal(_bits(got), _bf16_bits(y))
    if h % 16 == 0:
        q, _ = focus.rmsnorm_nvfp4(x.to(DEV), w.to(DEV), EPS, dequant=True)
        _check_nvfp4(q, y, True)


@pytest.mark.parametrize("h", [512, 4096, 40992])
@pytest.mark.parametrize("alias", ["residual", "x"])
def test_norm_in_place(focus, h, alias):
    x, r, w = _input(7, h, 1), _input(7, h, 2), _weight(h, 3)
    hh = ref.norm_h(x, r)
    y = ref.norm_y(hh, w, EPS)
    for call in (focus.rmsnorm, focus.rmsnorm_nvfp4, focus.rmsnorm_mxfp8):
        xd, rd = x.to(DEV), r.to(DEV)
        target = rd if alias == "residual" else xd
        got, res = call(xd, w.to(DEV), EPS, residual=rd, residual_out=target)
        assert res is target
        assert np.array_equal(_bits(target), _bf16_bits(hh))
        if call is focus.rmsnorm:
            assert np.array_equal(_bits(got), _bf16_bits(y))
        elif call is focus.rmsnorm_nvfp4:
            _check_nvfp4(got, y, False)
        else:
            _check_mxfp8(got, y, False)


@pytest.mark.parametrize("t", [1, 3, 1023, 8192])
def test_norm_batch_sizes_agree(focus, t):
    """A row's result does not depend on how many rows are in the call."""
    x, w = _input(t, 2048, 5), _weight(2048, 6)
    xd, wd = x.to(DEV), w.to(DEV)
    whole, _ = focus.rmsnorm_nvfp4(xd, wd, EPS, dequant=True)
    for i in sorted({0, t // 2, t - 1}):
        one, _ = focus.rmsnorm_nvfp4(xd[i:i + 1], wd, EPS, dequant=True)
        assert torch.equal(one.codes[0], whole.codes[i]) and torch.equal(one.s2[0], whole.s2[i])
    y = ref.norm_y(ref.norm_h(x, None), w, EPS)
    _check_nvfp4(whole, y, True)


def test_norm_extreme_rows(focus):
    """Large, tiny, infinite and NaN rows beside ordinary ones: each row's
    result is its own, and the ordinary rows are as without the others."""
    x, w = _input(12, 1024, 7), _weight(1024, 8)
    clean, _ = focus.rmsnorm_mxfp8(x.to(DEV), w.to(DEV), EPS, dequant=True)
    bad = x.clone()
    bad[2, 5] = float("inf")
    bad[4, 7] = float("nan")
    bad[6] = 3e38          # squares beyond binary32
    bad[8] *= 2.0 ** -120  # squares below binary32
    for call in (focus.rmsnorm, focus.rmsnorm_nvfp4, focus.rmsnorm_mxfp8):
        call(bad.to(DEV), w.to(DEV), EPS)
    got, _ = focus.rmsnorm_mxfp8(bad.to(DEV), w.to(DEV), EPS, dequant=True)
    keep = [0, 1, 3, 5, 7, 9, 10, 11]
    for a, b in zip(got[:3], clean[:3]):
        assert torch.equal(a[keep], b[keep])
    fin = [6, 8]
    y = ref.norm_y(ref.norm_h(bad[fin], None), w, EPS)
    codes, scales, _ = ref.mxfp8(y)
    assert np.array_equal(got.codes[fin].cpu().numpy(), codes)
    assert np.array_equal(got.scales[fin].cpu().numpy(), scales)
    # the bad rows show what they are: an infinity leaves NaN in its place (its
    # row's root is infinite), a NaN everywhere
    assert (got.scales[4] == 255).all() and torch.isnan(got.deq[4]).all()
    assert got.scales[2, 0] == 255 and torch.isnan(got.deq[2, :32]).all() and (got.deq[2, 32:] == 0).all()
    out, _ = focus.rmsnorm(bad.to(DEV), w.to(DEV), EPS)
    assert torch.isnan(out[4]).all() and torch.isnan(out[2, 5])
    q4, _ = focus.rmsnorm_nvfp4(bad.to(DEV), w.to(DEV), EPS)
    assert torch.isnan(q4.s2[[2, 4]]).all() and torch.isfinite(q4.s2[keep + fin]).all()


def test_silu_and_mxfp8_show_bad_values(focus):
    g, u = _input(5, 256, 7), _input(5, 256, 8)
    g[1, 40], u[2, 70], g[3, 3] = float("nan"), float("inf"), float("inf")
    q = focus.silu_mul_mxfp8(g.to(DEV), u.to(DEV), dequant=True)
    want = torch.zeros(5, 8, dtype=torch.bool)
    want[1, 1] = want[2, 2] = want[3, 0] = True
    assert torch.equal(q.scales.cpu() == 255, want)
    assert torch.equal(torch.isnan(q.deq.float().view(5, 8, 32)).all(-1).cpu(), want)
    s2 = focus.silu_mul_nvfp4(g.to(DEV), u.to(DEV)).s2
    assert torch.equal(torch.isfinite(s2).cpu(), torch.tensor([True, False, False, False, True]))
    x = focus.quantize_mxfp8(u.to(DEV))
    assert (x.scales == 255).sum() == 1 and x.scales[2, 2] == 255


# --------------------------------------------------------------------------
# gated activation
# --------------------------------------------------------------------------

def test_silu_every_gate_value(focus):
    """All finite BF16 gates, times 1 and times a value with a full
    significand: the binary32 contract bit for bit, and the formula in 64
    bits."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    v = v.reshape(-1, 32)  # 2 * 255 * 128 of them
    for uv in (1.0, 1.9921875):
        u = torch.full_like(v, uv)
        y = ref.silu_y(v, u)
        got = focus.silu_mul(v.to(DEV), u.to(DEV))
        g64 = v.double().numpy()
        # exp(-g) beyond binary32 gives sigmoid 0 in the contract, where the
        # formula gives less than 2^-127
        with np.errstate(over="ignore"):
            exact = g64 / (1.0 + np.exp(-g64)) * uv
        assert np.array_equal(_bits(got), _bf16_bits(y))
        tol = np.abs(exact) * (2.0 ** -8 + 6 * 2.0 ** -24) + 2.0 ** -120
        out = got.cpu().double().numpy()
        # a BF16 result overflows from (2 - 2^-8) * 2^127 on: the exact value
        # of a gate above 2^127 times 1.99 lies beyond it, and infinity is its
        # correct rounding there
        over = np.abs(exact) >= (2 - 2.0 ** -8) * 2.0 ** 127
        assert np.isinf(out[over]).all() and (uv == 1.0 or over.any())
        assert (np.abs(out - exact)[~over] <= tol[~over]).all()


SILU = [(1, 32), (1, 14336), (3, 160), (17, 4128), (5, 28672), (130, 512), (2, 32768 + 32)]


@pytest.mark.parametrize("layout", ["dense", "halves", "apart"])
@pytest.mark.parametrize("t,h", SILU)
def test_silu(focus, t, h, layout):
    g, u = _input(t, h, h, 1.0), _input(t, h, h + 1, 1.0)
    g[0, :32] = 0
    if layout == "dense":
        gd, ud = g.to(DEV), u.to(DEV)
    elif layout == "halves":
        both = torch.cat([g, u], 1).to(DEV)
        gd, ud = both[:, :h], both[:, h:]
    else:  # rows 8 and 24 elements further apart than they are long
        gb = torch.full((t, h + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
        ub = torch.full((t, h + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
        gd, ud = gb[:, :h], ub[:, 8:h + 8]
        gd.copy_(g)
        ud.copy_(u)
    y = ref.silu_y(g, u)
    assert np.array_equal(_bits(focus.silu_mul(gd, ud)), _bf16_bits(y))
    for deq in (False, True):
        _check_nvfp4(focus.silu_mul_nvfp4(gd, ud, dequant=deq), y, deq)
        _check_mxfp8(focus.silu_mul_mxfp8(gd, ud, dequant=deq), y, deq)


def test_silu_zero_and_saturated_rows(focus):
    g, u = _input(6, 256, 3), _input(6, 256, 4)
    g[1] = 0
    u[2] = 0
    g[3] = -200.0   # sigmoid 0: signed zeros
    g[4] = 200.0
    y = ref.silu_y(g, u)
    _check_nvfp4(focus.silu_mul_nvfp4(g.to(DEV), u.to(DEV), dequant=True), y, True)
    _check_mxfp8(focus.silu_mul_mxfp8(g.to(DEV), u.to(DEV), dequant=True), y, True)


# --------------------------------------------------------------------------
# MXFP8
# --------------------------------------------------------------------------

@pytest.mark.parametrize("t,h", [(1, 32), (7, 96), (300, 4096), (3, 40000)])
def test_quantize_mxfp8(focus, t, h):
    x = _input(t, h, h)
    x[0, :32] = 0
    _check_mxfp8(focus.quantize_mxfp8(x.to(DEV)), x.float().numpy(), False)
    _check_mxfp8(focus.quantize_mxfp8(x.to(DEV), dequant=True), x.float().numpy(), True)


def test_quantize_mxfp8_every_value(focus):
    """Every finite BF16 value in the place after its block's maximum, for
    maxima over the whole exponent range: rounding, saturation, subnormal
    codes and the scale's lower limit."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    n = v.numel()
    for e in (-133, -126, -119, -20, 0, 8, 127):
        top = torch.full((n, 1), 1.9921875, dtype=torch.float64) * 2.0 ** e
        x = torch.zeros(n, 32, dtype=torch.bfloat16)
        x[:, 0] = top[:, 0].to(torch.bfloat16)
        x[:, 1] = v
        # larger values become the maximum themselves, and are then as valid
        q = focus.quantize_mxfp8(x.to(DEV), dequant=True)
        _check_mxfp8(q, x.float().numpy(), True)


# --------------------------------------------------------------------------
# buffers, streams, graphs
# --------------------------------------------------------------------------

def _buffers(focus, t, h, fmt):
    pad = 64
    def u8(n):
        return torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)
    raw = {"codes": u8(t * h if fmt == "mxfp8" else t * h // 2), "scales": u8(t * h // (32 if fmt == "mxfp8" else 16)),
           "deq": u8(2 * t * h), "s2": u8(4 * t)}
    def body(k):
        return raw[k][pad:-pad]
    q = focus.Quantized(body("codes").view(t, -1), body("scales").view(t, -1),
                        body("deq").view(torch.bfloat16).view(t, h),
                        body("s2").view(torch.float32) if fmt == "nvfp4" else None)
    return raw, q, pad


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("t,h", [(3, 96), (5, 4128)])
def test_outputs_stay_inside_their_buffers(focus, fmt, t, h):
    x, w, u = _input(t, h, 1).to(DEV), _weight(h, 2).to(DEV), _input(t, h, 3).to(DEV)
    norm = focus.rmsnorm_nvfp4 if fmt == "nvfp4" else focus.rmsnorm_mxfp8
    silu = focus.silu_mul_nvfp4 if fmt == "nvfp4" else focus.silu_mul_mxfp8
    calls = [lambda q: norm(x, w, EPS, dequant=True, out=q)[0], lambda q: silu(x, u, dequant=True, out=q)]
    if fmt == "mxfp8":
        calls.append(lambda q: focus.quantize_mxfp8(x, dequant=True, out=q))
    for call in calls:
        raw, q, pad = _buffers(focus, t, h, fmt)
        got = call(q)
        fresh = call(None)
        for a, b in zip(got, fresh):
            assert (a is None) == (b is None)
            if a is not None:
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        for k, v in raw.items():
            if k == "s2" and fmt == "mxfp8":
                assert (v == 0xA5).all()
            assert (v[:pad] == 0xA5).all() and (v[-pad:] == 0xA5).all(), k


def test_refusals_leave_outputs_alone(focus):
    x, w = _input(4, 64, 1).to(DEV), _weight(64, 2).to(DEV)
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    bad = [
        lambda: focus.rmsnorm(x, w[:32], out=out),
        lambda: focus.rmsnorm(x, w, 0.0, out=out),
        lambda: focus.rmsnorm(x, w, float("nan"), out=out),
        lambda: focus.rmsnorm(x, w.float(), out=out),
        lambda: focus.rmsnorm(x[:, ::2], w[:32], out=out),
        lambda: focus.rmsnorm(x.t(), w, out=out),
        lambda: focus.rmsnorm(x, w, residual=x[:2], out=out),
        lambda: focus.rmsnorm(x, w, residual_out=out, out=out),
        lambda: focus.rmsnorm(x, w, out=out[:2]),
        lambda: focus.rmsnorm(x[0], w, out=out),
        lambda: focus.rmsnorm_mxfp8(x[:, :48].contiguous(), w[:48]),
        lambda: focus.rmsnorm_nvfp4(x, w, dequant=True, out=focus.Quantized(
            torch.empty(4, 32, dtype=torch.uint8, device=DEV), torch.empty(4, 4, dtype=torch.uint8, device=DEV),
            None, torch.empty(4, device=DEV))),
        lambda: focus.silu_mul(x, x[:, ::2], out=out),
        lambda: focus.silu_mul(x, x[:2], out=out),
        lambda: focus.silu_mul(x, x.cpu(), out=out),
        lambda: focus.silu_mul(x.t(), x.t(), out=out),
        lambda: focus.silu_mul(x[:1].expand(4, 64), x, out=out),   # rows 0 apart
        lambda: focus.silu_mul(torch.empty(4, 68, dtype=torch.bfloat16, device=DEV)[:, :64], x, out=out),
        lambda: focus.silu_mul(torch.empty(4, 80, dtype=torch.bfloat16, device=DEV)[:, 1:65], x, out=out),
        lambda: focus.silu_mul_mxfp8(x[:, :48], x[:, :48]),
        lambda: focus.quantize_mxfp8(x[:, :32]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, focus.FocusError)):
            print("refusal", i, flush=True)
            call()
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def test_empty(focus):
    w = _weight(64, 1).to(DEV)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    y, h = focus.rmsnorm(x, w, residual=x)
    assert y.shape == (0, 64) and h.shape == (0, 64)
    q, _ = focus.rmsnorm_nvfp4(x, w)
    assert q.codes.shape == (0, 32) and q.s2.shape == (0,)
    assert focus.silu_mul_mxfp8(x, x).codes.shape == (0, 64)
    assert focus.quantize_mxfp8(x).scales.shape == (0, 2)


def test_another_stream_and_graph(focus):
    """On a stream of its own, and captured: every replay, with eager work
    between, gives the eager results."""
    t, h = 9, 4096
    x, r, w = _input(t, h, 1).to(DEV), _input(t, h, 2).to(DEV), _weight(h, 3).to(DEV)
    both = _input(t, 2 * h, 4).to(DEV)
    names = ("rmsnorm", "rmsnorm_nvfp4", "rmsnorm_mxfp8")

    def run():
        outs = []
        for n in names:
            a, b = getattr(focus, n)(x, w, EPS, residual=r)
            outs += [a] if n == "rmsnorm" else [a.codes, a.scales]
            outs.append(b)
        outs.append(focus.silu_mul(both[:, :h], both[:, h:]))
        for q in (focus.silu_mul_nvfp4(both[:, :h], both[:, h:]), focus.silu_mul_mxfp8(both[:, :h], both[:, h:]),
                  focus.quantize_mxfp8(x)):
            outs += [q.codes, q.scales]
        return outs

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
        for t_ in caught:
            t_.zero_()
        run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, caught):
            assert torch.equal(a, b)


@pytest.mark.parametrize("t,h", [(560_000, 4096), (70, 36_700_160)])
def test_offsets_past_32_bits(focus, t, h):
    """More than 2^31 elements: the last rows equal those of the same call on
    these rows alone."""
    def rows(p, n):
        return p[t - n:].clone()

    g = torch.Generator(device=DEV).manual_seed(h)
    x = torch.randn(t, h, device=DEV, dtype=torch.bfloat16, generator=g)
    r = torch.randn(t, h, device=DEV, dtype=torch.bfloat16, generator=g)
    w = torch.randn(h, device=DEV, dtype=torch.bfloat16, generator=g)
    n = 3

    def same(big, small):
        for a, b in zip(big, small):
            if a is not None:
                assert torch.equal(a[t - n:], b)

    y, res = focus.rmsnorm(x, w, EPS, residual=r)
    y1, res1 = focus.rmsnorm(rows(x, n), w, EPS, residual=rows(r, n))
    same((y, res), (y1, res1))
    del y, res
    for call in (focus.rmsnorm_nvfp4, focus.rmsnorm_mxfp8):
        q, _ = call(x, w, EPS, residual=r)
        same(q, call(rows(x, n), w, EPS, residual=rows(r, n))[0])
        del q
    same((focus.silu_mul(x, r),), (focus.silu_mul(rows(x, n), rows(r, n)),))
    for call in (focus.silu_mul_nvfp4, focus.silu_mul_mxfp8):
        same(call(x, r, dequant=True), call(rows(x, n), rows(r, n), dequant=True))
    same(focus.quantize_mxfp8(x, dequant=True), focus.quantize_mxfp8(rows(x, n), dequant=True))


def test_two_streams_at_once(focus):
    """No call keeps anything another could use."""
    ins = [(torch.randn(t, h, device=DEV).to(torch.bfloat16), torch.randn(t, h, device=DEV).to(torch.bfloat16),
            torch.randn(h, device=DEV).to(torch.bfloat16)) for t, h in ((1, 4096), (300, 8192), (4096, 2048))]

    def run():
        out = []
        for x, r, w in ins:
            y, res = focus.rmsnorm(x, w, EPS, residual=r)
            q, _ = focus.rmsnorm_nvfp4(x, w, EPS, dequant=True)
            p = focus.silu_mul_mxfp8(x, r, dequant=True)
            out += [y, res, q.codes, q.scales, q.s2, q.deq, p.codes, p.scales, p.deq]
        return out

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for s, out in zip(streams, got):
            with torch.cuda.stream(s):
                out += run()
    torch.cuda.synchronize()
    for out in got:
        for i, y in enumerate(out):
            assert torch.equal(y, want[i % len(want)])
