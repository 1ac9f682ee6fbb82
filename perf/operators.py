"""Measured cases of the decoder-layer operators around the 4-bit formats:
root-mean-square norm and gated activation with quantized outputs, and the
linear layers with 4-bit weights and 8- or 16-bit activations.

``run`` has two forms.  With ``own`` false it computes an operator from
elementary torch operations in binary32 (binary64 where a rounding decides
which code is stored: the sum of squares, the exponential, quotients), with
``own`` true it makes the calls of ``fp4_post_weight_amd``.
"""
import math

import torch

own = False

EPS = 1e-5

# The outputs an operator can have: BF16; NVFP4 (E2M1 codes, one E4M3 scale
# per 16, one FP32 scale per token), returned as its dequantized values and
# the token scales; MXFP8 (E4M3 codes, one E8M0 scale per 32), returned as
# code values and scale values.


def listed():
    return [
        # norm before q, k, v of one decoded token of a 2048-wide model, into
        # the NVFP4 linear layer
        {"name": "norm nvfp4 1x2048", "op": "norm", "tokens": 1, "hidden": 2048, "out": "nvfp4", "residual": True},
        # norm of an 8192-wide model's batch of odd length, 16-bit output
        {"name": "norm bf16 1003x8192", "op": "norm", "tokens": 1003, "hidden": 8192, "out": "bf16",
         "residual": True},
        # prefill of a 4096-wide model, into the MXFP4 linear layer
        {"name": "norm mxfp8 8192x4096", "op": "norm", "tokens": 8192, "hidden": 4096, "out": "mxfp8",
         "residual": True},
        # gated activation of one decoded token
        {"name": "silu mxfp8 1x14336", "op": "silu", "tokens": 1, "hidden": 14336, "out": "mxfp8", "halves": False},
        # gate and up as the halves of one product's rows, odd batch
        {"name": "silu mxfp8 333x28672 halves", "op": "silu", "tokens": 333, "hidden": 28672, "out": "mxfp8",
         "halves": True},
        # prefill, into the NVFP4 linear layer
        {"name": "silu nvfp4 8192x14336", "op": "silu", "tokens": 8192, "hidden": 14336, "out": "nvfp4",
         "halves": False},
        # one decoded token through a square projection
        {"name": "mx linear 1x4096x4096", "op": "mx", "M": 1, "N": 4096, "K": 4096, "y": "bf16"},
        # a decode batch of odd size through gate or up
        {"name": "mx linear 100x14336x4096", "op": "mx", "M": 100, "N": 14336, "K": 4096, "y": "bf16"},
        # prefill through gate or up
        {"name": "mx linear 8192x14336x4096", "op": "mx", "M": 8192, "N": 14336, "K": 4096, "y": "bf16"},
        # weight-only, one token through down
        {"name": "w4a16 nvfp4 1x4096x14336", "op": "w4a16", "M": 1, "N": 4096, "K": 14336, "format": "nvfp4",
         "y": "bf16"},
        # weight-only, a few tokens through the widest matrix
        {"name": "w4a16 mxfp4 8x28672x8192", "op": "w4a16", "M": 8, "N": 28672, "K": 8192, "format": "mxfp4",
         "y": "bf16"},
        # weight-only, a decode batch through merged q, k, v, FP32 result
        {"name": "w4a16 nvfp4 61x6144x4096", "op": "w4a16", "M": 61, "N": 6144, "K": 4096, "format": "nvfp4",
         "y": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "silu", "mx", "w4a16"])
    if op in ("norm", "silu"):
        out = rng.choice(["bf16", "nvfp4", "mxfp8"])
        # whole scale blocks; BF16 rows come in vectors of 8
        unit = {"bf16": 8, "nvfp4": 16, "mxfp8": 32}[out]
        hidden = unit * _log_int(rng, 1024 // unit, 28672 // unit)
        tokens = _log_int(rng, 1, 8192)
        tokens = max(1, min(tokens, 8192 * 4096 // hidden))
        if op == "norm":
            return {"op": op, "tokens": tokens, "hidden": hidden, "out": out, "residual": rng.random() < 0.75}
        return {"op": op, "tokens": tokens, "hidden": hidden, "out": out, "halves": rng.random() < 0.5}
    fmt = "mxfp4" if op == "mx" else rng.choice(["nvfp4", "mxfp4"])
    unit = 16 if fmt == "nvfp4" else 32
    N = _log_int(rng, 500, 28672)
    K = unit * _log_int(rng, 1024 // unit, 14336 // unit)
    M = _log_int(rng, 1, 8192 if op == "mx" else 128)
    M = max(1, min(M, 8192 * 14336 * 4096 // (N * K)))
    y = rng.choice(["bf16", "fp32"])
    if op == "mx":
        return {"op": op, "M": M, "N": N, "K": K, "y": y}
    return {"op": op, "M": M, "N": N, "K": K, "format": fmt, "y": y}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _device():
    return torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _hidden_states(gen, tokens, hidden):
    """Hidden states: token-dependent size, a few channels far above the rest."""
    x = _normal(gen, tokens, hidden)
    channel = torch.exp(0.5 * _normal(gen, hidden))
    channel[torch.randint(0, hidden, (max(1, hidden // 512),), generator=gen, device=gen.device)] *= 12.0
    return x * channel * torch.exp(0.3 * _normal(gen, tokens, 1))


def _e2m1_codes(x):
    """Codes (0..15) of the nearest E2M1 values, ties to the even mantissa."""
    mag = x.abs().clamp(max=6.0)
    step = torch.where(mag < 2.0, 0.5, torch.where(mag < 4.0, 1.0, 2.0))
    v = torch.round(mag / step) * step
    code = torch.where(v < 2.0, v * 2.0, torch.where(v < 4.0, v + 2.0, v / 2.0 + 4.0)).to(torch.uint8)
    return code | (torch.signbit(x).to(torch.uint8) << 3)


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _weights(gen, N, K, fmt):
    """Stored 4-bit weights of a normal matrix: codes, scale bytes, s2."""
    w = _normal(gen, N, K) * 0.02
    if fmt == "mxfp4":
        b = w.view(N, K // 32, 32)
        e = torch.floor(torch.log2(b.abs().amax(-1))).clamp(-125.0, 127.0) - 2.0
        codes = _e2m1_codes(b / torch.exp2(e)[..., None]).view(N, K)
        return _pack(codes), (e + 127.0).to(torch.uint8), None
    s2 = w.abs().max() / 2688.0
    b = w.view(N, K // 16, 16)
    S = (b.abs().amax(-1) / (6.0 * s2)).clamp(2.0 ** -6, 448.0).to(torch.float8_e4m3fn)
    codes = _e2m1_codes(b / (S.float() * s2)[..., None]).view(N, K)
    return _pack(codes), S.view(torch.uint8), s2.reshape(1)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case)
    if case["op"] == "norm":
        t, h = case["tokens"], case["hidden"]
        st["x"] = _hidden_states(gen, t, h).to(torch.bfloat16)
        st["res"] = (4.0 * _hidden_states(gen, t, h)).to(torch.bfloat16) if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * _normal(gen, h)).to(torch.bfloat16)
    elif case["op"] == "silu":
        t, h = case["tokens"], case["hidden"]
        if case["halves"]:
            both = (1.5 * _normal(gen, t, 2 * h)).to(torch.bfloat16)
            st["gate"], st["up"] = both[:, :h], both[:, h:]
        else:
            st["gate"] = (1.5 * _normal(gen, t, h)).to(torch.bfloat16)
            st["up"] = (1.5 * _normal(gen, t, h)).to(torch.bfloat16)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["codes"], st["scales"], st["s2"] = _weights(gen, N, K, case.get("format", "mxfp4"))
        x = _hidden_states(gen, M, K)
        if case["op"] == "mx":
            b = x.view(M, K // 32, 32)
            e = torch.floor(torch.log2(b.abs().amax(-1))).clamp(-119.0, 127.0) - 8.0
            q = (b / torch.exp2(e)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            st["xc"] = q.view(M, K).view(torch.uint8)
            st["xs"] = (e + 127.0).to(torch.uint8)
        else:
            st["x"] = x.to(torch.bfloat16)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _quotient(a, b):
    """The binary32 quotient, rounded once."""
    return (a.double() / b.double()).float()


def _plain_nvfp4(y):
    t, h = y.shape
    s2 = _quotient(y.abs().amax(-1), torch.full((1,), 2688.0, device=y.device))
    b = y.view(t, h // 16, 16)
    amax = b.abs().amax(-1)
    q = _quotient(amax, 6.0 * s2[:, None])
    q = torch.where(q == 0, torch.ones_like(q), q).clamp(2.0 ** -6, 448.0)
    S = q.to(torch.float8_e4m3fn).float()
    codes = _e2m1_codes(_quotient(b, (S * s2[:, None])[..., None]))
    deq = (_e2m1_values(codes) * S[..., None]) * s2[:, None, None]
    return deq.view(t, h).to(torch.bfloat16), s2


def _plain_mxfp8(y):
    t, h = y.shape
    b = y.view(t, h // 32, 32)
    amax = b.abs().amax(-1)
    _, ex = torch.frexp(amax)
    e = (ex.float() - 9.0).clamp(-127.0, 127.0)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    S = torch.exp2(e.double())
    q = (b.double() / S[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(t, h), (e + 127.0).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_out(y, out):
    if out == "bf16":
        return y.to(torch.bfloat16)
    return _plain_nvfp4(y) if out == "nvfp4" else _plain_mxfp8(y)


def _e2m1_values(codes):
    c = (codes & 7).float()
    v = torch.where(c < 4.0, c * 0.5, torch.where(c < 6.0, c - 2.0, 2.0 * c - 8.0))
    return torch.where(codes > 7, -v, v)


def _plain_weight(st):
    c = st["codes"]
    w = _e2m1_values(torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1))
    if st.get("format", "mxfp4") == "mxfp4":
        s = torch.exp2(st["scales"].float() - 127.0)
    else:
        s = st["scales"].view(torch.float8_e4m3fn).float()
    return (w.view(*s.shape, -1) * s[..., None]).view(w.shape)


def _plain(st):
    if st["op"] == "norm":
        x, res = st["x"], st["res"]
        h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
        ms = h.double().square().mean(-1, keepdim=True) + EPS
        y = (h.float() * ms.rsqrt().float()) * st["weight"].float()
        y = _plain_out(y, st["out"])
        return y if res is None else (y, h)
    if st["op"] == "silu":
        g, u = st["gate"].float(), st["up"].float()
        sig = _quotient(torch.ones_like(g), 1.0 + torch.exp(-g.double()).float())
        return _plain_out((g * sig) * u, st["out"])
    w = _plain_weight(st)
    if st["op"] == "mx":
        s = torch.exp2(st["xs"].float() - 127.0)
        x = st["xc"].view(torch.float8_e4m3fn).float()
        x = (x.view(*s.shape, 32) * s[..., None]).view(x.shape)
    else:
        x = st["x"].float()
    y = x @ w.t()
    if st["s2"] is not None:
        y = y * st["s2"]
    return y.to(torch.bfloat16) if st["y"] == "bf16" else y


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own_out(q, out):
    if out == "bf16":
        return q
    if out == "nvfp4":
        return q.deq, q.s2
    return q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)


def _own(st):
    import fp4_post_weight_amd as focus
    if st["op"] == "norm":
        if st["out"] == "bf16":
            y, h = focus.rmsnorm(st["x"], st["weight"], EPS, residual=st["res"])
        elif st["out"] == "nvfp4":
            y, h = focus.rmsnorm_nvfp4(st["x"], st["weight"], EPS, residual=st["res"], dequant=True)
        else:
            y, h = focus.rmsnorm_mxfp8(st["x"], st["weight"], EPS, residual=st["res"])
        y = _own_out(y, st["out"])
        return y if st["res"] is None else (y, h)
    if st["op"] == "silu":
        if st["out"] == "bf16":
            return focus.silu_mul(st["gate"], st["up"])
        if st["out"] == "nvfp4":
            return _own_out(focus.silu_mul_nvfp4(st["gate"], st["up"], dequant=True), "nvfp4")
        return _own_out(focus.silu_mul_mxfp8(st["gate"], st["up"]), "mxfp8")
    dtype = torch.bfloat16 if st["y"] == "bf16" else torch.float32
    w = focus.Quantized(st["codes"], st["scales"], None, st["s2"])
    if st["op"] == "mx":
        return focus.mxfp4_linear(focus.Quantized(st["xc"], st["xs"], None, None), w, out_dtype=dtype)
    return focus.w4a16_linear(st["x"], w, out_dtype=dtype)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "silu"):
        n = case["tokens"] * case["hidden"]
        out = {"bf16": 2.0, "nvfp4": 0.5 + 1 / 16 + 2.0, "mxfp8": 1 + 1 / 32}[case["out"]]
        if case["op"] == "norm":
            return {"bytes": n * ((6.0 if case["residual"] else 2.0) + out) + 2 * case["hidden"], "flops": 8.0 * n}
        return {"bytes": n * (4.0 + out), "flops": 8.0 * n}
    M, N, K = case["M"], case["N"], case["K"]
    w = N * K * (0.5 + (1 / 32 if case.get("format", "mxfp4") == "mxfp4" else 1 / 16))
    x = M * K * (33 / 32 if case["op"] == "mx" else 2.0)
    return {"bytes": w + x + M * N * (2 if case["y"] == "bf16" else 4), "flops": 2.0 * M * N * K}


_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_out(y, out):
    """y in binary64 -> the operator's outputs, every step in binary64."""
    if out == "bf16":
        return y
    rows, cols = y.shape
    if out == "nvfp4":
        s2 = y.abs().amax(1) / 2688.0
        blocks = y.reshape(rows, cols // 16, 16)
        scale = blocks.abs().amax(2) / (6.0 * s2[:, None])
        scale = scale.clamp(2.0 ** -6, 448.0)
        # E4M3: three mantissa bits, nearest, ties to even
        unit = torch.exp2(torch.floor(torch.log2(scale)) - 3.0)
        scale = torch.round(scale / unit) * unit
        full = (scale * s2[:, None])[..., None]
        ratio = (blocks / full).clamp(-6.0, 6.0)
        grid = torch.tensor(_LEVELS, dtype=torch.float64, device=y.device)
        mid = (grid[1:] + grid[:-1]) / 2
        level = grid[torch.bucketize(ratio.abs().contiguous(), mid)]
        return (torch.copysign(level, ratio) * full).reshape(rows, cols), s2
    blocks = y.reshape(rows, cols // 32, 32)
    power = torch.exp2((torch.floor(torch.log2(blocks.abs().amax(2))) - 8.0).clamp(-127.0, 127.0))
    ratio = (blocks / power[..., None]).clamp(-448.0, 448.0)
    unit = torch.exp2((torch.floor(torch.log2(ratio.abs().clamp(min=2.0 ** -30))) - 3.0).clamp(min=-9.0))
    return (torch.round(ratio / unit) * unit).reshape(rows, cols), power


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        x = st["x"].double()
        total = x if st["res"] is None else x + st["res"].double()
        # the stored residual is BF16, and the norm is the stored residual's
        stored = total.to(torch.bfloat16).double()
        root = torch.sqrt((stored * stored).sum(1) / case["hidden"] + EPS)
        y = _exact_out(stored / root[:, None] * st["weight"].double(), case["out"])
        return y if st["res"] is None else (y, total)
    if case["op"] == "silu":
        g = st["gate"].double()
        return _exact_out(st["up"].double() * g * torch.sigmoid(g), case["out"])
    codes = st["codes"].long()
    table = torch.tensor(_LEVELS + [-v for v in _LEVELS], dtype=torch.float64, device=codes.device)
    w = torch.empty(case["N"], case["K"], dtype=torch.float64, device=codes.device)
    w[:, 0::2], w[:, 1::2] = table[codes % 16], table[codes // 16]
    if case.get("format", "mxfp4") == "mxfp4":
        w *= torch.pow(2.0, st["scales"].double() - 127.0).repeat_interleave(32, 1)
    else:
        w *= st["scales"].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * st["s2"].double()
    if case["op"] == "mx":
        x = st["xc"].view(torch.float8_e4m3fn).double()
        x = x * torch.pow(2.0, st["xs"].double() - 127.0).repeat_interleave(32, 1)
    else:
        x = st["x"].double()
    return torch.mm(x, w.t().contiguous())
