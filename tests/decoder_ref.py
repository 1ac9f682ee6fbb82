"""Plain references of the decoder-layer operators, on the CPU: the contract
of include/focus_nvfp4.h step by step (binary32 steps formed in numpy float32,
binary64 where the contract says so), and the linear layers' sums in
binary64.  Nothing here calls the library."""
import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float64)


def e4m3_table():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return t


E4M3 = e4m3_table()


def bf16_round(a):
    """float32 array -> nearest BF16 (ties to even), as float32."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def norm_h(x, res):
    """The summed row h (float32 holding BF16 values)."""
    x = x.float().numpy()
    return x if res is None else bf16_round(x + res.float().numpy())


def norm_y(h, w, eps):
    """binary32 y of the norm of h."""
    h64 = h.astype(np.float64)
    ms = (h64 * h64).sum(-1, keepdims=True) / h.shape[-1]
    rs = (1.0 / np.sqrt(ms + np.float64(np.float32(eps)))).astype(np.float32)
    return (h * rs) * w.float().numpy()[None]


def silu_y(g, u):
    """binary32 y of the gated activation."""
    g, u = g.float().numpy(), u.float().numpy()
    with np.errstate(over="ignore"):
        e = np.exp(-g.astype(np.float64)).astype(np.float32)
        sig = np.float32(1.0) / (np.float32(1.0) + e)
    return (g * sig) * u


def e2m1_code(x):
    """Codes of the nearest E2M1 value (ties to the even code), |x| clamped to 6."""
    mag = np.minimum(np.abs(x.astype(np.float64)), 6.0)
    mid = (E2M1[1:8] + E2M1[:7]) / 2
    code = np.searchsorted(mid, mag, side="left")  # on a midpoint: the lower code
    tie = (code < 7) & (mag == mid[np.minimum(code, 6)]) & (code % 2 == 1)
    code = code + tie
    return (code | (np.signbit(x).astype(np.int64) << 3)).astype(np.uint8)


def nvfp4(y):
    """Per-token NVFP4 of binary32 rows -> codes [T, H/2], scale bytes, s2, deq (float32)."""
    t, h = y.shape
    amax = np.abs(y).max(-1)
    s2 = amax / np.float32(2688.0)
    b = y.reshape(t, h // 16, 16)
    bm = np.abs(b).max(-1)
    zero = s2 == 0
    with np.errstate(divide="ignore", invalid="ignore"):
        q = bm / (np.float32(6.0) * s2)[:, None]
        q = np.where(q == 0, np.float32(1.0), q)
        q = np.minimum(np.maximum(q, np.float32(2.0 ** -6)), np.float32(448.0)).astype(np.float32)
        q[zero] = 1.0
        byte = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        S = E4M3[byte].astype(np.float32)
        d = (S * s2[:, None])[..., None]
        x = np.minimum(np.maximum(b / d, np.float32(-6.0)), np.float32(6.0))
    x = np.where(zero[:, None, None], b, x)  # a zero row keeps its signs
    codes = e2m1_code(x)
    deq = bf16_round((E2M1[codes].astype(np.float32) * S[..., None]) * s2[:, None, None]).reshape(t, h)
    codes = codes.reshape(t, h)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), byte.reshape(t, h // 16), s2, deq


def mxfp8(y):
    """MXFP8 of binary32 rows -> codes [T, H], scale bytes [T, H/32], deq (float32)."""
    t, h = y.shape
    b = y.reshape(t, h // 32, 32)
    bm = np.abs(b).max(-1)
    _, ex = np.frexp(bm)
    e = np.where(bm == 0, 0, np.maximum(ex.astype(np.int64) - 9, -127))
    e = np.where(np.isfinite(bm), e, 128)  # scale byte 255, NaN
    x = np.clip(np.ldexp(b.astype(np.float64), -e[..., None]), -448.0, 448.0)
    # x is a binary32 value or, below 2^-126, far under half the smallest code
    codes = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    deq = bf16_round(np.ldexp(E4M3[codes], e[..., None]).astype(np.float32))
    deq[e == 128] = np.nan
    return codes.reshape(t, h), (e + 127).astype(np.uint8), deq.reshape(t, h)


# --------------------------------------------------------------------------
# linear layers
# --------------------------------------------------------------------------

def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)


def weight_values(codes, scales, fmt):
    """binary64 c * S of stored weights (NVFP4 without s2)."""
    w = E2M1[unpack(codes)]
    s = np.ldexp(1.0, scales.astype(np.int64) - 127) if fmt == "mxfp4" else E4M3[scales]
    n = w.shape[1] // s.shape[1] if s.shape[1] else 1
    return w * np.repeat(s, n, 1)


def mxfp8_values(codes, scales):
    return E4M3[codes] * np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32, 1)


def _exponent(values, least):
    """floor(log2 |v|) of code values, at least `least` (zeros and subnormals)."""
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(values)))
    return np.maximum(e, least)


def mx_truncation(xc, xs, wc, ws):
    """Bound of the block-scaled product's truncation, [M, N]: in each group of
    8 consecutive k every product loses less than 2^-13 * 2^E, E the group's
    largest sum of the operands' exponents."""
    xe = _exponent(E4M3[xc], -6) + np.repeat(xs.astype(np.float64) - 127, 32, 1)
    we = _exponent(E2M1[unpack(wc)], 0) + np.repeat(ws.astype(np.float64) - 127, 32, 1)
    M, K = xe.shape
    out = np.zeros((M, we.shape[0]))
    for g in range(0, K, 8):
        E = (xe[:, None, g:g + 8] + we[None, :, g:g + 8]).max(-1)
        out += 8 * np.exp2(E - 13)
    return out
