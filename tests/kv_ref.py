"""Plain reference of the paged 8-bit cache and of the attention over it, on the
CPU: the contract of include/focus_nvfp4.h token by token (binary32 steps in
numpy float32 where a rounding decides a code, binary64 elsewhere).  Nothing
here calls the library."""
import numpy as np
import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


class Cache:
    """codes k [pages, heads, page, dim], v [pages, heads, dim, page], scale bytes."""

    def __init__(self, pages, heads, page, dim, fill=0):
        self.k = np.full((pages, heads, page, dim), fill, np.uint8)
        self.v = np.full((pages, heads, dim, page), fill, np.uint8)
        self.ks = np.full((pages, heads), fill, np.uint8)
        self.vs = np.full((pages, heads), fill, np.uint8)
        self.page = page

    def copy(self):
        c = Cache.__new__(Cache)
        c.k, c.v, c.ks, c.vs, c.page = self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy(), self.page
        return c

    def tensors(self, dev):
        return [torch.from_numpy(a).to(dev) for a in (self.k, self.ks, self.v, self.vs)]

    def key(self, p, h, t):
        return E4M3[self.k[p, h, t]] * 2.0 ** (int(self.ks[p, h]) - 127)

    def value(self, p, h, t):
        return E4M3[self.v[p, h, :, t]] * 2.0 ** (int(self.vs[p, h]) - 127)


def code(x):
    """E4M3 codes of float32 values at most 448 in magnitude; non-finite: 0x7F."""
    c = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(np.isfinite(x), c, np.uint8(0x7F))


def exponent(x):
    """The least e with max|x| <= 448 * 2^e over the finite values, in [-127, 119]."""
    a = np.abs(x[np.isfinite(x)]).astype(np.float64)
    top = a.max() if a.size else 0.0
    e = -127
    while e < 119 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def turn(x, rope, pos):
    """x [heads, dim] float32 turned by the table's row, each step binary32."""
    h = x.shape[1] // 2
    if pos < rope.shape[0]:
        c, s = rope[pos, :h], rope[pos, h:]
    else:
        c = s = np.full(h, np.nan, np.float32)
    a, b = x[:, :h], x[:, h:]
    with np.errstate(all="ignore"):
        return np.concatenate([a * c - b * s, b * c + a * s], 1)


def rows_of(b, lengths, cu):
    """(row, position) pairs of sequence b."""
    lo, hi = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
    first = int(lengths[b]) - (hi - lo)
    return [(r, first + r - lo) for r in range(lo, hi)]


def place(cache, table, b, pos):
    """(page, offset) of a token, or None if it has no page."""
    j = pos // cache.page
    if pos < 0 or j >= table.shape[1] or not 0 <= table[b, j] < cache.k.shape[0]:
        return None
    return int(table[b, j]), pos % cache.page


def write(cache, table, lengths, cu, k, v, rope=None):
    """k, v: float32 arrays [tokens, heads, dim] of BF16 values."""
    heads = k.shape[1]
    for b in range(len(lengths)):
        parts = {}
        for r, pos in rows_of(b, lengths, cu):
            at = place(cache, table, b, pos)
            if at is not None:
                kk = turn(k[r], rope, pos) if rope is not None else k[r]
                parts.setdefault((pos // cache.page, at[0]), []).append((at[1], kk, v[r]))
        for (_, p), toks in parts.items():
            for h in range(heads):
                for which, codes, scales in ((1, cache.k, cache.ks), (2, cache.v, cache.vs)):
                    x = np.stack([t[which][h] for t in toks])
                    e, held = exponent(x), toks[0][0]
                    old = int(scales[p, h]) - 127
                    mem = codes[p, h] if which == 1 else codes[p, h].T  # [page, dim]
                    if held > 0:
                        e = max(e, old)
                        if e != old:
                            moved = E4M3[mem[:held]] * 2.0 ** (old - e)
                            mem[:held] = np.where(np.isnan(moved), mem[:held], code(moved))
                    with np.errstate(all="ignore"):
                        q = np.clip(x.astype(np.float64) * 2.0 ** -e, -448.0, 448.0)
                        q = np.where(np.isfinite(x), q, np.nan)
                    for i, t in enumerate(toks):
                        mem[t[0]] = code(q[i])
                    scales[p, h] = e + 127


def read(cache, table, lengths, cu, tokens, heads, dim):
    """Values [tokens, heads, dim] twice and which rows belong to a sequence."""
    k, v = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads, dim))
    mine = np.zeros(tokens, bool)
    for b in range(len(lengths)):
        for r, pos in rows_of(b, lengths, cu):
            mine[r] = True
            at = place(cache, table, b, pos)
            for h in range(heads):
                if at is not None:
                    k[r, h], v[r, h] = cache.key(at[0], h, at[1]), cache.value(at[0], h, at[1])
                elif pos >= 0:
                    k[r, h] = v[r, h] = np.nan
    return k, v, mine


def attention(cache, table, lengths, cu, q, rope=None, scale=None, softcap=0.0, window=0, parts=1):
    """q: float32 [tokens, heads, dim] of BF16 values.  Returns (y, tol, mine):
    binary64 results and how far the library's may be from them.

    With u = 2^-24: a score's error d_s is the queries' rounding (turned: 2^-11
    of an element and three binary32 roundings; else exact), the binary32
    sum of dim products on the matrix cores (at most (1.25 dim + 4) 2^-23 of
    the products' magnitudes), four roundings of the score itself and, capped,
    8 u of the cap (tanh from an exponential and a reciprocal of 1 ulp each).
    A probability is then off by exp(d_s) - 1, the exponential's 2 ulp and the
    rounding of its argument, |s - m| u; in the numerator also by its rounding to
    BF16 (2^-8; 2^-16 in two parts), and with one part in the sum as well, which
    adds up what the numerator takes: with weights p (1 + d), |d| <= 2^-8, both
    are off by at most 2^-8 of their magnitudes.  Sums over n keys add (1.25 n + 8) 2^-23
    (chunks and wavefronts included).  The quotient takes both sums' errors,
    and the result one rounding to BF16."""
    tokens, heads, dim = q.shape
    kvh = cache.k.shape[1]
    group = heads // kvh
    scale = dim ** -0.5 if scale is None else scale
    u = 2.0 ** -24
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    mine = np.zeros(tokens, bool)
    for b in range(len(lengths)):
        n = int(lengths[b])
        rows = rows_of(b, lengths, cu)
        if not rows:
            continue
        low = 0 if window <= 0 else max(0, rows[0][1] - window + 1)
        span = range(low, n)
        keys = np.full((kvh, len(span), dim), np.nan)
        vals = np.full((kvh, len(span), dim), np.nan)
        for i, j in enumerate(span):
            at = place(cache, table, b, j)
            if at is not None:
                keys[:, i] = E4M3[cache.k[at[0], :, at[1]]] * 2.0 ** (cache.ks[at[0]].astype(float) - 127)[:, None]
                vals[:, i] = E4M3[cache.v[at[0], :, :, at[1]]] * 2.0 ** (cache.vs[at[0]].astype(float) - 127)[:, None]
        for r, pos in rows:
            mine[r] = True
            first = max(low, pos - window + 1) if window > 0 else 0
            if pos < 0:
                continue
            x = q[r].astype(np.float64)
            if rope is not None:
                h = dim // 2
                if pos < rope.shape[0]:
                    c, s = rope[pos, :h].astype(np.float64), rope[pos, h:].astype(np.float64)
                else:
                    c = s = np.full(h, np.nan)
                mag = np.abs(x)
                x = np.concatenate([x[:, :h] * c - x[:, h:] * s, x[:, h:] * c + x[:, :h] * s], 1)
                near = np.concatenate([mag[:, :h] * abs(c) + mag[:, h:] * abs(s), mag[:, h:] * abs(c) + mag[:, :h] * abs(s)], 1)
                dq = 2.0 ** -11 * np.abs(x) + 3 * u * near
            else:
                dq = np.zeros_like(x)
            for hh in range(heads):
                kk, vv = keys[hh // group, first - low:pos + 1 - low], vals[hh // group, first - low:pos + 1 - low]
                with np.errstate(all="ignore"):
                    s = scale * (kk @ x[hh])
                    ds = abs(scale) * (np.abs(kk) @ dq[hh] + (1.25 * dim + 4) * 2 * u * (np.abs(kk) @ np.abs(x[hh])))
                    ds = ds + 4 * u * np.abs(s)
                    if softcap > 0:
                        s = softcap * np.tanh(s / softcap)
                        ds = ds + 8 * u * softcap + 4 * u * np.abs(s)
                    m = np.max(s)
                    p = np.exp(s - m)
                    # base 2: s and m are log2(e) times larger
                    eps = np.expm1(ds + (np.abs(s - m) + np.abs(s) + np.abs(m)) * 2 * u) + 4 * u
                    total = p.sum()
                    sums = (1.25 * len(s) + 8) * 2 * u
                    num = np.abs(vv).T @ (p * (eps + 2.0 ** (-8 * parts))) + sums * (np.abs(vv).T @ p)
                    den = (p * eps).sum() + sums * total + (2.0 ** -8 * total if parts == 1 else 0.0)
                    yy = (vv.T @ p) / total
                    y[r, hh] = yy
                    t = (num + np.abs(yy) * den) / max(total - den, 1e-300)
                    tol[r, hh] = t * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(yy) + 2.0 ** -133
    return y, tol, mine


def close(got, want, tol, mine):
    """Asserts results [tokens, heads, dim] within tol, NaN exactly where wanted."""
    got = got.astype(np.float64)[mine]
    want, tol = want[mine], tol[mine]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    worst = np.max(np.abs(got - want)[ok] / np.maximum(tol[ok], 1e-300)) if ok.any() else 0.0
    assert worst <= 1.0, f"off by {worst} of the tolerance"
