"""Binary64 attention over the paged cache with the bounds that the kernels hold
sequence by sequence: 64 rows or fewer (tokens times query heads of a cache's
head, or one token) meet two parts of the probabilities and of turned queries,
more rows one.  For caches whose tokens all have pages and positions in the
rotation's table; scores are finite.  Nothing here calls the library."""
import numpy as np

import kv_ref as ref

U = 2.0 ** -24


def attention(c, table, lengths, cu, q, rope=None, scale=None, softcap=0.0, window=0):
    """q: float32 [tokens, heads, dim] of BF16 values.  Returns (y, tol, mine),
    as ref.attention does.

    With u = 2^-24.  A query's element turns by three binary32 roundings of its
    two products' magnitudes; stored in FP16 it is off by half a step, 2^-11 of
    itself, and with the rest in FP16 too by 2^-22 of itself and 2^-25 of a row's
    largest element's 2^-14 (the row is brought to 2^14 and beyond).  Without a
    table it is exact.  The score is the matrix cores' sum of dim products,
    or twice as many in two parts: (1.25 dim parts + 4) 2 u of their magnitudes,
    and 4 u of itself in its factor.

    A cap's slope is at most 1, so a capped score is off by no more of that.  The
    cap itself adds an error relative to the result.  Its argument x is off by
    4 u of itself (two roundings, the factor's two), and x tanh'(x) <= tanh(x).
    Below |x| = 0.75 a polynomial, 0.55 u off, is added to the score: with its
    roundings, which count for a fifth of theirs, within 4 u.  Beyond it is
    1 - 2 / (e + 1), e = exp(2 x): the exponential's argument is off by 2 u of
    itself and the exponential by 2 ulp, so that e is off by (4 |x| + 4) u e, the
    sum by u and the reciprocal by 2 ulp of itself: 2 / (e + 1) by
    2 / (e + 1) ((4 |x| + 4) e / (e + 1) + 5) u, which is at most 17 u of tanh|x|,
    at x = -0.75.  The difference and the product with the cap (two roundings
    itself) add 4 u: 25 u, taken as 26.

    A probability is then off by exp(ds) - 1, the exponential's 2 ulp and the
    rounding of its argument (to base 2: of s, m and s - m); in the numerator
    also by its rounding to BF16, 2^-8, in two parts 2^-16, and with one part in
    the sum as well, which adds up what the numerator takes.  Sums over n keys
    add (1.25 n parts + 8) 2 u of the magnitudes.  The quotient takes both sums'
    errors, and the result one rounding to BF16."""
    tokens, heads, dim = q.shape
    kvh = c.k.shape[1]
    group = heads // kvh
    scale = dim ** -0.5 if scale is None else scale
    y, tol, mine = np.zeros(q.shape), np.zeros(q.shape), np.zeros(tokens, bool)
    for b in range(len(lengths)):
        rows = ref.rows_of(b, lengths, cu)
        if not rows:
            continue
        parts = 2 if len(rows) == 1 or len(rows) * group <= 64 else 1
        at = np.array([ref.place(c, table, b, j) for j in range(int(lengths[b]))])
        page, off = at[:, 0], at[:, 1]
        keys = ref.E4M3[c.k[page, :, off]] * 2.0 ** (c.ks[page].astype(float) - 127)[..., None]
        vals = ref.E4M3[c.v[page, :, :, off]] * 2.0 ** (c.vs[page].astype(float) - 127)[..., None]
        for r, pos in rows:
            mine[r] = True
            lo = max(0, pos - window + 1) if window > 0 else 0
            x = q[r].astype(np.float64)
            dx = np.zeros_like(x)
            if rope is not None:
                h = dim // 2
                cs, sn = rope[pos, :h].astype(np.float64), rope[pos, h:].astype(np.float64)
                a, d = x[:, :h], x[:, h:]
                near = np.concatenate([abs(a * cs) + abs(d * sn), abs(d * cs) + abs(a * sn)], 1)
                x = np.concatenate([a * cs - d * sn, d * cs + a * sn], 1)
                dx = 3 * U * near + 2.0 ** (-11 * parts) * (np.abs(x) + 3 * U * near)
                dx = dx + 2.0 ** -39 * np.abs(x).max(1, keepdims=True)
            for i in range(heads):
                k, v = keys[lo:pos + 1, i // group], vals[lo:pos + 1, i // group]
                s = scale * (k @ x[i])
                ds = abs(scale) * (np.abs(k) @ (dx[i] + (1.25 * dim * parts + 4) * 2 * U * (np.abs(x[i]) + dx[i]))) + 4 * U * np.abs(s)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                    ds = ds + 26 * U * np.abs(s)
                m = s.max()
                p = np.exp(s - m)
                eps = np.expm1(ds + (np.abs(s - m) + np.abs(s) + np.abs(m)) * 2 * U) + 4 * U
                total, sums = p.sum(), (1.25 * len(s) * parts + 8) * 2 * U
                num = np.abs(v).T @ (p * (eps + 2.0 ** (-8 * parts))) + sums * (np.abs(v).T @ p)
                den = (p * eps).sum() + sums * total + (2.0 ** -8 * total if parts == 1 else 0.0)
                y[r, i] = v.T @ p / total
                with np.errstate(over="ignore"):  # scores of which nothing is left: no bound
                    t = (num + np.abs(y[r, i]) * den) / max(total - den, 1e-300)
                tol[r, i] = t * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y[r, i]) + 2.0 ** -133
    return y, tol, mine
