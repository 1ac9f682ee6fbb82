"""The paged 8-bit cache of keys and values and the attention over it, against
the plain reference of kv_ref (MI355X only, marker gpu)."""
import numpy as np
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def focus():
    import fp4_post_weight_amd as f
    f._lib.lib()
    return f


def bf16(x):
    return x.to(torch.bfloat16)


def table_for(rng, counts, pages, width=None, fill=0):
    """A page table whose sequences own counts[b] random distinct pages."""
    width = max(list(counts) + [1]) if width is None else width
    t = np.full((len(counts), width), fill, np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(counts):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make_cache(focus, c):
    return focus.KVCache(*c.tensors(DEV))


def same(cache, want):
    """The device cache equals the reference's, NaN codes as NaN."""
    for got, w in ((cache.k_codes, want.k), (cache.v_codes, want.v)):
        got = got.cpu().numpy()
        diff = (got != w) & ~(((got & 0x7F) == 0x7F) & ((w & 0x7F) == 0x7F))
        assert not diff.any(), f"{np.count_nonzero(diff)} codes differ, first at {np.argwhere(diff)[0]}"
    assert np.array_equal(cache.k_scales.cpu().numpy(), want.ks)
    assert np.array_equal(cache.v_scales.cpu().numpy(), want.vs)


def angles(positions, dim):
    f = 10000.0 ** (-np.arange(0, dim, 2) / dim)
    a = np.arange(positions)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def np32(t):
    return t.float().numpy()


# --------------------------------------------------------------------------
# the table of angles
# --------------------------------------------------------------------------

@pytest.mark.parametrize("positions,dim", [(1, 64), (77, 128), (131072, 128), (300, 2)])
def test_rope_table(focus, positions, dim):
    t = focus.rope_table(positions, dim, base=500000.0).cpu().numpy()
    f = np.array([500000.0 ** (-2.0 * i / dim) for i in range(dim // 2)])
    a = np.arange(positions)[:, None] * f
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    # the angle is rounded once on both sides, the functions to 2 ulp of
    # binary64, the result once to binary32
    tol = 2.0 ** -24 * np.abs(want) + 2.0 ** -50 + 2.0 ** -149
    assert (np.abs(t - want) <= tol).all()


def test_rope_table_own_frequencies(focus):
    f = torch.tensor([0.5, 0.0, 3.0, 1e-9], dtype=torch.float64, device=DEV)
    t = focus.rope_table(5, 8, inv_freq=f).cpu().numpy()
    a = np.arange(5)[:, None] * f.cpu().numpy()
    assert np.allclose(t, np.concatenate([np.cos(a), np.sin(a)], 1), rtol=0, atol=2.0 ** -24)
    assert focus.rope_table(0, 64).shape == (0, 64)


# --------------------------------------------------------------------------
# write
# --------------------------------------------------------------------------

def run_write(focus, cache, want, table, lengths, cu, k, v, rope=None, tokens=None, apart=True):
    """One write on the device and in the reference; k, v BF16 [T, heads, dim]."""
    T, heads, dim = k.shape
    if apart:  # parts of a wider product's rows
        wide = torch.randn(T, 2 * heads * dim + 24).to(torch.bfloat16)
        wide[:, 8:8 + heads * dim], wide[:, 16 + heads * dim:16 + 2 * heads * dim] = k.view(T, -1), v.view(T, -1)
        wide = wide.to(DEV)
        kd, vd = wide[:, 8:8 + heads * dim], wide[:, 16 + heads * dim:16 + 2 * heads * dim]
    else:
        kd, vd = k.view(T, -1).to(DEV), v.view(T, -1).to(DEV)
    batch = focus.KVBatch(dev(table), dev(np.asarray(lengths, np.int32)),
                          None if cu is None else dev(np.asarray(cu, np.int32)), T)
    focus.kv_cache_write(cache, batch, kd, vd, rope=None if rope is None else dev(rope))
    ref.write(want, table, lengths, cu, np32(k), np32(v), rope)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rope", [False, True])
def test_write_grows(focus, dim, page, rope):
    """Prompts, chunks behind them, then single tokens, with growing and
    shrinking magnitudes, so that pages change their exponent."""
    heads, pages = 3, 24
    g = torch.Generator().manual_seed(dim + page)
    rng = np.random.default_rng(page)
    want = ref.Cache(pages, heads, page, dim, fill=0x55)
    cache = make_cache(focus, want)
    table = table_for(rng, [5, 1, 7, 3], pages)
    rows = np.array([2 * page + 3, 1, 3 * page, page - 1])
    lengths = np.zeros(4, np.int64)
    angle = angles(7 * page, dim) if rope else None
    for step, size in enumerate([1.0, 30.0, 0.01, 5.0, 900.0]):
        if step == 1:
            rows = np.array([page // 2, 0, page + 5, 1])
        lengths = lengths + (rows if step < 2 else 1)
        lengths = np.minimum(lengths, [5 * page, page, 7 * page, 3 * page])
        cu = np.concatenate([[0], np.cumsum(rows)]) if step < 2 else None
        T = int(rows.sum()) if step < 2 else 4
        k = bf16(size * torch.randn(T, heads, dim, generator=g))
        v = bf16(size * torch.randn(T, heads, dim, generator=g) * torch.tensor([1.0, 1e-6, 1e9])[:, None])
        run_write(focus, cache, want, table, lengths, cu, k, v, angle)
        same(cache, want)


@pytest.mark.parametrize("dim,page,heads", [(64, 16, 1), (128, 64, 8), (128, 128, 2)])
def test_write_odd_places(focus, dim, page, heads):
    """Empty sequences, rows before position 0, tokens past the table and
    entries that are no page are left out, and rows of no sequence are not read."""
    rng = np.random.default_rng(5)
    g = torch.Generator().manual_seed(5)
    pages = 16
    want = ref.Cache(pages, heads, page, dim, fill=0x31)
    cache = make_cache(focus, want)
    table = table_for(rng, [3, 3, 3, 3], pages)
    table[1, 1] = -1
    table[2, 0] = pages
    table[2, 2] = 2 ** 31 - 1
    rows = np.array([0, 3 * page, 3 * page - 2, page + 9, 0])
    table = np.concatenate([table, table[:1]])
    # sequence 3 is shorter than its rows; sequence 1 ends behind its table
    lengths = np.array([7, 3 * page + 4, 3 * page - 1, page + 3, 0])
    cu = 3 + np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1]) + 5
    k, v = bf16(torch.randn(T, heads, dim, generator=g)), bf16(torch.randn(T, heads, dim, generator=g))
    batch = focus.KVBatch(dev(table), dev(lengths.astype(np.int32)), dev(cu.astype(np.int32)), T)
    focus.kv_cache_write(cache, batch, k.view(T, -1).to(DEV), v.view(T, -1).to(DEV))
    ref.write(want, table, lengths, cu, np32(k), np32(v))
    same(cache, want)


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16)])
def test_write_values_at_the_ends(focus, dim, page):
    """Zeros, subnormals, the largest BF16, values next to 448 * 2^e, infinities
    and NaN; then a token that moves the page's exponent over them."""
    heads = 6
    want = ref.Cache(3, heads, page, dim)
    cache = make_cache(focus, want)
    g = torch.Generator().manual_seed(1)
    k = torch.randn(page - 1, heads, dim, generator=g)
    k[:, 0] = 0.0
    k[:, 1] *= 2.0 ** -131
    k[:, 2] *= 2.0 ** 126
    k[0, 2, 0] = 3.3895313892515355e38  # the largest BF16
    k[:, 3] = k[:, 3].clamp(-1, 1)
    k[3, 3, 7] = 1.75  # 448 * 2^-8 exactly
    k[:, 4] = k[:, 4].clamp(-1, 1)
    k[3, 4, 7] = 1.7578125  # one BF16 step above
    k[1, 5, 3], k[2, 5, 4], k[3, 5, 5] = float("inf"), float("-inf"), float("nan")
    k = bf16(k)
    v = k.flip(0)
    table = np.array([[1, 2]], np.int32)
    n = page - 1
    run_write(focus, cache, want, table, [n], [0, n], k, v, apart=False)
    same(cache, want)
    assert (want.ks[1, 3], want.ks[1, 4]) == (119, 120)
    for size in (1e-3, 2.0 ** 20):
        one = bf16(size * torch.randn(1, heads, dim, generator=g))
        want2 = want.copy()
        cache2 = make_cache(focus, want2)
        run_write(focus, cache2, want2, table, [n + 1], None, one, one)
        same(cache2, want2)


def test_write_turn_past_the_table(focus):
    want = ref.Cache(4, 2, 16, 64)
    cache = make_cache(focus, want)
    g = torch.Generator().manual_seed(2)
    k, v = bf16(torch.randn(40, 2, 64, generator=g)), bf16(torch.randn(40, 2, 64, generator=g))
    run_write(focus, cache, want, np.array([[3, 1, 2]], np.int32), [40], [0, 40], k, v, angles(21, 64))
    same(cache, want)
    assert (want.k[1, 0, 5:] == 0x7F).all() and (want.k[1, 0, :5] != 0x7F).any()


def test_write_same_twice_and_many_sequences(focus):
    """300 sequences (more than a wavefront finds at once); the same call again
    changes nothing."""
    rng = np.random.default_rng(7)
    g = torch.Generator().manual_seed(7)
    n, page, dim, heads = 300, 16, 64, 2
    lengths = rng.integers(1, 60, n)
    rows = np.minimum(rng.integers(0, 40, n), lengths)
    rows[::7] = 0
    counts = -(-lengths // page)
    want = ref.Cache(int(counts.sum()) + 3, heads, page, dim, fill=0x3A)
    cache = make_cache(focus, want)
    table = table_for(rng, counts, want.k.shape[0], fill=-1)
    cu = np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1])
    k, v = bf16(torch.randn(T, heads, dim, generator=g)), bf16(torch.randn(T, heads, dim, generator=g))
    run_write(focus, cache, want, table, lengths, cu, k, v)
    same(cache, want)
    run_write(focus, cache, want.copy(), table, lengths, cu, k, v)
    same(cache, want)


# --------------------------------------------------------------------------
# read
# --------------------------------------------------------------------------

def filled(rng, pages, heads, page, dim, spread=6, nan=0.0):
    """A cache of random codes (NaN codes with probability nan) and scales."""
    c = ref.Cache(pages, heads, page, dim)
    for codes in (c.k, c.v):
        codes[...] = rng.integers(0, 256, codes.shape)
        codes[(codes & 0x7F) == 0x7F] ^= 0x40
        # mostly ordinary sizes
        codes[...] = np.where(rng.random(codes.shape) < 0.7, (codes & 0x87) | 0x30, codes)
        if nan:
            codes[rng.random(codes.shape) < nan] = 0x7F
    for s in (c.ks, c.vs):
        s[...] = rng.integers(121 - spread, 121, s.shape)
    return c


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_read(focus, dim, page):
    rng = np.random.default_rng(dim + page)
    heads, pages = 3, 20
    c = filled(rng, pages, heads, page, dim, spread=110, nan=0.01)
    c.ks[:3], c.vs[:3] = 0, 254
    table = table_for(rng, [4, 1, 5, 4, 2], pages)
    table[3, 2] = -7
    rows = np.array([3 * page + 5, 1, 0, 4 * page - 3, page + 4])
    lengths = np.array([3 * page + 5, page, 4 * page, 4 * page - 1, page - 2])  # the last: rows before position 0
    cu = 2 + np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1]) + 3
    cache = make_cache(focus, c)
    batch = focus.KVBatch(dev(table), dev(lengths.astype(np.int32)), dev(cu.astype(np.int32)), T)
    outs = [torch.full((T, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    got = focus.kv_cache_read(cache, batch, *outs)
    wk, wv, mine = ref.read(c, table, lengths, cu, T, heads, dim)
    for g, w in zip(got, (wk, wv)):
        g = g.cpu()
        assert (g[~mine] == 7.0).all()
        w = torch.from_numpy(w).to(torch.float32).to(torch.bfloat16)[mine]
        g = g[mine]
        assert torch.equal(torch.isnan(g), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(g.float(), nan=1.0), torch.nan_to_num(w.float(), nan=1.0))


def test_read_single_rows_and_round_trip(focus):
    """What a write stored comes back; without cu_tokens each sequence's last token."""
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(3)
    heads, dim, page = 8, 128, 64
    want = ref.Cache(12, heads, page, dim)
    cache = make_cache(focus, want)
    table = table_for(rng, [3, 4, 1], 12)
    lengths, cu = [130, 256, 1], [0, 130, 386, 387]
    k, v = bf16(torch.randn(387, heads, dim, generator=g)), bf16(torch.randn(387, heads, dim, generator=g))
    run_write(focus, cache, want, table, lengths, cu, k, v)
    same(cache, want)
    batch = focus.KVBatch(dev(table), dev(np.array(lengths, np.int32)), dev(np.array(cu, np.int32)), 387)
    kk, vv = focus.kv_cache_read(cache, batch)
    # a code is within 2^-4 of its value, or 2^-10 of a scale that is at most 2^-7.8 of the largest value
    for got, x in ((kk, k), (vv, v)):
        err = (got.cpu().float() - x.float()).abs()
        assert (err <= 2.0 ** -4 * x.float().abs() + 2.0 ** -10 * x.float().abs().max() / 224).all()
    last = focus.KVBatch(dev(table), dev(np.array(lengths, np.int32)))
    k1, v1 = focus.kv_cache_read(cache, last)
    assert torch.equal(k1, kk[[129, 385, 386]]) and torch.equal(v1, vv[[129, 385, 386]])


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

def run_attention(focus, c, table, lengths, cu, q, rope=None, out=None, apart=False, **kw):
    T, heads, dim = q.shape
    cache = make_cache(focus, c)
    batch = focus.KVBatch(dev(table), dev(np.asarray(lengths, np.int32)),
                          None if cu is None else dev(np.asarray(cu, np.int32)), T)
    qd = q.view(T, -1).to(DEV)
    if apart:
        wide = torch.zeros(T, heads * dim + 40, dtype=torch.bfloat16, device=DEV)
        wide[:, 16:16 + heads * dim] = qd
        qd = wide[:, 16:16 + heads * dim]
    y = focus.kv_attention(cache, batch, qd, rope=None if rope is None else dev(rope), out=out, **kw)
    return y.float().cpu().numpy().reshape(T, heads, dim)


def check_attention(focus, c, table, lengths, cu, q, rope=None, parts=1, apart=False, **kw):
    got = run_attention(focus, c, table, lengths, cu, q, rope, apart=apart, **kw)
    y, tol, mine = ref.attention(c, table, lengths, cu, np32(q), rope, parts=parts, **kw)
    ref.close(got, y, tol, mine)
    return got


def queries(seed, T, heads, dim, size=1.0):
    return bf16(size * torch.randn(T, heads, dim, generator=torch.Generator().manual_seed(seed)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kvh,group", [(2, 4), (1, 1), (3, 7), (1, 16), (1, 21)])
def test_decode(focus, dim, page, kvh, group):
    rng = np.random.default_rng(page + group)
    lengths = [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 700, 0]
    counts = [-(-n // page) for n in lengths]
    c = filled(rng, sum(counts), kvh, page, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    q = queries(group, len(lengths), kvh * group, dim, 0.5)
    got = check_attention(focus, c, table, lengths, None, q, parts=2, apart=True)
    assert (got[-1] == 0).all()  # a sequence without tokens


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rope,softcap,window", [(True, 0.0, 0), (False, 20.0, 0), (False, 0.0, 1), (True, 30.0, 100),
                                                 (False, 0.0, 64), (False, 0.0, 2 ** 31 - 1), (True, 0.0, 333)])
def test_decode_options(focus, dim, rope, softcap, window):
    rng = np.random.default_rng(window % 1000)
    lengths = [1, 65, 100, 101, 333, 334, 1500, 900]
    page = 32
    counts = [-(-n // page) for n in lengths]
    c = filled(rng, sum(counts), 2, page, dim)
    table = table_for(rng, counts, sum(counts), width=60, fill=-1)
    if 0 < window < 1000:  # pages that left the window are gone
        for b, n in enumerate(lengths):
            table[b, :max(0, n - window) // page] = 2 ** 30
    q = queries(3, len(lengths), 8, dim, 1.0)
    check_attention(focus, c, table, lengths, None, q, angles(1400, dim) if rope else None, parts=2, softcap=softcap,
                    window=window, scale=0.1)


@pytest.mark.parametrize("dim,kvh,group", [(64, 2, 4), (128, 1, 8), (128, 3, 1), (64, 1, 5)])
@pytest.mark.parametrize("rope,softcap,window", [(False, 0.0, 0), (True, 25.0, 0), (True, 0.0, 70), (False, 0.0, 1)])
def test_ragged(focus, dim, kvh, group, rope, softcap, window):
    """Long and short sequences, empty ones, rows before position 0, rows of no sequence."""
    rng = np.random.default_rng(dim + group)
    page = 16
    rows = np.array([300, 1, 0, 5, 131, 64, 40, 1])
    lengths = np.array([300, 500, 80, 77, 420, 64, 25, 900])
    counts = [-(-n // page) for n in lengths]
    c = filled(rng, sum(counts), kvh, page, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    cu = 2 + np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1]) + 3
    q = queries(1, T, kvh * group, dim, 0.7)
    out = torch.full((T, kvh * group * dim), 5.0, dtype=torch.bfloat16, device=DEV)
    got = check_attention_into(focus, c, table, lengths, cu, q, angles(800, dim) if rope else None, out, softcap, window)
    assert (got[:2] == 5.0).all() and (got[-3:] == 5.0).all()
    assert (got[cu[6]:cu[6] + 15] == 0).all()  # 40 rows of a sequence of 25 tokens


def check_attention_into(focus, c, table, lengths, cu, q, rope, out, softcap, window):
    got = run_attention(focus, c, table, lengths, cu, q, rope, out=out, apart=True, softcap=softcap, window=window)
    y, tol, mine = ref.attention(c, table, lengths, cu, np32(q), rope, softcap=softcap, window=window)
    ref.close(got, y, tol, mine)
    return got


@pytest.mark.parametrize("rows", [2, 3, 8, 16, 17, 64, 65, 200])
def test_rows_per_sequence(focus, rows):
    """Both sides of every kernel's limits on rows, by one key more than the rows and by many."""
    rng = np.random.default_rng(rows)
    lengths = np.array([rows, rows + 1, rows + 600])
    counts = [-(-n // 64) for n in lengths]
    c = filled(rng, sum(counts), 1, 64, 128)
    table = table_for(rng, counts, sum(counts))
    cu = np.arange(4) * rows
    for group in (1, 4):
        check_attention(focus, c, table, lengths, cu, queries(rows, 3 * rows, group, 128))


def test_nan_shows_where_it_is_seen(focus):
    """NaN keys and values reach the rows that see their token and no others;
    behind the last token, and in pages that no row sees, they reach none."""
    rng = np.random.default_rng(11)
    for rows, window in ((1, 0), (6, 0), (6, 40), (90, 0), (90, 33)):
        c = filled(rng, 12, 2, 32, 128)
        lengths, cu = np.array([181, 150]), np.array([0, rows, 2 * rows])
        table = table_for(rng, [6, 6], 12)
        tail = table[0, 5]
        c.k[tail, :, 181 % 32:], c.v[tail, :, :, 181 % 32:] = 0x7F, 0xFF
        # tokens 178 of sequence 0 (a key) and 148 and 130 of sequence 1 (a value each)
        c.k[tail, 0, 178 % 32, 5] = 0x7F
        c.v[table[1, 4], 1, 9, 148 % 32] = 0xFF
        c.v[table[1, 4], 0, 3, 130 % 32] = 0x7F
        c.k[table[1, 5]] = 0x7F  # a page behind the end
        q = queries(rows, 2 * rows, 8, 128)
        got = check_attention(focus, c, table, lengths, cu if rows > 1 else None, q, window=window)
        assert np.isnan(got).any() and not np.isnan(got).all()


def test_pages_that_are_not_there(focus):
    """Rows that see a token without a page are NaN, others are not."""
    rng = np.random.default_rng(12)
    c = filled(rng, 12, 1, 16, 64)
    table = table_for(rng, [6, 6], 12)
    table[0, 2], table[1, 3] = -1, 12
    for rows in (1, 3, 80):
        for lengths in ([96, 96], [90, 50], [120, 97]):  # the last: past the table
            cu = None if rows == 1 else np.array([0, rows, 2 * rows])
            q = queries(rows, 2 * rows, 4, 64)
            for window in (0, 20):
                check_attention(focus, c, table, np.array(lengths), cu, q, window=window)


@pytest.mark.parametrize("rows", [1, 70])
def test_queries_at_the_ends(focus, rows):
    """Queries of zeros, of very small and very large size with keys of the
    opposite one, infinite and NaN ones: each shows in its own row."""
    rng = np.random.default_rng(13)
    c = filled(rng, 10, 1, 64, 128)
    c.ks[:] = 10
    table = table_for(rng, [5, 5], 10)
    lengths = np.array([300, 290])
    q = queries(4, 2 * rows, 6, 128).float()
    q[:, 0] = 0.0
    q[:, 1] *= 2.0 ** 110
    q[:, 2] *= 2.0 ** -130
    q[0, 3, 7] = float("inf")
    q[-1, 3, 7] = float("nan")
    q[:, 4, 1:] *= 2.0 ** -40
    q = bf16(q)
    got = check_attention(focus, c, table, lengths, None if rows == 1 else np.array([0, rows, 2 * rows]), q)
    assert np.isnan(got[0, 3]).all() and np.isnan(got[-1, 3]).all() and not np.isnan(got[:, 5]).any()


@pytest.mark.parametrize("rows", [1, 70])
def test_values_of_any_scale(focus, rows):
    """Pages of very large values that get no weight do not cost the others'
    precision, and values at the ends of E8M0 come out."""
    rng = np.random.default_rng(14)
    c = filled(rng, 8, 1, 64, 64, spread=1)
    table = np.arange(8, dtype=np.int32)[None]
    c.vs[:, 0] = [127, 200, 120, 60, 127, 127, 20, 127]
    # page 1, of large values: keys far from the queries
    c.k[:, 0] &= 0x7F
    c.k[1, 0] |= 0x80
    c.k[3, 0] |= 0x80
    q = bf16(3.0 + torch.rand(rows, 2, 64, generator=torch.Generator().manual_seed(5)))
    check_attention(focus, c, table, np.array([500]), None if rows == 1 else np.array([0, rows]), q)
    c.vs[:] = 0
    check_attention(focus, c, table, np.array([500]), None if rows == 1 else np.array([0, rows]), q)


def test_long_sequences_and_workspaces(focus):
    """Sequences of very different lengths, with the full workspace, part of it
    and none, through the C ABI: each within the bound, equal calls equal."""
    rng = np.random.default_rng(15)
    lengths = np.array([9000, 3, 2500, 640])
    page, heads, dim = 64, 2, 128
    counts = [-(-n // page) for n in lengths]
    c = filled(rng, sum(counts), heads, page, dim)
    table = table_for(rng, counts, sum(counts))
    q = queries(6, 4, 8, dim)
    y, tol, mine = ref.attention(c, table, lengths, None, np32(q), parts=2)
    cache, batch = make_cache(focus, c), focus.KVBatch(dev(table), dev(lengths.astype(np.int32)))
    need = focus.kv_attention_workspace_bytes(cache, batch, 8)
    assert need > 0
    lib = focus._lib.lib()
    qd = q.view(4, -1).to(DEV)
    seen = []
    for size in (need, need, need // 3, need // 20, 0):
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.empty(4, 8 * dim, dtype=torch.bfloat16, device=DEV)
        focus._lib.check(lib.focus_kv_attention(cache._desc, batch._desc, qd.data_ptr(), 8 * dim, 8, None, 0,
                                                dim ** -0.5, 0.0, 0, out.data_ptr(), ws.data_ptr() if size else None,
                                                size, torch.cuda.current_stream().cuda_stream))
        ref.close(out.float().cpu().numpy().reshape(4, 8, dim), y, tol, mine)
        seen.append(out)
    assert torch.equal(seen[0], seen[1])


def test_many_sequences(focus):
    """More sequences than a wavefront holds, some without rows."""
    rng = np.random.default_rng(16)
    n, page = 200, 16
    lengths = rng.integers(1, 90, n)
    lengths[50] = 1500
    counts = -(-lengths // page)
    c = filled(rng, int(counts.sum()), 1, page, 64)
    table = table_for(rng, counts, int(counts.sum()), fill=-1)
    check_attention(focus, c, table, lengths, None, queries(1, n, 2, 64), parts=2)
    rows = np.where(rng.random(n) < 0.2, 0, np.minimum(rng.integers(1, 9, n), lengths))
    rows[50], rows[120], lengths[120] = 400, 50, 60
    rows = np.minimum(rows, lengths)
    cu = np.concatenate([[0], np.cumsum(rows)])
    check_attention(focus, c, table, lengths, cu, queries(2, int(cu[-1]), 2, 64))


def test_offsets_past_32_bits(focus):
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    heads, dim, page, pages = 8, 128, 128, 33000  # 4.3 GB each
    cache = focus.KVCache.zeros(pages, heads, dim, page, device=DEV)
    g = torch.Generator().manual_seed(8)
    T = 150
    k, v = bf16(torch.randn(T, heads, dim, generator=g)), bf16(torch.randn(T, heads, dim, generator=g))
    table = np.array([[32999, 32900]], np.int32)
    near = np.array([[1, 0]], np.int32)
    small = ref.Cache(2, heads, page, dim)
    ref.write(small, near, [T], [0, T], np32(k), np32(v))
    cu = dev(np.array([0, T], np.int32))
    batch = focus.KVBatch(dev(table), dev(np.array([T], np.int32)), cu, T)
    focus.kv_cache_write(cache, batch, k.view(T, -1).to(DEV), v.view(T, -1).to(DEV))
    for p, s in ((32999, 1), (32900, 0)):
        assert np.array_equal(cache.k_codes[p].cpu().numpy(), small.k[s])
        assert np.array_equal(cache.v_codes[p].cpu().numpy(), small.v[s])
    q = queries(9, T, 16, dim)
    y, tol, mine = ref.attention(small, near, [T], [0, T], np32(q))
    got = focus.kv_attention(cache, batch, q.view(T, -1).to(DEV))
    ref.close(got.float().cpu().numpy().reshape(T, 16, dim), y, tol, mine)
    one = focus.KVBatch(dev(table), dev(np.array([T], np.int32)))
    got = focus.kv_attention(cache, one, q[-1:].view(1, -1).to(DEV))
    ref.close(got.float().cpu().numpy().reshape(1, 16, dim), y[-1:], tol[-1:], mine[-1:])
    kk, vv = focus.kv_cache_read(cache, batch)
    wk, wv, _ = ref.read(small, near, [T], [0, T], T, heads, dim)
    assert np.array_equal(kk.float().cpu().numpy(), wk) and np.array_equal(vv.float().cpu().numpy(), wv)


def test_nothing_to_do(focus):
    cache = focus.KVCache.zeros(4, 2, 64, 16, device=DEV)
    empty = focus.KVBatch(torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    z = torch.zeros(0, 128, dtype=torch.bfloat16, device=DEV)
    focus.kv_cache_write(cache, empty, z, z)
    assert focus.kv_attention(cache, empty, z).shape == (0, 128)
    assert focus.kv_cache_read(cache, empty)[0].shape == (0, 2, 64)
    # sequences without rows: rows of no sequence stay
    none = focus.KVBatch(torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.tensor([5, 9], dtype=torch.int32, device=DEV),
                         torch.zeros(3, dtype=torch.int32, device=DEV), 4)
    out = torch.full((4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    q = torch.ones(4, 128, dtype=torch.bfloat16, device=DEV)
    focus.kv_cache_write(cache, none, q, q)
    focus.kv_attention(cache, none, q, out=out)
    torch.cuda.synchronize()
    assert (out == 3.0).all() and int(cache.k_codes.sum()) == 0
    # a table without columns: nothing has a page
    bare = focus.KVBatch(torch.zeros(1, 0, dtype=torch.int32, device=DEV), torch.tensor([5], dtype=torch.int32, device=DEV))
    assert torch.isnan(focus.kv_attention(cache, bare, q[:1])).all()
