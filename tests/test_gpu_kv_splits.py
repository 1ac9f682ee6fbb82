"""Attention over the paged cache where the keys are split: ranges across
sequences, pieces of sequences, tiles of many rows over few workgroups; and
batches whose row offsets make no sense (MI355X only, marker gpu)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from test_gpu_kv import DEV, angles, bf16, check_attention, dev, filled, focus, make_cache, np32, queries, run_attention, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (64, 4000)])
def test_ranges_across_sequences(focus, dim, window):
    """So many heads that a workgroup's range of keys spans sequences, some of
    them a few tokens long, one without rows and one without tokens."""
    rng = np.random.default_rng(dim)
    lengths = np.array([3, 5000, 1, 900, 0, 64, 7000, 17, 2600])
    counts = [-(-n // 64) for n in lengths]
    c = filled(rng, sum(counts), 64, 64, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    check_attention(focus, c, table, lengths, None, queries(1, len(lengths), 64, dim), angles(6000, dim), parts=2, window=window)
    rows = np.array([1, 2, 1, 9, 0, 1, 3, 4, 1])
    cu = np.concatenate([[0], np.cumsum(rows)])
    check_attention(focus, c, table, lengths, cu, queries(2, int(cu[-1]), 64, dim), parts=1, window=window)


@pytest.mark.parametrize("dim", [64, 128])
def test_tiles_per_sequence_in_ranges(focus, dim):
    """More than 16 rows per sequence and head, pieces of each 16-row tile."""
    rng = np.random.default_rng(dim + 1)
    lengths = np.array([4000, 130, 5555])
    counts = [-(-n // 128) for n in lengths]
    c = filled(rng, sum(counts), 2, 128, dim)
    table = table_for(rng, counts, sum(counts))
    cu = np.array([0, 3, 6, 10])
    check_attention(focus, c, table, lengths, cu, queries(3, 10, 2 * 13, dim))  # 39, 39 and 52 rows
    check_attention(focus, c, table, lengths, None, queries(4, 3, 2 * 40, dim), parts=2)


@pytest.mark.parametrize("dim,kvh,group", [(128, 1, 4), (64, 2, 3), (128, 2, 1)])
@pytest.mark.parametrize("rope,softcap,window", [(True, 0.0, 0), (False, 20.0, 0), (False, 0.0, 1500)])
def test_many_rows_split(focus, dim, kvh, group, rope, softcap, window):
    rng = np.random.default_rng(dim + group)
    lengths = np.array([5000, 2, 3100, 700])
    rows = np.array([130, 1, 300, 90])
    counts = [-(-n // 32) for n in lengths]
    c = filled(rng, sum(counts), kvh, 32, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    lengths[1] = 1
    cu = np.concatenate([[0], np.cumsum(rows)])
    q = queries(5, int(cu[-1]), kvh * group, dim, 0.7)
    check_attention(focus, c, table, lengths, cu, q, angles(5000, dim) if rope else None, softcap=softcap, window=window)


def test_many_rows_split_nan_and_lost_pages(focus):
    """NaN values and pages that are not there, in pieces of a tile's keys."""
    rng = np.random.default_rng(9)
    n, rows = 4100, 80
    c = filled(rng, 70, 1, 64, 64)
    table = table_for(rng, [65], 70)
    c.v[table[0, 3], 0, 5, 7] = 0x7F     # seen by every row
    c.v[table[0, 63], 0, 9, 40] = 0xFF   # token 4072: seen by the last rows
    c.v[table[0, 64], 0, 2, 10:] = 0x7F  # behind the end
    q = queries(6, rows, 2, 64)
    got = check_attention(focus, c, table, np.array([n]), np.array([0, rows]), q)
    assert np.isnan(got[:, :, 5]).all() and np.isnan(got[-1, :, 9]).all() and not np.isnan(got[0, :, 9]).any()
    table[0, 63] = 70
    check_attention(focus, c, table, np.array([n]), np.array([0, rows]), q)
    check_attention(focus, c, table, np.array([n]), np.array([0, rows]), q, window=50)


def test_workspaces_of_any_size(focus):
    """Many rows and single ones beside each other, with workspaces from none to
    the full one: every result within the bound."""
    rng = np.random.default_rng(10)
    lengths, rows = np.array([4000, 2500, 3000]), np.array([100, 1, 5])
    counts = [-(-n // 64) for n in lengths]
    c = filled(rng, sum(counts), 1, 64, 128)
    table = table_for(rng, counts, sum(counts))
    cu = np.concatenate([[0], np.cumsum(rows)])
    T, heads, dim = int(cu[-1]), 4, 128
    q = queries(7, T, heads, dim)
    y, tol, mine = ref.attention(c, table, lengths, cu, np32(q))
    cache = make_cache(focus, c)
    batch = focus.KVBatch(dev(table), dev(lengths.astype(np.int32)), dev(cu.astype(np.int32)), T)
    need = focus.kv_attention_workspace_bytes(cache, batch, heads)
    qd = q.view(T, -1).to(DEV)
    for size in (0, 16, need // 50, need // 7, need // 2, need):
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.empty(T, heads * dim, dtype=torch.bfloat16, device=DEV)
        focus._lib.check(focus._lib.lib().focus_kv_attention(
            cache._desc, batch._desc, qd.data_ptr(), heads * dim, heads, None, 0, dim ** -0.5, 0.0, 0, out.data_ptr(),
            ws.data_ptr() if size else None, size, torch.cuda.current_stream().cuda_stream))
        ref.close(out.float().cpu().numpy().reshape(T, heads, dim), y, tol, mine)


def test_offsets_that_make_no_sense(focus):
    """Row offsets that fall, leave the tensors or count rows twice, and
    lengths below 0 or past every table, lead to no access outside the
    tensors: pages and rows beyond what they could mean keep their bytes, and a
    sound batch after them gives its results."""
    rng = np.random.default_rng(11)
    pages, page, dim, heads, T = 12, 16, 64, 2, 50
    c = filled(rng, pages, 1, page, dim)
    cache = make_cache(focus, c)
    table = rng.permutation(pages - 2).astype(np.int32)[:8].reshape(4, 2) + 1  # pages 0 and 11 belong to no one
    q = queries(8, T, heads, dim).view(T, -1).to(DEV)
    kv = queries(9, T, 1, dim).view(T, -1).to(DEV)
    big = 2 ** 31 - 1
    for cu in ([0, 40, 10, 45, 50], [50, 0, 50, 0, 50], [-5, 20, 20, 999, 7], [big, -big, big, 0, big]):
        for lengths in ([20, 30, 32, 1], [-3, big, 0, 31], [-big, -1, big, big]):
            b = focus.KVBatch(dev(table), dev(np.array(lengths, np.int32)), dev(np.array(cu, np.int32)), T)
            focus.kv_cache_write(cache, b, kv, kv)
            focus.kv_cache_read(cache, b)
            focus.kv_attention(cache, b, q)
            focus.kv_attention(cache, b, q, window=5)
    torch.cuda.synchronize()
    for p in (0, 11):
        assert np.array_equal(cache.k_codes[p].cpu().numpy(), c.k[p]) and np.array_equal(cache.v_codes[p].cpu().numpy(), c.v[p])
    check_attention(focus, c, table, np.array([20, 30, 32, 1]), np.array([0, 5, 20, 45, 46]), queries(8, T, heads, dim))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
def test_wide_windows_and_rows_before_the_first(focus, window):
    """Rows at negative positions beside rows that see keys, under windows wider
    than any sequence."""
    rng = np.random.default_rng(12)
    c = filled(rng, 8, 1, 64, 64)
    table = table_for(rng, [4, 4], 8)
    for rows in (3, 90):
        lengths, cu = np.array([rows - 2, rows + 40]), np.array([0, rows, 2 * rows])
        got = check_attention(focus, c, table, lengths, cu, queries(rows, 2 * rows, 2, 64), window=window)
        assert (got[:2] == 0).all() and (got[2:] != 0).any()


def test_tables_rows_apart(focus):
    """A page table that is part of a wider one."""
    rng = np.random.default_rng(13)
    c = filled(rng, 12, 2, 16, 64)
    wide = rng.permutation(12).astype(np.int32).reshape(2, 6)
    lengths = np.array([40, 29])
    q = queries(1, 2, 4, 64)
    cache = make_cache(focus, c)
    batch = focus.KVBatch(dev(wide)[:, 2:5], dev(lengths.astype(np.int32)))
    got = focus.kv_attention(cache, batch, q.view(2, -1).to(DEV))
    y, tol, mine = ref.attention(c, wide[:, 2:5], lengths, None, np32(q), parts=2)
    ref.close(got.float().cpu().numpy().reshape(2, 4, 64), y, tol, mine)
    kk, _ = focus.kv_cache_read(cache, batch)
    assert np.array_equal(kk.float().cpu().numpy(), ref.read(c, wide[:, 2:5], lengths, None, 2, 2, 64)[0])


@pytest.mark.parametrize("dim,softcap,window", [(64, 0.0, 0), (128, 0.0, 0), (64, 25.0, 0), (128, 0.0, 2100)])
def test_many_and_few_rows_split_together(focus, dim, softcap, window):
    """Sequences with many rows whose keys are split, beside so many single
    tokens that theirs are cut into ranges; then the batch again without the
    ones or the others."""
    rng = np.random.default_rng(dim + 14)
    lengths = np.concatenate([rng.integers(2000, 3000, 24), [2500, 1900]])
    rows = np.concatenate([np.ones(24, int), [70, 300]])
    order = rng.permutation(26)
    lengths, rows = lengths[order], rows[order]
    counts = [-(-n // 64) for n in lengths]
    c = filled(rng, sum(counts), 8, 64, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    for kept in (rows, np.where(rows == 1, 1, 0), np.where(rows == 1, 0, rows)):
        cu = np.concatenate([[0], np.cumsum(kept)])
        check_attention(focus, c, table, lengths, cu, queries(15, int(cu[-1]), 16, dim), softcap=softcap, window=window)


def test_rope_table_of_no_positions(focus):
    c = make_cache(focus, filled(np.random.default_rng(16), 2, 1, 16, 64))
    batch = focus.KVBatch(torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV))
    x, none = torch.zeros(1, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 64, device=DEV)
    with pytest.raises(ValueError):
        focus.kv_attention(c, batch, x, rope=none)
    with pytest.raises(ValueError):
        focus.kv_cache_write(c, batch, x, x, rope=none)


@pytest.mark.parametrize("dim,kvh,heads,rows,lengths", [
    (64, 2, 8, [400, 1, 129], [410, 30, 1000]),       # 128-row tiles: few, short keys
    (128, 2, 8, [400, 1, 129], [410, 30, 1000]),
    (128, 8, 32, [1100], [1150]),                     # more of them than compute units
    (64, 8, 32, [1100, 1], [1150, 70]),
    (64, 8, 64, [1200], [1200]),                      # 256-row tiles beside the same keys
    (128, 8, 64, [1200], [1200]),
])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_tiles_of_either_height(focus, dim, kvh, heads, rows, lengths, softcap):
    rng = np.random.default_rng(17)
    lengths = np.array(lengths)
    counts = [-(-n // 16) for n in lengths]
    c = filled(rng, sum(counts), kvh, 16, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    cu = np.concatenate([[0], np.cumsum(rows)])
    check_attention(focus, c, table, lengths, cu, queries(18, int(cu[-1]), heads, dim), angles(1200, dim), softcap=softcap)


def test_row_counts_that_are_none(focus):
    table, lengths = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    cu = torch.zeros(2, dtype=torch.int32, device=DEV)
    for tokens in (-1, 2 ** 30 + 1, 1 << 70):
        with pytest.raises(ValueError):
            focus.KVBatch(table, lengths, cu, tokens)
    with pytest.raises(TypeError):
        focus.KVBatch(table, lengths, cu, 1.0)
