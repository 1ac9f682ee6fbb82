"""Sequences with few rows keep turned queries and probabilities in two parts,
alone and beside sequences with many (MI355X only, marker gpu)."""
import numpy as np
import pytest

import kv_bounds as bounds
import kv_ref as ref
from test_gpu_kv import angles, filled, focus, np32, queries, run_attention, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kvh,group", [(1, 1), (2, 4), (1, 21)])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (20.0, 0), (0.0, 100)])
def test_turned_queries_of_single_tokens(focus, dim, kvh, group, softcap, window):
    rng = np.random.default_rng(dim + group)
    lengths = np.array([1, 63, 64, 65, 300, 700])
    counts = [-(-n // 32) for n in lengths]
    c = filled(rng, sum(counts), kvh, 32, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    q, rope = queries(group, len(lengths), kvh * group, dim, 2.0), angles(700, dim)
    got = run_attention(focus, c, table, lengths, None, q, rope, softcap=softcap, window=window)
    ref.close(got, *bounds.attention(c, table, lengths, None, np32(q), rope, softcap=softcap, window=window))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (20.0, 150)])
def test_few_rows_beside_many(focus, dim, rope, softcap, window):
    """Each sequence of a batch holds its own bound."""
    rng = np.random.default_rng(dim + 2)
    rows = np.array([1, 130, 3, 16, 1, 70, 9])
    lengths = np.array([500, 200, 3, 333, 64, 400, 129])
    counts = [-(-n // 16) for n in lengths]
    c = filled(rng, sum(counts), 2, 16, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    cu = np.concatenate([[0], np.cumsum(rows)])
    q, angle = queries(4, int(cu[-1]), 8, dim, 1.5), angles(500, dim) if rope else None
    got = run_attention(focus, c, table, lengths, cu, q, angle, softcap=softcap, window=window)
    ref.close(got, *bounds.attention(c, table, lengths, cu, np32(q), angle, softcap=softcap, window=window))


@pytest.mark.parametrize("dim", [64, 128])
def test_turned_queries_split_over_the_keys(focus, dim):
    rng = np.random.default_rng(dim + 3)
    lengths = np.array([5000, 17, 2600])
    counts = [-(-n // 64) for n in lengths]
    c = filled(rng, sum(counts), 1, 64, dim)
    table = table_for(rng, counts, sum(counts), fill=-1)
    rope = angles(5000, dim)
    for rows in ([1, 1, 1], [3, 4, 1]):
        cu = np.concatenate([[0], np.cumsum(rows)])
        q = queries(5, int(cu[-1]), 8, dim, 1.5)
        got = run_attention(focus, c, table, lengths, None if max(rows) == 1 else cu, q, rope)
        ref.close(got, *bounds.attention(c, table, lengths, cu, np32(q), rope))
