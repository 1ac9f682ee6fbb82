"""Attention over values and scores at the ends of what the cache holds (MI355X
only, marker gpu)."""
import numpy as np
import pytest

import kv_ref as ref
from test_gpu_kv import bf16, check_attention, filled, focus, table_for  # noqa: F401
import torch

pytestmark = pytest.mark.gpu


def e4m3(x):
    return ref.code(np.float32(x)).item()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,heads", [(1, 2), (3, 2), (70, 2), (1, 40), (130, 2)])
@pytest.mark.parametrize("softcap", [0.0, 1e4])
def test_large_values_behind_small_scores(focus, dim, rows, heads, softcap):
    """Values of 2^116 to 2^117 whose keys' scores are 7.9 above (base 2) those of
    the sequence's first 128 tokens: their mean is finite, and so are the sums of
    900 of them with weights up to 1."""
    rng = np.random.default_rng(dim)
    n, page = 900, 64
    c = filled(rng, 15, 1, page, dim)
    c.ks[:] = 127
    c.k[:] = 0
    table = table_for(rng, [15], 15)
    # 5.5 / log(2) = 7.93
    c.k[table[0, 2:]] = e4m3(0.6875)
    size = 2.0 ** rng.uniform(0, 1, c.v.shape) * np.where(rng.random(c.v.shape) < 0.7, 1.0, -1.0)
    c.v[:] = ref.code(size.astype(np.float32))
    c.vs[:] = 127 + 116
    c.vs[table[0, 1]] = 127
    q = torch.ones(rows, heads, dim, dtype=torch.bfloat16)
    got = check_attention(focus, c, table, np.array([n]), None if rows == 1 else np.array([0, rows]), q,
                          scale=8.0 / dim, softcap=softcap)
    assert np.isfinite(got).all()


@pytest.mark.parametrize("rows", [1, 70])
def test_largest_value_alone(focus, rows):
    """A token that has all the weight holds the largest value that the cache can,
    448 * 2^119."""
    rng = np.random.default_rng(3)
    c = filled(rng, 2, 1, 64, 64)
    c.ks[:] = 127
    c.k[:] = 0
    table = np.array([[0, 1]], np.int32)
    c.k[1, 0, 5] = e4m3(16.0)
    c.v[:], c.vs[0], c.vs[1] = e4m3(1.0), 127, 127 + 119
    c.v[1] = e4m3(0.0)
    c.v[1, 0, :, 5] = e4m3(448.0)
    q = torch.ones(rows, 2, 64, dtype=torch.bfloat16)
    # 128 above in base e: every other weight is below 2^-184
    got = check_attention(focus, c, table, np.array([128]), None if rows == 1 else np.array([0, rows]), q)
    seen = got if rows == 1 else got[-1:]
    assert (seen == 448.0 * 2.0 ** 119).all()


def test_smallest_values(focus):
    """Subnormal values come out: weights below 1 do not take them away."""
    rng = np.random.default_rng(4)
    for rows in (1, 70):
        c = filled(rng, 8, 1, 64, 64, spread=1)
        c.vs[:] = 0
        c.v[:] = (c.v & 0x80) | 0x7E  # 448 * 2^-127
        q = bf16(torch.rand(rows, 2, 64, generator=torch.Generator().manual_seed(6)))
        table = np.arange(8, dtype=np.int32)[None]
        got = check_attention(focus, c, table, np.array([500]), None if rows == 1 else np.array([0, rows]), q)
        assert (got != 0).any()
