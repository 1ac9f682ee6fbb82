"""Caps of the attention's scores over all of their range: a score is capped with
an error relative to itself, whatever the cap (MI355X only, marker gpu)."""
import numpy as np
import pytest
import torch

import kv_bounds as bounds
import kv_ref as ref
from test_gpu_kv import filled, focus, np32, queries, run_attention, table_for  # noqa: F401

pytestmark = pytest.mark.gpu

CAPS = [1e-42, 1e-3, 1.0, 30.0, 1e3, 1e5, 1e6, 1e8, 1e10, 1e30, 2.4e38, 3.4028234e38]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 70])
def test_caps_of_any_size(focus, dim, rows):
    rng = np.random.default_rng(dim + rows)
    lengths = np.array([150, 90])
    c = filled(rng, 8, 2, 32, dim, spread=3)
    table = table_for(rng, [5, 3], 8)
    cu = None if rows == 1 else np.array([0, rows, 2 * rows])
    q = queries(rows, 2 * rows, 4, dim, 0.5)
    plain = bounds.attention(c, table, lengths, cu, np32(q))
    for cap in CAPS:
        print("cap", cap, flush=True)
        want = bounds.attention(c, table, lengths, cu, np32(q), softcap=float(np.float32(cap)))
        got = run_attention(focus, c, table, lengths, cu, q, softcap=cap)
        ref.close(got, *want)
        if cap <= 1.0:  # a cap that does nothing would show
            assert (np.abs(want[0] - plain[0]) > want[1] + plain[1]).any()
    ref.close(run_attention(focus, c, table, lengths, cu, q), *plain)


@pytest.mark.parametrize("rows", [1, 70])
def test_scores_around_the_cap(focus, rows):
    """Scores from far below the cap to far beyond it; a NaN query's row is NaN."""
    rng = np.random.default_rng(5)
    c = filled(rng, 6, 1, 64, 64, spread=3)
    table = table_for(rng, [6], 6)
    cu = None if rows == 1 else np.array([0, rows])
    q = queries(7, rows, 6, 64)
    size = torch.tensor([2.0 ** -20, 2.0 ** -6, 0.5, 4.0, 64.0, 2.0 ** 20])
    q = (q.float() * size[None, :, None]).to(torch.bfloat16)
    got = run_attention(focus, c, table, [380], cu, q, softcap=5.0)
    ref.close(got, *bounds.attention(c, table, [380], cu, np32(q), softcap=5.0))
    q[0, 1, 3], q[0, 2, 3] = float("inf"), float("nan")
    for cap in (5.0, 1e9):
        got = run_attention(focus, c, table, [380], cu, q, softcap=cap)
        assert np.isnan(got[0, 2]).all() and not np.isnan(got[0, [0, 3, 4, 5]]).any()


def test_negative_scale_and_window(focus):
    """A cap is odd: a negative scale gives the scores' mirror images."""
    rng = np.random.default_rng(6)
    c = filled(rng, 12, 1, 16, 128, spread=3)
    table = table_for(rng, [12], 12)
    for rows in (1, 70):
        cu = None if rows == 1 else np.array([0, rows])
        q = queries(8, rows, 4, 128, 0.5)
        for cap in (2.0, 1e7):
            got = run_attention(focus, c, table, [190], cu, q, softcap=cap, scale=-0.05, window=77)
            ref.close(got, *bounds.attention(c, table, [190], cu, np32(q), softcap=cap, scale=-0.05, window=77))
