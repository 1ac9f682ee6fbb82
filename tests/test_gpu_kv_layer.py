"""A layer's cache after prompts and steps, both scales of every page (MI355X
only, marker gpu)."""
import numpy as np
import pytest
import torch

from test_gpu_kv_serving import DEV, Layer, dev, focus, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32)])
def test_scales_of_keys_and_values(focus, dim, page):
    """Both scales of every page, those that grow with later tokens among them."""
    layer = Layer(focus, dim=dim, page=page, pages=24, seed=3)
    table = np.random.default_rng(5).permutation(24).astype(np.int32).reshape(3, 8)
    rows = [5, page + 3, 2 * page]
    lengths, cu = np.array(rows), np.concatenate([[0], np.cumsum(rows)])
    p, y, _ = layer(focus.KVBatch(dev(table), dev(lengths), dev(cu), int(cu[-1])), tokens(1, int(cu[-1])))
    layer.check(table, lengths, cu, p, y)
    for step in range(page + 2):
        lengths = lengths + 1
        p, y, _ = layer(focus.KVBatch(dev(table), dev(lengths)), tokens(2 + step, 3) * (1 + step % 3))
        layer.check(table, lengths, None, p, y, parts=2)
        assert np.array_equal(layer.cache.v_scales.cpu().numpy(), layer.ref.vs)
        assert np.array_equal(layer.cache.k_scales.cpu().numpy(), layer.ref.ks)
