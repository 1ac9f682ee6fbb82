"""Integers of the cache's and the attention's calls that no C integer holds
(MI355X only, marker gpu)."""
import pytest
import torch

from test_gpu_kv_serving import DEV, dev, focus  # noqa: F401

pytestmark = pytest.mark.gpu


def test_integers_past_64_bits(focus):
    """They are refused, not cut: 2^64 + 5 is no window of 5."""
    c = focus.KVCache.zeros(4, 2, 64, 16, device=DEV)
    b = focus.KVBatch(dev([[0, 1], [2, 3]]), dev([3, 4]))
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device=DEV)
    for n in (2 ** 64, 2 ** 64 + 5, 2 ** 63, -2 ** 64, -2 ** 63 - 1):
        with pytest.raises(ValueError):
            focus.kv_attention(c, b, x, window=n)
        with pytest.raises(ValueError):
            focus.kv_attention_workspace_bytes(c, b, n)
    for n in (2 ** 31, 2 ** 63 - 1, -1):
        with pytest.raises(focus.FocusError):
            focus.kv_attention(c, b, x, window=n)
