"""Handles of the paged cache hold a descriptor that is packed once: what it was
packed of cannot be exchanged under it (CPU only)."""
import pytest
import torch

import fp4_post_weight_amd as focus

FIELDS = {"KVCache": ("k_codes", "k_scales", "v_codes", "v_scales", "pages", "kv_heads", "head_dim", "page_tokens", "device"),
          "KVBatch": ("page_table", "lengths", "cu_tokens", "sequences", "tokens", "device")}


@pytest.mark.parametrize("kind,name", [(k, n) for k, names in FIELDS.items() for n in names])
def test_attributes_are_read_only(kind, name):
    handle = object.__new__(getattr(focus, kind))
    for value in (None, 3, torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(AttributeError):
            setattr(handle, name, value)
    with pytest.raises(AttributeError):
        delattr(handle, name)


@pytest.mark.parametrize("kind", FIELDS)
def test_no_other_attributes(kind):
    handle = object.__new__(getattr(focus, kind))
    with pytest.raises(AttributeError):
        handle.anything = 1
