"""The cache's and the attention's C ABI and binding refuse bad arguments on the
host before any HIP call (CPU only: no call here reaches a kernel launch)."""
import ctypes as ct
import os

import numpy as np
import pytest
import torch

import kv_ref as ref
from fp4_post_weight_amd import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_RANGE = 0, 1, 2, 3, 4, 5
FAKE = 0x10000  # never dereferenced
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfocus_nvfp4.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def cache(**kw):
    d = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, pages=10, kv_heads=2, head_dim=64, page_tokens=16)
    return _lib.KVCacheDesc(**{**d, **kw})


def batch(**kw):
    d = dict(page_table=FAKE, table_stride=5, max_pages=5, lengths=FAKE, cu_tokens=FAKE, sequences=3, tokens=7)
    return _lib.KVBatchDesc(**{**d, **kw})


def calls(lib):
    """The three calls with good arguments besides the descriptors."""
    yield lambda c, b: lib.focus_kv_cache_write(c, b, FAKE, 128, FAKE, 128, None, 0, None)
    yield lambda c, b: lib.focus_kv_cache_read(c, b, FAKE, FAKE, None)
    yield lambda c, b: lib.focus_kv_attention(c, b, FAKE, 256, 4, None, 0, 0.1, 0.0, 0, FAKE, None, 0, None)


def test_descriptor_layout():
    assert ct.sizeof(_lib.KVCacheDesc) == 8 * 8 and _lib.KVCacheDesc.pages.offset == 32
    assert ct.sizeof(_lib.KVBatchDesc) == 7 * 8 and _lib.KVBatchDesc.cu_tokens.offset == 32


def test_descriptors(lib):
    for f in calls(lib):
        assert f(None, batch()) == ERR_NULL and f(cache(), None) == ERR_NULL
        for bad in (dict(pages=-1), dict(kv_heads=0), dict(head_dim=96), dict(head_dim=0), dict(page_tokens=8),
                    dict(page_tokens=48), dict(page_tokens=256), dict(pages=0)):
            assert f(cache(**bad), batch()) == ERR_SHAPE, bad
        for bad in (dict(pages=1 << 31), dict(kv_heads=1025)):
            assert f(cache(**bad), batch()) == ERR_RANGE, bad
        for bad in (dict(sequences=-1), dict(tokens=-1), dict(max_pages=-1), dict(table_stride=4),
                    dict(cu_tokens=None)):
            assert f(cache(), batch(**bad)) == ERR_SHAPE, bad
        for bad in (dict(sequences=(1 << 20) + 1), dict(tokens=1 << 31), dict(max_pages=(1 << 26) + 1, table_stride=1 << 27),
                    dict(table_stride=1 << 40)):
            assert f(cache(), batch(**bad)) == ERR_RANGE, bad
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert f(cache(**{name: None}), batch()) == ERR_NULL, name
        for name in ("page_table", "lengths"):
            assert f(cache(), batch(**{name: None})) == ERR_NULL, name
        for bad in (dict(k_codes=FAKE + 8), dict(v_codes=FAKE + 4)):
            assert f(cache(**bad), batch()) == ERR_ALIGN, bad
        for bad in (dict(page_table=FAKE + 2), dict(lengths=FAKE + 1), dict(cu_tokens=FAKE + 2)):
            assert f(cache(), batch(**bad)) == ERR_ALIGN, bad
        # more threads than a launch has: 2^30 tokens of 1024 heads
        assert f(cache(kv_heads=1024), batch(tokens=1 << 30)) in (ERR_RANGE, ERR_SHAPE)
        # nothing to do
        nothing = dict(page_table=None, lengths=None, cu_tokens=None)
        assert f(cache(), batch(sequences=0, tokens=0, **nothing)) == OK
        assert f(cache(k_codes=None, pages=0), batch(sequences=0, tokens=0, **nothing)) == OK
        assert f(cache(), batch(tokens=0)) == OK


def test_write_arguments(lib):
    f = lib.focus_kv_cache_write
    c, b = cache(), batch()
    #           k     ks   v     vs   rope  n  stream
    assert f(c, b, None, 128, FAKE, 128, None, 0, None) == ERR_NULL
    assert f(c, b, FAKE, 128, None, 128, None, 0, None) == ERR_NULL
    assert f(c, b, FAKE, 120, FAKE, 128, None, 0, None) == ERR_SHAPE
    assert f(c, b, FAKE, 128, FAKE, 132, None, 0, None) == ERR_SHAPE
    assert f(c, b, FAKE, 1 << 60, FAKE, 128, None, 0, None) == ERR_SHAPE
    assert f(c, b, FAKE + 8, 128, FAKE, 128, None, 0, None) == ERR_ALIGN
    assert f(c, b, FAKE, 128, FAKE + 2, 128, None, 0, None) == ERR_ALIGN
    assert f(c, b, FAKE, 128, FAKE, 128, FAKE + 4, 9, None) == ERR_ALIGN
    assert f(c, b, FAKE, 128, FAKE, 128, FAKE, -1, None) == ERR_SHAPE
    r = lib.focus_kv_cache_read
    assert r(c, b, None, FAKE, None) == ERR_NULL and r(c, b, FAKE, None, None) == ERR_NULL
    assert r(c, b, FAKE + 8, FAKE, None) == ERR_ALIGN and r(c, b, FAKE, FAKE + 4, None) == ERR_ALIGN


def test_attention_arguments(lib):
    f = lib.focus_kv_attention
    c, b = cache(), batch()

    def g(q=FAKE, qs=256, heads=4, rope=None, n=0, scale=0.1, cap=0.0, window=0, y=FAKE, ws=None, size=0):
        return f(c, b, q, qs, heads, rope, n, scale, cap, window, y, ws, size, None)
    assert g(q=None) == ERR_NULL and g(y=None) == ERR_NULL
    assert g(heads=0) == ERR_SHAPE and g(heads=3) == ERR_SHAPE and g(heads=-2) == ERR_SHAPE
    assert g(heads=65538, qs=1 << 23) == ERR_RANGE
    assert g(qs=248) == ERR_SHAPE and g(qs=260) == ERR_SHAPE
    assert g(rope=FAKE, n=-1) == ERR_SHAPE and g(rope=FAKE + 8, n=5) == ERR_ALIGN
    for bad in (INF, -INF, NAN):
        assert g(scale=bad) == ERR_RANGE and g(cap=bad) == ERR_RANGE
    assert g(cap=-1.0) == ERR_RANGE and g(window=-1) == ERR_RANGE and g(window=1 << 31) == ERR_RANGE
    assert g(size=-1, ws=FAKE) == ERR_RANGE and g(ws=FAKE + 8, size=64) == ERR_ALIGN
    assert g(q=FAKE + 8) == ERR_ALIGN and g(y=FAKE + 8) == ERR_ALIGN


def test_rope_without_positions(lib):
    """A table of no positions would be read at its first."""
    assert lib.focus_kv_cache_write(cache(), batch(), FAKE, 128, FAKE, 128, FAKE, 0, None) == ERR_SHAPE
    assert lib.focus_kv_attention(cache(), batch(), FAKE, 256, 4, FAKE, 0, 0.1, 0.0, 0, FAKE, None, 0, None) == ERR_SHAPE


def test_counts_past_32_bits(lib):
    """Batches whose tiles, rows or threads leave 32 bits are refused, and need
    no workspace."""
    c = cache(kv_heads=1)
    one = dict(cu_tokens=None, max_pages=1000, table_stride=1000)
    w = lib.focus_kv_attention_workspace_bytes
    f = lib.focus_kv_attention
    for n, heads in ((1 << 20, 65536), (1 << 20, 64), (1 << 19, 64)):
        b = batch(sequences=n, tokens=n, **one)
        assert w(c, b, heads) == 0
        assert f(c, b, FAKE, heads * 64, heads, None, 0, 0.1, 0.0, 0, FAKE, None, 0, None) == ERR_RANGE
    b = batch(sequences=4, tokens=1 << 30)
    assert f(c, b, FAKE, 64 * 4, 4, None, 0, 0.1, 0.0, 0, FAKE, None, 0, None) == ERR_RANGE
    assert f(cache(), batch(tokens=(1 << 30) + 1), FAKE, 256, 4, None, 0, 0.1, 0.0, 0, FAKE, None, 0, None) == ERR_RANGE
    assert lib.focus_rope_table(FAKE, (1 << 26) + 1, 64, FAKE, None) == ERR_RANGE


def test_attention_workspace(lib):
    f = lib.focus_kv_attention_workspace_bytes
    assert f(None, batch(), 4) == 0 and f(cache(), batch(), 3) == 0 and f(cache(), batch(tokens=0), 4) == 0
    # no sequence is longer than one chunk
    one = dict(cu_tokens=None, tokens=3)
    assert f(cache(), batch(**one), 4) == 0
    assert f(cache(), batch(max_pages=1000, table_stride=1000, **one), 4) > 0


def test_rope_table_arguments(lib):
    f = lib.focus_rope_table
    assert f(None, 4, 64, FAKE, None) == ERR_NULL and f(FAKE, 4, 64, None, None) == ERR_NULL
    assert f(FAKE, -1, 64, FAKE, None) == ERR_SHAPE and f(FAKE, 4, 63, FAKE, None) == ERR_SHAPE
    assert f(FAKE, 1 << 38, 64, FAKE, None) == ERR_RANGE
    assert f(FAKE + 4, 4, 64, FAKE, None) == ERR_ALIGN and f(FAKE, 4, 64, FAKE + 8, None) == ERR_ALIGN
    assert f(None, 0, 64, None, None) == OK and f(None, 4, 0, None, None) == OK


def test_binding_refuses_cpu_tensors():
    import fp4_post_weight_amd as focus
    z = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        focus.KVCache(z, z[:, :, 0, 0], z.transpose(2, 3), z[:, :, 0, 0])
    with pytest.raises(TypeError):
        focus.KVCache(z.float(), z, z, z)
    with pytest.raises(ValueError):
        focus.KVBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        focus.KVBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        focus.kv_cache_write(None, None, None, None)
    with pytest.raises(ValueError):
        focus.rope_table(4, 63)


# --------------------------------------------------------------------------
# the reference itself
# --------------------------------------------------------------------------

def test_reference_scale_rule():
    for top, e in ((448.0, 0), (448.0001, 1), (0.0, -127), (1.75, -8), (1.7578125, -7), (3.39e38, 119), (2.0 ** -140, -127),
                   (224.0, -1)):
        assert ref.exponent(np.array([0.0, -top, np.inf, np.nan], np.float32)) == e
    x = np.array([448.0, -448.0, 0.0, np.nan, np.inf, 1.0625, 1.1875, 2.0 ** -10, 2.0 ** -10 * 1.5], np.float32)
    assert np.array_equal(ref.E4M3[ref.code(x)], [448.0, -448.0, 0.0, np.nan, np.nan, 1.0, 1.25, 0.0, 2.0 ** -9], equal_nan=True)


def test_reference_attention_against_softmax():
    """The reference's attention is torch's softmax attention over the values
    that its read gives."""
    rng = np.random.default_rng(0)
    c = ref.Cache(6, 2, 16, 64)
    k, v = rng.standard_normal((70, 2, 64)).astype(np.float32), rng.standard_normal((70, 2, 64)).astype(np.float32)
    table = np.array([[4, 1, 0, 3, 2]], np.int32)
    ref.write(c, table, [70], [0, 70], k, v)
    kk, vv, _ = ref.read(c, table, [70], [0, 70], 70, 2, 64)
    assert np.abs(kk - k).max() < 0.3 and np.abs(vv - v).max() < 0.3
    q = torch.randn(20, 6, 64, generator=torch.Generator().manual_seed(1))
    y, tol, mine = ref.attention(c, table, [70], [0, 20], q.numpy(), window=33)
    assert mine.all() and (tol > 0).all() and (tol < 0.1).all()
    i = torch.arange(50, 70)[:, None]
    j = torch.arange(70)[None]
    for h in range(6):
        s = (q[:, h].double() @ torch.from_numpy(kk[:, h // 3]).t()) / 8.0
        s = s.masked_fill((j > i) | (j <= i - 33), -INF)
        want = torch.softmax(s, -1) @ torch.from_numpy(vv[:, h // 3])
        assert np.allclose(y[:, h], want.numpy(), rtol=1e-12, atol=1e-13)


def test_packed_descriptors():
    """The bytes that the handles hold are the structures'."""
    c, b = cache(), batch()
    assert _lib.pack_kv_cache(*(getattr(c, n) or 0 for n, _ in c._fields_)) == bytes(c)
    assert _lib.pack_kv_batch(*(getattr(b, n) or 0 for n, _ in b._fields_)) == bytes(b)
