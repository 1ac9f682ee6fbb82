"""Row offsets and lengths that make no sense: outputs, workspaces and the cache
keep every byte around what the calls own, also where keys are split over
workgroups and where offsets count rows so often that counts of keys leave 32
bits (MI355X only, marker gpu)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from test_gpu_kv import DEV, check_attention, dev, filled, focus, make_cache, queries  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD = 1 << 16
BIG = 2 ** 31 - 1


class Guarded:
    """`size` bytes between two guards, all of one pattern."""

    def __init__(self, size):
        self.buf = torch.full((2 * GUARD + (size + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device=DEV)
        self.size = size

    def bf16(self, *shape):
        return self.buf[GUARD:GUARD + self.size].view(torch.bfloat16).view(shape)

    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def check(self):
        assert bool((self.buf[:GUARD] == 0xA5).all()) and bool((self.buf[GUARD + self.size:] == 0xA5).all())


def attend(focus, cache, batch, q, heads, y, ws, size, window=0):
    dim = cache.head_dim
    focus._lib.check(focus._lib.lib().focus_kv_attention(
        cache._desc, batch._desc, q.data_ptr(), heads * dim, heads, None, 0, dim ** -0.5, 0.0, window, y.ptr(),
        ws.ptr() if size else None, size, torch.cuda.current_stream().cuda_stream))


OFFSETS = [[0, 40, 10, 45, 50], [50, 0, 50, 0, 50], [-5, 20, 20, 999, 7], [BIG, -BIG, BIG, 0, BIG], [0, 300, 0, 300, 300],
           [299, 300, 299, 300, 1]]


@pytest.mark.parametrize("cu", OFFSETS)
def test_guards_of_write_and_read(focus, cu):
    rng = np.random.default_rng(11)
    pages, page, dim, T = 12, 16, 64, 50
    c = filled(rng, pages, 2, page, dim)
    cache = make_cache(focus, c)
    table = rng.permutation(pages - 2).astype(np.int32)[:8].reshape(4, 2) + 1  # pages 0 and 11 belong to no one
    free = [p for p in range(pages) if p not in table]
    kv = queries(9, T, 2, dim).view(T, -1).to(DEV)
    for lengths in ([20, 30, 32, 1], [-3, BIG, 0, 31], [-BIG, -1, BIG, BIG]):
        b = focus.KVBatch(dev(table), dev(np.array(lengths, np.int32)), dev(np.array(cu, np.int32)), T)
        focus.kv_cache_write(cache, b, kv, kv)
        k, v = Guarded(2 * T * 2 * dim), Guarded(2 * T * 2 * dim)
        focus.kv_cache_read(cache, b, k.bf16(T, 2, dim), v.bf16(T, 2, dim))
        k.check()
        v.check()
    for got, want in ((cache.k_codes, c.k), (cache.v_codes, c.v), (cache.k_scales, c.ks), (cache.v_scales, c.vs)):
        assert np.array_equal(got[free].cpu().numpy(), want[free])


@pytest.mark.parametrize("cu", OFFSETS)
@pytest.mark.parametrize("heads", [2, 16])
def test_guards_of_split_attention(focus, cu, heads):
    """A table of 4800 tokens, so that keys of few and of many rows are split."""
    rng = np.random.default_rng(12)
    pages, page, dim, T = 40, 16, 64, 300
    c = filled(rng, pages, 1, page, dim)
    cache = make_cache(focus, c)
    table = rng.integers(0, pages, (4, 300)).astype(np.int32)
    q = queries(8, T, heads, dim).view(T, -1).to(DEV)
    split = []
    for lengths in ([4800, 3000, 4000, 2000], [-3, BIG, 0, 4500], [-BIG, -1, BIG, BIG]):
        b = focus.KVBatch(dev(table), dev(np.array(lengths, np.int32)), dev(np.array(cu, np.int32)), T)
        need = focus.kv_attention_workspace_bytes(cache, b, heads)
        split.append(need)
        for size in (need, need // 3, 0):
            for window in (0, 2500):
                y, ws = Guarded(2 * T * heads * dim), Guarded(size)
                attend(focus, cache, b, q, heads, y, ws, size, window)
                y.check()
                ws.check()
    assert min(split) > 0
    check_attention(focus, c, table, np.array([4800, 3000, 4000, 20]), np.array([0, 3, 80, 90, 91]),
                    queries(8, 91, heads, dim))


def test_counts_that_leave_32_bits(focus):
    """One row counted by nine sequences: their tiles' steps are 2^32 + 16384, so
    that sums over the sequences wrap, to negative ones in between.  The tables
    name one page everywhere."""
    sequences, page, dim, heads = 18, 128, 64, 512
    rng = np.random.default_rng(13)
    cache = make_cache(focus, filled(rng, 1, 1, page, dim))
    table = torch.zeros(sequences, 1 << 23, dtype=torch.int32, device=DEV)
    lengths = torch.full((sequences,), 1 << 30, dtype=torch.int32, device=DEV)
    lengths[16] = 512 * 64
    cu = torch.arange(sequences + 1, device=DEV, dtype=torch.int32) % 2
    b = focus.KVBatch(table, lengths, cu, 1)
    need = focus.kv_attention_workspace_bytes(cache, b, heads)
    assert need > 0
    q = queries(14, 1, heads, dim).view(1, -1).to(DEV)
    y, ws = Guarded(2 * heads * dim), Guarded(need)
    attend(focus, cache, b, q, heads, y, ws, need)
    y.check()
    ws.check()
    # the same tensors in a sound batch
    one = focus.KVBatch(table[16:17], lengths[16:17])
    got = focus.kv_attention(cache, one, q)
    assert bool(torch.isfinite(got).all())
