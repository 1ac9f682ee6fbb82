"""A decoder layer's attention part as a serving program runs it: norm, the
merged q, k, v product on 4-bit weights, the cache's write with the rotation,
attention, the o product -- prompts, then steps of single tokens, eager, as
captured graphs and on other streams.  MI355X only (marker gpu)."""
import numpy as np
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


@pytest.fixture(scope="module")
def focus():
    import fp4_post_weight_amd as f
    f._lib.lib()
    return f


class Layer:
    def __init__(self, focus, hidden=512, heads=8, kv_heads=2, dim=64, page=16, pages=40, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.focus, self.heads, self.kv_heads, self.dim = focus, heads, kv_heads, dim
        w = torch.randn((heads + 2 * kv_heads) * dim, hidden, generator=g) * hidden ** -0.5
        self.qkv = focus.quantize_mx(w.to(torch.bfloat16).to(DEV), dequant=False)
        w = torch.randn(hidden, heads * dim, generator=g) * (heads * dim) ** -0.5
        self.o = focus.quantize_mx(w.to(torch.bfloat16).to(DEV), dequant=False)
        self.norm = (1 + 0.2 * torch.randn(hidden, generator=g)).to(torch.bfloat16).to(DEV)
        self.rope = focus.rope_table(page * pages, dim, base=10000.0, device=DEV)
        self.cache = focus.KVCache.zeros(pages, kv_heads, dim, page, device=DEV)
        self.ref = ref.Cache(pages, kv_heads, page, dim)

    def __call__(self, batch, x):
        f, n = self.focus, self.heads * self.dim
        m = self.kv_heads * self.dim
        h, _ = f.rmsnorm(x, self.norm, EPS)
        p = f.w4a16_linear(h, self.qkv)
        f.kv_cache_write(self.cache, batch, p[:, n:n + m], p[:, n + m:], rope=self.rope)
        y = f.kv_attention(self.cache, batch, p[:, :n], rope=self.rope)
        return p, y, f.w4a16_linear(y, self.o)

    def check(self, table, lengths, cu, p, y, parts=1):
        T = p.shape[0]
        p = p.float().cpu().numpy().reshape(T, -1, self.dim)
        q, k, v = p[:, :self.heads], p[:, self.heads:self.heads + self.kv_heads], p[:, self.heads + self.kv_heads:]
        rope = self.rope.cpu().numpy()
        ref.write(self.ref, table, lengths, cu, k, v, rope)
        assert np.array_equal(self.cache.k_codes.cpu().numpy(), self.ref.k)
        assert np.array_equal(self.cache.v_codes.cpu().numpy(), self.ref.v)
        assert np.array_equal(self.cache.k_scales.cpu().numpy(), self.ref.ks)
        want, tol, mine = ref.attention(self.ref, table, lengths, cu, q, rope, parts=parts)
        ref.close(y.float().cpu().numpy().reshape(T, self.heads, self.dim), want, tol, mine)


def dev(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


def tokens(seed, n, hidden=512):
    return torch.randn(n, hidden, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def test_prompts_then_tokens(focus):
    layer = Layer(focus)
    table = np.random.default_rng(0).permutation(40).astype(np.int32).reshape(4, 10)
    rows = [33, 1, 100, 17]
    cu = np.concatenate([[0], np.cumsum(rows)])
    lengths = np.array(rows)
    p, y, o = layer(focus.KVBatch(dev(table), dev(lengths), dev(cu), int(cu[-1])), tokens(1, int(cu[-1])))
    layer.check(table, lengths, cu, p, y)
    assert o.shape == (151, 512) and torch.isfinite(o).all()
    for step in range(20):
        lengths = lengths + 1
        p, y, _ = layer(focus.KVBatch(dev(table), dev(lengths)), tokens(2 + step, 4))
        layer.check(table, lengths, None, p, y, parts=2)
    # a chunk of one beside tokens of the others
    rows = [1, 30, 1, 1]
    lengths = lengths + rows
    cu = np.concatenate([[0], np.cumsum(rows)])
    p, y, _ = layer(focus.KVBatch(dev(table), dev(lengths), dev(cu), 33), tokens(99, 33))
    layer.check(table, lengths, cu, p, y)


@pytest.mark.parametrize("dim,window", [(64, 0), (128, 300)])
def test_graph_of_a_step(focus, dim, window):
    """A captured step of single tokens, replayed while the lengths grow in
    place, against the same steps run eagerly on a second cache; two graphs of
    the same layer in turn."""
    rng = np.random.default_rng(1)
    page, heads, n = 64, 4, 5
    start = np.array([700, 3, 64, 1200, 1])
    table = rng.permutation(5 * 20).astype(np.int32).reshape(5, 20)
    caches = []
    g = torch.Generator().manual_seed(3)
    T = int(start.sum())
    k, v = (torch.randn(T, 2 * dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    cu = dev(np.concatenate([[0], np.cumsum(start)]))
    for _ in range(2):
        c = focus.KVCache.zeros(100, 2, dim, page, device=DEV)
        focus.kv_cache_write(c, focus.KVBatch(dev(table), dev(start), cu, T), k, v)
        caches.append(c)
    lengths = dev(start)
    x = torch.randn(n, (heads + 4) * dim, generator=g).to(torch.bfloat16).to(DEV)
    rope = focus.rope_table(2000, dim, device=DEV)
    table_d = dev(table)

    def step(cache, lengths):
        b = focus.KVBatch(table_d, lengths)
        focus.kv_cache_write(cache, b, x[:, heads * dim:(heads + 2) * dim], x[:, (heads + 2) * dim:], rope=rope)
        return focus.kv_attention(cache, b, x[:, :heads * dim], rope=rope, window=window)

    eager_lengths = dev(start)
    lengths.add_(1)
    eager_lengths.add_(1)
    step(caches[0], lengths)  # warm-up; a step repeated leaves the cache as it is
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step(caches[0], lengths)
        graphs.append((graph, y))
    for i in range(6):
        graph, y = graphs[i % 2]
        graph.replay()
        want = step(caches[1], eager_lengths)
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        assert torch.equal(caches[0].k_codes, caches[1].k_codes) and torch.equal(caches[0].v_codes, caches[1].v_codes)
        assert torch.equal(caches[0].k_scales, caches[1].k_scales) and torch.equal(caches[0].v_scales, caches[1].v_scales)
        lengths.add_(1)
        eager_lengths.add_(1)
        x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))


def test_two_streams(focus):
    """Calls on two streams at once, each on its own batch of one cache."""
    rng = np.random.default_rng(4)
    dim, heads = 128, 16
    c = focus.KVCache.zeros(128, 2, dim, 32, device=DEV)
    table = rng.permutation(128).astype(np.int32).reshape(4, 32)
    g = torch.Generator().manual_seed(5)
    n = 1000
    k, v = (torch.randn(4 * n, 2 * dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    lengths = np.full(4, n)
    focus.kv_cache_write(c, focus.KVBatch(dev(table), dev(lengths), dev(np.arange(5) * n), 4 * n), k, v)
    one = focus.KVBatch(dev(table), dev(lengths))
    many = focus.KVBatch(dev(table), dev(lengths), dev(np.arange(5) * 300), 1200)
    q1 = torch.randn(4, heads * dim, generator=g).to(torch.bfloat16).to(DEV)
    q2 = torch.randn(1200, heads * dim, generator=g).to(torch.bfloat16).to(DEV)
    w1, w2 = focus.kv_attention(c, one, q1), focus.kv_attention(c, many, q2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = [focus.kv_attention(c, one, q1), focus.kv_attention(c, many, q2), focus.kv_attention(c, one, q1)]
        torch.cuda.synchronize()
        for r in got:
            assert torch.equal(r[0], w1) and torch.equal(r[1], w2) and torch.equal(r[2], w1)


def test_binding_refusals(focus):
    c = focus.KVCache.zeros(4, 2, 64, 16, device=DEV)
    b = focus.KVBatch(dev([[0, 1], [2, 3]]), dev([3, 4]))
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device=DEV)
    bad = [lambda: focus.KVCache(c.k_codes, c.k_scales, c.k_codes, c.v_scales),
           lambda: focus.KVCache(c.k_codes, c.k_scales[:3], c.v_codes, c.v_scales),
           lambda: focus.KVCache.zeros(4, 2, 80, 16, device=DEV),
           lambda: focus.KVCache.zeros(4, 2, 64, 24, device=DEV),
           lambda: focus.KVBatch(dev([[0, 1]]), dev([3, 4])),
           lambda: focus.KVBatch(dev([[0, 1], [2, 3]]), dev([3, 4]), tokens=3),
           lambda: focus.KVBatch(dev([[0, 1], [2, 3]]), dev([3, 4]), dev([0, 1, 2])),
           lambda: focus.KVBatch(dev([[0, 1], [2, 3]]), dev([3, 4]), dev([0, 1]), 2),
           lambda: focus.KVBatch(dev([[0, 2], [1, 3]]).t(), dev([3, 4])),
           lambda: focus.kv_cache_write(c, b, x[:1], x),
           lambda: focus.kv_cache_write(c, b, x, x[:, :64]),
           lambda: focus.kv_cache_write(c, b, x, x, rope=torch.zeros(5, 128, device=DEV)),
           lambda: focus.kv_cache_write(c, b, x, x.cpu()),
           lambda: focus.kv_attention(c, b, x[:, :64]),
           lambda: focus.kv_attention(c, b, x, out=x[:1]),
           lambda: focus.kv_attention(c, b, torch.zeros(2, 132, dtype=torch.bfloat16, device=DEV)[:, :128]),
           lambda: focus.kv_cache_read(c, b, x[:1])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    for f in (lambda: focus.kv_cache_write(c, b, x.float(), x), lambda: focus.kv_attention(c, b, x.half()),
              lambda: focus.KVBatch(dev([[0, 1], [2, 3]]).long(), dev([3, 4])), lambda: focus.kv_attention(b, c, x)):
        with pytest.raises(TypeError):
            f()
    for kw in (dict(softcap=-1.0), dict(window=-1), dict(scale=float("nan"))):
        with pytest.raises(focus.FocusError):
            focus.kv_attention(c, b, x, **kw)
