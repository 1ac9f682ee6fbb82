"""Measured cases of the paged 8-bit cache of keys and values: writing a step's
keys and values into it, reading it back, and the attention over it.

``run`` has two forms.  With ``own`` false it computes an operator from
elementary torch operations in binary32, rounded once at the end, with ``own``
true it makes the calls of ``fp4_post_weight_amd``.

The cache.  A page holds ``page`` consecutive tokens of one sequence; per page
and key/value head it has E4M3 codes of the keys [page, head_dim], E4M3 codes
of the values [head_dim, page] and one E8M0 scale byte for each of the two:
    S = 2^e, e the least integer with max|x| <= 448 * 2^e, -127 <= e <= 119
    code = E4M3(clamp(x / S, -448, 448)), nearest, ties to even
over the page's tokens; a page that gains tokens keeps the larger exponent, and
its older codes move to it (E4M3(code * 2^(e_old - e))).

The batch.  Sequence b has rows cu[b] .. cu[b+1]-1 of the step's tensors; they
are its last ones, row cu[b+1]-1 at position lengths[b]-1, and token j of the
sequence lies in page table[b, j // page] at j % page.

Rotation (where a table is given): the pairs (x[i], x[i + head_dim/2]) of the
keys, and of the queries, turn by the angle of their position, whose cosines
and sines are the table's row.
"""
import math
import random

import torch

own = False


# rows: the most new tokens of a sequence (0: every token, of a read); singles:
# how many sequences have one row; pattern: seed of the lengths and rows.

def listed():
    return [
        # one decoded token of a small model's layer goes into the cache
        {"name": "write 1 seq, 8x64", "op": "write", "sequences": 1, "longest": 77, "rows": 1, "singles": 1,
         "kv_heads": 8, "head_dim": 64, "page": 16, "rope": True, "pattern": 1},
        # a decode batch of 128 requests of different lengths
        {"name": "write 128 seqs, 8x128", "op": "write", "sequences": 128, "longest": 4096, "rows": 1, "singles": 128,
         "kv_heads": 8, "head_dim": 128, "page": 64, "rope": True, "pattern": 2},
        # prompts of different lengths, some of them chunks behind earlier ones
        {"name": "write prompts up to 8191, 8x128", "op": "write", "sequences": 7, "longest": 8191, "rows": 8191,
         "singles": 0, "kv_heads": 8, "head_dim": 128, "page": 64, "rope": True, "pattern": 3},
        # a short prefix is taken out again
        {"name": "read 333 tokens, 8x64", "op": "read", "sequences": 1, "longest": 333, "rows": 0, "singles": 0,
         "kv_heads": 8, "head_dim": 64, "page": 16, "pattern": 4},
        # 16 long requests move to another device or format
        {"name": "read 16 seqs up to 16384, 8x128", "op": "read", "sequences": 16, "longest": 16384, "rows": 0,
         "singles": 0, "kv_heads": 8, "head_dim": 128, "page": 128, "pattern": 5},
        # one decoded token of a short conversation
        {"name": "decode 1 x 333, 32/8x128", "op": "attention", "sequences": 1, "longest": 333, "rows": 1,
         "singles": 1, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "rope": True, "window": 0, "cap": 0.0,
         "pattern": 6},
        # one decoded token behind a long document
        {"name": "decode 1 x 131072, 64/8x128", "op": "attention", "sequences": 1, "longest": 131072, "rows": 1,
         "singles": 1, "heads": 64, "kv_heads": 8, "head_dim": 128, "page": 64, "rope": True, "window": 0, "cap": 0.0,
         "pattern": 7},
        # a decode batch of requests of very different lengths
        {"name": "decode 64 up to 16384, 32/8x128", "op": "attention", "sequences": 64, "longest": 16384, "rows": 1,
         "singles": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 32, "rope": False, "window": 0,
         "cap": 0.0, "pattern": 8},
        # a decode batch with a sliding window and capped scores, narrow heads
        {"name": "decode 33 up to 5000, 32/8x64, window 1000, cap 30", "op": "attention", "sequences": 33,
         "longest": 5000, "rows": 1, "singles": 33, "heads": 32, "kv_heads": 8, "head_dim": 64, "page": 16,
         "rope": True, "window": 1000, "cap": 30.0, "pattern": 9},
        # a long prompt in one piece
        {"name": "prompt 8192, 32/8x128", "op": "attention", "sequences": 1, "longest": 8192, "rows": 8192,
         "singles": 0, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "rope": True, "window": 0, "cap": 0.0,
         "pattern": 10},
        # chunks of prompts behind what the cache already holds of them
        {"name": "chunks of 5 up to 700 of 8192, 64/8x128", "op": "attention", "sequences": 5, "longest": 8192,
         "rows": 700, "singles": 0, "heads": 64, "kv_heads": 8, "head_dim": 128, "page": 128, "rope": False,
         "window": 0, "cap": 0.0, "pattern": 11},
        # a serving step: requests that decode beside prompts that come in
        {"name": "mixed 43 up to 2000, 32/8x64", "op": "attention", "sequences": 43, "longest": 2000, "rows": 500,
         "singles": 40, "heads": 32, "kv_heads": 8, "head_dim": 64, "page": 16, "rope": True, "window": 0, "cap": 0.0,
         "pattern": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    c = {"op": rng.choice(["write", "read", "attention", "attention"])}
    c["kv_heads"] = rng.choice([1, 2, 4, 5, 8, 8])
    c["head_dim"] = rng.choice([64, 128])
    c["page"] = rng.choice([16, 32, 64, 128])
    c["pattern"] = rng.randrange(1 << 30)
    width = c["kv_heads"] * c["head_dim"]
    if c["op"] != "attention":
        c["sequences"] = _log_int(rng, 1, 128)
        # at most about 262144 tokens of 1024 in the cache
        c["longest"] = _log_int(rng, 1, max(1, min(16384, 262144 * 1024 // (width * c["sequences"]))))
        c["rows"] = c["singles"] = 0
        if c["op"] == "write":
            c["rope"] = rng.random() < 0.7
            c["rows"] = rng.choice([1, _log_int(rng, 1, min(8192, c["longest"]))])
            c["rows"] = max(1, min(c["rows"], 16384 // c["sequences"]))
            c["singles"] = c["sequences"] if c["rows"] == 1 else rng.randrange(c["sequences"])
        return c
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 7, 8])
    c["sequences"] = _log_int(rng, 1, 64)
    # the cache as a padded batch: at most 64 x 16384 tokens of 1024 values
    c["longest"] = _log_int(rng, 1, max(1, min(131072, 64 * 16384 * 1024 // (width * c["sequences"]))))
    # rows x keys x heads: at most 8192 x 8192 x 32
    most = 8192 * 8192 * 32 // (c["sequences"] * c["longest"] * c["heads"])
    c["rows"] = rng.choice([1, _log_int(rng, 1, max(1, min(8192, c["longest"], most)))])
    c["singles"] = c["sequences"] if c["rows"] == 1 else rng.randrange(c["sequences"])
    c["rope"] = rng.random() < 0.5
    c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    return c


def _shape(case):
    """(rows, lengths) of every sequence, from the case alone."""
    rng = random.Random(case["pattern"])
    n, longest = case["sequences"], case["longest"]
    lengths = [longest] + [rng.randint(1, longest) for _ in range(n - 1)]
    if case["op"] == "read":
        return list(lengths), lengths
    rows = [1 if i >= n - case["singles"] else min(lengths[i], case["rows"] if i == 0 else rng.randint(1, case["rows"]))
            for i in range(n)]
    return rows, lengths


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _device():
    return torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _exponent(amax):
    """The scale exponent of a page whose largest magnitude is amax."""
    f, x = torch.frexp(amax)
    e = x.float() - 9.0 + (f > 0.875).float()
    return torch.where(amax == 0, torch.full_like(e, -127.0), e).clamp(-127.0, 119.0)


def _pages(gen, pages, heads, page, dim):
    """Pages full of stored tokens: codes [pages, heads, page, dim], exponents."""
    x = _normal(gen, pages, heads, page, dim)
    x.mul_(torch.exp(0.4 * _normal(gen, heads, 1, dim)))
    e = _exponent(x.abs().amax((2, 3)))
    codes = x.mul_(torch.exp2(-e)[..., None, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127.0).to(torch.uint8)


def _table_of_angles(positions, dim, dev):
    freq = 500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=dev) / dim)
    angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, lengths = _shape(case)
    page, dim, kvh = case["page"], case["head_dim"], case["kv_heads"]
    counts = [-(-n // page) for n in lengths]
    total, width = sum(counts), max(counts)
    st = dict(case)
    st["tokens"] = sum(rows)
    # pages lie anywhere in the cache; entries behind a sequence's last page are 0
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(counts), width, dtype=torch.int32, device=dev)
    held = torch.arange(width, device=dev)[None] < torch.tensor(counts, device=dev)[:, None]
    table[held] = order
    st["table"] = table
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    at = [0]
    for n in rows:
        at.append(at[-1] + n)
    st["cu"] = torch.tensor(at, dtype=torch.int32, device=dev)
    st["kc"], st["ks"] = _pages(gen, total, kvh, page, dim)
    vc, st["vs"] = _pages(gen, total, kvh, page, dim)
    st["vc"] = vc.transpose(2, 3).contiguous()
    st["angles"] = _table_of_angles(case["longest"], dim, dev) if case.get("rope") else None
    T = st["tokens"]
    if case["op"] == "write":
        # k and v as parts of one product's rows
        both = _normal(gen, T, 2 * kvh * dim) * torch.exp(0.4 * _normal(gen, 2 * kvh * dim))
        both = (both * torch.exp(0.3 * _normal(gen, T, 1))).to(torch.bfloat16)
        st["k"], st["v"] = both[:, :kvh * dim], both[:, kvh * dim:]
    if case["op"] == "attention":
        st["q"] = (1.5 * _normal(gen, T, case["heads"] * dim)).to(torch.bfloat16)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _places(st):
    """Sequence and position of every row."""
    row = torch.arange(st["tokens"], device=st["cu"].device)
    seq = torch.searchsorted(st["cu"][1:], row.to(torch.int32), right=True)
    return seq, st["lengths"][seq].long() - st["cu"][seq + 1] + row


def _turn(x, angles, pos):
    """x [rows, heads, dim] turned by the angles of its positions."""
    half = x.shape[-1] // 2
    c, s = angles[pos, None, :half], angles[pos, None, half:]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127.0)[..., None, None]


def _plain_write(st):
    page, dim, kvh = st["page"], st["head_dim"], st["kv_heads"]
    seq, pos = _places(st)
    at, off = st["table"][seq, pos // page].long(), pos % page
    first = st["lengths"].long() - (st["cu"][1:] - st["cu"][:-1])
    first_page = st["table"][torch.arange(len(first), device=first.device), first // page].long()
    older = torch.arange(page, device=first.device)[None] < (first % page)[:, None]
    k = st["k"].float().view(-1, kvh, dim)
    k = k if st["angles"] is None else _turn(k, st["angles"], pos)
    v = st["v"].float().view(-1, kvh, dim)
    # the values' codes with their tokens in rows: a view of [dim, page]
    k_codes, v_codes = st["kc"], st["vc"].transpose(2, 3)
    _plain_write_one(k, k_codes, st["ks"], at, off, first, first_page, older, page)
    _plain_write_one(v, v_codes, st["vs"], at, off, first, first_page, older, page)
    return _stored(st)


def _plain_write_one(x, codes, scales, at, off, first, first_page, older, page):
    index = at[:, None].expand(-1, x.shape[1])
    amax = torch.zeros(scales.shape, device=x.device).scatter_reduce_(0, index, x.abs().amax(-1), "amax")
    e = _exponent(amax)
    # the first page of a sequence's new tokens may hold older ones
    e_old = scales[first_page].float() - 127.0
    e_first = torch.where((first % page > 0)[:, None], torch.maximum(e[first_page], e_old), e[first_page])
    e[first_page] = e_first
    old = codes[first_page]
    moved = old.view(torch.float8_e4m3fn).float() * torch.exp2(e_old - e_first)[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[first_page] = torch.where(older[:, None, :, None], moved, old)
    new = (x * torch.exp2(-e[at])[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    codes[at, :, off] = new.view(torch.uint8)
    scales[at] = (e[at] + 127.0).to(torch.uint8)


def _stored(st):
    return {"k": st["kc"].view(torch.float8_e4m3fn), "ks": st["ks"].view(torch.float8_e8m0fnu),
            "v": st["vc"].view(torch.float8_e4m3fn), "vs": st["vs"].view(torch.float8_e8m0fnu)}


def _plain_read(st):
    seq, pos = _places(st)
    at, off = st["table"][seq, pos // st["page"]].long(), pos % st["page"]
    k = st["kc"][at, :, off].view(torch.float8_e4m3fn).float() * torch.exp2(st["ks"][at].float() - 127.0)[..., None]
    v = st["vc"][at, :, :, off].view(torch.float8_e4m3fn).float() * torch.exp2(st["vs"][at].float() - 127.0)[..., None]
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_attention(st):
    page, dim, kvh = st["page"], st["head_dim"], st["kv_heads"]
    group = st["heads"] // kvh
    n = st["sequences"]
    seq, pos = _places(st)
    q = st["q"].float().view(-1, st["heads"], dim)
    q = q if st["angles"] is None else _turn(q, st["angles"], pos)
    # rows and cache as padded batches: [n, kvh, rows, group, dim] and [n, kvh, keys, dim]
    most = st["rows"]
    slot = torch.arange(st["tokens"], device=q.device) - st["cu"][seq]
    qb = torch.zeros(n, most, kvh, group, dim, device=q.device)
    qb[seq, slot] = q.view(-1, kvh, group, dim)
    qb = qb.permute(0, 2, 1, 3, 4).reshape(n, kvh, most * group, dim)
    table = st["table"].long()
    keys = table.shape[1] * page
    k = _values(st["kc"][table], st["ks"][table]).transpose(1, 2).reshape(n, kvh, keys, dim)
    s = torch.matmul(qb, k.transpose(2, 3).contiguous()).mul_(dim ** -0.5)
    del k
    if st["cap"] > 0:
        s = s.div_(st["cap"]).tanh_().mul_(st["cap"])
    rows = st["cu"][1:] - st["cu"][:-1]
    last = (st["lengths"] - rows)[:, None] + torch.arange(most, device=q.device)
    j = torch.arange(keys, device=q.device)
    seen = (j <= last[..., None]) & (j < st["lengths"][:, None, None])
    if st["window"] > 0:
        seen &= j > last[..., None] - st["window"]
    s = s.view(n, kvh, most, group, keys).masked_fill_(~seen[:, None, :, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(st["vc"][table], st["vs"][table]).permute(0, 2, 1, 4, 3).reshape(n, kvh, keys, dim)
    y = torch.matmul(p.view(n, kvh, most * group, keys), v).view(n, kvh, most, group, dim).div_(total)
    y = y.permute(0, 2, 1, 3, 4)[seq, slot]
    return y.reshape(st["tokens"], st["heads"] * dim).to(torch.bfloat16)


def _plain(st):
    if st["op"] == "write":
        return _plain_write(st)
    return _plain_read(st) if st["op"] == "read" else _plain_attention(st)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own(st):
    import fp4_post_weight_amd as focus
    cache = focus.KVCache(st["kc"], st["ks"], st["vc"], st["vs"])
    # one row per sequence needs no cu
    batch = focus.KVBatch(st["table"], st["lengths"]) if st["rows"] == 1 else \
        focus.KVBatch(st["table"], st["lengths"], st["cu"], st["tokens"])
    if st["op"] == "write":
        focus.kv_cache_write(cache, batch, st["k"], st["v"], rope=st["angles"])
        return _stored(st)
    if st["op"] == "read":
        return focus.kv_cache_read(cache, batch)
    return focus.kv_attention(cache, batch, st["q"], rope=st["angles"], window=st["window"], softcap=st["cap"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------

def work(case):
    rows, lengths = _shape(case)
    page, width = case["page"], case["kv_heads"] * case["head_dim"]
    tokens = sum(rows)
    turned = tokens * case["head_dim"] * 4 if case.get("rope") else 0
    if case["op"] in ("write", "read"):
        # k and v in 16 bits on one side, 8 bits and the scales on the other
        pages = sum((n - 1) // page - (n - r) // page + 1 for r, n in zip(rows, lengths))
        return {"bytes": tokens * width * 6 + 2 * pages * case["kv_heads"] + turned, "flops": 8.0 * tokens * width}
    pairs = held = 0
    for r, n in zip(rows, lengths):
        w = case["window"] or n
        # row i sees the keys up to its position, w at most
        seen = [min(p + 1, w) for p in range(n - r, n)]
        pairs += sum(seen)
        held += min(n, w + r - 1)
    pages = sum(-(-n // page) for n in lengths)
    size = 2 * (held * width + pages * case["kv_heads"]) + 4 * tokens * case["heads"] * case["head_dim"] + turned
    return {"bytes": size, "flops": 4.0 * pairs * case["heads"] * case["head_dim"]}


def _grid(x):
    """The nearest E4M3 values of x (binary64), ties to even."""
    x = x.clamp(-448.0, 448.0)
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(x / unit) * unit


def _power(top):
    """2^e of the least e with top <= 448 * 2^e, within E8M0 and 119."""
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0))
    # the logarithm is off by a rounding at most: settle it by the products
    e = torch.where(top <= 448.0 * torch.exp2(e - 1.0), e - 1.0, e)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1.0, e)
    return torch.exp2(e.clamp(-127.0, 119.0))


def _rotated(x, st, pos):
    if st["angles"] is None:
        return x
    c, s = st["angles"][pos].double().chunk(2, -1)
    z = torch.complex(*x.chunk(2, -1)) * torch.complex(c, s)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_write(st, rows, lengths):
    page, kvh, dim = st["page"], st["kv_heads"], st["head_dim"]
    out = {}
    for name, codes, scales in (("k", st["kc"], st["ks"]), ("v", st["vc"], st["vs"])):
        values = codes.view(torch.float8_e4m3fn).double()
        power = torch.pow(2.0, scales.double() - 127.0)
        tokens = values if name == "k" else values.transpose(2, 3)
        x = st[name].double().view(-1, kvh, dim)
        begin = 0
        for b, (r, n) in enumerate(zip(rows, lengths)):
            pos = torch.arange(n - r, n, device=x.device)
            part = x[begin:begin + r]
            part = _rotated(part, st, pos) if name == "k" else part
            begin += r
            first = (n - r) // page
            for p in range(first, (n - 1) // page + 1):
                where = int(st["table"][b, p])
                lo, hi = max(n - r, p * page), min(n, (p + 1) * page)
                mine = part[lo - (n - r):hi - (n - r)]
                now = _power(mine.abs().amax((0, 2)))
                held = lo - p * page
                if held > 0:
                    now = torch.maximum(now, power[where])
                    tokens[where, :, :held] = _grid(tokens[where, :, :held] * (power[where] / now)[:, None, None])
                tokens[where, :, held:hi - p * page] = _grid(mine / now[None, :, None]).transpose(0, 1)
                power[where] = now
        out[name], out[name + "s"] = values, power
    return out


def exact(case, seed):
    st = prepare(case, seed)
    rows, lengths = _shape(case)
    if case["op"] == "write":
        return _exact_write(st, rows, lengths)
    page, kvh, dim = case["page"], case["kv_heads"], case["head_dim"]
    group = case["heads"] // kvh if case["op"] == "attention" else 0
    parts = []
    begin = 0
    for b, (r, n) in enumerate(zip(rows, lengths)):
        where = st["table"][b, :-(-n // page)].long()
        k = st["kc"][where].view(torch.float8_e4m3fn).double() * torch.pow(2.0, st["ks"][where].double() - 127.0)[..., None, None]
        v = st["vc"][where].view(torch.float8_e4m3fn).double() * torch.pow(2.0, st["vs"][where].double() - 127.0)[..., None, None]
        # [tokens, heads, dim]
        k = k.permute(0, 2, 1, 3).reshape(-1, kvh, dim)[:n]
        v = v.permute(0, 3, 1, 2).reshape(-1, kvh, dim)[:n]
        if case["op"] == "read":
            parts.append((k, v))
            continue
        pos = torch.arange(n - r, n, device=k.device)
        q = _rotated(st["q"][begin:begin + r].double().view(r, -1, dim), st, pos)
        begin += r
        j = torch.arange(n, device=k.device)[None]
        hidden = j > pos[:, None]
        if case["window"]:
            hidden |= j <= pos[:, None] - case["window"]
        y = torch.empty(r, kvh * group, dim, dtype=torch.float64, device=k.device)
        for h in range(kvh * group):
            s = torch.mm(q[:, h].contiguous(), k[:, h // group].t().contiguous()) / math.sqrt(dim)
            if case["cap"]:
                s = torch.tanh(s / case["cap"]) * case["cap"]
            p = torch.softmax(s.masked_fill_(hidden, -math.inf), -1)
            y[:, h] = torch.mm(p, v[:, h // group].contiguous())
        parts.append(y.reshape(r, -1))
    if case["op"] == "read":
        return torch.cat([k for k, _ in parts]), torch.cat([v for _, v in parts])
    return torch.cat(parts)
