"""Workloads of the long-context operators: block bounds, block selection, attention over the
selected blocks, and attention of a batch that shares a prefix, all beside the compressed cache.

Codes follow include/tq.h: bit planes [row][head][plane][slot][16] (4-bit values as nibbles
[row][head][slot][64]), float32 norms, and optionally a block table that maps a sequence's
tokens to pages of a pool.
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128
BLOCK = 64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELEM = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ constants of the codes

@functools.lru_cache(None)
def _matrices():
    """(rotation, sketch) in 64 bits: the sign-fixed Q of a Gaussian matrix, and a Gaussian."""
    g = np.random.default_rng(42).standard_normal((D, D))
    q, r = np.linalg.qr(g)
    return q * np.where(np.diag(r) < 0, -1.0, 1.0), np.random.default_rng(43).standard_normal((D, D))


@functools.lru_cache(None)
def _levels(bits):
    """Lloyd-Max levels of a coordinate of a uniform point on the sphere, by k-means on a grid."""
    t = (np.arange(200000) + 0.5) / 200000 * 1.6 - 0.8
    w = np.exp((D - 3) / 2 * np.log1p(-t * t))
    w0, w1 = np.concatenate([[0], np.cumsum(w)]), np.concatenate([[0], np.cumsum(w * t)])
    c = np.linspace(-2.5, 2.5, 1 << bits) / math.sqrt(D)
    for _ in range(3000):
        e = np.concatenate([[0], np.searchsorted(t, (c[1:] + c[:-1]) / 2), [len(t)]])
        n = np.diff(w1[e]) / np.diff(w0[e])
        if np.max(np.abs(n - c)) < 1e-12:
            break
        c = n
    return 0.5 * (c - c[::-1])


@functools.lru_cache(None)
def _on_gpu(name, dtype):
    a = {"pi": lambda: _matrices()[0], "s": lambda: _matrices()[1]}.get(name) or (lambda: _levels(int(name)))
    return torch.tensor(a(), dtype=dtype, device=DEV)


# ------------------------------------------------------------------ making inputs

def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _lens(n, low, high):
    """Ragged lengths in [low, high], the longest first; the same for every seed."""
    v = np.random.default_rng(2005 + n).integers(low, high, n, endpoint=True)
    v[0] = high
    return [int(x) for x in v]


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pack(bits):
    w = (1 << torch.arange(8, device=DEV)).to(torch.uint8)
    return (bits.to(torch.uint8).reshape(*bits.shape[:-1], D // 8, 8) * w).sum(-1, dtype=torch.uint8)


def _keys(rows, heads, tokens, gen):
    """Keys as long contexts have them: a drift from block to block and four loud channels."""
    x = torch.randn(rows, heads, tokens, D, generator=gen, device=DEV)
    nb = -(-tokens // BLOCK)
    drift = 0.5 * torch.randn(rows, heads, nb, 1, D, generator=gen, device=DEV)
    x += drift.expand(-1, -1, -1, BLOCK, -1).reshape(rows, heads, nb * BLOCK, D)[:, :, :tokens]
    x[..., torch.randperm(D, generator=gen, device=DEV)[:4]] *= 10
    return x


def _codes(rows, heads, cap, kbits, vbits, gen):
    """Codes of `cap` random tokens for each (row, head): the key's planes, signs and norms and
    the value's codes and norms, every slot written (slots past a length hold stale tokens)."""
    pi, s = _on_gpu("pi", torch.float32), _on_gpu("s", torch.float32)
    kc, vc = _on_gpu(str(kbits - 1), torch.float32), _on_gpu(str(vbits), torch.float32)
    m = s @ pi.T
    parts = []
    for r in range(rows):
        x = _keys(1, heads, cap, gen)[0].to(torch.bfloat16).float()
        xn = x.norm(dim=-1)
        y = (x / xn[..., None]) @ pi.T
        i = torch.bucketize(y, (kc[1:] + kc[:-1]) / 2)
        rho = y - kc[i]
        kidx = torch.stack([_pack((i >> p) & 1) for p in range(kbits - 1)], 1)
        sgn, rn = _pack(rho @ m.T >= 0), rho.norm(dim=-1) * xn
        del x, y, rho, i
        v = torch.randn(heads, cap, D, generator=gen, device=DEV).to(torch.bfloat16).float()
        vn = v.norm(dim=-1)
        j = torch.bucketize((v / vn[..., None]) @ pi.T, (vc[1:] + vc[:-1]) / 2)
        vidx = (j[..., 0::2] | (j[..., 1::2] << 4)).to(torch.uint8) if vbits == 4 else \
            torch.stack([_pack((j >> p) & 1) for p in range(vbits)], 1)
        parts.append((kidx, sgn, xn, rn, vidx, vn))
    names = ("kidx", "sgn", "xn", "rn", "vidx", "vn")
    return {k: torch.stack(t) for k, t in zip(names, zip(*parts))}


def _slots(name, t):
    """The dimension of an array of _codes (or of the bounds) that counts slots."""
    return t.dim() - (1 if name in ("xn", "rn", "vn") else 3 if name == "bounds" else 2)


def _to_pages(arrays, page, gen, before=()):
    """Pools and block tables for the flat arrays (and those of `before`, which come first in the
    same pool): the pages lie in a random order. -> pool, [tables]"""
    pool, tables = {}, []
    groups = list(before) + [arrays]
    for name in arrays:
        pages = []
        for g in groups:
            t = g[name]
            d = _slots(name, t)
            per = page // BLOCK if name == "bounds" else page
            t = t.unflatten(d, (t.shape[d] // per, per))
            pages.append(t.movedim(d, 1).flatten(0, 1))
        pool[name] = torch.cat(pages)
    order = torch.randperm(next(iter(pool.values())).shape[0], generator=gen, device=DEV)
    for name, t in pool.items():
        pool[name] = torch.empty_like(t).index_copy_(0, order, t)
    at = 0
    for g in groups:
        t = next(iter(g.values()))
        name = next(iter(g))
        rows, n = t.shape[0], t.shape[_slots(name, t)] // (page // BLOCK if name == "bounds" else page)
        tables.append(order[at:at + rows * n].view(rows, n).to(torch.int32))
        at += rows * n
    return pool, tables


def _round_up(n, to):
    return -(-n // to) * to


def _kept(scores, blocks, keep, first, last):
    """The blocks that a selection keeps, ascending, -1 behind them: `first` and `last` blocks of
    each sequence always, then the largest scores, ties to the lowest index."""
    nb = scores.shape[-1]
    at = torch.arange(nb, device=DEV)
    n = blocks.view(-1, 1, 1)
    forced = (at < first) | (at >= n - last)
    key = torch.where(at >= n, -math.inf, torch.where(forced, math.inf, scores))
    got = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :keep]
    got = torch.sort(torch.where(got < n, got, nb), dim=-1)[0]
    got = torch.where(got < nb, got, -1).to(torch.int32)
    return torch.nn.functional.pad(got, (0, keep - got.shape[-1]), value=-1)


def _bounds_of(x):
    """bf16 bounds [rows][heads][blocks][2][128] of whole blocks of bf16 values."""
    t = x.to(torch.bfloat16).unflatten(2, (-1, BLOCK))
    return torch.stack([t.amin(3), t.amax(3)], 3)


# ------------------------------------------------------------------ cases

def listed():
    b = dict(op="bounds", paged=0)
    s = dict(op="select", paged=0, first=1, last=2, dtype="bf16")
    a = dict(op="sparse", paged=0, out="bf16", dtype="bf16")
    p = dict(op="prefix", paged=0, out="bf16", dtype="bf16")
    return [
        # a serving step's new key of each of 32 sequences, folded into its block: launch-bound
        dict(b, name="bounds_append_b32", batch=32, kv=4, tokens=1, low=4096, high=16383, dtype="bf16"),
        # the prefill of one long context: bound by reading the keys
        dict(b, name="bounds_prefill_262k", batch=1, kv=8, tokens=262144, low=0, high=0, dtype="bf16"),
        # a ragged chunk of odd lengths behind odd histories, in a paged pool
        dict(b, name="bounds_ragged_f16_paged", batch=3, kv=4, tokens=5003, low=1, high=3333, dtype="f16", paged=256),
        # one sequence of 32K tokens
        dict(s, name="select_32k", batch=1, kv=4, group=7, low=32768, high=32768, keep=64),
        # one long context: the bounds of 4096 blocks a head
        dict(s, name="select_262k", batch=1, kv=8, group=4, low=262144, high=262144, keep=128),
        # a ragged serving batch
        dict(s, name="select_b32_paged", batch=32, kv=4, group=7, low=4096, high=16384, keep=32, dtype="f16", paged=256),
        # 8192 of 262144 tokens, 3-bit keys and 2-bit values
        dict(a, name="sparse_262k_keep128", batch=1, kv=8, group=4, low=262144, high=262144, keep=128, kbits=3, vbits=2),
        # 2048 tokens of each sequence of a ragged serving batch
        dict(a, name="sparse_b32_keep32_paged", batch=32, kv=4, group=7, low=4096, high=16384, keep=32, kbits=4, vbits=4, paged=256),
        # a short system prompt and four young sequences: latency
        dict(p, name="prefix_b4_1k", batch=4, kv=4, group=7, prefix=1000, low=1, high=100, kbits=3, vbits=4, out="f16"),
        # a serving batch behind one document
        dict(p, name="prefix_b32_32k", batch=32, kv=4, group=7, prefix=32768, low=1, high=512, kbits=3, vbits=4),
        # a few questions about one very long document
        dict(p, name="prefix_b8_262k", batch=8, kv=8, group=4, prefix=262144, low=0, high=1024, kbits=3, vbits=2),
        # a large batch, prefix and own tokens in one paged pool
        dict(p, name="prefix_b64_64k_paged", batch=64, kv=4, group=7, prefix=65536, low=16, high=1024, kbits=4, vbits=4, paged=256),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "prefix"])
    c = dict(op=op, kv=rng.choice([1, 2, 4, 8]), paged=rng.choice([0, 0, 64, 256]), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "bounds":
        c["batch"] = _log(rng, 1, 32)
        c["tokens"] = 1 if rng.random() < 0.3 else _log(rng, 2, 1500000 // (c["batch"] * c["kv"]))
        c["low"] = rng.randint(0, 3000)
        c["high"] = c["low"] + rng.randint(0, 5000)
        return c
    c["batch"], c["group"] = _log(rng, 1, 48), rng.randint(1, 8)
    if op == "select":
        c["high"] = _log(rng, 2500, min(262144, 2097152 // (c["batch"] * c["kv"])))
        c["low"] = rng.randint(1, c["high"])
        c["first"], c["last"] = rng.randint(0, 3), rng.randint(0, 4)
        c["keep"] = c["first"] + c["last"] + _log(rng, 4, min(256, c["high"] // (2 * BLOCK)))   # fewer than there are
        return c
    c["kbits"], c["vbits"], c["out"] = rng.randint(2, 5), rng.randint(1, 4), rng.choice(["bf16", "f16"])
    if op == "sparse":
        c["high"] = _log(rng, 100, min(131072, 1000000 // (c["batch"] * c["kv"])))
        c["low"] = rng.randint(0, c["high"])
        c["keep"] = _log(rng, 1, 160)
        return c
    c["prefix"] = _log(rng, 64, min(131072, 1000000 // c["kv"], 12000000 // (c["kv"] * c["batch"])))
    c["high"] = _log(rng, 1, 1500)
    c["low"] = rng.randint(0, c["high"])
    return c


# ------------------------------------------------------------------ inputs and handles

def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    batch, kv, page = c["batch"], c["kv"], c["paged"]
    st = {"case": c}
    lens = _lens(batch, c["low"], c["high"])
    if c["op"] == "bounds":
        # histories of `low` to `high` tokens whose bounds are there, and a chunk behind them
        tokens = c["tokens"]
        counts = _lens(batch, (tokens + 1) // 2, tokens)
        cap = _round_up(c["high"] + tokens, page or BLOCK)
        st["x"] = _keys(batch, kv, tokens, gen).to(TYPES[c["dtype"]])
        st["pos"], st["count"] = _int32(lens), _int32(counts)
        base = _keys(batch, kv, _round_up(c["high"] + 1, BLOCK), gen)
        arrays = {"bounds": torch.zeros(batch, kv, cap // BLOCK, 2, D, dtype=torch.bfloat16, device=DEV)}
        made = _bounds_of(base)[:, :, :cap // BLOCK]
        arrays["bounds"][:, :, :made.shape[2]] = made
    elif c["op"] == "select":
        cap = _round_up(c["high"], page or BLOCK)
        st["lens"] = _int32(lens)
        st["q"] = torch.randn(batch, kv * c["group"], D, generator=gen, device=DEV).to(TYPES[c["dtype"]])
        arrays = {"bounds": torch.cat([_bounds_of(_keys(1, kv, cap, gen)) for _ in range(batch)])}
    else:
        cap = _round_up(max(c["high"], 1), page or BLOCK)
        st["lens"] = _int32(lens)
        st["q"] = torch.randn(batch, kv * c["group"], D, generator=gen, device=DEV).to(TYPES[c["dtype"]])
        arrays = _codes(batch, kv, cap, c["kbits"], c["vbits"], gen)
        if c["op"] == "sparse":
            nb = (st["lens"].long() + BLOCK - 1) // BLOCK
            st["list"] = _kept(torch.rand(batch, kv, cap // BLOCK, generator=gen, device=DEV), nb, c["keep"], 1, 2)
    before = ()
    if c["op"] == "prefix":
        pcap = _round_up(c["prefix"], page or BLOCK)
        before = (_codes(1, kv, pcap, c["kbits"], c["vbits"], gen),)
        st["plen"] = _int32([c["prefix"]])
        st["prefix"], st["pcap"], st["ptable"] = before[0], pcap, None
    st["arrays"], st["table"], st["cap"] = arrays, None, cap
    if page:
        pool, tables = _to_pages(arrays, page, gen, before)
        st["arrays"], st["table"] = pool, tables[-1]
        if before:
            st["prefix"], st["ptable"] = pool, tables[0]
    if own:
        _handles(st)
    return st


@functools.lru_cache(None)
def _codec(keys, bits):
    from kv_cache_quantization_gb300 import _binding as B, api
    pi, s = _matrices()
    return api.Codec(B.TQ_PROD, bits, pi, s, _levels(bits - 1)) if keys else api.Codec(B.TQ_MSE, bits, pi, None, _levels(bits))


def _handles(st):
    """What a program of this framework keeps: codecs, cache objects, plans, output buffers."""
    from kv_cache_quantization_gb300 import api
    c, a = st["case"], st["arrays"]
    batch, kv, page = c["batch"], c["kv"], c["paged"]

    def pages(table, pool):
        return api.Pages(table, page, next(iter(pool.values())).shape[0]) if page else None

    at = pages(st["table"], a)
    if c["op"] in ("bounds", "select"):
        st["blocks"] = api.BlockBounds(a["bounds"], at)
        if c["op"] == "select":
            st["plan"] = api.SparsePlan(batch, kv * c["group"], kv, st["cap"], c["high"], c["keep"], c["first"], c["last"],
                                        q_dtype=st["q"].dtype)
            st["out"] = st["plan"].new_list()
        return
    st["kc"], st["vc"] = _codec(True, c["kbits"]), _codec(False, c["vbits"])

    def caches(x, p):
        return (api.ProdCache(x["kidx"], x["sgn"], x["xn"], x["rn"], p), api.MSECache(x["vidx"], x["vn"], c["vbits"], p))

    st["k"], st["v"] = caches(a, at)
    if c["op"] == "sparse":
        st["plan"] = api.SparsePlan(batch, kv * c["group"], kv, st["cap"], max(c["high"], 1), c["keep"], 0, 0,
                                    q_dtype=st["q"].dtype, out_dtype=TYPES[c["out"]])
    else:
        st["pk"], st["pv"] = caches(st["prefix"], pages(st["ptable"], st["prefix"]))
        st["plan"] = api.PrefixPlan(batch, kv * c["group"], kv, st["cap"], max(c["high"], 1), st["pcap"], c["prefix"],
                                    q_dtype=st["q"].dtype, out_dtype=TYPES[c["out"]])
    st["out"] = st["plan"].new_out()


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        from kv_cache_quantization_gb300 import api
        if op == "bounds":
            api.block_bounds(st["x"], st["blocks"], st["pos"], st["count"])
            return st["arrays"]["bounds"]
        if op == "select":
            return st["plan"].select(st["q"], st["blocks"], st["lens"], st["out"])
        if op == "sparse":
            return st["plan"].run(st["kc"], st["vc"], st["q"], st["k"], st["v"], st["lens"], st["list"], st["out"])
        return st["plan"].run(st["kc"], st["vc"], st["q"], st["pk"], st["pv"], st["plen"], st["k"], st["v"], st["lens"], st["out"])
    return {"bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse, "prefix": _plain_prefix}[op](st)


def _flat(arrays, table, names):
    """The arrays `names` in the flat layout, gathered from a pool where there is a table."""
    if table is None:
        return [arrays[n] for n in names]
    out = []
    for n in names:
        t = arrays[n][table.long()]                      # [row][page][head]...
        out.append(t.movedim(1, _slots(n, t) - 1).flatten(_slots(n, t) - 1, _slots(n, t)))
    return out


def _outward(x, up):
    """bf16 numbers nearest to x that are not below it (up) or not above it."""
    u = x.float().contiguous().view(torch.int32)
    cut = u & -65536
    away = ((u & 65535) != 0) & ((u >= 0) if up else (u < 0))
    return torch.where(away, cut + 65536, cut).view(torch.float32).to(torch.bfloat16)


def _plain_bounds(st):
    x, pos, count = st["x"].float(), st["pos"].long(), st["count"].long()
    batch, kv, tokens, _ = x.shape
    table, pool, nb = st["table"], st["arrays"]["bounds"], st["cap"] // BLOCK
    nt = (tokens + BLOCK - 2) // BLOCK + 1                # blocks that a chunk can touch
    slot = torch.arange(nt * BLOCK, device=DEV) - (pos % BLOCK)[:, None]      # token of each slot
    there = (slot >= 0) & (slot < count[:, None])
    got = x.gather(2, slot.clamp(0, tokens - 1)[:, None, :, None].expand(batch, kv, -1, D)).unflatten(2, (nt, BLOCK))
    m = there.view(batch, 1, nt, BLOCK, 1)
    lo, hi = torch.where(m, got, math.inf).amin(3), torch.where(m, got, -math.inf).amax(3)
    blk = (pos // BLOCK)[:, None] + torch.arange(nt, device=DEV)
    touched = there.view(batch, nt, BLOCK).any(-1)
    anew = there.view(batch, nt, BLOCK)[:, :, 0]          # slot 0 begins a block
    safe = blk.clamp(max=nb - 1)
    if table is None:
        row, at = torch.arange(batch, device=DEV)[:, None].expand(-1, nt), safe
    else:
        per = nb // table.shape[1]
        row, at = table.long().gather(1, safe // per), safe % per
    old = pool[row, :, at].transpose(1, 2)                # [batch][head][block][2][128]
    keep = ~anew[:, None, :, None, None]
    new = torch.stack([_outward(lo, False), _outward(hi, True)], 3)
    both = torch.stack([torch.minimum(old[..., 0, :], new[..., 0, :]), torch.maximum(old[..., 1, :], new[..., 1, :])], 3)
    new = torch.where(keep, both, new).transpose(1, 2)
    pool[row[touched], :, at[touched]] = new[touched]
    return pool


def _plain_select(st):
    c = st["case"]
    (b,) = _flat(st["arrays"], st["table"], ("bounds",))
    q = st["q"].double().unflatten(1, (c["kv"], c["group"]))
    both = torch.cat([q.clamp(max=0), q.clamp(min=0)], -1)               # of the lower and the upper bounds
    scores = (both @ b.double().flatten(3).transpose(2, 3)).amax(2)
    return _kept(scores, (st["lens"].long() + BLOCK - 1) // BLOCK, c["keep"], c["first"], c["last"])


def _bits(planes):
    return ((planes[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).flatten(-2)


def _index(codes, bits, dim):
    """Level indices from planes (stacked at `dim`) or nibbles."""
    if bits == 4 and codes.shape[-1] == 64:
        return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    w = (1 << torch.arange(codes.shape[dim], device=DEV, dtype=torch.int32))
    return (_bits(codes).int().movedim(dim, -1) * w).sum(-1, dtype=torch.int32)


def _rotated(st):
    c = st["case"]
    q = st["q"].float().unflatten(1, (c["kv"], c["group"]))
    return q @ _on_gpu("pi", torch.float32).T, q @ _on_gpu("s", torch.float32).T


def _logits(qp, qs, index, sgn, xn, rn, kbits):
    """Scores of rows of queries [..., rows, 128] with tokens [..., tokens, ...], scaled."""
    kc = _on_gpu(str(kbits - 1), torch.float32)
    main = qp @ kc[index].transpose(-1, -2)
    sketch = qs @ (2.0 * _bits(sgn).float() - 1.0).transpose(-1, -2)
    return (main * xn[..., None, :] + sketch * (math.sqrt(math.pi / 2) / D * rn[..., None, :])) / math.sqrt(D)


def _finish(p, vindex, vn, vbits):
    """Rotated output rows (not divided) of weights p with tokens of values."""
    return (p * vn[..., None, :]) @ _on_gpu(str(vbits), torch.float32)[vindex]


def _out(acc, total, c):
    o = torch.where(total > 0, acc / total, 0.0) @ _on_gpu("pi", torch.float32)
    return o.reshape(c["batch"], c["kv"] * c["group"], D).to(TYPES[c["out"]])


NAMES = ("kidx", "sgn", "xn", "rn", "vidx", "vn")


def _plain_sparse(st):
    c, lst = st["case"], st["list"].long()
    flat = _flat(st["arrays"], st["table"], NAMES)
    there = lst >= 0

    def take(name, t):
        d = _slots(name, t)
        t = t.unflatten(d, (-1, BLOCK))
        shape = [1] * t.dim()
        shape[0], shape[1], shape[d] = lst.shape
        size = list(t.shape)
        size[d] = lst.shape[2]
        return t.gather(d, lst.clamp(min=0).view(shape).expand(size)).flatten(d, d + 1)

    kidx, sgn, xn, rn, vidx, vn = (take(n, t) for n, t in zip(NAMES, flat))
    token = (lst[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(2)
    ok = (there[..., None].expand(*lst.shape, BLOCK).flatten(2) & (token < st["lens"].view(-1, 1, 1)))[:, :, None]
    qp, qs = _rotated(st)
    s = torch.where(ok, _logits(qp, qs, _index(kidx, c["kbits"] - 1, 2), sgn, xn, rn, c["kbits"]), -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    return _out(_finish(p, _index(vidx, c["vbits"], 2), vn, c["vbits"]), total, c)


def _plain_prefix(st):
    c = st["case"]
    qp, qs = _rotated(st)                                                 # [batch][kv][group][128]
    rows = [t.transpose(0, 1).flatten(1, 2) for t in (qp, qs)]            # [kv][batch·group][128]
    kidx, sgn, xn, rn, vidx, vn = (t[0] for t in _flat(st["prefix"], st["ptable"], NAMES))
    shared = _logits(*rows, _index(kidx, c["kbits"] - 1, 1), sgn, xn, rn, c["kbits"])
    shared = torch.where(torch.arange(st["pcap"], device=DEV) < st["plen"], shared, -math.inf)
    okidx, osgn, oxn, orn, ovidx, ovn = _flat(st["arrays"], st["table"], NAMES)
    mine = _logits(qp, qs, _index(okidx, c["kbits"] - 1, 2), osgn, oxn, orn, c["kbits"])
    mine = torch.where(torch.arange(st["cap"], device=DEV) < st["lens"].view(-1, 1, 1, 1), mine, -math.inf)
    shared = shared.unflatten(1, (c["batch"], c["group"])).transpose(0, 1)
    top = torch.maximum(shared.amax(-1, keepdim=True), mine.amax(-1, keepdim=True)).clamp(min=-1e30)
    ps, pm = torch.exp(shared - top), torch.exp(mine - top)
    total = ps.sum(-1, keepdim=True) + pm.sum(-1, keepdim=True)
    acc = _finish(ps.transpose(0, 1).flatten(1, 2), _index(vidx, c["vbits"], 1), vn, c["vbits"])
    acc = acc.unflatten(1, (c["batch"], c["group"])).transpose(0, 1)
    acc = acc + _finish(pm, _index(ovidx, c["vbits"], 2), ovn, c["vbits"])
    return _out(acc, total, c)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    batch, kv = c["batch"], c["kv"]
    lens = _lens(batch, c["low"], c["high"])
    if c["op"] == "bounds":
        counts = _lens(batch, (c["tokens"] + 1) // 2, c["tokens"])
        n, w = sum(counts), 0
        for p, k in zip(lens, counts):      # each touched block is written, one that goes on is read
            w += (p + k - 1) // BLOCK - p // BLOCK + 1 + (1 if p % BLOCK else 0)
        return {"bytes": kv * (n * D * ELEM[c["dtype"]] + w * 2 * D * 2), "flops": 2 * kv * n * D}
    rows = batch * kv * c["group"]
    if c["op"] == "select":
        n = sum(-(-x // BLOCK) for x in lens)
        return {"bytes": kv * n * 2 * D * 2 + rows * D * ELEM[c["dtype"]] + batch * kv * c["keep"] * 4,
                "flops": 2 * 2 * D * kv * n * c["group"]}
    token = (c["kbits"] - 1) * 16 + 16 + 8 + c["vbits"] * 16 + 4
    io = rows * D * (ELEM[c["dtype"]] + ELEM[c["out"]])
    each = 2 * 3 * D * c["group"]           # scores with two halves of the code, and values
    if c["op"] == "sparse":
        n = sum(x if -(-x // BLOCK) <= c["keep"] else (c["keep"] - 1) * BLOCK + (x - 1) % BLOCK + 1 for x in lens)
        return {"bytes": kv * n * token + io + batch * kv * c["keep"] * 4, "flops": each * kv * n}
    return {"bytes": kv * (sum(lens) + c["prefix"]) * token + io,
            "flops": each * kv * (sum(lens) + batch * c["prefix"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    f64 = torch.float64
    batch, kv, group = c["batch"], c["kv"], c.get("group")
    lens = st["lens"].tolist() if "lens" in st else None

    def pieces(arrays, table, b, h, blocks, name):
        """The slots of the listed 64-token blocks of sequence b, head h, token after token."""
        t = arrays[name]
        if table is None:
            one = t[b, h]
        else:
            one = t[table[b].long(), h]
            d = _slots(name, t) - 2
            one = one.movedim(0, d).flatten(d, d + 1)
        d = _slots(name, t) - 2
        one = one.movedim(d, 0)
        return one.unflatten(0, (-1, BLOCK))[blocks].flatten(0, 1) if name != "bounds" else one

    if c["op"] == "bounds":
        pool, table = st["arrays"]["bounds"].double(), st["table"]
        flat = pool.clone()
        for b, (p, n) in enumerate(zip(st["pos"].tolist(), st["count"].tolist())):
            x = st["x"][b, :, :n].double()
            for blk in range(p // BLOCK, (p + n - 1) // BLOCK + 1):
                t0, t1 = blk * BLOCK - p, (blk + 1) * BLOCK - p
                lo, hi = x[:, max(t0, 0):t1].amin(1), x[:, max(t0, 0):t1].amax(1)
                per = st["cap"] // BLOCK // (1 if table is None else table.shape[1])
                row, at = (b, blk) if table is None else (int(table[b, blk // per]), blk % per)
                if t0 < 0:
                    lo, hi = torch.minimum(lo, pool[row, :, at, 0]), torch.maximum(hi, pool[row, :, at, 1])
                flat[row, :, at, 0], flat[row, :, at, 1] = lo, hi
        return flat
    if c["op"] == "select":
        got = torch.full((batch, kv, c["keep"]), -1, dtype=torch.int32)
        for b in range(batch):
            n = -(-lens[b] // BLOCK)
            for h in range(kv):
                t = pieces(st["arrays"], st["table"], b, h, None, "bounds")[:n].double()
                q = st["q"][b, h * group:(h + 1) * group, None].double()
                s = torch.maximum(q * t[:, 0], q * t[:, 1]).sum(-1).amax(0).tolist()
                sure = set(range(min(c["first"], n))) | set(range(max(0, n - c["last"]), n))
                rest = sorted((i for i in range(n) if i not in sure), key=lambda i: (-s[i], i))
                kept = sorted(sure | set(rest[:c["keep"] - len(sure)])) if n > c["keep"] else range(n)
                got[b, h, :len(kept)] = torch.tensor(list(kept), dtype=torch.int32)
        return got.to(DEV)
    pi, s = (torch.tensor(m, device=DEV) for m in _matrices())
    kl, vl = (torch.tensor(_levels(n), device=DEV) for n in (c["kbits"] - 1, c["vbits"]))
    shift = torch.arange(8, device=DEV, dtype=torch.uint8)

    def bits(t):
        return (t.unsqueeze(-1).bitwise_right_shift(shift) % 2).reshape(*t.shape[:-1], D).long()

    def tokens(arrays, table, b, h, n, blocks=None):
        """Dequantised keys and values [n][128] of a sequence's tokens, or of those of some blocks."""
        blocks = torch.arange(-(-n // BLOCK), device=DEV) if blocks is None else blocks
        live = (blocks[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten() < n
        kidx, sgn, xn, rn, vidx, vn = (pieces(arrays, table, b, h, blocks, x)[live] for x in NAMES)
        i = sum(bits(kidx[:, p]) << p for p in range(c["kbits"] - 1))
        if c["vbits"] == 4:
            j = torch.stack([vidx % 16, vidx // 16], 2).reshape(-1, D).long()
        else:
            j = sum(bits(vidx[:, p]) << p for p in range(c["vbits"]))
        k = xn.double()[:, None] * (kl[i] @ pi) + rn.double()[:, None] * math.sqrt(math.pi / 2) / D * ((2 * bits(sgn) - 1).to(f64) @ s)
        return k, vn.double()[:, None] * (vl[j] @ pi)

    out = torch.zeros(batch, kv * group, D, dtype=f64, device=DEV)
    for h in range(kv):
        shared = tokens(st["prefix"], st["ptable"], 0, h, c["prefix"]) if c["op"] == "prefix" else None
        for b in range(batch):
            if c["op"] == "prefix":
                k, v = (torch.cat(p) for p in zip(shared, tokens(st["arrays"], st["table"], b, h, lens[b])))
            else:
                lst = st["list"][b, h].long()
                k, v = tokens(st["arrays"], st["table"], b, h, lens[b], lst[lst >= 0])
            if len(k):
                q = st["q"][b, h * group:(h + 1) * group].double()
                out[b, h * group:(h + 1) * group] = torch.softmax(q @ k.T / math.sqrt(D), -1) @ v
    return out
