"""Workloads of what stands around the compressed cache when prompts are taken in and tokens are
drafted: rotary positions of queries and keys, attention of packed prompts on exact keys and values,
attention of a tree of drafted tokens over the compressed cache, keeping the accepted ones of them,
and copying pages.

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
NAMES = ("kidx", "sgn", "xn", "rn", "vidx", "vn")


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


def _lens(n, low, high, salt=0):
    """Ragged lengths in [low, high], the longest first; the same for every seed."""
    v = np.random.default_rng(2005 + n + salt).integers(low, high, n, endpoint=True)
    v[0] = high
    return [int(x) for x in v]


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(lens):
    return _int32(np.concatenate([[0], np.cumsum(lens)]).tolist())


def _round_up(n, to):
    return -(-n // to) * to


def _loud(shape, gen, dtype):
    """Vectors whose channels have scales of their own, four of them loud."""
    x = torch.randn(*shape, D, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(D, generator=gen, device=DEV))
    x[..., torch.randperm(D, generator=gen, device=DEV)[:4]] *= 5
    return x.to(dtype)


def _pack(bits):
    w = (1 << torch.arange(8, device=DEV)).to(torch.uint8)
    return (bits.to(torch.uint8).reshape(*bits.shape[:-1], D // 8, 8) * w).sum(-1, dtype=torch.uint8)


def _codes(rows, heads, cap, kbits, vbits, gen):
    """Codes of `cap` random tokens for each (row, head): the key's planes, signs and norms and
    the value's codes and norms, every slot written (slots past a length hold stale tokens)."""
    pi, s = _on_gpu("pi", torch.float32), _on_gpu("s", torch.float32)
    kc, vc = _on_gpu(str(kbits - 1), torch.float32), _on_gpu(str(vbits), torch.float32)
    m = s @ pi.T
    parts = []
    for r in range(rows):
        x = _loud((heads, cap), gen, torch.bfloat16).float()
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
    return {k: torch.stack(t) for k, t in zip(NAMES, zip(*parts))}


def _noise(rows, heads, slots, kbits, vbits, gen):
    """Arrays of the same layout with random bits and norms, for calls that only move codes."""
    def byte(*shape):
        return torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)

    def norm():
        return 1 + torch.rand(rows, heads, slots, generator=gen, device=DEV)

    vidx = byte(rows, heads, slots, 64) if vbits == 4 else byte(rows, heads, vbits, slots, 16)
    return dict(zip(NAMES, (byte(rows, heads, kbits - 1, slots, 16), byte(rows, heads, slots, 16), norm(), norm(),
                            vidx, norm())))


def _slots(name, t):
    """The dimension of an array of _codes that counts slots."""
    return t.dim() - (1 if name in ("xn", "rn", "vn") else 2)


def _to_pages(arrays, page, gen):
    """Pool and block table for the flat arrays: the pages lie in a random order."""
    pool, rows, per = {}, arrays["xn"].shape[0], arrays["xn"].shape[2] // page
    order = torch.randperm(rows * per, generator=gen, device=DEV)
    for name, t in arrays.items():
        d = _slots(name, t)
        t = t.unflatten(d, (per, page)).movedim(d, 1).flatten(0, 1)
        pool[name] = torch.empty_like(t).index_copy_(0, order, t)
    return pool, order.view(rows, per).to(torch.int32)


def _tree(batch, nodes, gen):
    """Ancestor masks of drafted trees, bit j of node i: i attends node j (itself among them). A
    node's parent is one of the eight before it."""
    up = torch.randint(0, 8, (batch, nodes), generator=gen, device=DEV)
    at = torch.arange(nodes, device=DEV)
    parent = torch.where(at > 0, (at - 1 - up).clamp(min=0), -1)
    step = (parent[..., None] == at).double()                    # node -> its parent
    eye = torch.eye(nodes, dtype=torch.float64, device=DEV)
    reach = ((eye + step) > 0).double()
    for _ in range(max(1, math.ceil(math.log2(nodes + 1)))):
        reach = ((reach @ reach) > 0).double()
    return (reach.long() << at).sum(-1)                          # (bit 63 makes the number negative)


# ------------------------------------------------------------------ cases

def listed():
    r = dict(op="rotary", inter=False, scaling="none")
    p = dict(op="prompt", causal=True, fused=False)
    t = dict(op="tree", paged=0, out="bf16", dtype="bf16")
    return [
        # a decode step's queries and keys of 32 sequences anywhere in long contexts: launch-bound
        dict(r, name="rotary_step_b32", batch=32, tokens=1, kv=4, group=7, rd=128, low=4096, high=262143, dtype="bf16"),
        # a long prompt in fp16, neighbouring pairs of three quarters of the head, scaled by parts
        dict(r, name="rotary_prompt_131k", batch=1, tokens=131072, kv=8, group=4, rd=96, low=0, high=131071, dtype="f16", inter=True, scaling="parts"),
        # a few young conversations: latency, ragged
        dict(p, name="prompt_short_b4", batch=4, kv=4, group=7, qlow=1, qhigh=300, hlow=0, hhigh=0, dtype="f16", fused=True),
        # the whole prompt of one long context: bound by the matrix products
        dict(p, name="prompt_32k", batch=1, kv=4, group=7, qlow=32768, qhigh=32768, hlow=0, hhigh=0, dtype="bf16", fused=True),
        # one new token each of 8 sequences with exact keys: bound by reading them
        dict(p, name="prompt_step_b8_8k", batch=8, kv=4, group=7, qlow=1, qhigh=1, hlow=8191, hhigh=8191, dtype="bf16"),
        # 16 drafted tokens behind one context
        dict(t, name="tree_32k_n16", batch=1, kv=4, group=7, nodes=16, low=32768, high=32768, kbits=3, vbits=4),
        # 8 drafted tokens of each sequence of a ragged serving batch
        dict(t, name="tree_b32_n8_paged", batch=32, kv=4, group=7, nodes=8, low=4096, high=16384, kbits=4, vbits=4, paged=256),
        # 64 drafted tokens behind one very long context
        dict(t, name="tree_262k_n64", batch=1, kv=8, group=4, nodes=64, low=262144, high=262144, kbits=3, vbits=2),
        # what a serving batch keeps of 16 drafted tokens each: launch-bound
        dict(op="keep", name="keep_b32", batch=32, kv=4, nodes=16, most=5, low=1000, high=2000, kbits=4, vbits=4, paged=256),
        # the accepted path of 64 drafted tokens in each of 512 short sequences
        dict(op="keep", name="keep_b512", batch=512, kv=8, nodes=64, most=16, low=100, high=400, kbits=3, vbits=2, paged=0),
        # the last page of each of eight sequences, for their forks
        dict(op="copy", name="copy_8_pages", kv=4, page=256, pairs=8, pool=300, kbits=4, vbits=4),
        # moving half a pool
        dict(op="copy", name="copy_2048_pages", kv=8, page=256, pairs=2048, pool=4096, kbits=3, vbits=2),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "tree", "tree", "keep", "copy"])
    kv, group = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    bits = dict(kbits=rng.randint(2, 5), vbits=rng.randint(1, 4))
    if op == "copy":
        page = rng.choice([64, 128, 256])
        pairs = _log(rng, 1, 300000 // (page * kv))
        return dict(op=op, kv=kv, page=page, pairs=pairs, pool=2 * pairs + rng.randint(0, 50), **bits)
    batch = _log(rng, 1, 48)
    if op == "keep":
        low = rng.randint(0, 1500)
        nodes = rng.randint(2, 64)
        return dict(op=op, kv=kv, batch=batch, nodes=nodes, most=rng.randint(1, max(1, nodes // 2)), low=low,
                    high=low + rng.randint(0, 1500), paged=rng.choice([0, 64, 128, 256]), **bits)
    if op == "rotary":
        tokens = 1 if rng.random() < 0.3 else _log(rng, 2, 3000000 // (batch * kv * (group + 1)))
        low = rng.randint(0, 200000)
        return dict(op=op, kv=kv, group=group, batch=batch, tokens=tokens, rd=2 * rng.randint(1, 64), low=low,
                    high=low + rng.randint(0, 800000), dtype=rng.choice(["bf16", "f16", "f32"]),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "parts"]))
    if op == "prompt":
        kind = rng.choice(["step", "chunk", "whole", "whole"])
        most = 4e9 / (batch * kv * group)                       # pairs of a query and a key
        if kind == "whole":
            high = _log(rng, 2, min(16384, math.sqrt(2 * most)))
            hist = 0
        else:
            hist = _log(rng, 16, min(65536, most, 8000000 / (batch * kv)))
            high = 1 if kind == "step" else _log(rng, 2, min(512, max(2, most / hist)))
        return dict(op=op, kv=kv, group=group, batch=batch, qlow=rng.randint(1, high), qhigh=high,
                    hlow=rng.randint(0, hist), hhigh=hist, causal=kind == "step" or rng.random() < 0.8,
                    dtype=rng.choice(["bf16", "f16"]), fused=hist == 0 and rng.random() < 0.5)
    high = _log(rng, 100, min(131072, 1000000 // (batch * kv)))
    return dict(op=op, kv=kv, group=group, batch=batch, nodes=_log(rng, 1, 64), low=rng.randint(0, high), high=high,
                paged=rng.choice([0, 0, 64, 256]), dtype=rng.choice(["bf16", "f16", "f32"]),
                out=rng.choice(["bf16", "f16"]), **bits)


# ------------------------------------------------------------------ inputs and handles

def prepare(case, seed):
    st = {"case": dict(case)}
    {"rotary": _make_rotary, "prompt": _make_prompt, "tree": _make_tree, "keep": _make_keep, "copy": _make_copy}[case["op"]](
        st, st["case"], _gen(seed))
    if own:
        _handles(st)
    return st


def _make_rotary(st, c, gen):
    """Queries and keys as projections leave them, [batch][tokens][heads][128], seen head by head;
    a prompt's positions run on from its first one, a step's lie anywhere."""
    b, n, dtype = c["batch"], c["tokens"], TYPES[c["dtype"]]
    both = torch.randn(b, n, c["kv"] * (c["group"] + 1), D, generator=gen, device=DEV).to(dtype).transpose(1, 2)
    st["q"], st["k"] = both[:, :c["kv"] * c["group"]], both[:, c["kv"] * c["group"]:]
    first = torch.randint(c["low"], max(c["low"], c["high"] - n + 1) + 1, (b, 1), generator=gen, device=DEV)
    st["at"] = (first + torch.arange(n, device=DEV)).to(torch.int32)
    st["outs"] = [torch.empty(b, n, x.shape[1], D, dtype=dtype, device=DEV).transpose(1, 2) for x in (st["q"], st["k"])]


def _make_prompt(st, c, gen):
    """Packed queries, keys and values [tokens][heads][128], views of one projection where fused."""
    hq, kv, dtype = c["kv"] * c["group"], c["kv"], TYPES[c["dtype"]]
    nq = _lens(c["batch"], c["qlow"], c["qhigh"])
    nk = [a + b for a, b in zip(nq, _lens(c["batch"], c["hlow"], c["hhigh"], 7))]
    st["nq"], st["nk"] = nq, nk
    st["qat"], st["kat"] = _starts(nq), _starts(nk)
    if c["fused"]:
        x = torch.empty(sum(nq), hq + 2 * kv, D, dtype=dtype, device=DEV)
        st["q"], st["k"], st["v"] = x.split([hq, kv, kv], 1)
        st["k"].copy_(_loud((sum(nk), kv), gen, dtype))
    else:
        st["q"], st["v"] = (torch.empty(sum(n), h, D, dtype=dtype, device=DEV) for n, h in ((nq, hq), (nk, kv)))
        st["k"] = _loud((sum(nk), kv), gen, dtype)
    st["q"].copy_(torch.randn(sum(nq), hq, D, generator=gen, device=DEV))
    st["v"].copy_(torch.randn(sum(nk), kv, D, generator=gen, device=DEV))


def _make_tree(st, c, gen):
    lens = _lens(c["batch"], c["low"], c["high"])
    st["lens"], st["cap"] = _int32(lens), _round_up(c["high"] + c["nodes"], c["paged"] or BLOCK)
    st["q"] = torch.randn(c["batch"], c["nodes"], c["kv"] * c["group"], D, generator=gen, device=DEV).to(TYPES[c["dtype"]])
    st["tree"] = _tree(c["batch"], c["nodes"], gen)
    st["arrays"], st["table"] = _codes(c["batch"], c["kv"], st["cap"], c["kbits"], c["vbits"], gen), None
    if c["paged"]:
        st["arrays"], st["table"] = _to_pages(st["arrays"], c["paged"], gen)


def _make_keep(st, c, gen):
    """Accepted nodes per sequence, ascending, −1 behind them: the first few nodes of the tree or
    nodes beyond the slots that are filled, so that a pass can be repeated."""
    b, most, nodes = c["batch"], c["most"], c["nodes"]
    st["lens"], st["cap"] = _int32(_lens(b, c["low"], c["high"])), _round_up(c["high"] + nodes, c["paged"] or BLOCK)
    at = torch.arange(most, device=DEV)
    stay = torch.randint(0, most + 1, (b, 1), generator=gen, device=DEV)
    far = most + torch.sort(torch.rand(b, nodes, generator=gen, device=DEV), dim=1)[1][:, :most] % max(1, nodes - most)
    far = torch.sort(far, dim=1)[0]
    n = torch.randint(1, most + 1, (b, 1), generator=gen, device=DEV)
    st["keep"] = torch.where(at < n, torch.where(at < stay, at, far), -1).to(torch.int32)
    st["arrays"], st["table"] = _noise(b, c["kv"], st["cap"], c["kbits"], c["vbits"], gen), None
    if c["paged"]:
        st["arrays"], st["table"] = _to_pages(st["arrays"], c["paged"], gen)


def _make_copy(st, c, gen):
    st["arrays"] = _noise(c["pool"], c["kv"], c["page"], c["kbits"], c["vbits"], gen)
    st["arrays"]["bounds"] = torch.randn(c["pool"], c["kv"], c["page"] // BLOCK, 2, D, generator=gen, device=DEV).to(torch.bfloat16)
    order = torch.randperm(c["pool"], generator=gen, device=DEV).to(torch.int32)
    st["src"], st["dst"] = order[:c["pairs"]].contiguous(), order[c["pairs"]:2 * c["pairs"]].contiguous()


@functools.lru_cache(None)
def _codec(keys, bits):
    from kv_cache_quantization_gb300 import _binding as B, api
    pi, s = _matrices()
    return api.Codec(B.TQ_PROD, bits, pi, s, _levels(bits - 1)) if keys else api.Codec(B.TQ_MSE, bits, pi, None, _levels(bits))


#: base, factor, length that the frequencies were made for, and its turns between which scaling by parts blends.
BASE, FACTOR, LENGTH, LOW, HIGH, MAGNITUDE = 500000.0, 8.0, 32768, 1.0, 32.0, 1.2


def _handles(st):
    """What a program of this framework keeps: codecs, cache objects, plans, output buffers."""
    from kv_cache_quantization_gb300 import api
    c = st["case"]
    if c["op"] == "rotary":
        more = {} if c["scaling"] == "none" else dict(factor=FACTOR)
        if c["scaling"] == "parts":
            more |= dict(original_len=LENGTH, low_turns=LOW, high_turns=HIGH, magnitude=MAGNITUDE)
        st["rotary"] = api.Rotary(c["rd"], BASE, c["inter"], **more)
        return
    if c["op"] == "prompt":
        st["plan"] = api.PromptPlan(c["batch"], c["kv"] * c["group"], c["kv"], sum(st["nq"]), sum(st["nk"]), max(st["nk"]),
                                    causal=c["causal"], dtype=st["q"].dtype)
        st["out"] = st["plan"].new_out()
        return
    a = st["arrays"]
    at = api.Pages(st["table"], c["paged"], a["xn"].shape[0]) if c.get("paged") else None
    st["k"] = api.ProdCache(a["kidx"], a["sgn"], a["xn"], a["rn"], at)
    st["v"] = api.MSECache(a["vidx"], a["vn"], c["vbits"], at)
    if c["op"] == "copy":
        st["blocks"] = api.BlockBounds(a["bounds"])
    if c["op"] == "tree":
        st["kc"], st["vc"] = _codec(True, c["kbits"]), _codec(False, c["vbits"])
        st["plan"] = api.TreePlan(c["batch"], c["nodes"], c["kv"] * c["group"], c["kv"], st["cap"], c["high"] + c["nodes"],
                                  q_dtype=st["q"].dtype, out_dtype=TYPES[c["out"]])
        st["out"] = st["plan"].new_out()


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        from kv_cache_quantization_gb300 import api
        if op == "rotary":
            return st["rotary"].apply(st["q"], st["k"], st["at"], *st["outs"])
        if op == "prompt":
            return st["plan"].run(st["q"], st["k"], st["v"], st["qat"], st["kat"], st["out"])
        if op == "tree":
            return st["plan"].run(st["kc"], st["vc"], st["q"], st["k"], st["v"], st["lens"], st["tree"], st["out"])
        if op == "keep":
            api.keep_tokens(st["k"], st["v"], st["lens"], st["keep"])
        else:
            api.copy_pages(st["src"], st["dst"], st["k"], st["v"], st["blocks"])
        return st["arrays"]
    return {"rotary": _plain_rotary, "prompt": _plain_prompt, "tree": _plain_tree, "keep": _plain_keep, "copy": _plain_copy}[op](st)


def _frequencies(c):
    f = BASE ** (-torch.arange(0, c["rd"], 2, dtype=torch.float64, device=DEV) / c["rd"])
    if c["scaling"] == "linear":
        f = f / FACTOR
    if c["scaling"] == "parts":
        g = ((LENGTH * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * g + f / FACTOR * (1 - g)
    return f, MAGNITUDE if c["scaling"] == "parts" else 1.0


def _plain_rotary(st):
    c, rd = st["case"], st["case"]["rd"]
    f, magnitude = _frequencies(c)
    angle = (st["at"].double()[..., None] * f)[:, None]                  # (64 bits: positions are far)
    cos, sin = (magnitude * torch.cos(angle)).float(), (magnitude * torch.sin(angle)).float()

    def turned(x):
        y = x.float()
        a, b = (y[..., :rd:2], y[..., 1:rd:2]) if c["inter"] else (y[..., :rd // 2], y[..., rd // 2:rd])
        u, v = a * cos - b * sin, a * sin + b * cos
        head = torch.stack([u, v], -1).flatten(-2) if c["inter"] else torch.cat([u, v], -1)
        return torch.cat([head, y[..., rd:]], -1).to(x.dtype)

    return turned(st["q"]), turned(st["k"])


def _padded(x, starts, lens):
    """Packed rows [tokens][heads][128] as [batch][heads][longest][128], zeros behind a sequence."""
    at = torch.arange(max(max(lens), 1), device=DEV)
    there = at < _int32(lens)[:, None]
    got = x[torch.where(there, starts[:-1, None].long() + at, 0)].float()
    return torch.where(there[..., None, None], got, 0.0).transpose(1, 2)


def _plain_prompt(st):
    c = st["case"]
    batch, kv, group, nq, nk = c["batch"], c["kv"], c["group"], st["nq"], st["nk"]
    q, k, v = (_padded(st[n], at, lens) for n, at, lens in (("q", st["qat"], nq), ("k", st["kat"], nk), ("v", st["kat"], nk)))
    q = q.unflatten(1, (kv, group))
    longest, keys = q.shape[3], k.shape[2]
    column, lens = torch.arange(keys, device=DEV), _int32(nk).view(-1, 1, 1)
    behind = (_int32(nk) - _int32(nq)).view(-1, 1, 1)
    out = torch.empty_like(q)
    chunk = max(1, int(2e9 / (batch * kv * group * keys)))               # rows whose scores are held at a time
    for i in range(0, longest, chunk):
        part = q[:, :, :, i:i + chunk].flatten(2, 3)
        row = torch.arange(i, min(i + chunk, longest), device=DEV).view(1, -1, 1)
        ok = column < (torch.minimum(lens, row + behind + 1) if c["causal"] else lens.expand(-1, row.shape[1], 1))
        s = (part @ k.transpose(2, 3)).unflatten(2, (group, -1)) / math.sqrt(D)
        s = torch.where(ok[:, None, None], s, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
        total = p.sum(-1, keepdim=True)
        o = (p.flatten(2, 3) @ v).unflatten(2, (group, -1))
        out[:, :, :, i:i + chunk] = torch.where(total > 0, o / total, 0.0)
    rows = torch.arange(longest, device=DEV) < _int32(nq)[:, None]
    return out.flatten(1, 2).transpose(1, 2)[rows].to(st["q"].dtype)


def _flat(arrays, table, names=NAMES):
    """The arrays in the flat layout, gathered from a pool where there is a table."""
    if table is None:
        return [arrays[n] for n in names]
    got = {n: arrays[n][table.long()] for n in names}                    # [row][page][head]...
    return [t.movedim(1, _slots(n, t) - 1).flatten(_slots(n, t) - 1, _slots(n, t)) for n, t in got.items()]


def _bits(planes):
    return ((planes[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).flatten(-2)


def _index(codes, bits, dim):
    """Level indices from planes (stacked at `dim`) or nibbles."""
    if bits == 4 and codes.shape[-1] == 64:
        return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    w = (1 << torch.arange(codes.shape[dim], device=DEV, dtype=torch.int32))
    return (_bits(codes).int().movedim(dim, -1) * w).sum(-1, dtype=torch.int32)


def _plain_tree(st):
    c = st["case"]
    kv, group, nodes = c["kv"], c["group"], c["nodes"]
    kidx, sgn, xn, rn, vidx, vn = _flat(st["arrays"], st["table"])
    q = st["q"].float().unflatten(2, (kv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)      # [b][kv][nodes · group][128]
    pi, sk = _on_gpu("pi", torch.float32), _on_gpu("s", torch.float32)
    main = (q @ pi.T) @ _on_gpu(str(c["kbits"] - 1), torch.float32)[_index(kidx, c["kbits"] - 1, 2)].transpose(2, 3)
    sketch = (q @ sk.T) @ (2.0 * _bits(sgn).float() - 1.0).transpose(2, 3)
    s = (main * xn[:, :, None] + sketch * (math.sqrt(math.pi / 2) / D * rn[:, :, None])) / math.sqrt(D)
    drafted = torch.arange(st["cap"], device=DEV) - st["lens"].view(-1, 1, 1)                # [b][1][tokens]
    seen = (st["tree"][..., None] >> drafted.clamp(0, 63)) & 1 == 1
    ok = torch.where(drafted < 0, True, seen & (drafted < nodes))[:, None, :, None].expand(-1, -1, -1, group, -1)
    s = torch.where(ok.flatten(2, 3), s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p * vn[:, :, None]) @ _on_gpu(str(c["vbits"]), torch.float32)[_index(vidx, c["vbits"], 2)]
    o = torch.where(total > 0, o / total, 0.0) @ pi
    return o.unflatten(2, (nodes, group)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(TYPES[c["out"]])


def _plain_keep(st):
    """Tokens pos + keep[i] to pos + i in every array, all of them read before any is written."""
    batch, most = st["keep"].shape
    pos, keep, table = st["lens"].long()[:, None], st["keep"].long(), st["table"]
    kept, i = keep >= 0, torch.arange(most, device=DEV)
    row = torch.arange(batch, device=DEV)[:, None].expand(-1, most)

    def place(at):
        if table is None:
            return row[kept], at[kept]
        page = st["case"]["paged"]
        return table.long().gather(1, at // page)[kept], (at % page)[kept]

    r0, s0 = place(pos + keep.clamp(min=0))
    r1, s1 = place(pos + i)
    for name, t in st["arrays"].items():
        t = t.movedim(_slots(name, t), 1)
        t[r1, s1] = t[r0, s0]
    return st["arrays"]


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for t in st["arrays"].values():
        t.index_copy_(0, dst, t.index_select(0, src))
    return st["arrays"]


# ------------------------------------------------------------------ work

def _token_bytes(c):
    return (c["kbits"] - 1) * 16 + 16 + 8 + c["vbits"] * 16 + 4


def work(case):
    c = case
    if c["op"] == "copy":
        return {"bytes": 2 * c["pairs"] * c["kv"] * (c["page"] * _token_bytes(c) + c["page"] // BLOCK * 2 * D * 2) + 8 * c["pairs"], "flops": 0}
    batch, kv = c["batch"], c["kv"]
    if c["op"] == "keep":       # about half of the entries are there, and half of those move
        return {"bytes": batch * kv * (c["most"] + 3) // 4 * 2 * _token_bytes(c) + 4 * batch * (c["most"] + 1), "flops": 0}
    hq = kv * c["group"]
    if c["op"] == "rotary":
        n = batch * c["tokens"]
        return {"bytes": 2 * n * (hq + kv) * D * ELEM[c["dtype"]] + 4 * n, "flops": 3 * n * (hq + kv) * c["rd"]}
    if c["op"] == "prompt":
        nq = _lens(batch, c["qlow"], c["qhigh"])
        nk = [a + b for a, b in zip(nq, _lens(batch, c["hlow"], c["hhigh"], 7))]
        pairs = sum(a * b - a * (a - 1) // 2 if c["causal"] else a * b for a, b in zip(nq, nk))
        return {"bytes": ELEM[c["dtype"]] * D * (2 * sum(nq) * hq + 2 * sum(nk) * kv) + 8 * (batch + 1), "flops": 4 * D * hq * pairs}
    n = sum(_lens(batch, c["low"], c["high"])) + batch * c["nodes"]
    rows = batch * c["nodes"] * hq
    return {"bytes": kv * n * _token_bytes(c) + rows * D * (ELEM[c["dtype"]] + ELEM[c["out"]]) + 8 * batch * c["nodes"],
            "flops": 2 * 3 * D * c["group"] * c["nodes"] * kv * n}      # scores with two halves of the code, and values


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "prompt": _exact_prompt, "tree": _exact_tree, "keep": _exact_keep, "copy": _exact_copy}[case["op"]](
        st, st["case"])


def _exact_rotary(st, c):
    """Pairs as complex numbers times exp(i · position · frequency)."""
    rd, half = c["rd"], c["rd"] // 2
    i = np.arange(half)
    f = np.exp(-2.0 * i / rd * np.log(BASE))
    size = 1.0
    if c["scaling"] == "linear":
        f = f / FACTOR
    elif c["scaling"] == "parts":
        turns = LENGTH / (2 * np.pi / f)
        share = np.where(turns <= LOW, 0.0, np.where(turns >= HIGH, 1.0, (turns - LOW) / (HIGH - LOW)))
        f, size = (1 - share) * (f / FACTOR) + share * f, MAGNITUDE
    turn = torch.polar(torch.full((1,), size, dtype=torch.float64, device=DEV),
                       st["at"].double()[:, None, :, None] * torch.tensor(f, device=DEV))
    first = torch.arange(half, device=DEV) * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else half)
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double().contiguous()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_prompt(st, c):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for nq, nk in zip(st["nq"], st["nk"]):
        for h in range(c["kv"] * c["group"]):
            k, v = (st[n][k0:k0 + nk, h // c["group"]].double() for n in ("k", "v"))
            for i in range(0, nq, 2048):
                rows = torch.arange(i, min(i + 2048, nq), device=DEV)
                end = min(nk, int(rows[-1]) + 1 + nk - nq) if c["causal"] else nk
                s = st["q"][q0 + rows, h].double() @ k[:end].T / math.sqrt(D)
                if c["causal"]:
                    s.masked_fill_(torch.arange(end, device=DEV) > (rows + nk - nq)[:, None], -math.inf)
                out[q0 + rows, h] = torch.softmax(s, -1) @ v[:end]
        q0, k0 = q0 + nq, k0 + nk
    return out


def _exact_tree(st, c):
    pi, sk = (torch.tensor(m, device=DEV) for m in _matrices())
    kl, vl = (torch.tensor(_levels(n), device=DEV) for n in (c["kbits"] - 1, c["vbits"]))
    shift = torch.arange(8, device=DEV, dtype=torch.uint8)

    def bits(t):
        return (t.unsqueeze(-1).bitwise_right_shift(shift) % 2).reshape(*t.shape[:-1], D).long()

    out = torch.zeros(*st["q"].shape, dtype=torch.float64, device=DEV)
    group = c["group"]
    for b, hist in enumerate(st["lens"].tolist()):
        n = hist + c["nodes"]
        at = torch.arange(n, device=DEV)
        masks = [[True] * hist + [(int(m) >> j) & 1 == 1 for j in range(c["nodes"])] for m in st["tree"][b].tolist()]
        mask = torch.tensor(masks, device=DEV)
        for h in range(c["kv"]):
            if st["table"] is None:
                row, slot = torch.full_like(at, b), at
            else:
                row, slot = st["table"][b].long()[at // c["paged"]], at % c["paged"]
            a = st["arrays"]
            kidx = a["kidx"][row, h, :, slot]
            i = sum(bits(kidx[:, p]) << p for p in range(c["kbits"] - 1))
            if c["vbits"] == 4:
                x = a["vidx"][row, h, slot]
                j = torch.stack([x % 16, x // 16], 2).reshape(-1, D).long()
            else:
                x = a["vidx"][row, h, :, slot]
                j = sum(bits(x[:, p]) << p for p in range(c["vbits"]))
            xn, rn, vn = (a[m][row, h, slot].double()[:, None] for m in ("xn", "rn", "vn"))
            sign = (2 * bits(a["sgn"][row, h, slot]) - 1).double()
            k = xn * (kl[i] @ pi) + rn * math.sqrt(math.pi / 2) / D * (sign @ sk)
            v = vn * (vl[j] @ pi)
            q = st["q"][b, :, h * group:(h + 1) * group].double()
            s = torch.where(mask[:, None], q @ k.T / math.sqrt(D), -math.inf)
            out[b, :, h * group:(h + 1) * group] = torch.softmax(s, -1) @ v
    return out


def _exact_keep(st, c):
    new = {n: t.clone() for n, t in st["arrays"].items()}
    for b, (pos, keep) in enumerate(zip(st["lens"].tolist(), st["keep"].tolist())):
        for i, j in enumerate(keep):
            if j < 0:
                continue
            for n, t in st["arrays"].items():
                (r0, s0), (r1, s1) = ((b, x) if st["table"] is None else (int(st["table"][b, x // c["paged"]]), x % c["paged"])
                                      for x in (pos + j, pos + i))
                if _slots(n, t) == 3:
                    new[n][r1, :, :, s1] = t[r0, :, :, s0]
                else:
                    new[n][r1, :, s1] = t[r0, :, s0]
    return {n: t.double() if t.is_floating_point() else t for n, t in new.items()}


def _exact_copy(st, c):
    new = {n: t.clone() for n, t in st["arrays"].items()}
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        for n, t in st["arrays"].items():
            new[n][b] = t[a]
    return {n: t.double() if t.is_floating_point() else t for n, t in new.items()}
