"""Attention of drafted tokens over the compressed cache (include/tq.h: tq_tree_attention) against its
definition in 64 bits (longctx_ref.py)."""
import math

import numpy as np
import pytest
import torch

import longctx_ref as ref
from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import D, caches, capture, codec, flags, gen, hide, i32, parts, table, up64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


def trees(batch, nodes, kind, seed=0):
    """Masks as Python numbers [batch][nodes]: random trees, a chain, or any bits at all."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(batch):
        row = []
        for i in range(nodes):
            if kind == "any":
                row.append(int(rng.integers(0, 1 << 32)) << 32 | int(rng.integers(0, 1 << 32)))
            else:
                up = i - 1 if kind == "chain" else int(rng.integers(-1, i))
                row.append((row[up] if up >= 0 else 0) | 1 << i)
        out.append(row)
    return out


def masks(rows):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in rows], dtype=torch.int64, device="cuda")


def queries(batch, nodes, heads, dtype, seed):
    return torch.randn(batch, nodes, heads, D, generator=gen(seed), device="cuda").to(dtype)


def run_tree(kbits, vbits, batch, kv, group, lens, nodes, rows, paged=0, q_dtype=torch.bfloat16,
             out_dtype=torch.float16, seed=0, scale=None, own_pages=False):
    kc, vc = codec("k", kbits), codec("v", vbits)
    used = [n + nodes for n in lens]
    cap = up64(max(used))
    kp = vp = None
    if paged:
        cap = -(-cap // paged) * paged
        kp = vp = table(batch, cap // paged, paged, seed + 2)
        if own_pages:
            cap = -(-cap // (3 * paged)) * 3 * paged
            kp, vp = table(batch, cap // paged, paged, seed + 2), table(batch, cap // (3 * paged), 3 * paged, seed + 9)
    k = caches(batch, kv, cap, kbits, vbits, seed + 4, kp, used)[0]
    v = caches(batch, kv, cap, kbits, vbits, seed + 4, vp, used)[1]
    hide(kp, used)
    if vp is not kp:
        hide(vp, used)
    q = queries(batch, nodes, kv * group, q_dtype, seed + 5)
    plan = api.TreePlan(batch, nodes, kv * group, kv, cap, max(used), q_dtype, out_dtype, scale)
    out = plan.new_out().fill_(7)
    plan.run(kc, vc, q, k, v, i32(lens), masks(rows), out)
    check_tree(kc, vc, q, k, v, lens, rows, out, group, scale)
    return kc, vc, q, k, v, plan, out


def check_tree(kc, vc, q, k, v, lens, rows, out, group, scale=None):
    kv, nodes = q.shape[2] // group, q.shape[1]
    for b, n in enumerate(lens):
        row = rows[b if len(rows) > 1 else 0]
        for h in range(kv):
            heads = slice(h * group, (h + 1) * group)
            p = parts(k, v, kc, vc, b, h, torch.arange(n + nodes, device="cuda"))
            for i in range(nodes):
                there = torch.tensor([True] * n + [bool(row[i] >> j & 1) for j in range(nodes)], device="cuda")
                r, err = ref.attend(q[b, i, heads], [t[there] for t in p], kc, vc, scale, out.dtype == torch.float16)
                ref.check_rows(out[b, i, heads], r, err, f"sequence {b}, node {i}, KV head {h}")


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kbits,vbits", [(k, v) for k in (2, 3, 4, 5) for v in (1, 2, 3, 4)])
def test_tree_bit_widths(kbits, vbits, out_dtype):
    run_tree(kbits, vbits, 2, 1, 3, [5, 250], 6, trees(2, 6, "tree"), out_dtype=out_dtype, seed=10 * kbits + vbits)
    assert flags() == 0


@pytest.mark.parametrize("batch,kv,group,lens,nodes,kind", [
    (1, 1, 1, [0], 1, "chain"),                    # one token that attends itself
    (1, 2, 7, [1], 64, "tree"),                    # four row tiles of one sequence, no full tile of history
    (2, 1, 8, [0, 64], 16, "any"),                 # rows of 128, rows that attend nothing among them
    (3, 2, 7, [127, 128, 129], 5, "tree"),         # drafted tokens on both sides of a tile's border
    (2, 1, 5, [100, 1], 64, "any"),
    (2, 2, 4, [63, 1000], 33, "chain"),
    (1, 1, 8, [20011], 9, "tree"),                 # many splits
    (3, 1, 2, [65, 0, 300], 1, "chain"),           # single tokens
])
@pytest.mark.parametrize("paged", [0, 64, 192])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_tree_shapes(batch, kv, group, lens, nodes, kind, paged, out_dtype):
    run_tree(3, 4, batch, kv, group, lens, nodes, trees(batch, nodes, kind, nodes), paged, out_dtype=out_dtype,
             seed=nodes + paged, own_pages=paged == 64)
    assert flags() == 0


@pytest.mark.parametrize("q_dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_tree_types(q_dtype, out_dtype):
    run_tree(4, 2, 2, 2, 4, [9, 70], 7, trees(2, 7, "tree"), 0, q_dtype, out_dtype, seed=7, scale=0.05)


@pytest.mark.parametrize("batch,kv,group,nodes,kbits,vbits", [(29, 1, 5, 9, 3, 4), (30, 2, 7, 9, 4, 2), (3, 8, 8, 64, 2, 1)])
@pytest.mark.parametrize("q_dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16),
                                               (torch.float16, torch.bfloat16)])
def test_many_rows(batch, kv, group, nodes, kbits, vbits, q_dtype, out_dtype):
    """More rows than 8 for each SM: kernels of their own before and after the attention (1305 rows is no
    multiple of 8)."""
    lens = [(37 * b) % 150 for b in range(batch)]
    run_tree(kbits, vbits, batch, kv, group, lens, nodes, trees(batch, nodes, "any", batch), 0, q_dtype, out_dtype, seed=batch)
    assert flags() == 0


@pytest.mark.parametrize("batch,group", [(300, 8), (257, 5), (2, 8)])
def test_ragged_batches_are_taken_by_length(batch, group):
    """Large batches' items are taken by length: equal lengths, none at all, one much longer than the
    others; then the same call replayed with other lengths."""
    nodes, kv = (2, 1) if batch > 2 else (64, 8)
    lens = [(61 * b) % 7 * 40 for b in range(batch)]
    lens[batch // 2] = 3000
    rows = trees(batch, nodes, "any", batch)
    kc, vc, q, k, v, plan, out = run_tree(3, 2, batch, kv, group, lens, nodes, rows, seed=batch)
    tree, n, side = masks(rows), i32(lens), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = plan.new_out()
    with torch.cuda.stream(side):
        g = capture(lambda: plan.run(kc, vc, q, k, v, n, tree, o), side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out)
    other = [x // (1 + b % 3) for b, x in enumerate(lens)]
    n.copy_(i32(other))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check_tree(kc, vc, q, k, v, other, rows, o, group)
    assert flags() == 0


@pytest.mark.parametrize("batch", [2048, 2049, 5000])
def test_more_sequences_than_are_ranked(batch):
    """Large ragged batches with one long sequence, ranked by length and not."""
    kc, vc = codec("k", 3), codec("v", 2)
    lens = [(61 * b) % 11 * 6 for b in range(batch)]
    lens[batch // 3] = 1500
    cap = up64(1502)
    some = [0, 1, batch // 3 - 1, batch // 3, batch // 3 + 1, 2047, batch - 1] + list(range(5, batch, batch // 20))
    k, v = api.ProdCache.empty(batch, 1, cap, 3), api.MSECache.empty(batch, 1, cap, 2)
    few = caches(len(some), 1, cap, 3, 2, 5)
    for c, f in ((k, few[0]), (v, few[1])):
        for t, x in ((c.idx, f.idx), (c.xnorm, f.xnorm)) + (((c.sgn, f.sgn), (c.rnorm, f.rnorm)) if c is k else ()):
            t.zero_()
            t[some] = x
    q = queries(batch, 2, 8, torch.bfloat16, 6)
    rows = trees(batch, 2, "any", batch)
    plan = api.TreePlan(batch, 2, 8, 1, cap, 1502, out_dtype=torch.bfloat16)
    out = plan.run(kc, vc, q, k, v, i32(lens), masks(rows), plan.new_out())
    pick = lambda c: type(c)(*[t[some] for t in ((c.idx, c.sgn, c.xnorm, c.rnorm) if c is k else (c.idx, c.xnorm))],
                             *(() if c is k else (2,)))
    check_tree(kc, vc, q[some], pick(k), pick(v), [lens[b] for b in some], [rows[b] for b in some], out[some], 8)
    assert out.isfinite().all() and flags() == 0


@pytest.mark.parametrize("nodes", [15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("first", [0, 1, 15, 16, 17, 111, 112, 113, 127])
def test_every_place_of_the_drafted_tokens_in_a_tile(first, nodes):
    run_tree(3, 2, 1, 1, 2, [128 + first], nodes, trees(1, nodes, "any", first), seed=first)


def test_rows_that_attend_nothing_are_zero():
    nodes = 12
    rows = [[0] * nodes, [0 if i % 3 else 1 << i for i in range(nodes)]]
    kc, vc, q, k, v, plan, out = run_tree(3, 4, 2, 2, 3, [0, 0], nodes, rows)
    assert not out[0].any() and not out[1, 1].any() and out[1, 3].any()
    # bits past the drafted tokens name nothing
    more = masks([[m | (1 << 64) - (1 << nodes) for m in row] for row in rows])
    assert torch.equal(plan.run(kc, vc, q, k, v, i32([0, 0]), more, plan.new_out()), out)


def test_one_tree_for_all_sequences():
    rows = trees(1, 10, "tree", 3)
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 3, 2, 4, [40, 0, 300], 10, rows * 3)
    assert torch.equal(plan.run(kc, vc, q, k, v, i32([40, 0, 300]), masks(rows), plan.new_out()), out)


def test_masked_tokens_do_not_show():
    """Codes, infinite and NaN norms of drafted tokens that a node does not attend change nothing."""
    nodes, lens = 8, [130, 3]
    rows = [[1 << i | 1 for i in range(nodes)] for _ in lens]
    kc, vc, q, k, v, plan, out = run_tree(3, 4, 2, 2, 3, lens, nodes, rows)
    for b, n in enumerate(lens):
        for i, x in ((2, math.nan), (5, math.inf), (6, -math.inf)):
            for t in (k.xnorm, k.rnorm, v.xnorm):
                t[b, :, n + i] = x
            k.idx[b, :, :, n + i] ^= 255
    got = plan.run(kc, vc, q, k, v, i32(lens), masks(rows), plan.new_out())
    keep = [i for i in range(nodes) if i not in (2, 5, 6)]
    assert torch.equal(got[:, keep], out[:, keep])


def test_a_chain_equals_causal_prefill_attention():
    """Nodes in a chain are a causal chunk: tq_prefill_attention (its own kernels, fp32 output)."""
    kc, vc = codec("k", 3), codec("v", 2)
    lens, nodes = [200, 31], 9
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 2, 2, 4, lens, nodes, trees(2, nodes, "chain"))
    cap = k.capacity
    pre = api.PrefillPlan(2, nodes, 8, 2, cap, max(lens) + nodes)
    want = pre.run(kc, vc, q, k, v, i32(lens), pre.new_out())
    off = (out.double() - want.double()).norm(dim=-1) / want.double().norm(dim=-1)
    assert float(off.max()) < 4e-3


def test_histories_over_the_plan_are_clamped_and_flagged():
    kc, vc, q, k, v, _, _ = run_tree(3, 2, 2, 1, 2, [250, 100], 4, trees(2, 4, "chain"))
    plan = api.TreePlan(2, 4, 2, 1, k.capacity, 104)
    out = plan.run(kc, vc, q, k, v, i32([250, 100]), masks(trees(2, 4, "chain")), plan.new_out())
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW
    check_tree(kc, vc, q, k, v, [100, 100], trees(2, 4, "chain"), out, 2)
    out = plan.run(kc, vc, q, k, v, i32([-5, 100]), masks(trees(2, 4, "chain")), plan.new_out())
    check_tree(kc, vc, q, k, v, [0, 100], trees(2, 4, "chain"), out, 2)
    assert flags() == 0


def test_bad_pages_are_left_out_and_flagged():
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 2, 1, 2, [200, 100], 8, trees(2, 8, "tree"), 64)
    k.pages.block_table[0, 1] = k.pages.num_pages
    got = plan.run(kc, vc, q, k, v, i32([200, 100]), masks(trees(2, 8, "tree")), plan.new_out())
    assert flags() == B.TQ_FLAG_PAGE
    assert torch.equal(got[1], out[1]) and got[0].isfinite().all() and not torch.equal(got[0], out[0])


def test_draft_verify_keep_loop():
    """Steps of a program that drafts: rotary positions by depth, appends behind the history, attention
    of the tree, the accepted path kept, and a decode step over what is there, on forked pages."""
    kc, vc = codec("k", 3), codec("v", 4)
    batch, kv, group, page, nodes = 3, 2, 4, 64, 9
    pages = table(batch, 8, page, 1, spare=6)
    k, v = api.ProdCache.empty_paged(pages, kv, 3), api.MSECache.empty_paged(pages, kv, 4)
    rot = api.Rotary(128)
    rng = np.random.default_rng(3)
    lens = [100, 0, 250]

    def codes(b, at):
        """Codes and norms of tokens `at` of sequence b."""
        at = torch.tensor(at, dtype=torch.long, device="cuda")
        page, slot = pages.block_table[b].long()[at // 64], at % 64
        return [t[page, :, :, slot] for t in (k.idx,)] + [t[page, :, slot] for t in (k.sgn, k.xnorm, k.rnorm, v.idx, v.xnorm)]

    x = torch.randn(2, batch, kv, max(lens), D, generator=gen(1), device="cuda").bfloat16()
    at = torch.arange(max(lens), dtype=torch.int32, device="cuda").expand(batch, -1)
    rot.apply(x[0], None, at)
    api.quantize_prod(kc, x[0], k, count=i32(lens))
    api.quantize_mse(vc, x[1], v, count=i32(lens))
    written = [codes(b, list(range(n))) for b, n in enumerate(lens)]
    plan = api.TreePlan(batch, nodes, kv * group, kv, pages.capacity, pages.capacity)
    for step in range(6):
        rows = trees(batch, nodes, "tree", step)
        depth = [[bin(m).count("1") - 1 for m in row] for row in rows]
        at = i32([[n + d for d in row] for n, row in zip(lens, depth)])
        q = queries(batch, nodes, kv * group, torch.bfloat16, 10 + step)
        x = torch.randn(2, batch, kv, nodes, D, generator=gen(20 + step), device="cuda").bfloat16()
        rot.apply(q.transpose(1, 2), x[0], at)
        pos = i32(lens)
        api.quantize_prod(kc, x[0], k, pos=pos)
        api.quantize_mse(vc, x[1], v, pos=pos)
        out = plan.run(kc, vc, q, k, v, pos, masks(rows), plan.new_out())
        check_tree(kc, vc, q, k, v, lens, rows, out, group)
        # the path to a node of each sequence is accepted
        ends = [row[int(rng.integers(0, nodes))] for row in rows]
        paths = [[j for j in range(nodes) if end >> j & 1] for end in ends]
        written = [[torch.cat(p) for p in zip(w, codes(b, [n + j for j in path]))]
                   for b, (w, n, path) in enumerate(zip(written, lens, paths))]
        api.keep_tokens(k, v, pos, i32([p + [-1] * (nodes - len(p)) for p in paths]))
        lens = [n + len(p) for n, p in zip(lens, paths)]
    # the cache holds the codes of the kept tokens, in order, and nothing of what was left behind
    for b, n in enumerate(lens):
        assert all(torch.equal(x, y) for x, y in zip(codes(b, list(range(n))), written[b]))
    q = torch.randn(batch, kv * group, D, generator=gen(99), device="cuda").bfloat16()
    dec = api.DecodePlan(batch, kv * group, kv, pages.capacity, pages.capacity, out_dtype=torch.float32)
    want = dec.run(kc, vc, q, k, v, i32(lens), dec.new_out())
    # a fork: the last page of sequence 2 is copied, the others are shared
    spare = [p for p in range(pages.num_pages) if p not in pages.block_table.flatten().tolist()]
    last = lens[2] // page
    bt = pages.block_table[2:3].clone()
    api.copy_pages(bt[0, last:last + 1].contiguous(), i32([spare[0]]), k, v)
    bt[0, last] = spare[0]
    fork = api.Pages(bt, page, pages.num_pages)
    fk = api.ProdCache(k.idx, k.sgn, k.xnorm, k.rnorm, fork)
    fv = api.MSECache(v.idx, v.xnorm, 4, fork)
    one = api.DecodePlan(1, kv * group, kv, pages.capacity, pages.capacity, out_dtype=torch.float32)
    a = one.run(kc, vc, q[2:3], fk, fv, i32(lens[2:3]), one.new_out())
    off = (a - want[2:3]).norm(dim=-1) / want[2:3].norm(dim=-1)
    assert float(off.max()) < 4e-3
    assert flags() == 0


def test_graph_stream_and_two_plans():
    lens, nodes = [500, 64], 7
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 2, 2, 4, lens, nodes, trees(2, nodes, "tree"))
    tree, n = masks(trees(2, nodes, "tree")), i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = plan.new_out()
    plan.run(kc, vc, q, k, v, n, tree, o, stream=side)
    side.synchronize()
    assert torch.equal(o, out)
    with torch.cuda.stream(side):
        g = capture(lambda: plan.run(kc, vc, q, k, v, n, tree, o), side)
    q.copy_(queries(2, nodes, 8, q.dtype, 77))
    n.copy_(i32([333, 501]))
    tree.copy_(masks(trees(2, nodes, "any", 5)))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for t in (k.xnorm, k.rnorm, v.xnorm):
        assert t[1, :, 64 + nodes:].isnan().all()        # (sequence 1 is longer than its codes: NaN)
    check_tree(kc, vc, q[:1], k, v, [333], trees(2, nodes, "any", 5)[:1], o[:1], 4)
    # two plans on two streams, many calls in flight
    other = api.TreePlan(2, nodes, 8, 2, k.capacity, max(lens) + nodes, out_dtype=torch.float16)
    n.copy_(i32(lens))
    tree.copy_(masks(trees(2, nodes, "tree")))
    alone = plan.run(kc, vc, q, k, v, n, tree, plan.new_out()).clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[plan.new_out() for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for p, s, os in zip((plan, other), streams, outs):
            p.run(kc, vc, q, k, v, n, tree, os[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, alone) for os in outs for x in os)
    flags()


def test_replays_and_streams_raise_no_flags():
    """A captured call replayed with other lengths and trees is right in every sequence; neither that nor
    calls of two plans on two streams raise a flag; histories past the plan's bound raise theirs."""
    lens, nodes, other = [700, 64, 1], 7, [333, 600, 0]
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 3, 2, 4, [700] * 3, nodes, trees(3, nodes, "tree"), seed=31)
    rows, new = trees(3, nodes, "tree", 1), trees(3, nodes, "any", 2)
    tree, n, o = masks(rows), i32(lens), plan.new_out()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = capture(lambda: plan.run(kc, vc, q, k, v, n, tree, o), side)
    assert flags() == 0
    q.copy_(queries(3, nodes, 8, q.dtype, 32))
    n.copy_(i32(other))
    tree.copy_(masks(new))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check_tree(kc, vc, q, k, v, other, new, o, 4)
    assert flags() == 0
    n.copy_(i32(lens))
    tree.copy_(masks(rows))
    plans = [plan, api.TreePlan(3, nodes, 8, 2, k.capacity, 700 + nodes, out_dtype=torch.float16)]
    alone = plan.run(kc, vc, q, k, v, n, tree, plan.new_out()).clone()
    streams = [torch.cuda.Stream() for _ in plans]
    outs = [[plan.new_out() for _ in range(10)] for _ in plans]
    torch.cuda.synchronize()
    for i in range(10):
        for p, s, os in zip(plans, streams, outs):
            p.run(kc, vc, q, k, v, n, tree, os[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, alone) for os in outs for x in os)
    assert flags() == 0
    n.copy_(i32([700, 701, 0]))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check_tree(kc, vc, q, k, v, [700, 700, 0], rows, o, 4)
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW


def test_offsets_past_32_bits():
    """Value codes of more than 4 GiB, drafted tokens at their end."""
    kc, vc = codec("k", 2), codec("v", 4)
    n, kv = 1 << 20, 72
    k, v = caches(1, kv, n, 2, 4, 1)
    assert v.idx.numel() > 1 << 32
    q = queries(1, 3, kv, torch.bfloat16, 2)
    lens, rows = [n - 3], [[1, 3, 5]]
    plan = api.TreePlan(1, 3, kv, kv, n, n)
    out = plan.run(kc, vc, q, k, v, i32(lens), masks(rows), plan.new_out())
    for h in (0, kv - 1):
        p = parts(k, v, kc, vc, 0, h, torch.arange(n, device="cuda"))
        for i in range(3):
            there = torch.arange(n, device="cuda") < n - 3
            there[n - 3:] = torch.tensor([bool(rows[0][i] >> j & 1) for j in range(3)], device="cuda")
            r, err = ref.attend(q[0, i, h:h + 1], [t[there] for t in p], kc, vc)
            ref.check_rows(out[0, i, h:h + 1], r, err, f"head {h}, node {i}")
    assert flags() == 0


def test_refusals_on_the_gpu():
    lens, nodes = [10, 20], 4
    rows = trees(2, nodes, "tree")
    kc, vc, q, k, v, plan, out = run_tree(3, 2, 2, 2, 4, lens, nodes, rows)
    n, tree = i32(lens), masks(rows)
    other = caches(2, 2, k.capacity + 64, 3, 2, 1)
    for bad in (lambda: plan.run(kc, vc, q.float(), k, v, n, tree, out), lambda: plan.run(kc, vc, q[:, :3], k, v, n, tree, out),
                lambda: plan.run(kc, vc, q, k, v, n.long(), tree, out), lambda: plan.run(kc, vc, q, k, v, n, tree.int(), out),
                lambda: plan.run(kc, vc, q, k, v, n, tree[:, :3], out), lambda: plan.run(kc, vc, q, *other, n, tree, out),
                lambda: plan.run(kc, vc, q, k, v, n, tree.cpu(), out), lambda: plan.run(kc, vc, q, k, v, n, tree, out.float()),
                lambda: plan.run(codec("k", 4), vc, q, k, v, n, tree, out),
                lambda: plan.run(kc, codec("v", 4), q, k, v, n, tree, out)):
        with pytest.raises(ValueError):
            bad()
    assert flags() == 0
