"""Operators of long contexts at values and layouts where they can go wrong: infinite and tiny
values in a selection, long even tails, block tables of their own for keys and values, bad pages,
refusals; against the definitions in 64 bits (longctx_ref.py)."""
import math

import pytest
import torch

import longctx_ref as ref
from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import (D, blank, caches, check_prefix, check_select, check_sparse, codec, flags,
                              flat_bounds, hide, i32, lists_of, parts, queries, run_select, table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("n", [64, 1500])
@pytest.mark.parametrize("where", ["first", "middle", "last", "all over"])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("group", [1, 4])
def test_select_with_infinite_bounds_that_no_query_uses(group, side, where, n):
    """A channel's lower (upper) bound is infinite in some blocks and every query of the group is
    positive (negative) there: the blocks' scores are finite, and the largest of all."""
    blocks = blank(1, 1, 64 * n, None, 1)
    blocks.bounds[..., 1, :] += 2
    q = queries(1, group, torch.float32, 2)
    q[..., 5] = 1.0 if side == 0 else -1.0
    at = {"first": [1, 2], "middle": [n // 2], "last": [n - 2], "all over": [3, n // 3, n // 2, n - 5]}[where]
    for i in at:
        blocks.bounds[0, 0, i] = torch.where(q[0, 0] < 0, -9.0, 9.0)
        blocks.bounds[0, 0, i, side, 5] = -math.inf if side == 0 else math.inf
    keep = 16
    _, got = run_select(q, blocks, [64 * n], keep, 0, 1, group, 1, 64 * n)
    assert set(at) <= set(got[0, 0].tolist())
    check_select(q, blocks, [64 * n], keep, 0, 1, group, 1, got)
    assert flags() == 0


@pytest.mark.parametrize("q_size,b_size", [(1e-30, 1e-16), (1e-25, 1e-18), (1e-28, 1e-12), (2e-38, 1.0)])
@pytest.mark.parametrize("group", [1, 5])
def test_select_with_products_that_32_bits_do_not_hold(group, q_size, b_size):
    """Products of queries and bounds of 1e-46 (0 in 32 bits), 1e-43 and 1e-40 (subnormal) and about
    the smallest normal number: the order is that of 64 bits all the same."""
    n = 300
    blocks = blank(1, 2, 64 * n, None, 1)
    blocks.bounds[..., 1, :] += 1
    blocks.bounds *= b_size
    q = queries(1, 2 * group, torch.float32, 2, q_size)
    _, got = run_select(q, blocks, [64 * n - 7], 24, 1, 2, group, 2, 64 * n)
    check_select(q, blocks, [64 * n - 7], 24, 1, 2, group, 2, got)
    assert flags() == 0


@pytest.mark.parametrize("what", ["queries", "bounds", "queries but one"])
def test_select_among_zeros(what):
    """Zero queries, or zero bounds, score every block 0: the lowest numbers stay.  One query of
    1e-45 among zero ones decides."""
    n = 500
    blocks = blank(1, 1, 64 * n, None, 1)
    q = queries(1, 4, torch.float32, 2)
    if what == "bounds":
        blocks.bounds.zero_()
    else:
        q.zero_()
        if what == "queries but one":
            q[0, 2, 77] = 1e-45
            blocks.bounds[0, 0, :, 1, 77] = 1e-3 * (1 + torch.randperm(n, device="cuda").bfloat16())
    _, got = run_select(q, blocks, [64 * n], 40, 2, 1, 4, 1, 64 * n)
    check_select(q, blocks, [64 * n], 40, 2, 1, 4, 1, got)
    if what != "queries but one":
        assert got[0, 0].tolist() == list(range(39)) + [499]


# ------------------------------------------------------------------ attention

def alike(t, b, h):
    """Every token of (b, h) gets the codes and norms of its first one."""
    x = t[b, h]
    if x.dim() == 3:
        x[:] = x[:, :1].clone()
    else:
        x[:] = x[:1].clone()


@pytest.mark.parametrize("tail", [23.3, 24.6, 25.1])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_a_peak_before_a_long_even_tail(out_dtype, tail):
    """One token of weight 1 and then 65535 equal ones of weight 2^-tail, in one item: the tail's sum
    counts in full, although fp16 holds numbers around 2^-24 as 0, 2^-24 or 2^-23.

    Off by at most, relative to the values' norm V: the output's rounding; the values' levels; the
    tail's sum n · 2^-tail times twice the error of its one score (2^-18, or 2^-9 with single fp16
    operands, of the sum of its terms' sizes: three roundings of 2^-21 or 2^-11, the levels, 32-bit
    sums); each weight's rounding, 2^-25 of a weight taken 2^7 times as large, in the same direction
    n times; and 2^-23 of the accumulator for each of 4096 matrix instructions."""
    n, batch, heads, group = 65536, 16, 152, 8       # 128 rows of each of 152 heads: an item a head
    kc, vc = codec("k", 3), codec("v", 2)
    k, v = caches(1, heads, n, 3, 2, 1)
    q = queries(batch, heads * group, torch.float32, 2)
    pi, sk = (torch.tensor(m, device="cuda") for m in (kc.pi, kc.s))
    size = {}
    for h in (0, heads - 1):
        for t in (k.idx, k.sgn, k.xnorm, k.rnorm, v.idx, v.xnorm):
            alike(t, 0, h)
        # the norms of a key scale its score: token 0's is 0, the others' are -tail·ln 2
        c, s, xn, rn = ref.key_parts(k, kc, 0, h, torch.arange(1, device="cuda"))
        rows = q[:, h * group:(h + 1) * group]
        y, z = rows.double() @ pi.T, rows.double() @ sk.T
        one = (xn * (y @ c[0]) + ref.QJL * rn * (z @ s[0])) / math.sqrt(D)
        by = -tail * math.log(2) / one
        rows *= by[..., None].float()
        terms = (xn * (y * c[0]).abs().sum(-1) + ref.QJL * rn * z.abs().sum(-1)) / math.sqrt(D)
        size[h] = float((terms * by.abs()).max())
        k.xnorm[0, h, 0] = k.rnorm[0, h, 0] = 0.0
        v.idx[0, h, :, 0] = 255 - v.idx[0, h, :, 1]      # the peak's value is another one
        v.xnorm[0, h] = 10.0
    plan = api.PrefixPlan(batch, heads * group, heads, 64, 0, n, n, torch.float32, out_dtype)
    own = caches(batch, heads, 64, 3, 2, 3)
    out = plan.run(kc, vc, q, k, v, i32([n]), *own, i32([0] * batch), plan.new_out())
    pairs = out_dtype == torch.float16
    for h in size:
        rows = slice(h * group, (h + 1) * group)
        r, _ = ref.attend(q[:, rows].reshape(-1, D), parts(k, v, kc, vc, 0, h, torch.arange(n, device="cuda")),
                          kc, vc, pairs=pairs)
        off = (out[:, rows].reshape(-1, D).double() - r).norm(dim=-1).max()
        score = 2.0 ** (-18 if pairs else -9) * size[h]
        most = 10.0 * (torch.finfo(out_dtype).eps / 2 + ref.level_error(vc) + 2 * n * 2.0 ** -tail * score
                       + n * 2.0 ** -32 + 4096 * 2.0 ** -23)
        assert float(off) <= most, (h, float(off), most)
    assert flags() == 0


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_scores_so_large_that_32_bits_hold_them_to_units(out_dtype):
    """Base-2 scores of 2^20 to 2^30 whose maximum grows by 0 to 5 steps of 32 bits in the second
    tile: such scores are known to some units only, so the weights of the two tokens that share the
    maximum are anything, but the row is finite and lies between their values."""
    batch, n = 304, 256            # (two items an SM, so that an item has both tiles)
    kc, vc = codec("k", 3), codec("v", 2)
    k, v = caches(batch, 1, n, 3, 2, 1)
    k.xnorm.zero_()
    k.rnorm.zero_()
    v.xnorm.fill_(1.0)
    top = (37, 37 + 128)           # the same lane of either tile
    b = torch.arange(batch, device="cuda")
    q = torch.empty(batch, 1, D, device="cuda")
    c = ref.key_parts(k, kc, 0, 0, torch.tensor([37], device="cuda"))[0][0]
    for t in (k.idx, k.sgn):
        for i in top:
            t[:, :, ..., i, :] = t[:1, :, ..., 37, :]
    v.xnorm[:, 0, top[0]] = v.xnorm[:, 0, top[1]] = 8.0
    k.xnorm[:, 0, top[0]] = 1.0
    k.xnorm[:, 0, top[1]] = 1.0 + 2.0 ** -23 * (b % 6)
    one = (c @ c) / math.sqrt(D) / math.log(2)             # base-2 score of q = Π^T c
    want = 2.0 ** (20 + 10 * b.double() / batch)
    q[:, 0] = ((want / one)[:, None] * (c @ torch.tensor(kc.pi, device="cuda"))).float()
    lens = i32([n] * batch)
    plan = api.PrefixPlan(batch, 1, 1, n, n, 64, 0, torch.float32, out_dtype)
    out = plan.run(kc, vc, q, *caches(1, 1, 64, 3, 2, 3), i32([0]), k, v, lens, plan.new_out())
    assert out.isfinite().all(), (~out.isfinite()).any(-1).any(-1).nonzero().flatten().tolist()[:20]
    cv = torch.stack([ref.value_parts(v, vc, i, 0, torch.tensor(top, device="cuda"))[0] for i in range(batch)])
    most = 8.0 * cv.norm(dim=-1).amax(-1)
    assert bool((out[:, 0].double().norm(dim=-1) <= most * (1 + 2.0 ** -7)).all())
    assert flags() == 0


# ------------------------------------------------------------------ refusals

def test_arrays_and_tables_of_the_host_are_refused():
    """Block tables, norms and signs that lie on the host, or of another capacity: refused before
    anything is launched, by every call."""
    kc, vc = codec("k", 3), codec("v", 2)
    there = api.Pages(torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2), 64, 4)
    host = api.Pages(torch.arange(4, dtype=torch.int32).view(2, 2), 64, 4)
    k, v = caches(2, 2, 128, 3, 2, 1)
    pk, pv = caches(2, 2, 128, 3, 2, 1, there)
    q, n = queries(2, 4, torch.bfloat16, 1), i32([100, 3])
    sp, pr = api.SparsePlan(2, 4, 2, 128, 128, 1, 0, 0), api.PrefixPlan(2, 4, 2, 128, 128, 128, 128)
    lst, out = sp.new_list(), sp.new_out()
    lst.zero_()

    def sparse(a, b):
        sp.run(kc, vc, q, a, b, n, lst, out)

    def prefix(a, b):
        pr.run(kc, vc, q, a, b, i32([50]), k, v, n, out)

    for run in (sparse, prefix):
        run(k, v)
        run(pk, pv)
        bad = [(api.ProdCache(pk.idx, pk.sgn, pk.xnorm, pk.rnorm, host), pv),
               (pk, api.MSECache(pv.idx, pv.xnorm, 2, host)),
               (api.ProdCache(k.idx, k.sgn, k.xnorm, k.rnorm.cpu()), v),
               (api.ProdCache(k.idx, k.sgn[:, :, :64].contiguous(), k.xnorm, k.rnorm), v),
               (k, api.MSECache(v.idx, v.xnorm.cpu(), 2)),
               (k, api.MSECache(v.idx.int(), v.xnorm, 2))]
        for a, b in bad:
            with pytest.raises(ValueError):
                run(a, b)
    blocks = api.BlockBounds.empty_paged(there, 2)
    sp.select(q, blocks, n, lst)
    api.block_bounds(torch.zeros(2, 2, 3, D, device="cuda"), blocks)
    blocks.pages = host
    with pytest.raises(ValueError):
        sp.select(q, blocks, n, lst)
    with pytest.raises(ValueError):
        api.block_bounds(torch.zeros(2, 2, 3, D, device="cuda"), blocks)
    torch.cuda.synchronize()
    assert flags() == 0


def test_a_refused_step_writes_nothing():
    """Every argument of SparsePlan.step is checked before the appends: a refused step leaves codes,
    norms and bounds as they are."""
    kc, vc = codec("k", 3), codec("v", 2)
    k, v = caches(2, 2, 128, 3, 2, 1)
    blocks = blank(2, 2, 128, None, 2)
    plan = api.SparsePlan(2, 4, 2, 128, 128, 1, 0, 0, out_dtype=torch.float16)
    g = torch.randn(2, 2, D, device="cuda").half()
    good = dict(kc=kc, vc=vc, q=queries(2, 4, torch.bfloat16, 1), k_new=g, v_new=g.clone(), k=k, v=v,
                blocks=blocks, pos=i32([70, 3]), seq_lens=i32([71, 4]), block_list=plan.new_list(),
                out=plan.new_out())
    arrays = (k.idx, k.sgn, k.xnorm, k.rnorm, v.idx, v.xnorm, blocks.bounds)
    before = [t.clone() for t in arrays]
    odd = torch.zeros(2 * 2 * D + 8, device="cuda").half()
    bad = dict(kc=[vc, codec("k", 4)], vc=[kc, codec("v", 4)], q=[good["q"].half(), good["q"][:1]],
               k_new=[g[:1], g.double(), torch.cat([g, g]), odd[1:1 + 2 * 2 * D].view(2, 2, D), g.cpu()],
               v_new=[g[:, :1], g.long(), g.transpose(1, 2).contiguous().transpose(1, 2), g[..., :64]],
               k=[caches(2, 2, 64, 3, 2, 1)[0]], v=[caches(1, 2, 128, 3, 2, 1)[1]],
               blocks=[blank(2, 2, 64, None, 2)], pos=[i32([70, 3]).long(), i32([1]), i32([1, 2]).cpu()],
               seq_lens=[i32([71]), i32([71, 4]).float()], block_list=[plan.new_list()[:1]],
               out=[plan.new_out().float()])
    for name, values in bad.items():
        for x in values:
            with pytest.raises(ValueError):
                plan.step(**{**good, name: x})
    torch.cuda.synchronize()
    for t, b in zip(arrays, before):
        assert torch.equal(t, b)
    plan.step(**good)
    assert flags() == 0 and not torch.equal(k.sgn, before[1])
    strided = torch.randn(2, 2, 2 * D, device="cuda").half()[..., :D]      # rows of a wider tensor
    plan.step(**{**good, "k_new": strided, "v_new": strided})
    one = [t.clone() for t in arrays]
    plan.step(**{**good, "k_new": strided.contiguous(), "v_new": strided.contiguous()})
    for t, b in zip(arrays, one):
        assert torch.equal(t, b)


# ------------------------------------------------------------------ pages

def two_tables(rows, heads, cap, kbits, vbits, kpage, vpage, seed, used):
    """Keys and values with block tables (0: flat) and page sizes of their own."""
    def pages(page, s):
        return table(rows, cap // page, page, s) if page else None

    k = caches(rows, heads, cap, kbits, vbits, seed, pages(kpage, seed + 1), used)[0]
    v = caches(rows, heads, cap, kbits, vbits, seed + 2, pages(vpage, seed + 3), used)[1]
    for c in (k, v):
        hide(c.pages, used)
    return k, v


@pytest.mark.parametrize("kpage,vpage", [(64, 192), (192, 64), (0, 64), (384, 0), (64, 64)])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_keys_and_values_behind_tables_of_their_own(kpage, vpage, out_dtype):
    kc, vc = codec("k", 3), codec("v", 4)
    batch, kv, group, cap = 3, 2, 5, 1152
    lens, plen = [1000, 65, 0], 700
    k, v = two_tables(batch, kv, cap, 3, 4, kpage, vpage, 1, lens)
    pk, pv = two_tables(1, kv, 768, 3, 4, kpage, vpage, 9, [plen])
    q = queries(batch, kv * group, torch.bfloat16, 2)
    pr = api.PrefixPlan(batch, kv * group, kv, cap, cap, 768, 768, out_dtype=out_dtype)
    out = pr.run(kc, vc, q, pk, pv, i32([plen]), k, v, i32(lens), pr.new_out())
    check_prefix(kc, vc, q, (pk, pv), (k, v), out, plen, lens, kv, group)
    sp = api.SparsePlan(batch, kv * group, kv, cap, cap, 7, 0, 0, out_dtype=out_dtype)
    lst = lists_of(lens, kv, 7, 3)
    out = sp.run(kc, vc, q, k, v, i32(lens), lst, sp.new_out())
    check_sparse(kc, vc, q, k, v, lst, lens, out, group)
    assert flags() == 0


@pytest.mark.parametrize("value", [-1, 0, 1 << 30])
@pytest.mark.parametrize("which", ["keys", "values", "both", "same table"])
@pytest.mark.parametrize("page", [64, 192])
def test_attention_leaves_bad_pages_out(page, which, value):
    """Entries of the block tables that are no page, in the middle and at the end of the prefix and
    of a sequence: their tokens are left out of numerator and denominator, and the flag is raised."""
    kc, vc = codec("k", 4), codec("v", 2)
    batch, kv, group, cap = 2, 2, 4, 1152
    lens, plen = [1100, 300], 1000
    if which == "same table":
        k, v = caches(batch, kv, cap, 4, 2, 1, table(batch, cap // page, page, 2), lens)
        pk, pv = caches(1, kv, cap, 4, 2, 7, table(1, cap // page, page, 8), [plen])
        hide(k.pages, lens)
        hide(pk.pages, [plen])
    else:
        k, v = two_tables(batch, kv, cap, 4, 2, page, page, 1, lens)
        pk, pv = two_tables(1, kv, cap, 4, 2, page, page, 7, [plen])
    q = queries(batch, kv * group, torch.bfloat16, 2)
    n, pn = i32(lens), i32([plen])
    pr = api.PrefixPlan(batch, kv * group, kv, cap, cap, cap, cap, out_dtype=torch.float16)
    sp = api.SparsePlan(batch, kv * group, kv, cap, cap, 9, 0, 0, out_dtype=torch.float16)
    lst = lists_of(lens, kv, 9, 3)
    lst[0, :, 3] = 192 // 64           # a block of page 1 (192) or 3 (64)
    bad = [1, (1000 - 1) // page]
    if page == 64:
        bad.append(3)
    gone = (k, pk) if which == "keys" else (v, pv) if which == "values" else (k, v, pk, pv)
    seen = list({id(c.pages): c.pages for c in gone}.values())
    good = [p.block_table.clone() for p in seen]
    for p in seen:
        p.block_table[0, bad] = value if value < 0 else p.num_pages + value if value < 1000 else value
    o1 = pr.run(kc, vc, q, pk, pv, pn, k, v, n, pr.new_out())
    assert flags() == B.TQ_FLAG_PAGE
    o2 = sp.run(kc, vc, q, k, v, n, lst, sp.new_out())
    assert flags() == B.TQ_FLAG_PAGE
    for p, t in zip(seen, good):
        p.block_table.copy_(t)

    def there(at, b):
        keep = torch.ones_like(at, dtype=torch.bool)
        for i in bad if b == 0 else []:
            keep &= at // page != i
        return at[keep]

    for h in range(kv):
        rows = slice(h * group, (h + 1) * group)
        shared = parts(pk, pv, kc, vc, 0, h, there(torch.arange(plen, device="cuda"), 0))
        for b, m in enumerate(lens):
            own = parts(k, v, kc, vc, b, h, there(torch.arange(m, device="cuda"), b))
            r, err = ref.attend(q[b, rows], [torch.cat(t) for t in zip(shared, own)], kc, vc, pairs=True)
            ref.check_rows(o1[b, rows], r, err, f"prefix, sequence {b}, KV head {h}")
            at = [torch.arange(64 * i, min(64 * i + 64, m), device="cuda") for i in lst[b, h].tolist()
                  if 0 <= i and 64 * i < m]
            at = there(torch.cat(at), b) if at else torch.zeros(0, dtype=torch.long, device="cuda")
            r, err = ref.attend(q[b, rows], parts(k, v, kc, vc, b, h, at), kc, vc, pairs=True)
            ref.check_rows(o2[b, rows], r, err, f"list, sequence {b}, KV head {h}")


@pytest.mark.parametrize("value", [-1, 0, 1 << 30])
@pytest.mark.parametrize("page", [64, 256])
def test_bounds_and_selection_pass_bad_pages_over(page, value):
    """tq_block_bounds leaves such a page's blocks out and writes the others; tq_block_select scores
    them -inf, so they come last (also among each other, where only they are left)."""
    batch, kv, group, tokens = 2, 2, 3, 64 * 40 - 5
    cap = 64 * 40
    pages = table(batch, cap // page, page, 5)
    blocks = blank(batch, kv, cap, pages, 1)
    old = blocks.bounds.clone()
    x = 3 * torch.randn(batch, kv, tokens, D, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    good = pages.block_table.clone()
    bad = [1, 2, 5]
    pages.block_table[0, bad] = value if value < 0 else pages.num_pages + value if value < 1000 else value
    api.block_bounds(x, blocks)
    assert flags() == B.TQ_FLAG_PAGE
    broken = pages.block_table.clone()
    pages.block_table.copy_(good)
    want = ref.bounds(x, [0, 0], [tokens] * 2, torch.zeros_like(flat_bounds(blocks)))
    got, was = flat_bounds(blocks), flat_bounds(api.BlockBounds(old, pages))
    out = torch.zeros(batch, 40, dtype=torch.bool, device="cuda")
    for i in bad:
        out[0, i * page // 64:(i + 1) * page // 64] = True
    for b in range(batch):
        assert torch.equal(got[b][:, out[b]], was[b][:, out[b]])
        assert torch.equal(got[b][:, ~out[b]], want[b][:, ~out[b]])
    q = queries(batch, kv * group, torch.bfloat16, 2)
    gone = int(out[0].sum())
    for keep in (7, 40 - gone, 40 - gone + 2, 39):
        pages.block_table.copy_(broken)
        plan, lst = run_select(q, blocks, [tokens] * 2, keep, 1, 2, group, kv, cap)
        assert flags() == (B.TQ_FLAG_PAGE if keep < 40 else 0)
        pages.block_table.copy_(good)
        flat = flat_bounds(blocks).clone()
        for b in range(batch):
            for h in range(kv):
                t = flat[b, h].clone()
                t[out[b], 0], t[out[b], 1] = math.inf, -math.inf      # (scores -inf)
                w = ref.select(q[b, h * group:(h + 1) * group], t, 40, keep, 1, 2)
                assert lst[b, h].tolist() == w, (keep, b, h)


# ------------------------------------------------------------------ a captured step

@pytest.mark.parametrize("kbits,vbits,page", [(3, 4, 0), (5, 2, 128)])
def test_a_captured_step_replayed(kbits, vbits, page):
    """SparsePlan.step captured once with its counters, replayed on new inputs across block and page
    borders: caches, bounds, lists and rows are those of the same steps called eagerly."""
    kc, vc = codec("k", kbits), codec("v", vbits)
    batch, kv, group, cap, keep = 3, 2, 4, 1024, 5
    lens = [1000, 125, 0]

    def state():
        p = table(batch, cap // page, page, 4) if page else None
        k, v = caches(batch, kv, cap, kbits, vbits, 1, p)
        blocks = blank(batch, kv, cap, p, 2)
        blocks.bounds[..., 1, :] += 3
        plan = api.SparsePlan(batch, kv * group, kv, cap, cap, keep, 1, 1, out_dtype=torch.float16)
        return dict(plan=plan, k=k, v=v, blocks=blocks, pos=i32(lens), n=i32([x + 1 for x in lens]),
                    q=torch.zeros(batch, kv * group, D, device="cuda").bfloat16(),
                    kn=torch.zeros(batch, kv, D, device="cuda").half(),
                    vn=torch.zeros(batch, kv, D, device="cuda").half(), lst=plan.new_list(), out=plan.new_out())

    def step(s):
        s["plan"].step(kc, vc, s["q"], s["kn"], s["vn"], s["k"], s["v"], s["blocks"], s["pos"], s["n"], s["lst"],
                       s["out"])
        s["pos"] += 1
        s["n"] += 1

    def feed(s, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        for f in ("q", "kn", "vn"):
            s[f].copy_(torch.randn(s[f].shape, generator=g, device="cuda"))

    a, b = state(), state()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    step(b)                    # (warmed, then as it was)
    fresh = state()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(b)
    for f in ("pos", "n"):
        b[f].copy_(fresh[f])
    for x, y in ((b["k"], fresh["k"]), (b["v"], fresh["v"])):
        for f in ("idx", "sgn", "xnorm", "rnorm"):
            if hasattr(x, f):
                getattr(x, f).copy_(getattr(y, f))
    b["blocks"].bounds.copy_(fresh["blocks"].bounds)
    for i in range(8):
        feed(a, i)
        feed(b, i)
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for f in ("pos", "n", "lst", "out"):
            assert torch.equal(a[f], b[f]), (i, f)
    for f in ("idx", "sgn", "xnorm", "rnorm"):
        assert torch.equal(getattr(a["k"], f), getattr(b["k"], f)), f
    assert torch.equal(a["v"].idx, b["v"].idx) and torch.equal(a["blocks"].bounds, b["blocks"].bounds)
    now = [x + 8 for x in lens]
    check_select(b["q"], b["blocks"], now, keep, 1, 1, group, kv, b["lst"])
    check_sparse(kc, vc, b["q"], b["k"], b["v"], b["lst"], now, b["out"], group)
    assert flags() == 0
