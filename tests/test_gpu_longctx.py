"""Operators of long contexts (include/tq.h: tq_prefix_attention, tq_block_bounds,
tq_block_select, tq_sparse_attention) against their definitions in 64 bits (longctx_ref.py)."""
import math

import numpy as np
import pytest
import torch

import longctx_ref as ref
from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api

pytestmark = pytest.mark.gpu

D = 128
_codecs = {}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


def codec(kind, bits):
    if (kind, bits) not in _codecs:
        _codecs[kind, bits] = api.Codec.prod(bits) if kind == "k" else api.Codec.mse(bits)
    return _codecs[kind, bits]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def flags():
    return api.device_status()[1]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table(rows, per_row, page, seed, spare=3):
    """A block table of rows × per_row pages in a shuffled order."""
    n = rows * per_row + spare
    t = np.random.default_rng(seed).permutation(n)[:rows * per_row].reshape(rows, per_row)
    return api.Pages(i32(t), page, n)


def caches(rows, heads, cap, kbits, vbits, seed, pages=None, used=None):
    """Caches of random codes: every bit pattern, norms as Gaussian keys have them; norms of slots
    at or past used[b] are NaN (they must not be read into anything)."""
    g = gen(seed)
    if pages is None:
        k, v = api.ProdCache.empty(rows, heads, cap, kbits), api.MSECache.empty(rows, heads, cap, vbits)
    else:
        k, v = api.ProdCache.empty_paged(pages, heads, kbits), api.MSECache.empty_paged(pages, heads, vbits)
    for t in (k.idx, k.sgn, v.idx):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t, low, high in ((k.xnorm, 6, 16), (k.rnorm, 2, 5), (v.xnorm, 6, 16)):
        t.copy_(low + (high - low) * torch.rand(t.shape, generator=g, device="cuda"))
    if used is not None:
        for b, n in enumerate(used):
            for t in (k.xnorm, k.rnorm, v.xnorm):
                if pages is None:
                    t[b, :, n:] = math.nan
                else:
                    pt = pages.page_tokens
                    for i, p in enumerate(pages.block_table[b].tolist()):
                        t[p, :, max(0, n - i * pt):] = math.nan
    return k, v


def hide(pages, used):
    """Table entries past the pages of the first used[b] tokens become -1: nothing may read them."""
    if pages is not None:
        for b, n in enumerate(used):
            pages.block_table[b, -(-n // pages.page_tokens):] = -1


def queries(batch, heads, dtype, seed, size=1.0):
    return (size * torch.randn(batch, heads, D, generator=gen(seed), device="cuda")).to(dtype)


def parts(k, v, kc, vc, b, h, at):
    return (*ref.key_parts(k, kc, b, h, at), *ref.value_parts(v, vc, b, h, at))


def up64(n):
    return max(-(-n // 64) * 64, 64)


# ------------------------------------------------------------------ shared prefix

def run_prefix(kbits, vbits, batch, kv, group, plen, lens, paged=0, q_dtype=torch.bfloat16,
               out_dtype=torch.float16, seed=0, size=1.0, scale=None):
    kc, vc = codec("k", kbits), codec("v", vbits)
    pcap, cap = up64(plen), up64(max(lens))
    pp = po = None
    if paged:
        pcap, cap = -(-pcap // paged) * paged, -(-cap // paged) * paged
        pp, po = table(1, pcap // paged, paged, seed + 1), table(batch, cap // paged, paged, seed + 2)
    pk, pv = caches(1, kv, pcap, kbits, vbits, seed + 3, pp, [plen])
    k, v = caches(batch, kv, cap, kbits, vbits, seed + 4, po, lens)
    hide(pp, [plen])
    hide(po, lens)
    q = queries(batch, kv * group, q_dtype, seed + 5, size)
    plan = api.PrefixPlan(batch, kv * group, kv, cap, max(lens), pcap, plen, q_dtype, out_dtype, scale)
    out = plan.run(kc, vc, q, pk, pv, i32([plen]), k, v, i32(lens), plan.new_out())
    return kc, vc, q, (pk, pv), (k, v), plan, out


def check_prefix(kc, vc, q, pre, mine, out, plen, lens, kv, group, scale=None):
    worst = 0.0
    for h in range(kv):
        shared = parts(*pre, kc, vc, 0, h, torch.arange(plen, device="cuda"))
        for b, n in enumerate(lens):
            own = parts(*mine, kc, vc, b, h, torch.arange(n, device="cuda"))
            rows = slice(h * group, (h + 1) * group)
            r, err = ref.attend(q[b, rows], [torch.cat(p) for p in zip(shared, own)], kc, vc, scale,
                                out.dtype == torch.float16)
            worst = max(worst, ref.check_rows(out[b, rows], r, err, f"sequence {b}, KV head {h}"))
    return worst


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kbits,vbits", [(k, v) for k in (2, 3, 4, 5) for v in (1, 2, 3, 4)])
def test_prefix_bit_widths(kbits, vbits, out_dtype):
    lens = [5, 130]
    a = run_prefix(kbits, vbits, 2, 1, 3, 200, lens, out_dtype=out_dtype, seed=10 * kbits + vbits)
    check_prefix(*a[:5], a[6], 200, lens, 1, 3)
    assert flags() == 0


@pytest.mark.parametrize("batch,kv,group,plen,lens", [
    (1, 1, 1, 1, [0]),
    (1, 2, 8, 0, [1]),
    (2, 1, 5, 0, [0, 64]),                                      # a row with no token at all
    (3, 2, 7, 127, [127, 128, 129]),
    (1, 4, 4, 129, [0]),
    (19, 2, 7, 1000, [(37 * i) % 300 for i in range(19)]),      # 133 rows: two row tiles
    (5, 1, 8, 20011, [1, 0, 700, 63, 65]),                      # many splits
])
@pytest.mark.parametrize("paged", [0, 64, 192])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_prefix_shapes(batch, kv, group, plen, lens, paged, out_dtype):
    a = run_prefix(3, 4, batch, kv, group, plen, lens, paged, out_dtype=out_dtype, seed=plen + paged)
    check_prefix(*a[:5], a[6], plen, lens, kv, group)
    assert flags() == 0


@pytest.mark.parametrize("q_dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_prefix_types(q_dtype, out_dtype):
    lens = [9, 70]
    a = run_prefix(4, 2, 2, 2, 4, 300, lens, 0, q_dtype, out_dtype, seed=7, scale=0.05)
    check_prefix(*a[:5], a[6], 300, lens, 2, 4, 0.05)


@pytest.mark.parametrize("size", [1e-12, 30.0, 1e15])
def test_prefix_query_sizes(size):
    """Queries of any size: the operand is scaled by a power of two of the row (tiny queries
    attend evenly; large ones pick single tokens)."""
    lens = [40]
    scale = 1.0 / size
    a = run_prefix(3, 2, 1, 1, 2, 300, lens, 0, torch.float32, seed=3, size=size, scale=scale)
    check_prefix(*a[:5], a[6], 300, lens, 1, 2, scale)


def test_prefix_value_norms():
    """Value norms from 2^-50 to 2^16 side by side, zeros among them: the weights of the value
    product are taken relative to score + log2 of the norm, so fp16 holds them."""
    kc, vc = codec("k", 3), codec("v", 4)
    k, v = caches(2, 1, 512, 3, 4, 1)
    pk, pv = caches(1, 1, 512, 3, 4, 2)
    e = torch.randint(-50, 17, v.xnorm.shape, generator=gen(3), device="cuda").float()
    v.xnorm.copy_(torch.exp2(e) * (torch.rand(e.shape, generator=gen(4), device="cuda") > 0.2))
    v.xnorm[1] = 0
    pv.xnorm[:, :, :] = 0
    q = queries(2, 4, torch.bfloat16, 5)
    plan = api.PrefixPlan(2, 4, 1, 512, 512, 512, 512, out_dtype=torch.bfloat16)
    lens = [500, 300]
    out = plan.run(kc, vc, q, pk, pv, i32([400]), k, v, i32(lens), plan.new_out())
    check_prefix(kc, vc, q, (pk, pv), (k, v), out, 400, lens, 1, 4)
    assert not out[1].any()      # zero values only: exactly zero
    assert flags() == 0


def test_prefix_equals_decode_over_one_cache():
    """Prefix and own tokens in one paged cache attended by tq_decode_attention (fp32 output, its
    own kernel) give the rows that the prefix call gives."""
    kc, vc = codec("k", 3), codec("v", 2)
    kv, group, page = 2, 4, 64
    plen, lens = 640, [64, 100, 1]
    pp = table(1, 10, page, 1, spare=10)
    free = [p for p in range(pp.num_pages) if p not in pp.block_table[0].tolist()]
    own = i32(free[:6]).view(3, 2)
    po = api.Pages(own, page, pp.num_pages)
    both = api.Pages(torch.cat([pp.block_table.expand(3, -1), own], 1), page, pp.num_pages)
    k, v = caches(None, kv, None, 3, 2, 4, pp)
    q = queries(3, kv * group, torch.float16, 6)

    def at(pages):
        return (api.ProdCache(k.idx, k.sgn, k.xnorm, k.rnorm, pages), api.MSECache(v.idx, v.xnorm, 2, pages))

    plan = api.PrefixPlan(3, kv * group, kv, 128, 100, 640, 640, torch.float16, torch.float16)
    got = plan.run(kc, vc, q, *at(pp), i32([plen]), *at(po), i32(lens), plan.new_out())
    dec = api.DecodePlan(3, kv * group, kv, 768, 768, torch.float16, torch.float32)
    want = dec.run(kc, vc, q, *at(both), i32([plen + n for n in lens]), dec.new_out())
    check_prefix(kc, vc, q, at(pp), at(po), got, plen, lens, kv, group)
    # both are within 1e-3 of the definition (the decode's bound, and fp16's operands here)
    off = (got.double() - want.double()).norm(dim=-1) / want.double().norm(dim=-1)
    assert float(off.max()) < 4e-3


def test_prefix_lengths_over_the_plan_are_clamped_and_flagged():
    a = run_prefix(3, 2, 2, 1, 2, 256, [64, 64], seed=5)
    kc, vc, q, pre, mine, plan, out = a
    assert flags() == 0
    again = plan.run(kc, vc, q, *pre, i32([300]), *mine, i32([64, 65]), plan.new_out())
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW
    assert torch.equal(out, again)


# ------------------------------------------------------------------ sparse attention

def check_sparse(kc, vc, q, k, v, lists, lens, out, group):
    for b, n in enumerate(lens):
        for h in range(lists.shape[1]):
            at = [np.arange(64 * i, min(64 * i + 64, n)) for i in lists[b, h].tolist()
                  if 0 <= i and 64 * i < n]
            at = torch.tensor(np.concatenate(at) if at else [], dtype=torch.long, device="cuda")
            rows = slice(h * group, (h + 1) * group)
            r, err = ref.attend(q[b, rows], parts(k, v, kc, vc, b, h, at), kc, vc,
                                pairs=out.dtype == torch.float16)
            ref.check_rows(out[b, rows], r, err, f"sequence {b}, KV head {h}")


def lists_of(lens, kv, keep, seed):
    """Random lists: any order, absent entries anywhere, out-of-range numbers, repeats."""
    rng = np.random.default_rng(seed)
    x = np.full((len(lens), kv, keep), -1)
    for b, n in enumerate(lens):
        nb = -(-n // 64)
        for h in range(kv):
            m = int(rng.integers(0, min(keep, nb) + 1))
            x[b, h, rng.permutation(keep)[:m]] = rng.permutation(nb)[:m]
            if keep > 3:
                x[b, h, 1] = x[b, h, 0]
                x[b, h, 2] = [nb, 1 << 30, -7][(b + h) % 3]
    return i32(x)


@pytest.mark.parametrize("batch,kv,group,lens,keep,paged,kbits,vbits", [
    (1, 1, 1, [1], 1, 0, 3, 4),
    (1, 1, 3, [100], 1, 0, 2, 1),
    (2, 2, 8, [0, 4000], 5, 0, 3, 2),
    (3, 4, 7, [129, 700, 5000], 16, 64, 4, 4),
    (3, 4, 7, [129, 700, 5000], 17, 256, 5, 3),
    (1, 8, 4, [70001], 300, 0, 3, 2),
    (40, 2, 5, [61 * i for i in range(40)], 9, 128, 4, 1),
])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_sparse_attention(batch, kv, group, lens, keep, paged, kbits, vbits, out_dtype):
    kc, vc = codec("k", kbits), codec("v", vbits)
    cap = up64(max(lens))
    pages = None
    if paged:
        cap = -(-cap // paged) * paged
        pages = table(batch, cap // paged, paged, 9)
    k, v = caches(batch, kv, cap, kbits, vbits, keep, pages, lens)
    hide(pages, lens)
    q = queries(batch, kv * group, torch.bfloat16, 1)
    lst = lists_of(lens, kv, keep, 2)
    plan = api.SparsePlan(batch, kv * group, kv, cap, max(lens), keep, 0, 0, out_dtype=out_dtype)
    out = plan.run(kc, vc, q, k, v, i32(lens), lst, plan.new_out())
    check_sparse(kc, vc, q, k, v, lst, lens, out, group)
    assert flags() == 0


def test_sparse_bad_page_is_skipped_and_flagged():
    kc, vc = codec("k", 3), codec("v", 2)
    pages = table(1, 4, 64, 1)
    k, v = caches(1, 1, 256, 3, 2, 3, pages)
    pages.block_table[0, 2] = pages.num_pages + 5
    q = queries(1, 2, torch.bfloat16, 1)
    plan = api.SparsePlan(1, 2, 1, 256, 256, 4, 0, 0, out_dtype=torch.float16)
    lens = i32([256])
    out = plan.run(kc, vc, q, k, v, lens, i32([[[0, 1, 3, -1]]]), plan.new_out())
    assert flags() == 0      # an entry that no listed token needs is not read
    got = plan.run(kc, vc, q, k, v, lens, i32([[[0, 1, 2, 3]]]), plan.new_out())
    assert flags() == B.TQ_FLAG_PAGE
    assert torch.allclose(got.float(), out.float(), rtol=4e-3, atol=4e-3)


# ------------------------------------------------------------------ block bounds

def special_(x, seed):
    """NaN, infinities and zeros of both signs among the values."""
    r = torch.rand(x.shape, generator=gen(seed), device="cuda")
    for i, v in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0)):
        x[(r > 0.01 * i) & (r < 0.01 * i + 0.01)] = v
    return x


def blank(batch, heads, cap, pages, seed):
    b = api.BlockBounds.empty(batch, heads, cap) if pages is None else \
        api.BlockBounds.empty_paged(pages, heads)
    b.bounds.copy_(torch.randn(b.bounds.shape, generator=gen(seed), device="cuda"))
    return b


def flat_bounds(b):
    if b.pages is None:
        return b.bounds
    return b.bounds[b.pages.block_table.long()].movedim(1, 2).flatten(2, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,heads,tokens,pos,count,paged", [
    (1, 1, 1, None, None, 0),
    (1, 2, 640, None, None, 0),
    (2, 3, 300, None, [0, 300], 0),
    (4, 2, 1, [0, 63, 64, 200], None, 64),
    (3, 4, 130, [1, 63, 700], [130, 2, 65], 192),
    (2, 1, 66, [62, 127], [66, 1], 0),
])
def test_block_bounds(dtype, batch, heads, tokens, pos, count, paged):
    cap = up64(max(pos or [0]) + tokens)
    pages = None
    if paged:
        cap = -(-cap // paged) * paged
        pages = table(batch, cap // paged, paged, 5)
    x = special_(3 * torch.randn(batch, heads, tokens, D, generator=gen(1), device="cuda"), 2).to(dtype)
    blocks = blank(batch, heads, cap, pages, 3)
    want = ref.bounds(x, pos or [0] * batch, count or [tokens] * batch, flat_bounds(blocks))
    spare = blocks.bounds.clone()
    whole = None if pages is None else pages.block_table.clone()
    hide(pages, [p + n for p, n in zip(pos or [0] * batch, count or [tokens] * batch)])
    api.block_bounds(x, blocks, None if pos is None else i32(pos), None if count is None else i32(count))
    if pages is not None:
        torch.cuda.synchronize()
        pages.block_table.copy_(whole)
    assert torch.equal(flat_bounds(blocks), want)
    if pages is not None:      # pages outside the table are left alone
        free = sorted(set(range(pages.num_pages)) - set(pages.block_table.flatten().tolist()))
        assert torch.equal(blocks.bounds[free], spare[free])
    assert flags() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_bounds_strides_and_alignment(dtype):
    """Token-major inputs, views that start at an odd element, and rows at an odd stride."""
    base = torch.randn(2 * 100 * 3 * 131 + 1, generator=gen(1), device="cuda").to(dtype)
    x = base[1:].view(2, 100, 3, 131)[..., 2:130].transpose(1, 2)      # [2, 3, 100, 128]
    for v in (x, torch.randn(2, 100, 3, D, generator=gen(2), device="cuda").to(dtype).transpose(1, 2),
              x[:1].expand(2, -1, -1, -1)):                            # a broadcast batch
        blocks = blank(2, 3, 128, None, 3)
        want = ref.bounds(v, [20, 0], [100, 100], blocks.bounds)
        api.block_bounds(v, blocks, i32([20, 0]))
        assert torch.equal(blocks.bounds, want)


def test_block_bounds_one_by_one_equal_a_prefill():
    x = torch.randn(2, 2, 200, D, generator=gen(1), device="cuda").half()
    a, b = blank(2, 2, 256, None, 2), blank(2, 2, 256, None, 2)
    api.block_bounds(x, a)
    at = i32([0, 0])
    for t in range(200):
        api.block_bounds(x[:, :, t:t + 1], b, pos=at)
        at += 1
    assert torch.equal(a.bounds, b.bounds)


def test_block_bounds_past_the_capacity():
    x = torch.randn(3, 1, 100, D, generator=gen(1), device="cuda").bfloat16()
    blocks = blank(3, 1, 128, None, 2)
    want = ref.bounds(x, [100, 0, 0], [28, 100, 0], blocks.bounds)
    api.block_bounds(x, blocks, i32([100, 0, -5]), i32([100, 1000, 100]))
    assert flags() == B.TQ_FLAG_POS_OVERFLOW
    assert torch.equal(blocks.bounds, want)


# ------------------------------------------------------------------ block selection

def run_select(q, blocks, lens, keep, first, last, group, kv, cap, max_len=None):
    plan = api.SparsePlan(len(lens), kv * group, kv, cap, max_len or max(max(lens), 1), keep, first,
                          last, q_dtype=q.dtype)
    out = plan.new_list()
    out.fill_(12345)
    return plan, plan.select(q, blocks, i32(lens), out)


def check_select(q, blocks, lens, keep, first, last, group, kv, got):
    flat = flat_bounds(blocks)
    for b, n in enumerate(lens):
        for h in range(kv):
            want = ref.select(q[b, h * group:(h + 1) * group], flat[b, h], -(-n // 64), keep, first, last)
            assert got[b, h].tolist() == want, (b, h)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,kv,group,lens,keep,first,last,paged", [
    (1, 1, 1, [64 * 7], 3, 0, 0, 0),
    (1, 2, 7, [64 * 40 - 5], 7, 1, 2, 0),
    (4, 2, 8, [0, 1, 640, 6400], 10, 3, 7, 64),      # all forced
    (4, 3, 3, [63, 64, 65, 64 * 300 + 1], 100, 0, 1, 128),
    (2, 1, 2, [64 * 5000, 64 * 131 + 2], 130, 2, 0, 0),
    (1, 1, 5, [64 * 33], 32, 1, 0, 0),
])
def test_block_select(dtype, batch, kv, group, lens, keep, first, last, paged):
    cap = up64(max(lens))
    pages = None
    if paged:
        cap = -(-cap // paged) * paged
        pages = table(batch, cap // paged, paged, 5)
    blocks = blank(batch, kv, cap, pages, 1)
    blocks.bounds[..., 1, :] += 2
    hide(pages, lens)
    q = queries(batch, kv * group, dtype, 2)
    _, got = run_select(q, blocks, lens, keep, first, last, group, kv, cap)
    check_select(q, blocks, lens, keep, first, last, group, kv, got)
    assert flags() == 0


def test_block_select_ties_and_near_ties():
    """Scores that differ by less than 32 bits hold, and blocks that are the same: the order is
    that of 64 bits, equal ones by the lower number."""
    n = 700
    blocks = blank(1, 2, 64 * n, None, 1)
    blocks.bounds[:, :, :] = blocks.bounds[:, :, :1]                 # every block alike
    blocks.bounds[0, 1, :, :, 0] = 256.0
    blocks.bounds[0, 1, :, :, 1] = torch.linspace(0, 699, n, device="cuda")[torch.randperm(
        n, generator=gen(3), device="cuda")][:, None].bfloat16()
    q = queries(1, 4, torch.float32, 2)
    q[0, 2:, 0] = 4096.0
    q[0, 2:, 1] = 2.0 ** -22
    _, got = run_select(q, blocks, [64 * n], 50, 2, 3, 2, 2, 64 * n)
    check_select(q, blocks, [64 * n], 50, 2, 3, 2, 2, got)
    assert got[0, 0].tolist() == list(range(47)) + [697, 698, 699]


@pytest.mark.parametrize("kind", ["zero queries", "infinite bounds", "NaN", "tiny"])
def test_block_select_odd_values(kind):
    n = 300
    blocks = blank(1, 1, 64 * n, None, 1)
    q = queries(1, 3, torch.float32, 2)
    if kind == "zero queries":
        q.zero_()
    elif kind == "infinite bounds":
        blocks.bounds[0, 0, 100:150, 1, 5] = math.inf
        blocks.bounds[0, 0, 120:180, 0, 9] = -math.inf
    elif kind == "NaN":
        blocks.bounds[0, 0, 10:60, 1] = math.nan
        blocks.bounds[0, 0, 10:60, 0] = math.nan
        q[0, 1, 3] = math.nan
    else:
        q *= 1e-30
        blocks.bounds *= 1e-8
    _, got = run_select(q, blocks, [64 * n], 64, 1, 1, 3, 1, 64 * n)
    check_select(q, blocks, [64 * n], 64, 1, 1, 3, 1, got)


def test_block_select_length_over_the_plan():
    blocks = blank(2, 1, 64 * 40, None, 1)
    q = queries(2, 2, torch.bfloat16, 2)
    plan, got = run_select(q, blocks, [64 * 30, 64 * 30], 8, 0, 1, 2, 1, 64 * 40)
    assert flags() == 0
    more = plan.select(q, blocks, i32([64 * 30, 64 * 31]), plan.new_list())
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW
    assert torch.equal(got, more)


# ------------------------------------------------------------------ used together, and otherwise

def test_sparse_step_loop():
    """A prefill's codes and bounds, then decode steps of SparsePlan.step (append, bounds, select,
    attend) on ragged sequences: lists and rows against the definitions on the cache as it is."""
    kc, vc = codec("k", 3), codec("v", 4)
    batch, kv, group, cap, keep = 3, 2, 4, 2048, 6
    k, v = api.ProdCache.empty(batch, kv, cap, 3), api.MSECache.empty(batch, kv, cap, 4)
    blocks = api.BlockBounds.empty(batch, kv, cap)
    x = torch.randn(batch, kv, 1500, D, generator=gen(1), device="cuda").bfloat16()
    y = torch.randn(batch, kv, 1500, D, generator=gen(2), device="cuda").bfloat16()
    lens = [1500, 703, 62]
    pos, now = i32(lens), i32([n + 1 for n in lens])
    api.quantize_prod(kc, x, k, count=pos)
    api.quantize_mse(vc, y, v, count=pos)
    api.block_bounds(x, blocks, count=pos)
    keys = [x[b, :, :n] for b, n in enumerate(lens)]
    plan = api.SparsePlan(batch, kv * group, kv, cap, cap, keep, 1, 1, out_dtype=torch.float16)
    out, lst = plan.new_out(), plan.new_list()
    for step in range(4):
        kn, vn = (torch.randn(batch, kv, D, generator=gen(10 + 2 * step + i), device="cuda").bfloat16()
                  for i in (0, 1))
        q = queries(batch, kv * group, torch.bfloat16, 50 + step)
        plan.step(kc, vc, q, kn, vn, k, v, blocks, pos, now, lst, out)
        lens = [n + 1 for n in lens]
        keys = [torch.cat([t, kn[b, :, None]], 1) for b, t in enumerate(keys)]
        for b, n in enumerate(lens):
            nb = -(-n // 64)
            padded = torch.nn.functional.pad(keys[b].float(), (0, 0, 0, nb * 64 - n), value=math.nan)
            t = padded.unflatten(1, (nb, 64))
            lo = torch.where(t.isnan(), math.inf, t).amin(2).bfloat16()
            hi = torch.where(t.isnan(), -math.inf, t).amax(2).bfloat16()
            assert torch.equal(blocks.bounds[b, :, :nb], torch.stack([lo, hi], 2))
        check_select(q, blocks, lens, keep, 1, 1, group, kv, lst)
        check_sparse(kc, vc, q, k, v, lst, lens, out, group)
        pos += 1
        now += 1
    assert flags() == 0


def test_all_blocks_listed_equal_the_dense_decode():
    """A list of every block attends what tq_decode_attention attends (fp32 output, its own
    kernel): both are near the definition, so they are near each other."""
    kc, vc = codec("k", 4), codec("v", 2)
    lens = [1000, 64, 1]
    k, v = caches(3, 2, 1024, 4, 2, 1, None, lens)
    q = queries(3, 10, torch.float16, 2)
    plan = api.SparsePlan(3, 10, 2, 1024, 1024, 16, 0, 0, torch.float16, torch.float16)
    lst = torch.arange(16, dtype=torch.int32, device="cuda").expand(3, 2, -1).contiguous()
    got = plan.run(kc, vc, q, k, v, i32(lens), lst, plan.new_out())
    dec = api.DecodePlan(3, 10, 2, 1024, 1024, torch.float16, torch.float32)
    want = dec.run(kc, vc, q, k, v, i32(lens), dec.new_out())
    off = (got.double() - want.double()).norm(dim=-1) / want.double().norm(dim=-1)
    assert float(off.max()) < 4e-3


def test_nan_queries_stay_in_their_rows():
    kc, vc = codec("k", 3), codec("v", 2)
    lens = [100, 200]
    k, v = caches(2, 1, 256, 3, 2, 1, None, lens)
    pk, pv = caches(1, 1, 192, 3, 2, 2)
    q = queries(2, 4, torch.float32, 3)
    plan = api.PrefixPlan(2, 4, 1, 256, 256, 192, 192, torch.float32, torch.float16)
    clean = plan.run(kc, vc, q, pk, pv, i32([150]), k, v, i32(lens), plan.new_out())
    q[1, 2, 7] = math.nan
    got = plan.run(kc, vc, q, pk, pv, i32([150]), k, v, i32(lens), plan.new_out())
    assert got[1, 2].isnan().all()
    got[1, 2] = clean[1, 2]
    assert torch.equal(got, clean)


def capture(fn, stream):
    g = torch.cuda.CUDAGraph()
    fn()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        fn()
    return g


def test_graphs_and_streams():
    """All four operators captured into one graph on a side stream and replayed on new inputs; the
    same calls on another stream than the current one; repeated calls give the same bits."""
    kc, vc = codec("k", 3), codec("v", 4)
    batch, kv, group, cap, keep = 4, 2, 7, 1024, 5
    lens = [1024, 800, 64, 3]
    k, v = caches(batch, kv, cap, 3, 4, 1, None, lens)
    pk, pv = caches(1, kv, 512, 3, 4, 2)
    x = torch.randn(batch, kv, cap, D, generator=gen(3), device="cuda").half()
    blocks = api.BlockBounds.empty(batch, kv, cap)
    q = queries(batch, kv * group, torch.float16, 4)
    sp = api.SparsePlan(batch, kv * group, kv, cap, cap, keep, 1, 1, torch.float16, torch.float16)
    pr = api.PrefixPlan(batch, kv * group, kv, cap, cap, 512, 512, torch.float16, torch.float16)
    n, pn = i32(lens), i32([500])
    lst, o1, o2 = sp.new_list(), sp.new_out(), pr.new_out()
    side = torch.cuda.Stream()

    def all_four(stream=None):
        api.block_bounds(x, blocks, count=n, stream=stream)
        sp.select(q, blocks, n, lst, stream=stream)
        sp.run(kc, vc, q, k, v, n, lst, o1, stream=stream)
        pr.run(kc, vc, q, pk, pv, pn, k, v, n, o2, stream=stream)

    all_four()
    torch.cuda.synchronize()
    first = [t.clone() for t in (blocks.bounds, lst, o1, o2)]
    side.wait_stream(torch.cuda.current_stream())
    all_four(stream=side)
    side.synchronize()
    for a, b in zip(first, (blocks.bounds, lst, o1, o2)):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        g = capture(all_four, side)
    for seed in (8, 9):
        q.copy_(queries(batch, kv * group, torch.float16, seed))
        x.copy_(torch.randn(x.shape, generator=gen(seed), device="cuda"))
        for t in (blocks.bounds, lst, o1, o2):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_select(q, blocks, lens, keep, 1, 1, group, kv, lst)
        check_sparse(kc, vc, q, k, v, lst, lens, o1, group)
        check_prefix(kc, vc, q, (pk, pv), (k, v), o2, 500, lens, kv, group)
    assert flags() == 0


def test_two_plans_at_once():
    """Two plans (a workspace each) on two streams, many calls in flight: rows as when alone."""
    kc, vc = codec("k", 3), codec("v", 2)
    lens = [640] * 6
    k, v = caches(6, 2, 640, 3, 2, 1)
    pk, pv = caches(1, 2, 4096, 3, 2, 2)
    q = [queries(6, 8, torch.bfloat16, s) for s in (3, 4)]
    plans = [api.PrefixPlan(6, 8, 2, 640, 640, 4096, 4096) for _ in q]
    n, pn = i32(lens), i32([4000])
    alone = [p.run(kc, vc, x, pk, pv, pn, k, v, n, p.new_out()).clone() for p, x in zip(plans, q)]
    streams = [torch.cuda.Stream() for _ in q]
    outs = [[p.new_out() for _ in range(20)] for p in plans]
    torch.cuda.synchronize()
    for i in range(20):
        for p, x, s, o in zip(plans, q, streams, outs):
            p.run(kc, vc, x, pk, pv, pn, k, v, n, o[i], stream=s)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        for t in o:
            assert torch.equal(a, t)


def test_growing_scores_move_the_reference():
    """Scores that rise along the sequence by far more than 2^8 a tile, and fall: the running
    reference follows, accumulators are scaled, and what was large first stays."""
    kc, vc = codec("k", 3), codec("v", 4)
    n = 1500
    for order in (1, -1):
        k, v = caches(1, 1, 1536, 3, 4, 1)
        ramp = torch.linspace(0.1, 60, 1536, device="cuda")
        k.xnorm.copy_(ramp if order == 1 else ramp.flip(0))
        k.rnorm.copy_(0.4 * k.xnorm)
        pk, pv = caches(1, 1, 1536, 3, 4, 2)
        pk.xnorm.copy_(ramp if order == 1 else ramp.flip(0))
        pk.rnorm.copy_(0.4 * pk.xnorm)
        for rows in (1, 8):
            q = queries(1, rows, torch.float32, 5, 4.0)
            for out_dtype in (torch.float16, torch.bfloat16):
                plan = api.PrefixPlan(1, rows, 1, 1536, 1536, 1536, 1536, torch.float32, out_dtype)
                out = plan.run(kc, vc, q, pk, pv, i32([n]), k, v, i32([n]), plan.new_out())
                check_prefix(kc, vc, q, (pk, pv), (k, v), out, n, [n], 1, rows)


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,group", [(4, 8), (5, 8), (8, 8), (9, 8), (16, 8), (17, 8)])
def test_rows_per_item(batch, group, out_dtype):
    """32, 40, 64, 72, 128 and 136 query rows of a KV head: a row in four lane groups, in two, in
    one, and in two row tiles."""
    lens = [(53 * i) % 90 for i in range(batch)]
    a = run_prefix(3, 2, batch, 1, group, 700, lens, out_dtype=out_dtype, seed=batch)
    check_prefix(*a[:5], a[6], 700, lens, 1, group)


def test_python_layer_refuses_on_the_gpu():
    kc, vc = codec("k", 3), codec("v", 2)
    k, v = caches(2, 2, 128, 3, 2, 1)
    q = queries(2, 4, torch.bfloat16, 1)
    n = i32([100, 3])
    plan = api.SparsePlan(2, 4, 2, 128, 128, 2, 0, 0)
    lst, out = plan.new_list(), plan.new_out()
    lst.zero_()
    plan.run(kc, vc, q, k, v, n, lst, out)
    bad = [(q.float(), k, v, n, lst, out), (q[:1], k, v, n, lst, out), (q, k, v, n.long(), lst, out),
           (q, k, v, n.cpu(), lst, out), (q, k, v, n, lst[:, :1], out), (q, k, v, n, lst, out.float()),
           (q.transpose(0, 1).contiguous().transpose(0, 1), k, v, n, lst, out),
           (q, api.ProdCache.empty(2, 2, 64, 3), v, n, lst, out),
           (q, api.ProdCache.empty(2, 2, 128, 4), v, n, lst, out),
           (q, k, api.MSECache.empty(1, 2, 128, 2), n, lst, out)]
    for args in bad:
        with pytest.raises(ValueError):
            plan.run(kc, vc, *args)
    with pytest.raises(ValueError):      # codecs in each other's place
        plan.run(vc, kc, q, k, v, n, lst, out)
    assert B.tq_sparse_attention(plan.desc, vc.handle, kc.handle, q, k.c(), v.c(), n, lst, 2, out,
                                 plan.workspace, plan.nbytes, None) == B.TQ_ERR_INVALID_ARG
    x = torch.randn(2, 2, 5, D, device="cuda")
    blocks = api.BlockBounds.empty(2, 2, 128)
    for args in ((x[..., :64], blocks), (x, api.BlockBounds.empty(2, 3, 128)), (x, blocks, n.long()),
                 (x.cpu(), blocks), (x, blocks, i32([1]))):
        with pytest.raises((ValueError, TypeError)):
            api.block_bounds(*args)
    with pytest.raises(TypeError):
        api.block_bounds(x.double(), blocks)


def test_offsets_past_32_bits():
    """A cache whose code arrays are longer than 4 GiB: the last sequence's last head lies behind
    that, and so do its blocks' bounds behind 2^29 elements."""
    kc, vc = codec("k", 3), codec("v", 2)
    batch, kv, cap = 17, 8, 1 << 20
    k, v = api.ProdCache.empty(batch, kv, cap, 3), api.MSECache.empty(batch, kv, cap, 2)
    assert k.idx.numel() > 1 << 32
    g = gen(1)
    n = cap - 5
    for t in (k.idx, k.sgn, v.idx):
        last = t[-1, -1]
        last.copy_(torch.randint(0, 256, last.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (k.xnorm, k.rnorm, v.xnorm):
        t[-1, -1] = 6 + 4 * torch.rand(cap, generator=g, device="cuda")
    lens = [0] * (batch - 1) + [n]
    q = queries(batch, 4 * kv, torch.bfloat16, 2)
    blocks = api.BlockBounds.empty(batch, kv, cap)
    blocks.bounds[-1, -1] = torch.randn(blocks.bounds.shape[2:], generator=g, device="cuda").bfloat16()
    plan = api.SparsePlan(batch, 4 * kv, kv, cap, cap, 6, 0, 1, out_dtype=torch.float16)
    lst = plan.select(q, blocks, i32(lens), plan.new_list())
    want = ref.select(q[-1, -4:], blocks.bounds[-1, -1], -(-n // 64), 6, 0, 1)
    assert lst[-1, -1].tolist() == want
    out = plan.run(kc, vc, q, k, v, i32(lens), lst, plan.new_out())
    at = torch.tensor([t for i in want for t in range(64 * i, min(64 * i + 64, n))], device="cuda")
    r, err = ref.attend(q[-1, -4:], parts(k, v, kc, vc, batch - 1, kv - 1, at), kc, vc, pairs=True)
    ref.check_rows(out[-1, -4:], r, err, "last head")
    assert not out[:-1].any() and flags() == 0
    x = torch.randn(1, kv, 3, D, generator=g, device="cuda").bfloat16().expand(batch, -1, -1, -1)
    pos = i32([0] * (batch - 1) + [n])
    api.block_bounds(x, blocks, pos, i32([0] * (batch - 1) + [3]))
    old = ref.bounds(x[-1:], [n], [3], blocks.bounds[-1:].clone())
    assert torch.equal(blocks.bounds[-1:], old)
