"""Moving codes inside a cache (include/tq.h: tq_copy_pages, tq_keep_tokens): every array afterwards is
what the definition makes of it, bit for bit."""
import numpy as np
import pytest
import torch

from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import caches, capture, flags, gen, i32, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


def arrays(k, v):
    return [k.idx, k.sgn, k.xnorm, k.rnorm, v.idx, v.xnorm]


def bounds(pages, heads, slots, seed):
    b = api.BlockBounds.empty(pages, heads, slots)
    b.bounds.copy_(torch.randn(b.bounds.shape, generator=gen(seed), device="cuda"))
    return b


# ------------------------------------------------------------------ pages

def run_copy(pairs, k, v, blocks=None, want=None):
    """Copies, and compares with copying the pairs `want` (all) one array at a time."""
    every = arrays(k, v) + ([blocks.bounds] if blocks else [])
    before = [t.clone() for t in every]
    src, dst = (i32([p[e] for p in pairs]) for e in (0, 1))
    api.copy_pages(src, dst, k, v, blocks)
    for t, old in zip(every, before):
        ref = old.clone()
        for a, b in (pairs if want is None else want):
            ref[b] = old[a]
        assert torch.equal(t, ref)


@pytest.mark.parametrize("kbits,vbits", [(2, 1), (3, 2), (4, 3), (5, 4)])
@pytest.mark.parametrize("heads,page", [(1, 64), (3, 192), (8, 256)])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_copy_pages(n, heads, page, kbits, vbits):
    """Few pages (many CTAs share one) and many; a source may be copied several times."""
    k, v = caches(100, heads, page, kbits, vbits, 1)
    order = np.random.default_rng(n).permutation(100).tolist()
    pairs = [(order[i // 2], order[50 + i]) for i in range(n)]
    run_copy(pairs, k, v, bounds(100, heads, page, 2))
    assert flags() == 0


def test_copy_many_small_pages():
    k, v = caches(6000, 1, 64, 3, 2, 1)
    order = np.random.default_rng(1).permutation(6000).tolist()
    run_copy(list(zip(order[:3000], order[3000:])), k, v)
    assert flags() == 0


def test_copy_parts_of_a_cache():
    """Keys alone, values alone, bounds alone: nothing else moves."""
    for which in range(3):
        k, v = caches(10, 2, 128, 3, 4, 1)
        b = bounds(10, 2, 128, 2)
        every = arrays(k, v) + [b.bounds]
        before = [t.clone() for t in every]
        api.copy_pages(i32([3]), i32([7]), *[x if i == which else None for i, x in enumerate((k, v, b))])
        for i, (t, old) in enumerate(zip(every, before)):
            if (0 if i < 4 else 1 if i < 6 else 2) == which:
                old[7] = old[3]
            assert torch.equal(t, old)


def test_copy_passes_over_and_refuses_pairs():
    k, v = caches(20, 2, 64, 4, 2, 1)
    run_copy([(-1, 4), (5, -1), (-1, -1), (2, 3), (6, 6)], k, v, want=[(2, 3)])
    assert flags() == 0
    for bad in ([(20, 4)], [(4, 20)], [(-2, 4)], [(4, -7)], [(2 ** 31 - 1, 5)], [(-2 ** 31, 5)]):
        run_copy(bad + [(1, 2)], k, v, want=[(1, 2)])
        assert flags() == B.TQ_FLAG_PAGE
    # a page that two pairs write, and one that is read and written
    run_copy([(1, 9), (2, 9), (3, 4)], k, v, want=[(3, 4)])
    assert flags() == B.TQ_FLAG_PAGE
    run_copy([(1, 2), (2, 3)], k, v, want=[(2, 3)])
    assert flags() == B.TQ_FLAG_PAGE
    run_copy([(1, 2), (2, 1)], k, v, want=[])
    assert flags() == B.TQ_FLAG_PAGE
    # neither a pair that is passed over nor a page copied to itself is in the way
    run_copy([(1, 2), (2, -1), (-1, 2), (2, 2), (1, 1)], k, v, want=[(1, 2)])
    assert flags() == 0
    api.copy_pages(i32([]), i32([]), k, v)


@pytest.mark.parametrize("at", [0, 299, 300, 700])
def test_copy_finds_a_clash_anywhere_in_a_long_list(at):
    k, v = caches(2000, 1, 64, 2, 1, 1)
    pairs = [(i, 1000 + i) for i in range(701)]
    pairs[at] = (at, 1000 + 350 if at != 350 else 1000)
    run_copy(pairs, k, v, want=[p for i, p in enumerate(pairs) if i not in (at, 350)])
    assert flags() == B.TQ_FLAG_PAGE


@pytest.mark.parametrize("n,heads,page", [(2000, 1, 64), (2100, 2, 64), (2300, 2, 64), (7000, 2, 192), (65536, 1, 64)])
def test_copy_long_lists(n, heads, page):
    """Clashes between pairs that lie far apart or side by side, bad pages, pairs that are passed over and
    pages onto themselves, in lists up to the longest; sources may repeat."""
    pages = 2 * n + 7
    k, v = caches(pages, heads, page, 2, 1, 1)
    b = bounds(pages, heads, page, 2)
    rng = np.random.default_rng(n)
    order = rng.permutation(pages)
    src, dst = order[:n].astype(np.int64), order[n:2 * n].astype(np.int64)
    src[rng.integers(0, n, n // 3)] = src[0]                # (a repeated source)
    used = rng.permutation(n)[:590]
    for i, j in zip(used[:100], used[100:200]):
        dst[i] = dst[j]                                     # two write one page
    for i in range(0, n - 1, max(n // 50, 2)):
        dst[i] = dst[i + 1]                                 # neighbours in the list
    for i, j in zip(used[200:300], used[300:400]):
        src[i] = dst[j]                                     # one reads what another writes
    dst[used[400:450]] = src[used[400:450]]                 # onto itself
    src[used[450:500]], dst[used[500:550]] = -1, -1
    src[used[550:560]], dst[used[560:570]], dst[used[570:580]], src[used[580:590]] = pages, pages + 5, -2, -2 ** 31
    moves = (src >= 0) & (dst >= 0) & (src != dst)
    writes = np.bincount(dst[moves & (dst < pages)], minlength=pages)
    reads = np.bincount(src[moves & (src < pages)], minlength=pages)
    good = [i for i in range(n) if moves[i] and src[i] < pages and dst[i] < pages and writes[dst[i]] == 1 and not reads[dst[i]]]
    assert n // 2 < len(good) < n - 300
    every = arrays(k, v) + [b.bounds]
    want = [t.clone() for t in every]
    at = torch.tensor(good, device="cuda")
    s, d = (torch.tensor(x, device="cuda") for x in (src, dst))
    for w, t in zip(want, every):
        w[d[at]] = t[s[at]]
    api.copy_pages(s.int(), d.int(), k, v, b)
    assert all(torch.equal(t, w) for t, w in zip(every, want))
    assert flags() == B.TQ_FLAG_PAGE
    # the good pairs alone, and into themselves again: nothing changes, nothing is flagged
    api.copy_pages(s[at].int(), d[at].int(), k, v, b)
    assert all(torch.equal(t, w) for t, w in zip(every, want))
    assert flags() == 0


def test_copy_long_lists_of_parts_of_a_cache():
    n = 5000
    order = np.random.default_rng(5).permutation(2 * n)
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (order[:n], order[n:]))
    k, v = caches(2 * n, 3, 64, 5, 4, 3)
    b = bounds(2 * n, 3, 64, 4)
    for which in range(3):
        every = arrays(k, v) + [b.bounds]
        want = [t.clone() for t in every]
        for i, t in enumerate(want):
            if (0 if i < 4 else 1 if i < 6 else 2) == which:
                t[dst.long()] = t[src.long()]
        api.copy_pages(src, dst, *[x if i == which else None for i, x in enumerate((k, v, b))])
        assert all(torch.equal(t, w) for t, w in zip(every, want))
    assert flags() == 0


def test_copy_offsets_past_32_bits():
    """A pool of more than 4 GiB of value codes."""
    n = 40000
    v = api.MSECache.empty(n, 8, 256, 4)
    assert v.idx.numel() > 1 << 32
    v.idx[1].copy_(torch.randint(0, 256, v.idx[1].shape, generator=gen(1), device="cuda", dtype=torch.uint8))
    v.xnorm[1] = 3
    api.copy_pages(i32([1]), i32([n - 1]), v=v)
    api.copy_pages(i32([n - 1]), i32([n // 2]), v=v)
    for i in (n - 1, n // 2):
        assert torch.equal(v.idx[i], v.idx[1]) and torch.equal(v.xnorm[i], v.xnorm[1])
    assert int((v.idx.view(n, -1).view(torch.int64) != 0).any(1).sum()) == 3
    assert flags() == 0


# ------------------------------------------------------------------ tokens

def kept(t, slots_dim, pages, pos, keep, skip=()):
    """Array t after the tokens were kept, from the definition."""
    old, new = t.movedim(slots_dim, 1).clone(), t.clone()
    view = new.movedim(slots_dim, 1)
    for b, (p, row) in enumerate(zip(pos, keep)):
        for i, j in enumerate(row):
            if j < 0 or (b, i) in skip:
                continue
            if pages is None:
                view[b, p + i] = old[b, p + j]
            else:
                pt, bt = pages.page_tokens, pages.block_table[b].tolist()
                view[bt[(p + i) // pt], (p + i) % pt] = old[bt[(p + j) // pt], (p + j) % pt]
    return new


def run_keep(k, v, pos, keep, skip=()):
    every = arrays(k, v)
    dims = [3, 2, 2, 2, 2 if v.bits == 4 else 3, 2]
    want = [kept(t, d, k.pages if i < 4 else v.pages, pos, keep, skip) for i, (t, d) in enumerate(zip(every, dims))]
    api.keep_tokens(k, v, i32(pos), i32(keep).view(len(pos), -1))
    for t, w in zip(every, want):
        assert torch.equal(t, w)


def make(batch, heads, cap, kbits, vbits, paged):
    """Flat, one table for both, or tables and page sizes of their own."""
    if not paged:
        return caches(batch, heads, cap, kbits, vbits, 1)
    kp = table(batch, cap // paged, paged, 5)
    vp = kp if paged != 64 else table(batch, cap // 192, 192, 6)
    return caches(batch, heads, cap, kbits, vbits, 1, kp)[0], caches(batch, heads, cap, kbits, vbits, 2, vp)[1]


@pytest.mark.parametrize("kbits,vbits", [(2, 1), (3, 2), (4, 3), (5, 4)])
@pytest.mark.parametrize("paged", [0, 64, 192])
@pytest.mark.parametrize("batch,heads,most", [(1, 1, 1), (3, 2, 5), (5, 4, 64)])
def test_keep_tokens(batch, heads, most, paged, kbits, vbits):
    """Ascending paths, lists in any order with repeats (all read first), and empty entries; across
    block and page borders."""
    k, v = make(batch, heads, 576, kbits, vbits, paged)
    rng = np.random.default_rng(most)
    pos = [int(x) for x in rng.integers(0, 512 - most, batch)]
    pos[0] = 190
    run_keep(k, v, pos, [sorted(rng.permutation(64)[:most].tolist()) for _ in pos])
    run_keep(k, v, pos, rng.integers(-1, most, (batch, most)).tolist())
    run_keep(k, v, pos, [[-1] * most for _ in pos])
    assert flags() == 0


def test_keep_from_far_behind():
    k, v = make(2, 2, 576, 3, 4, 192)
    run_keep(k, v, [0, 100], [[500, 3, 575], [475, 0, 300]])
    assert flags() == 0


def test_keep_past_the_capacity_and_bad_positions():
    k, v = make(3, 2, 128, 3, 4, 0)
    run_keep(k, v, [126, 120, 0], [[1, 0, 1], [7, 8, 2], [127, 128, 2 ** 31 - 1]], skip={(0, 2), (1, 1), (2, 1), (2, 2)})
    assert flags() == B.TQ_FLAG_POS_OVERFLOW
    run_keep(k, v, [-1, 2 ** 31 - 1, 5], [[1, 0], [0, 1], [3, 2]], skip={(0, 0), (0, 1), (1, 0), (1, 1)})
    assert flags() == B.TQ_FLAG_POS_OVERFLOW


@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_keep_leaves_out_bad_pages(which, bad):
    """A token whose page is bad in either cache stays in both."""
    k, v = make(2, 2, 576, 3, 2, 64)       # pages of 64 and of 192 tokens
    c, at = (k, 3) if which == "keys" else (v, 1)
    good = int(c.pages.block_table[0, at])
    c.pages.block_table[0, at] = bad
    before = [t.clone() for t in arrays(k, v)]
    api.keep_tokens(k, v, i32([190, 10]), i32([[9, 1, 0], [2, 0, 0]]))      # token 192 begins page 3 (1)
    c.pages.block_table[0, at] = good
    after = [t.clone() for t in arrays(k, v)]
    for t, old in zip(arrays(k, v), before):
        t.copy_(old)
    assert flags() == B.TQ_FLAG_PAGE
    dims = [3, 2, 2, 2, 3, 2]
    for i, (t, got) in enumerate(zip(arrays(k, v), after)):
        # of sequence 0 only entry 1 (token 191, onto itself) has good pages
        assert torch.equal(got, kept(t, dims[i], k.pages if i < 4 else v.pages, [190, 10], [[9, 1, 0], [2, 0, 0]],
                                     {(0, 0), (0, 2)}))


def test_graph_and_stream():
    k, v = caches(4, 2, 192, 3, 2, 1)
    pos, keep = i32([5, 60, 100, 0]), i32([[3, 1], [4, 4], [0, 9], [-1, 5]])
    src, dst = i32([0]), i32([3])
    side = torch.cuda.Stream()

    def both(stream=None):
        api.keep_tokens(k, v, pos, keep, stream=stream)
        api.copy_pages(src, dst, k, v, stream=stream)

    saved = [t.clone() for t in arrays(k, v)]

    def reset():
        for t, old in zip(arrays(k, v), saved):
            t.copy_(old)
        torch.cuda.synchronize()

    both()
    torch.cuda.synchronize()
    want = [t.clone() for t in arrays(k, v)]
    assert not torch.equal(want[0], saved[0])
    reset()
    both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, arrays(k, v)))
    with torch.cuda.stream(side):
        g = capture(both, side)
    reset()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, arrays(k, v)))
    assert flags() == 0


def test_refusals_on_the_gpu():
    k, v = caches(4, 2, 128, 3, 2, 1)
    other = caches(4, 3, 128, 3, 2, 1)[1]
    p, keep = i32([0] * 4), i32([[0]] * 4)
    b = bounds(4, 2, 64, 1)
    for bad in (lambda: api.keep_tokens(k, other, p, keep), lambda: api.keep_tokens(k, v, p.long(), keep),
                lambda: api.keep_tokens(k, v, p, keep[:3]), lambda: api.keep_tokens(k, v, p, keep[:, 0]),
                lambda: api.keep_tokens(k, v, i32([0] * 5), i32([[0]] * 5)), lambda: api.keep_tokens(k, v, p.cpu(), keep),
                lambda: api.copy_pages(p, p[:3], k, v), lambda: api.copy_pages(p, p, k, other),
                lambda: api.copy_pages(p, p), lambda: api.copy_pages(p, p, k, v, b),
                lambda: api.copy_pages(p.cpu(), p, k), lambda: api.copy_pages(p.long(), p.long(), k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.TQError):
        api.keep_tokens(k, v, p, i32([[0] * 65] * 4))
    assert flags() == 0
