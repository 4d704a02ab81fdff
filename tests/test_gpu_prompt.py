"""Attention of packed prompts on exact keys (include/tq.h: tq_prompt_attention) against its definition
in 64 bits."""
import math

import pytest
import torch

import longctx_ref as ref
from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import capture, flags, gen, i32, parts

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def attend(q, k, v, causal, scale, dtype):
    """Rows of queries q [nq, 128] over k, v [nk, 128] in 64 bits, and the standard deviation of the
    error (2-norm) that the kernel's roundings allow.

    Weights are off by at most u = eps/2 of the type, uniform and independent (standard deviation
    u / √3): u/√3 · √Σ p²‖v‖².  A score is off by at most 2^-20 of the sum of its products' sizes
    (32-bit sums of 128 exact products, the argument of the power, the power itself 2^-22), which
    moves a row by p·δ·(‖v‖ + ‖out‖) at most; taken as eight deviations, as are 2^-20 for the sums
    over keys and, in fp16, 2^-32 of the largest weight for each of those it holds as subnormals."""
    q, k, v = q.double(), k.double(), v.double()
    nq, nk = len(q), len(k)
    if nk == 0:
        return torch.zeros(nq, D, dtype=torch.float64, device=q.device), torch.zeros(nq, dtype=torch.float64, device=q.device)
    s = scale * (q @ k.T)
    if causal:
        s = s.masked_fill(torch.arange(nk, device=q.device) > (torch.arange(nq, device=q.device) + nk - nq)[:, None], -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)          # (a row without a key: zero)
    out = p @ v
    u = torch.finfo(dtype).eps / 2 / math.sqrt(3)
    size = v.norm(dim=-1)
    delta = 2.0 ** -20 * scale * (q.abs() @ k.abs().T) + 2.0 ** -22
    err = u * ((p * size) ** 2).sum(-1).sqrt()
    err = err + (p * delta * (size + out.norm(dim=-1, keepdim=True))).sum(-1) / 8 + 2.0 ** -20 * (p * size).sum(-1) / 8
    if dtype == torch.float16:
        err = err + 2.0 ** -32 * nk * size.max() / 8
    return out, err


def check(q, k, v, qs, ks, out, causal, scale=None):
    scale = scale or 1 / math.sqrt(D)
    group = q.shape[1] // k.shape[1]
    for b in range(len(qs) - 1):
        for h in range(q.shape[1]):
            kk, vv = (t[ks[b]:ks[b + 1], h // group] for t in (k, v))
            for i in range(qs[b], qs[b + 1], 2048):          # rows in parts: scores in 64 bits are large
                j = min(i + 2048, qs[b + 1])
                nk, behind = ks[b + 1] - ks[b], qs[b + 1] - j
                end = max(nk - behind, 0) if causal else nk
                r, err = attend(q[i:j, h], kk[:end], vv[:end], causal, scale, q.dtype)
                ref.check_rows(out[i:j, h], r, err, f"sequence {b}, head {h}, rows from {i - qs[b]}")


def inputs(nq, nk, kv, group, dtype, seed, fused=False, before=0, behind=0):
    """q, k, v with rows of no sequence (NaN) before and behind."""
    g = gen(seed)
    tq, tk = before + sum(nq) + behind, before + sum(nk) + behind
    hq = kv * group
    if fused:
        x = torch.randn(tq, hq + 2 * kv + 1, D, generator=g, device="cuda").to(dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + kv], x[:, hq + kv:hq + 2 * kv]
    else:
        q, k, v = (torch.randn(t, h, D, generator=g, device="cuda").to(dtype) for t, h in ((tq, hq), (tk, kv), (tk, kv)))
    for t, n in ((q, sum(nq)), (k, sum(nk)), (v, sum(nk))):
        t[:before] = math.nan
        t[before + n:] = math.nan
    return q, k, v


def run(nq, nk, kv, group, dtype, causal=True, seed=0, fused=False, before=0, behind=0, scale=None, longest=None):
    q, k, v = inputs(nq, nk, kv, group, dtype, seed, fused, before, behind)
    qs, ks = starts(nq, before), starts(nk, before)
    plan = api.PromptPlan(len(nq), kv * group, kv, len(q), len(k), max(nk) if longest is None else longest, causal, dtype, scale)
    out = plan.new_out().fill_(7)
    plan.run(q, k, v, i32(qs), i32(ks), out)
    check(q, k, v, qs, ks, out, causal, scale)
    assert (out[:before] == 7).all() and (out[before + sum(nq):] == 7).all()
    assert flags() == 0
    return q, k, v, qs, ks, plan, out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("group", range(1, 9))
def test_groups(group, causal, dtype):
    """Every group size, in one block of rows a CTA (few tokens) and in two."""
    run([5, 300, 1, 40], [5, 300, 1, 40], 2, group, dtype, causal, seed=group, fused=True)
    run([700, 129], [700, 129], 8, group, dtype, causal, seed=group)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [
    ([1], [1]),
    ([1], [2]),
    ([0, 1, 0], [5, 3, 0]),                        # no queries, no keys
    ([3, 2], [0, 0]),                              # queries without keys: zero rows
    ([10, 200, 7], [4, 120, 7]),                   # more queries than keys: causal rows without one
    ([1, 1, 1], [127, 128, 129]),
    ([18, 19, 36, 37], [1000, 1001, 18, 555]),
    ([127, 128, 129, 255], [127, 128, 129, 255]),
    ([64] * 3, [5000, 64, 300]),
    ([2] * 40, [50 + i for i in range(40)]),
])
def test_lengths(nq, nk, causal, dtype):
    for group in (1, 7):
        run(nq, nk, 2, group, dtype, causal, seed=len(nq) + group, before=3, behind=2)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,kv,group,nk", [(1, 1, 8, 20000), (3, 2, 7, 4097), (8, 4, 7, 8192), (1, 4, 1, 513)])
def test_single_tokens_behind_long_histories(batch, kv, group, nk, dtype):
    """Keys are split over CTAs; loose and tight bounds of the lengths."""
    lens = [nk - 7 * b for b in range(batch)]
    run([1] * batch, lens, kv, group, dtype, seed=batch)
    run([1] * batch, lens, kv, group, dtype, seed=batch, longest=4 * nk)
    run([1] * batch, lens, kv, group, dtype, seed=batch, longest=0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_prompts(dtype):
    run([5000, 3001], [5000, 3001], 4, 4, dtype, seed=1, fused=True)
    run([300], [9000], 1, 8, dtype, seed=2)
    run([4096], [4096], 1, 1, dtype, False, seed=3)


def test_scales():
    for scale in (0.01, 1.0):
        run([200, 50], [300, 50], 2, 3, torch.bfloat16, seed=4, scale=scale)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("order", [1, -1])
def test_growing_scores_move_the_reference(order, dtype):
    """Scores that rise along the keys by far more than 2^8 a tile, and fall."""
    nk = 1500
    for nq in (4, 600):
        q, k, v = inputs([nq], [nk], 1, 4, dtype, 5)
        ramp = torch.linspace(0.05, 12, nk, device="cuda")
        k.copy_(torch.randn(1, 1, D, generator=gen(6), device="cuda") * (ramp if order == 1 else ramp.flip(0))[:, None, None])
        plan = api.PromptPlan(1, 4, 1, nq, nk, nk, True, dtype)
        out = plan.run(q, k, v, i32([0, nq]), i32([0, nk]), plan.new_out())
        check(q, k, v, [0, nq], [0, nk], out, True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tail", [20.2, 24.6, 25.1])
def test_a_peak_before_a_long_even_tail(tail, dtype):
    """One key of weight 1 and then 65535 equal ones of weight 2^-tail: the tail's sum counts in full.
    Off by at most, relative to the values' norm 10: the output's rounding, the weights' rounding (in
    the same direction for all of the tail, whose share is n·2^-tail: two halves of a step), the
    score's 2^-20 of its 25 units of log 2, and 2^-32 of the largest weight for each key."""
    n = 65536
    q = torch.zeros(1, 2, D, dtype=dtype, device="cuda")
    k = torch.zeros(n, 2, D, dtype=dtype, device="cuda")
    v = torch.zeros(n, 2, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    scale = 1.0
    k[1:, :, 0] = -tail * math.log(2)
    v[0, :, 0], v[1:, :, 1] = 10, 10
    plan = api.PromptPlan(1, 2, 2, 1, n, n, True, dtype, scale)
    out = plan.run(q, k, v, i32([0, 1]), i32([0, n]), plan.new_out())
    r, _ = attend(q[:, 0], k[:, 0], v[:, 0], True, scale, dtype)
    share = float(r[0, 1]) / 10
    step = torch.finfo(dtype).eps / 2
    most = 10 * (step + 2 * step * share + share * 25 * 2.0 ** -18 + (n * 2.0 ** -32 if dtype == torch.float16 else 0) + 2.0 ** -20)
    assert float((out.double() - r).norm(dim=-1).max()) <= most


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("nq,nk,at", [(300, 300, 130), (300, 300, 299), (5, 900, 897), (2, 20000, 19999), (40, 40, 0), (700, 700, 255)])
def test_what_a_row_does_not_attend_does_not_show(nq, nk, at, which, bad, dtype):
    """An infinite or NaN key or value at a key that later rows attend: earlier rows keep every bit."""
    q, k, v = inputs([nq], [nk], 2, 3, dtype, 7)
    plan = api.PromptPlan(1, 6, 2, nq, nk, nk, True, dtype)
    n = (i32([0, nq]), i32([0, nk]))
    clean = plan.run(q, k, v, *n, plan.new_out())
    (k if which == "k" else v)[at, 1, 77] = bad
    got = plan.run(q, k, v, *n, plan.new_out())
    first = max(at - (nk - nq), 0)                # rows from this one on attend it
    assert torch.equal(got[:first], clean[:first])
    assert torch.equal(got[:, :3], clean[:, :3])  # the other KV head's
    if which == "v":
        assert not got[first:, 3:, 77].isfinite().any()
        got[first:, 3:, 77] = clean[first:, 3:, 77]
        assert torch.equal(got, clean)
    elif math.isnan(bad):
        assert got[first:, 3:].isnan().all()
    assert flags() == 0


def test_infinite_values_of_both_signs():
    """Rows that attend +∞ alone, −∞ too (NaN), and neither."""
    q, k, v = inputs([200], [200], 1, 2, torch.bfloat16, 8)
    clean = v.clone()
    v[50, 0, 3], v[190, 0, 3], v[195, 0, 3] = math.inf, math.inf, -math.inf
    plan = api.PromptPlan(1, 2, 1, 200, 200, 200)
    n = i32([0, 200])
    got = plan.run(q, k, v, n, n, plan.new_out())
    want = plan.run(q, k, clean, n, n, plan.new_out())
    assert (got[50:195, :, 3] == math.inf).all() and got[195:, :, 3].isnan().all()
    assert torch.equal(got[:50], want[:50])


def test_nan_queries_stay_in_their_rows():
    q, k, v = inputs([100, 30], [100, 30], 2, 4, torch.float16, 9)
    plan = api.PromptPlan(2, 8, 2, 130, 130, 100, dtype=torch.float16)
    n = i32([0, 100, 130])
    clean = plan.run(q, k, v, n, n, plan.new_out())
    q[55, 3, 1], q[129, 6] = math.nan, math.nan
    got = plan.run(q, k, v, n, n, plan.new_out())
    assert got[55, 3].isnan().all() and got[129, 6].isnan().all()
    got[55, 3], got[129, 6] = clean[55, 3], clean[129, 6]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_neighbours_do_not_show(dtype):
    """A sequence's rows do not depend on what is packed beside it, NaN and infinite among it."""
    q, k, v = inputs([77, 130, 60], [77, 130, 60], 2, 5, dtype, 10)
    plan = api.PromptPlan(3, 10, 2, 267, 267, 130, dtype=dtype)
    n = i32([0, 77, 207, 267])
    clean = plan.run(q, k, v, n, n, plan.new_out())
    check(q, k, v, [0, 77, 207, 267], [0, 77, 207, 267], clean, True)
    for t in (q, k, v):
        t[:77] = math.nan
        t[207:] = math.inf
    got = plan.run(q, k, v, n, n, plan.new_out())
    assert torch.equal(got[77:207], clean[77:207])


def test_a_prompt_in_chunks_equals_the_whole():
    """Chunks over the keys so far, each near the definition; the last one a single token."""
    n, kv, group = 500, 2, 4
    q, k, v = inputs([n], [n], kv, group, torch.bfloat16, 11)
    at = 0
    for chunk in (200, 100, 199, 1):
        plan = api.PromptPlan(1, 8, kv, chunk, at + chunk, at + chunk)
        out = plan.run(q[at:at + chunk], k[:at + chunk], v[:at + chunk], i32([0, chunk]), i32([0, at + chunk]), plan.new_out())
        check(q[at:at + chunk], k, v, [0, chunk], [0, at + chunk], out, True)
        at += chunk


def test_starts_that_do_not_ascend_are_clamped_and_flagged():
    q, k, v = inputs([100], [100], 1, 2, torch.bfloat16, 12)
    plan = api.PromptPlan(2, 2, 1, 100, 100, 100)
    good = i32([0, 60, 100])
    for bad in ([0, 60, 140], [-5, 60, 100], [0, 2 ** 31 - 1, 100], [90, 10, 100], [-2 ** 31, 0, -7]):
        for a, b in ((i32(bad), good), (good, i32(bad))):
            plan.run(q, k, v, a, b, plan.new_out())
            assert flags() == B.TQ_FLAG_LEN_OVERFLOW
    out = plan.run(q, k, v, i32([0, 60, 140]), i32([0, 60, 140]), plan.new_out())
    check(q, k, v, [0, 60, 100], [0, 60, 100], out, True)
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW


def test_no_keys_at_all_and_no_queries():
    q, k, v = inputs([5, 3], [0, 0], 2, 3, torch.bfloat16, 19)
    assert len(k) == 0
    out = torch.full((8, 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
    api.PromptPlan(2, 6, 2, 8, 0, 0).run(q, k, v, i32([0, 5, 8]), i32([0, 0, 0]), out)
    assert not out.any()
    q, k, v = inputs([0, 0], [5, 3], 2, 3, torch.bfloat16, 19)
    plan = api.PromptPlan(2, 6, 2, 0, 8, 5)
    plan.run(q, k, v, i32([0, 0, 0]), i32([0, 5, 8]), plan.new_out())
    assert flags() == 0


def test_queries_and_output_in_one_place():
    """A CTA reads its rows' queries before it writes them."""
    for nq, nk in (([300, 40], [300, 40]), ([1, 1], [5000, 70])):
        q, k, v = inputs(nq, nk, 2, 4, torch.float16, 20)
        plan = api.PromptPlan(2, 8, 2, sum(nq), sum(nk), max(nk), dtype=torch.float16)
        n = (i32(starts(nq)), i32(starts(nk)))
        want = plan.run(q, k, v, *n, plan.new_out())
        assert torch.equal(plan.run(q, k, v, *n, q), want)


def test_many_sequences():
    """More sequences than threads a block; all of one token, and none in most."""
    run([1] * 1000, [3] * 1000, 1, 2, torch.bfloat16, seed=13)
    lens = [0] * 900
    lens[0], lens[500], lens[899] = 40, 3, 200
    run(lens, lens, 1, 4, torch.float16, seed=14, before=1)


def test_graph_stream_and_two_plans():
    nq, nk = [1, 40, 3], [3000, 40, 500]
    q, k, v, qs, ks, plan, out = run(nq, nk, 2, 4, torch.bfloat16, seed=15)
    a, b = i32(qs), i32(ks)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = plan.new_out()
    plan.run(q, k, v, a, b, o, stream=side)
    side.synchronize()
    assert torch.equal(o, out)
    with torch.cuda.stream(side):
        g = capture(lambda: plan.run(q, k, v, a, b, o), side)
    q.copy_(torch.randn(q.shape, generator=gen(16), device="cuda"))
    a.copy_(i32([0, 20, 30, 44]))
    b.copy_(i32([0, 100, 3200, 3540]))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check(q, k, v, [0, 20, 30, 44], [0, 100, 3200, 3540], o, True)
    other = api.PromptPlan(3, 8, 2, len(q), len(k), max(nk))
    alone = plan.run(q, k, v, a, b, plan.new_out()).clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[plan.new_out() for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for p, s, os in zip((plan, other), streams, outs):
            p.run(q, k, v, a, b, os[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, alone) for os in outs for x in os)
    assert flags() == 0


def test_heads_before_tokens():
    """Views whose heads lie further apart than their tokens, of one sequence and of a step."""
    for nq, nk in (([300], [300]), ([1, 1], [2000, 700])):
        q, k, v, qs, ks, plan, out = run(nq, nk, 2, 3, torch.float16, seed=21)
        views = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
        assert all(t.stride(1) > t.stride(0) for t in views)
        assert torch.equal(plan.run(*views, i32(qs), i32(ks), plan.new_out()), out)
    assert flags() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,kv,group", [(40, 4, 7), (60, 4, 8), (9, 8, 5)])
def test_ragged_batches_of_few_rows(batch, kv, group, dtype):
    """More parts of keys than SMs, many of them empty: histories of 0 to 9000 keys, one of which is long;
    some sequences have more rows than a block."""
    g = torch.Generator().manual_seed(batch)
    nk = torch.randint(0, 900, (batch,), generator=g).tolist()
    nq = torch.randint(0, 4, (batch,), generator=g).tolist()
    nk[batch // 2] = 9000
    nq[batch // 2] = 2
    nk[1], nq[1] = 700, 50
    run(nq, nk, kv, group, dtype, seed=batch, before=2, behind=3)
    run(nq, nk, kv, group, dtype, causal=False, seed=batch + 1)


def test_two_blocks_of_rows_without_keys():
    """Long prompts, some of them without a key, in CTAs of two blocks of rows."""
    run([700, 700, 700, 40], [0, 700, 129, 0], 8, 7, torch.bfloat16, seed=22)
    run([700, 700, 700, 40], [0, 700, 129, 0], 8, 7, torch.float16, causal=False, seed=23)


def test_prompt_then_codes_then_decode():
    """A prompt as a program takes it in: positions, attention on exact keys, codes; then a decode step
    on the codes is near attention on the exact keys (as near as 5-bit keys and 4-bit values are)."""
    lens, kv, group = [200, 75], 2, 4
    q, k, v = inputs(lens, lens, kv, group, torch.bfloat16, 17, fused=True)
    qs = starts(lens)
    at = i32([i for n in lens for i in range(n)])[None]
    api.Rotary(128).apply(q.transpose(0, 1)[None], k.transpose(0, 1)[None], at)
    plan = api.PromptPlan(2, 8, 2, len(q), len(k), 200)
    out = plan.run(q, k, v, i32(qs), i32(qs), plan.new_out())
    check(q, k, v, qs, qs, out, True)
    kc, vc = api.Codec.prod(4), api.Codec.mse(4)
    kcache, vcache = api.ProdCache.empty(2, kv, 256, 4), api.MSECache.empty(2, kv, 256, 4)
    for b, n in enumerate(lens):
        rows = slice(qs[b], qs[b + 1])
        one = api.ProdCache(*[t[b:b + 1] for t in (kcache.idx, kcache.sgn, kcache.xnorm, kcache.rnorm)])
        api.quantize_prod(kc, k[rows].transpose(0, 1)[None], one)
        api.quantize_mse(vc, v[rows].transpose(0, 1)[None], api.MSECache(vcache.idx[b:b + 1], vcache.xnorm[b:b + 1], 4))
    last = torch.stack([q[e - 1] for e in qs[1:]])
    dec = api.DecodePlan(2, 8, 2, 256, 256, out_dtype=torch.float32)
    got = dec.run(kc, vc, last, kcache, vcache, i32(lens), dec.new_out())
    want = torch.stack([out[e - 1] for e in qs[1:]]).float()
    assert float((got - want).norm() / want.norm()) < 0.5
    assert flags() == 0


def test_prompt_codes_and_the_step_behind_them():
    """A prompt whose keys were turned where they lie is coded as the turned keys are by themselves, and a
    drafted token behind it attends those codes as their definition says."""
    lens, kv, group = [200, 75], 2, 4
    q, k, v = inputs(lens, lens, kv, group, torch.bfloat16, 29, fused=True)
    qs, rot = starts(lens), api.Rotary(128)
    at = i32([i for n in lens for i in range(n)])[None]
    raw_k = k.clone()
    rot.apply(q.transpose(0, 1)[None], k.transpose(0, 1)[None], at)
    plan = api.PromptPlan(2, 8, 2, len(q), len(k), 200)
    out = plan.run(q, k, v, i32(qs), i32(qs), plan.new_out())
    check(q, k, v, qs, qs, out, True)
    kc, vc = api.Codec.prod(4), api.Codec.mse(4)
    kcache, vcache = api.ProdCache.empty(2, kv, 256, 4), api.MSECache.empty(2, kv, 256, 4)
    for b, n in enumerate(lens):
        turned = torch.empty(1, kv, n, D, dtype=k.dtype, device="cuda")
        rot.apply(raw_k[qs[b]:qs[b + 1]].transpose(0, 1)[None], None, i32([list(range(n))]), turned)
        assert torch.equal(turned[0].transpose(0, 1), k[qs[b]:qs[b + 1]])
        one = api.ProdCache(*[t[b:b + 1] for t in (kcache.idx, kcache.sgn, kcache.xnorm, kcache.rnorm)])
        api.quantize_prod(kc, k[qs[b]:qs[b + 1]].transpose(0, 1)[None], one)
        api.quantize_mse(vc, v[qs[b]:qs[b + 1]].transpose(0, 1)[None], api.MSECache(vcache.idx[b:b + 1], vcache.xnorm[b:b + 1], 4))
        alone = api.ProdCache.empty(1, kv, 256, 4)
        api.quantize_prod(kc, turned, alone)
        for x, y, dim in ((alone.idx, one.idx, 3), (alone.sgn, one.sgn, 2), (alone.xnorm, one.xnorm, 2), (alone.rnorm, one.rnorm, 2)):
            assert torch.equal(x.narrow(dim, 0, n), y.narrow(dim, 0, n))
    # the last token of each prompt, as the one drafted token behind the others
    last = torch.stack([q[e - 1] for e in qs[1:]])[:, None].contiguous()
    step = api.TreePlan(2, 1, 8, 2, 256, 256, out_dtype=torch.float16)
    one = torch.ones(2, 1, dtype=torch.int64, device="cuda")
    got = step.run(kc, vc, last, kcache, vcache, i32([n - 1 for n in lens]), one, step.new_out())
    for b, n in enumerate(lens):
        for h in range(kv):
            p = parts(kcache, vcache, kc, vc, b, h, torch.arange(n, device="cuda"))
            r, err = ref.attend(last[b, 0, h * group:(h + 1) * group], p, kc, vc, None, True)
            ref.check_rows(got[b, 0, h * group:(h + 1) * group], r, err, f"sequence {b}, KV head {h}")
    assert flags() == 0


def test_offsets_past_32_bits():
    """Keys and values in rows more than 2^32 bytes long in all, queries at their end."""
    n, wide = 2100, 1 << 20
    x = torch.empty(n, wide, dtype=torch.bfloat16, device="cuda")
    k, v, q = (x[:, i * 1024:i * 1024 + 256].view(n, 2, D) for i in range(3))
    for i, t in enumerate((k, v, q)):
        t.copy_(torch.randn(n, 2, D, generator=gen(i), device="cuda"))
    plan = api.PromptPlan(1, 2, 2, n, n, n)
    out = plan.run(q, k, v, i32([0, n]), i32([0, n]), plan.new_out())
    check(q, k, v, [0, n], [0, n], out, True)


def test_refusals_on_the_gpu():
    q, k, v = inputs([10], [10], 2, 2, torch.bfloat16, 18)
    plan = api.PromptPlan(1, 4, 2, 10, 10, 10)
    n, out = i32([0, 10]), plan.new_out()
    odd = torch.empty(10, 2, 132, dtype=torch.bfloat16, device="cuda")[..., :D]      # strides of 132
    shifted = torch.empty(10 * 256 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(10, 2, D)
    for bad in (lambda: plan.run(q.float(), k, v, n, n, out), lambda: plan.run(q[:9], k, v, n, n, out),
                lambda: plan.run(q, k[:9], v, n, n, out), lambda: plan.run(q, k, v.half(), n, n, out),
                lambda: plan.run(q, k, v, n.long(), n, out), lambda: plan.run(q, k, v, n, n[:1], out),
                lambda: plan.run(q, k, v, n, n, out[:, ::2]), lambda: plan.run(q, k, v.cpu(), n, n, out),
                lambda: plan.run(q, k, v, n, n.cpu(), out), lambda: plan.run(q, odd, v, n, n, out),
                lambda: plan.run(q, k, shifted, n, n, out), lambda: plan.run(q, k[:, :1].expand(-1, 2, -1), v, n, n, out)):
        with pytest.raises((ValueError, B.TQError)):
            bad()
    assert flags() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,nk,group", [
    ([19, 3, 100], [60, 3, 100], 7),               # blocks of rows that are not full, rows 126 and 127 never are
    ([2, 18], [9000, 700], 7),                     # keys in parts
    ([5, 11], [5, 300], 3),                        # one tile, two streams of tiles
    ([700, 37, 600], [700, 37, 640], 5),           # two blocks of rows a CTA, the last of them in part
    ([1], [1], 8),
])
def test_values_given_back_in_blocks_that_are_not_full(nq, nk, group, dtype):
    """Infinite values at the ends of the sequences, in every quarter of the channels, which rows attend in
    different numbers: a row has those of the keys that it attends and keeps every other bit."""
    kv = 2 if sum(nq) < 500 else 8
    q, k, v = inputs(nq, nk, kv, group, dtype, 24, behind=2)
    qs, ks = starts(nq), starts(nk)
    plan = api.PromptPlan(len(nq), kv * group, kv, len(q), len(k), max(nk), True, dtype)
    n = (i32(qs), i32(ks))
    want = plan.run(q, k, v, *n, plan.new_out().fill_(7))
    check(q, k, v, qs, ks, want, True)
    for b, (m, rows) in enumerate(zip(nk, nq)):
        for i, c in enumerate((0, 31, 32, 50, 77, 95, 96, 127)):
            j = m - 1 - (5 * i) % min(rows, m)     # the last rows attend it
            v[ks[b] + j, 1, c] = math.inf
            for row in range(rows):
                if row + m - rows >= j:
                    want[qs[b] + row, group:2 * group, c] = math.inf
    assert torch.equal(plan.run(q, k, v, *n, plan.new_out().fill_(7)), want)
    assert flags() == 0


def test_output_beside_the_inputs_in_one_array():
    """An output in the room between two rows of keys is apart from them."""
    q, k, v = inputs([1], [90], 2, 4, torch.bfloat16, 25)
    n = (i32([0, 1]), i32([0, 90]))
    plan = api.PromptPlan(1, 8, 2, 1, 90, 90)
    want = plan.run(q, k, v, *n, plan.new_out())
    x = torch.full((90, 13, D), 3.0, dtype=torch.bfloat16, device="cuda")
    x[:, :2], x[:, 2:4] = k, v
    out = x[40, 5:13].view(1, 8, D)
    plan.run(q, x[:, :2], x[:, 2:4], *n, out)
    assert torch.equal(out, want)
    with pytest.raises(B.TQError):
        plan.run(q, x[:, :2], x[:, 2:4], *n, x[40, 3:11].view(1, 8, D))
    with pytest.raises(B.TQError):
        plan.run(x[40, 4:12].view(1, 8, D), k, v, *n, out)
    assert flags() == 0


@pytest.mark.parametrize("batch", [384, 385, 20000, 160000])
def test_more_sequences_than_a_block_looks_at_at_once(batch):
    """Single tokens that attend their one key are its value, bit for bit; the last sequence has none."""
    v = torch.randn(batch - 1, 1, D, generator=gen(26), device="cuda").bfloat16()
    q = torch.randn(batch - 1, 2, D, generator=gen(27), device="cuda").bfloat16()
    n = torch.arange(batch + 1, dtype=torch.int32, device="cuda").clamp(max=batch - 1)
    plan = api.PromptPlan(batch, 2, 1, batch - 1, batch - 1, 1)
    assert torch.equal(plan.run(q, v, v, n, n, plan.new_out()), v.expand(-1, 2, -1))
    # starts that do not ascend, anywhere in a long list
    n[batch - 5] = batch
    plan.run(q, v, v, n, n, plan.new_out())
    assert flags() == B.TQ_FLAG_LEN_OVERFLOW


def test_few_sequences_with_tokens_among_many():
    batch = 150000
    at = [0, 1, 383, 384, 390, 391, 392, 1000, 77777, 77778, batch - 392, batch - 1]
    lens = [0] * batch
    for i, b in enumerate(at):
        lens[b] = (3, 300, 1, 40, 18, 19)[i % 6]
    total = sum(lens)
    q, k, v = inputs([total], [total], 1, 7, torch.bfloat16, 28, before=2, behind=1)
    n = i32(starts(lens, 2))
    plan = api.PromptPlan(batch, 7, 1, len(q), len(k), 300)
    out = plan.run(q, k, v, n, n, plan.new_out().fill_(7))
    check(q, k, v, *[starts([lens[b] for b in at], 2)] * 2, out, True)
    assert (out[:2] == 7).all() and (out[-1:] == 7).all() and flags() == 0


def test_no_keys_in_arrays_of_any_strides():
    """Keys and values that are not there have no strides to be refused."""
    q, _, _ = inputs([5, 3], [0, 0], 2, 3, torch.bfloat16, 30)
    none = torch.empty(0, 2, 132, dtype=torch.bfloat16, device="cuda")[..., :D]
    out = torch.full((8, 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
    api.PromptPlan(2, 6, 2, 8, 0, 0).run(q, none, none, i32([0, 5, 8]), i32([0, 0, 0]), out)
    assert not out.any() and flags() == 0
