"""Refusals of the operators around prompts and drafted tokens (include/tq.h), and what of them is
host code: nothing is launched, so these run without a GPU."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_longctx_args import BAD, BAD_PAGES, OK16, OK256, desc, key, pages, value

INVALID, UNSUPPORTED = B.TQ_ERR_INVALID_ARG, B.TQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from kv_cache_quantization_gb300 import build
        build.build()
    return B.load()


# ------------------------------------------------------------------ rotary positions

def test_frequencies():
    """base^(−2i/n); divided by the factor; by parts between two numbers of turns.  A power of 64 bits
    is off by a few units in the last place, the blend by a few more."""
    def close(a, b):
        np.testing.assert_allclose(a, b, rtol=2.0 ** -48, atol=0)

    for n, base in ((128, 10000.0), (64, 500000.0), (2, 3.0), (126, 1e6)):
        f = base ** (-np.arange(0, n, 2) / n)
        close(api.Rotary(n, base).frequencies, f)
        close(api.Rotary(n, base, factor=8.0).frequencies, f / 8)
        r = api.Rotary(n, base, factor=4.0, original_len=8192, low_turns=1.0, high_turns=32.0)
        turns = 8192 * f / (2 * math.pi)
        close(r.frequencies[turns >= 32], f[turns >= 32])
        close(r.frequencies[turns <= 1], f[turns <= 1] / 4)
        share = np.clip((turns - 1) / 31, 0, 1)
        np.testing.assert_allclose(r.frequencies, share * f + (1 - share) * f / 4, rtol=1e-12)


def test_turns_are_exact():
    """f / 2π as a fraction of 2^64, off by less than two units, for frequencies of all sizes."""
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986")
    f = np.array([1.0, 1e-12, 0.1, 2 * math.pi, 1e6, 0.9999999999999999, 5e-324, 12345.678, -0.25, 0.0])
    r = api.Rotary(20, frequencies=f)
    for i, x in enumerate(f.tolist()):
        want = Decimal(x) / two_pi * (1 << 64)
        off = (Decimal(r._c.turns[i]) - want) % (1 << 64)
        assert min(off, (1 << 64) - off) < 2, x


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=-2), dict(base=0.0), dict(base=math.inf),
    dict(base=math.nan), dict(factor=0.0), dict(factor=-1.0), dict(factor=math.inf), dict(original_len=-1),
    dict(original_len=100, low_turns=4.0, high_turns=4.0), dict(original_len=100, low_turns=-1.0),
    dict(original_len=100, high_turns=math.nan), dict(original_len=100, high_turns=math.inf),
    dict(magnitude=math.inf), dict(magnitude=math.nan), dict(magnitude=1e39), dict(frequencies=[1.0] * 63),
    dict(frequencies=[math.nan] * 64), dict(frequencies=[1e7] * 64)])
def test_rotary_refuses(kw):
    with pytest.raises((B.TQError, ValueError)):
        api.Rotary(**kw)


def io(x=OK16, y=OK16 + 65536, heads=2, xs=(1024, 512, 128), ys=(1024, 512, 128)):      # [1][2][4][128] in the calls
    return B.tq_rotary_io(x, y, heads, *xs, *ys)


def test_rotary_apply_refuses():
    r = api.Rotary(128)._c

    def call(status, r=r, dtype=B.TQ_BF16, batch=1, tokens=4, at=OK16, at_b=4, q=io(), k=io(x=1 << 20, y=1 << 24)):
        assert B.tq_rotary_apply(r, dtype, batch, tokens, at, at_b, q, k, None) == status

    call(UNSUPPORTED, dtype=7)
    call(INVALID, batch=-1)
    call(INVALID, tokens=-1)
    call(INVALID, at=0)
    call(INVALID, at=OK16 + 2)
    call(INVALID, at_b=-1)
    call(INVALID, r=B.tq_rotary())
    call(INVALID, r=B.tq_rotary(130, 0, 1.0))
    for bad in (io(x=0), io(y=0), io(x=OK16 + 1), io(y=OK16 + 65537), io(heads=-1), io(xs=(1024, -1, 128)), io(ys=(1024, 512, -128)),
                io(y=OK16, ys=(1024, 512, 256)),                      # the input with other strides
                io(y=OK16 + 256), io(y=OK16 + 1984), io(x=OK16 + 1984, y=OK16),          # overlapping the input
                io(ys=(1024, 512, 64)), io(ys=(1024, 0, 128)), io(ys=(1024, 256, 128))):  # vectors over each other
        call(INVALID, q=bad)
        call(INVALID, k=bad)
    call(INVALID, dtype=B.TQ_F32, q=io(x=OK16 + 2))
    call(INVALID, q=io(), k=io())                                       # both sides' outputs in one place
    call(INVALID, q=io(), k=io(x=1 << 30, y=OK16))                      # over the other side's vectors
    call(INVALID, q=io(y=1 << 30), k=io(x=1 << 30, y=1 << 35))
    call(UNSUPPORTED, q=io(y=1 << 40, heads=(1 << 20) + 1), k=None)
    call(B.TQ_OK, q=None, k=None)               # nothing to do
    call(B.TQ_OK, batch=0)
    call(B.TQ_OK, tokens=0)
    call(B.TQ_OK, q=io(x=0, y=0, heads=0), k=None)
    call(INVALID, q=io(y=OK16 + 2046), k=None)          # one coordinate short of apart


def test_rotary_apply_refuses_one_side_over_part_of_the_other():
    """Outputs that share some heads with the other side's vectors, in place and out of place, in every
    layout of projections; [2][heads][4][128], strides in elements."""
    r = api.Rotary(128)._c
    row = 14 * 128                                                     # a fused row of 14 heads
    fused, heads_first = (4 * row, 128, row), (14 * 512, 512, 128)     # [2][4][14][128] and [2][14][4][128]

    def view(at, heads, s, y=None, ys=None):
        x = OK16 + 2 * at
        return io(x, x if y is None else y, heads, s, ys or s)

    def call(q, k, batch=2, tokens=4):
        assert B.tq_rotary_apply(r, B.TQ_BF16, batch, tokens, OK16, tokens, q, k, None) == INVALID

    for s in (fused, heads_first):
        h = s[1]
        call(view(0, 8, s), view(7 * h, 2, s))                         # one head of both
        call(view(2 * h, 8, s), view(0, 3, s))
        call(view(0, 8, s), view(7 * h + 64, 2, s))                    # half a head
        call(view(0, 8, s), view(8 * h, 2, s, OK16 + 14 * h))          # k's output over q's last heads
        call(view(0, 8, s, 1 << 30), view(0, 2, s, (1 << 30) + 14 * h))
        call(view(0, 8, s, 1 << 30), view(9 * h, 2, s, OK16 + 6 * h))
        call(view(0, 8, s, OK16 + 18 * h), view(9 * h, 2, s, 1 << 30))
        call(view(0, 8, s), view(7 * h, 2, s), batch=1)
    call(view(0, 8, fused), view(3 * row + 512, 2, (4 * row, 128, row)), tokens=4)       # q's row 3 from k's row 0
    # other strides: k's output, packed, among q's rows
    call(view(0, 8, fused), view(1 << 20, 2, (1024, 512, 128), OK16 + 2 * row, (1024, 512, 128)))
    # a side's own output over its input by one head of another token
    call(view(0, 8, fused, OK16 + 2 * 7 * 128), None)


def test_rotary_python_layer_refuses():
    r = api.Rotary(128)
    x, at = torch.zeros(2, 4, 5, 128), torch.zeros(2, 5, dtype=torch.int32)
    for bad in (lambda: r.apply(x, None, at.long()), lambda: r.apply(x, None, at[0]), lambda: r.apply(x[0], None, at),
                lambda: r.apply(x, None, at.t()), lambda: r.apply(x, None, at.t().contiguous().t())):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            bad()


# ------------------------------------------------------------------ drafted tokens

@pytest.mark.parametrize("d,status", BAD)
def test_tree_bad_descriptors(d, status):
    assert B.tq_tree_workspace_bytes(d, 4) == 0
    assert B.tq_tree_attention(d, 4, 1, 1, OK16, key(), value(), OK16, OK16, 4, OK16, OK256, 1 << 40, None) == status


def test_tree_refuses():
    d = desc()

    def call(status, d=d, nodes=4, q=OK16, k=key(), v=value(), lens=OK16, tree=OK16, tree_b=4, out=OK16, ws=OK256):
        assert B.tq_tree_attention(d, nodes, None, None, q, k, v, lens, tree, tree_b, out, ws, 1 << 40, None) == status

    call(INVALID, nodes=0)
    call(INVALID, nodes=-1)
    call(UNSUPPORTED, nodes=65)
    call(INVALID, tree=0)
    call(INVALID, tree=OK16 + 4)
    call(INVALID, tree_b=-1)
    call(INVALID, out=OK16 + 2)
    call(INVALID, out=0)
    call(INVALID, d=desc(mx=3))                           # no room for four drafted tokens
    call(UNSUPPORTED, d=desc(out=B.TQ_F32))
    call(UNSUPPORTED, d=desc(batch=1 << 18))              # 28 · 4 · 2^18 query rows
    for bad in (key(idx=0), key(sgn=OK16 + 8), key(xn=0), key(rn=OK16 + 4)):
        call(INVALID, k=bad)
    for bad in (value(idx=0), value(xn=OK16 + 4)):
        call(INVALID, v=bad)
    for p in BAD_PAGES:
        call(INVALID, k=key(p=pages(**p)))
        call(INVALID, v=value(p=pages(**p)))
    assert B.tq_tree_workspace_bytes(d, 64) > B.tq_tree_workspace_bytes(d, 1) > 0
    call(INVALID, d=desc(batch=0))                        # (the codecs; no sequences are nothing to split)
    assert B.tq_tree_workspace_bytes(desc(batch=0), 4) == B.tq_prefix_workspace_bytes(desc(batch=0), 128)
    with pytest.raises(ValueError):
        api.TreePlan(1, 65, 4, 4, 128, 128, device="cpu")
    with pytest.raises(ValueError):
        api.TreePlan(1, 8, 4, 4, 128, 7, device="cpu")
    with pytest.raises(ValueError):
        api.TreePlan(1, 8, 4, 4, 128, 128, out_dtype=torch.float32, device="cpu")


def test_tree_batches_that_are_ranked_hold_an_order():
    """Ranks cost the square of the sequences: above 2048 there are none.  (The rest of the workspace is
    256-byte aligned row operands, and records of 528 bytes.)"""
    for batch, ranked in ((2, False), (2048, True), (2049, False), (1 << 18, False)):
        rows = batch * 8 * 2
        front = -(-(rows * 516) // 256) * 256
        n = B.tq_tree_workspace_bytes(desc(batch=batch, hq=8, hkv=1, mx=1024, out=B.TQ_BF16), 2) - front
        assert n % (rows * 528) == (4 * batch if ranked else 0)


# ------------------------------------------------------------------ moving codes

def test_copy_pages_refuses():
    k, v, b = key(), value(), B.tq_block_cache(OK16)

    def call(status, k=k, kb=3, v=v, vb=2, b=b, heads=2, pages=9, tokens=64, src=OK16, dst=OK16, n=1):
        assert B.tq_copy_pages(k, kb, v, vb, b, heads, pages, tokens, src, dst, n, None) == status

    for kw in (dict(heads=0), dict(pages=0), dict(tokens=0), dict(tokens=100), dict(n=-1), dict(src=0), dict(dst=0), dict(src=OK16 + 2),
               dict(dst=OK16 + 1), dict(k=None, v=None, b=None), dict(k=key(idx=0)), dict(k=key(sgn=OK16 + 8)), dict(k=key(rn=0)),
               dict(v=value(idx=OK16 + 4)), dict(v=value(xn=0)), dict(b=B.tq_block_cache(0)), dict(b=B.tq_block_cache(OK16 + 2))):
        call(INVALID, **kw)
    for kw in (dict(kb=1), dict(kb=6), dict(vb=0), dict(vb=5), dict(n=65537), dict(heads=1 << 20, tokens=128)):
        call(UNSUPPORTED, **kw)
    call(B.TQ_OK, n=0)
    call(B.TQ_OK, n=0, k=None, kb=0)


def test_keep_tokens_refuses():
    def call(status, k=key(), kb=3, v=value(), vb=2, batch=2, heads=2, cap=4096, pos=OK16, keep=OK16, most=4):
        assert B.tq_keep_tokens(k, kb, v, vb, batch, heads, cap, pos, keep, most, None) == status

    for kw in (dict(batch=-1), dict(heads=0), dict(cap=0), dict(cap=100), dict(pos=0), dict(keep=0), dict(pos=OK16 + 2), dict(keep=OK16 + 1),
               dict(most=-1), dict(k=key(idx=0)), dict(k=key(sgn=0)), dict(k=key(xn=OK16 + 4)), dict(k=key(rn=0)), dict(v=value(idx=0)),
               dict(v=value(xn=OK16 + 8))):
        call(INVALID, **kw)
    for p in BAD_PAGES:
        call(INVALID, k=key(p=pages(**p)))
        call(INVALID, v=value(p=pages(**p)))
    for kw in (dict(kb=1), dict(kb=6), dict(vb=0), dict(vb=5), dict(most=65), dict(batch=1 << 30, heads=4)):
        call(UNSUPPORTED, **kw)
    call(B.TQ_OK, batch=0)
    call(B.TQ_OK, most=0)


# ------------------------------------------------------------------ prompts

def prompt(batch=2, hq=28, hkv=4, d=128, tq=1000, tk=2000, longest=900, causal=1, dtype=B.TQ_BF16):
    return B.tq_prompt_desc(batch, hq, hkv, d, tq, tk, longest, causal, 0.0, dtype)


PROMPT_BAD = [
    (prompt(d=64), UNSUPPORTED), (prompt(batch=-1), INVALID), (prompt(hkv=0), INVALID), (prompt(hkv=5), INVALID), (prompt(hq=0), INVALID),
    (prompt(hq=36), UNSUPPORTED), (prompt(tq=-1), INVALID), (prompt(tk=-1), INVALID), (prompt(longest=-1), INVALID),
    (prompt(dtype=B.TQ_F32), UNSUPPORTED), (prompt(dtype=9), UNSUPPORTED), (prompt(tq=(1 << 28) + 1), UNSUPPORTED),
    (prompt(tk=(1 << 28) + 1), UNSUPPORTED), (prompt(batch=(1 << 20) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("d,status", PROMPT_BAD)
def test_prompt_bad_descriptors(d, status):
    assert B.tq_prompt_workspace_bytes(d) == 0
    assert B.tq_prompt_attention(d, OK16, 3584, 128, OK16, 512, 128, OK16, 512, 128, OK16, OK16, OK16, OK256, 1 << 40, None) == status


def test_prompt_refuses():
    def call(status, d=prompt(), q=OK16, qt=3584, qh=128, k=OK16, kt=512, kh=128, v=OK16, vt=512, vh=128, qs=OK16, ks=OK16, out=OK16,
             ws=OK256, n=1 << 40):
        assert B.tq_prompt_attention(d, q, qt, qh, k, kt, kh, v, vt, vh, qs, ks, out, ws, n, None) == status

    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(q=OK16 + 8), dict(k=OK16 + 2), dict(v=OK16 + 4), dict(qt=3588), dict(qh=0), dict(kt=-512),
               dict(kh=132), dict(vt=64), dict(vh=-128), dict(qt=1 << 39), dict(qs=0), dict(ks=0), dict(qs=OK16 + 2), dict(ks=OK16 + 1),
               dict(out=0), dict(out=OK16 + 8), dict(ws=0), dict(ws=OK256 + 16), dict(n=0)):
        call(INVALID, **kw)
    call(B.TQ_OK, d=prompt(batch=0))
    call(B.TQ_OK, d=prompt(tq=0))


def test_prompt_workspaces():
    """Records for single tokens behind long histories, whose keys are split; none for whole prompts."""
    small = B.tq_prompt_workspace_bytes(prompt(batch=1, tq=1, tk=65536, longest=65536))
    assert small > B.tq_prompt_workspace_bytes(prompt(batch=1, tq=65536, tk=65536, longest=65536)) > 0
    with pytest.raises(ValueError):
        api.PromptPlan(1, 28, 4, 10, 10, 10, dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError):
        api.PromptPlan(1, 27, 4, 10, 10, 10, device="cpu")


def test_prompt_refuses_outputs_over_inputs():
    """Keys, values, and queries that are not the output themselves; [1000][28 or 4][128] rows in bytes
    from their starts."""
    def call(q=1 << 30, k=1 << 31, v=1 << 32, out=1 << 33, qt=3584, kt=512, vt=512, kh=128, d=prompt(tq=1000, tk=2000)):
        assert B.tq_prompt_attention(d, q, qt, 128, k, kt, kh, v, vt, 128, OK16, OK16, out, OK256, 1 << 40, None) == INVALID

    size = 1000 * 28 * 256
    call(k=1 << 33)
    call(v=1 << 33)
    call(k=(1 << 33) + size - 16)
    call(v=(1 << 33) - 2000 * 1024 + 16)
    call(q=(1 << 33) + 16)
    call(q=(1 << 33) + size - 256)
    call(q=1 << 33, qt=3712)                          # rows further apart than the output's
    call(k=(1 << 33) - 4096 * 255, kh=2000 * 128, kt=128, d=prompt(tq=1, tk=2000))    # heads first; one token into them
    fused = dict(qt=36 * 128, kt=36 * 128, vt=36 * 128, d=prompt(tq=1000, tk=1000))
    call(q=1 << 33, k=(1 << 33) + 28 * 256, v=(1 << 33) + 32 * 256, **fused)
    call(q=1 << 30, k=(1 << 30) + 28 * 256, v=(1 << 30) + 32 * 256, out=(1 << 30) + 999 * 36 * 256, **fused)
