"""Operators of long contexts at values and layouts where they can go wrong: infinite and tiny
values in a selection, against the definitions in 64 bits (longctx_ref.py)."""
import math

import pytest
import torch

import longctx_ref as ref
from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import blank, check_select, flags, queries, run_select

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
