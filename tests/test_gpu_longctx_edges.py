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
