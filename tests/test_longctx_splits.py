"""How the rows attention splits its tokens (host code): the pair of splits whose estimated time is
least, found at a cost that does not depend on how many shapes a program uses."""
import math
import time

import pytest

from kv_cache_quantization_gb300 import _binding as B

TILE, RECORDS, SMS = 128, 512, 152      # (a GB300's SMs, which the library assumes where there is no GPU)


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from kv_cache_quantization_gb300 import build
        build.build()
    return B.load()


def desc(batch, kv, group, own, out=B.TQ_BF16):
    return B.tq_attn_desc(batch, kv * group, kv, 128, max(-(-own // 64) * 64, 64), own, 0, 0.0, B.TQ_BF16, out)


def records(batch, kv, group, prefix, own):
    """Records of a row in the workspace: the sum of both splits."""
    rows = batch * kv * group
    n = B.tq_prefix_workspace_bytes(desc(batch, kv, group, own), prefix)
    head = -(-(rows * 512 + rows * 4) // 256) * 256
    assert (n - head) % (rows * 132 * 4) == 0
    return (n - head) // (rows * 132 * 4)


def makespan(n1, c1, n2, c2):
    rest, start = n1 % SMS, n1 // SMS * c1
    until = start + c1 if rest else start
    beside = (SMS - rest) * int(c1 / c2) if rest else 0
    return until if n2 <= beside else until + -(-(n2 - beside) // SMS) * c2


def ways(tiles):
    n = 1
    while True:
        yield max(-(-tiles // n), 1)
        if n >= tiles:
            return
        n = min(n + max(1, n // 8), tiles)


def best(batch, kv, group, prefix, own):
    """All pairs, most items first among equals."""
    pre, own = -(-prefix // TILE), -(-own // TILE)
    pu, ou = -(-batch * group // TILE) * kv, batch * kv
    f = 0.75 if batch * group <= TILE // 2 else 1.0
    top = None
    for sp in (ways(pre) if pre else [0]):
        for so in ways(own):
            if sp + so > RECORDS and (sp > 1 or so > 1):
                continue
            cp = f * -(-pre // sp) + 2 if sp else 0
            co = 0.75 * -(-own // so) + 2
            t = makespan(pu * sp, cp, ou * so, co) + (sp + so) / 64
            if top is None or t < top[0]:
                top = (t, sp + so)
    return top[1]


@pytest.mark.parametrize("batch,kv,group,prefix,own", [
    (1, 1, 1, 0, 0), (1, 1, 1, 1, 0), (4, 4, 7, 1000, 100), (32, 4, 7, 32768, 512), (32, 4, 7, 32768, 4096),
    (8, 8, 4, 262144, 1024), (64, 4, 7, 65536, 1024), (3, 2, 5, 129, 70000), (1, 8, 4, 0, 1 << 20),
    (200, 1, 8, 7001, 333), (17, 16, 1, 100003, 2049), (2, 1, 8, 1 << 22, 1 << 18),
])
def test_the_pair_of_least_estimated_time(batch, kv, group, prefix, own):
    assert records(batch, kv, group, prefix, own) == best(batch, kv, group, prefix, own)


def test_many_shapes_cost_what_one_costs():
    """A server that cycles through more shapes than any small cache holds: the host time of a call
    stays a few microseconds."""
    shapes = [(desc(1 + i, 8, 4, (1 << 20) - 640 * i), (1 << 23) - 1280 * i) for i in range(24)]
    least = math.inf
    for _ in range(20):
        t = time.perf_counter()
        for d, p in shapes:
            B.tq_prefix_workspace_bytes(d, p)
        least = min(least, time.perf_counter() - t)
    assert least / len(shapes) < 20e-6, least / len(shapes)
