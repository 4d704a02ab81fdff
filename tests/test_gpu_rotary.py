"""Rotary positions (include/tq.h: tq_rotary_apply) against their definition in 64 bits."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api
from test_gpu_longctx import capture, flags, gen, i32

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.load()
    yield
    torch.cuda.synchronize()


def angles(r, at):
    """cos and sin of position · frequency [batch, 1, tokens, rotary_dim / 2] in 64 bits."""
    a = at.double()[:, None, :, None] * torch.tensor(r.frequencies, device=at.device)
    return a.cos(), a.sin()


def check(r, x, y, c, s, what):
    """Every coordinate of y.  Off by at most, with sizes |a| + |b| of its pair: 2 units in the last
    place (2^-23 of 1) of a sine or cosine, 2^-25 from the angle's own rounding, 2^-24 from the
    magnitude's, 2^-24 from each product and sum, together less than 2^-21; and half a step of the
    type (for fp16 at least half a subnormal one)."""
    h = r.rotary_dim // 2
    z = x.double()
    a, b = (z[..., :2 * h:2], z[..., 1:2 * h:2]) if r.interleaved else (z[..., :h], z[..., h:2 * h])
    u, v = r.magnitude * (a * c - b * s), r.magnitude * (a * s + b * c)
    size = abs(r.magnitude) * (a.abs() + b.abs())
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if r.interleaved else (lambda p, q: torch.cat([p, q], -1))
    want, size = join(u, v), join(size, size)
    got = y.double()
    step = torch.finfo(y.dtype).eps / 2 * (want.abs() + 2.0 ** -21 * size)
    if y.dtype == torch.float16:
        step = step.clamp(min=2.0 ** -25)
    off = (got[..., :2 * h] - want).abs() - 2.0 ** -21 * size - step
    assert float(off.max()) <= 0, (what, float(off.max()))
    assert torch.equal(y[..., 2 * h:], x[..., 2 * h:]), what


def vectors(batch, heads, tokens, dtype, seed, layout="fused", extra=0):
    """[batch, heads, tokens, 128] in the layouts that projections leave."""
    g = gen(seed)
    if layout == "flat":
        return torch.randn(batch, heads, tokens, D, generator=g, device="cuda").to(dtype)
    if layout == "fused":          # heads of one token side by side
        return torch.randn(batch, tokens, heads + 3, D, generator=g, device="cuda").to(dtype)[:, :, 1:heads + 1].transpose(1, 2)
    # odd strides and an odd start
    x = torch.randn(batch * heads * tokens * 131 + 1, generator=g, device="cuda").to(dtype)
    return x[1:].view(batch, heads, tokens, 131)[..., :D]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd", [2, 6, 16, 64, 96, 126, 128])
@pytest.mark.parametrize("layout", ["flat", "fused", "odd"])
def test_rotary(layout, rd, interleaved, dtype):
    r = api.Rotary(rd, 10000.0, interleaved, magnitude=1.25)
    for batch, qh, kh, tokens in ((1, 1, 1, 1), (3, 7, 1, 37), (2, 12, 4, 130)):
        q, k = vectors(batch, qh, tokens, dtype, 1, layout), vectors(batch, kh, tokens, dtype, 2, layout)
        at = torch.randint(0, 300000, (batch, tokens), generator=gen(3), device="cuda", dtype=torch.int32)
        qo, ko = r.apply(q, k, at, torch.empty_like(q, memory_format=torch.contiguous_format), vectors(batch, kh, tokens, dtype, 4, layout))
        c, s = angles(r, at)
        check(r, q, qo, c, s, "q")
        check(r, k, ko, c, s, "k")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd,layout", [(128, "fused"), (96, "fused"), (64, "flat"), (30, "odd")])
def test_in_place_equals_out_of_place(rd, layout, interleaved, dtype):
    """Bit for bit; what lies around the vectors stays."""
    r = api.Rotary(rd, 500000.0, interleaved)
    q, k = vectors(2, 8, 33, dtype, 1, layout), vectors(2, 2, 33, dtype, 2, layout)
    at = i32([list(range(5, 38)), list(range(70000, 70033))])
    qo, ko = r.apply(q, k, at, torch.empty_like(q), torch.empty_like(k))
    base = q if q._base is None else q._base
    whole = base.clone()
    outside = torch.ones_like(whole, dtype=torch.bool)
    outside.as_strided(q.shape, q.stride(), q.storage_offset()).fill_(False)
    a, b = r.apply(q, k, at)
    assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(base[outside], whole[outside])


def test_far_and_negative_positions():
    """Angles at the ends of 32 bits, against turns computed with 60 digits."""
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    at = [2 ** 31 - 1, -2 ** 31, -1, 0, 1, 1 << 20, 262143, -77777777, 2 ** 31 - 7]
    f = np.array([1.0, 0.7071067811865476, 3.25, 1e-9, 123.456, 6.283185307179586, 2.5e5, -0.3])
    r = api.Rotary(16, frequencies=f)
    turn = [[float((Decimal(p) * Decimal(x) / (2 * pi)) % 1) for x in f.tolist()] for p in at]
    a = 2 * math.pi * torch.tensor(turn, dtype=torch.float64, device="cuda")[None, None]
    x = vectors(1, 2, len(at), torch.float32, 1, "flat")
    y, _ = r.apply(x, None, i32([at]), torch.empty_like(x))
    check(r, x, y, a.cos(), a.sin(), "far")


def test_scaled_frequencies():
    for more in (dict(factor=4.0), dict(factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0, magnitude=1.2)):
        r = api.Rotary(128, 500000.0, **more)
        x = vectors(1, 4, 50, torch.bfloat16, 1)
        at = torch.randint(0, 131072, (1, 50), generator=gen(2), device="cuda", dtype=torch.int32)
        y, _ = r.apply(x, None, at, torch.empty_like(x))
        check(r, x, y, *angles(r, at), more)


@pytest.mark.parametrize("tokens", [1, 5, 4000])
def test_one_row_of_positions_for_all(tokens):
    """Positions with a stride of 0, as a prompt's chunks of equal offsets have them; many heads, so
    that warps share a token's heads in every way."""
    r = api.Rotary(128)
    q, k = vectors(3, 40, tokens, torch.bfloat16, 1), vectors(3, 5, tokens, torch.bfloat16, 2)
    at = torch.arange(7, 7 + tokens, dtype=torch.int32, device="cuda")[None].expand(3, -1)
    qo, ko = r.apply(q, k, at, torch.empty_like(q), torch.empty_like(k))
    c, s = angles(r, at)
    check(r, q, qo, c, s, "q")
    check(r, k, ko, c, s, "k")


def test_special_values_stay_in_their_pairs():
    r = api.Rotary(64, interleaved=True)
    x = vectors(1, 3, 9, torch.float32, 1, "flat")
    at = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    clean, _ = r.apply(x, None, at, torch.empty_like(x))
    x[0, 1, 4, 10], x[0, 2, 5, 100] = math.nan, math.inf
    y, _ = r.apply(x, None, at, torch.empty_like(x))
    assert y[0, 1, 4, 10:12].isnan().all() and y[0, 2, 5, 100] == math.inf
    y[0, 1, 4, 10:12], y[0, 2, 5, 100] = clean[0, 1, 4, 10:12], clean[0, 2, 5, 100]
    assert torch.equal(y, clean)


def test_nothing_to_do():
    r = api.Rotary(128)
    x = torch.empty(2, 4, 0, D, device="cuda")
    r.apply(x, None, torch.empty(2, 0, dtype=torch.int32, device="cuda"))
    x = torch.empty(0, 4, 3, D, device="cuda")
    r.apply(x, None, torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    x = vectors(1, 2, 3, torch.float16, 1)
    none = x[:, :0]
    y, _ = r.apply(x, none, i32([[1, 2, 3]]), torch.empty_like(x))
    check(r, x, y, *angles(r, i32([[1, 2, 3]])), "no keys")


def test_graph_and_stream():
    r = api.Rotary(96, interleaved=True)
    q, k = vectors(2, 6, 11, torch.float16, 1), vectors(2, 2, 11, torch.float16, 2)
    at = i32([list(range(11)), list(range(50, 61))])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.apply(q, k, at, qo, ko, stream=side)
    side.synchronize()
    check(r, q, qo, *angles(r, at), "stream")
    with torch.cuda.stream(side):
        g = capture(lambda: r.apply(q, k, at, qo, ko), side)
    q.copy_(vectors(2, 6, 11, torch.float16, 5))
    at += 1000
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check(r, q, qo, *angles(r, at), "replay")
    check(r, k, ko, *angles(r, at), "replay")
    assert flags() == 0


def test_offsets_past_32_bits():
    """Queries of more than 2^32 elements apart."""
    x = torch.empty(1, 1, 2, (1 << 32) + D, dtype=torch.bfloat16, device="cuda")[..., :D]
    x.copy_(vectors(1, 1, 2, torch.bfloat16, 1))
    before = x.clone()
    r = api.Rotary(128)
    at = i32([[3, 4]])
    r.apply(x, None, at)
    check(r, before, x, *angles(r, at), "far apart")


def test_refusals_on_the_gpu():
    r = api.Rotary(128)
    x, at = vectors(2, 4, 5, torch.bfloat16, 1, "flat"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    room = torch.empty(2, 8, 5, D, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: r.apply(x, None, at.long()), lambda: r.apply(x, None, at[:1]), lambda: r.apply(x[..., :64], None, at),
                lambda: r.apply(x, None, at, x.float()), lambda: r.apply(x, x.float(), at),
                lambda: r.apply(x, None, at.cpu()), lambda: r.apply(x, None, at, torch.empty_like(x).cpu()),
                lambda: r.apply(x[:, :3], None, at, x[:, 1:]),                       # shifted by a head
                lambda: r.apply(x, None, at, room[:, :1].expand(-1, 4, -1, -1)),     # all heads in one place
                lambda: r.apply(x.transpose(-1, -2).contiguous().transpose(-1, -2), None, at)):
        with pytest.raises((ValueError, TypeError, B.TQError)):
            bad()


@pytest.mark.parametrize("layout", ["grouped", "alternating", "heads first"])
def test_sides_between_each_other_in_one_array(layout):
    """Queries, keys and outputs that are views of one array and apart: each is what separate arrays give,
    and the rest of the array stays."""
    r = api.Rotary(128)
    tokens = 9
    if layout == "grouped":          # the heads of a token: queries, keys, values, then room
        x = torch.randn(2, tokens, 20, D, generator=gen(1), device="cuda").bfloat16().transpose(1, 2)
        at = [slice(0, 6), slice(6, 8), slice(10, 16), slice(16, 18)]
    elif layout == "alternating":    # a query, a key and a value for each head, then their outputs
        x = torch.randn(2, tokens, 4, 5, D, generator=gen(1), device="cuda").bfloat16().view(2, tokens, 20, D).transpose(1, 2)
        at = [slice(i, None, 5) for i in (0, 1, 3, 4)]
    else:
        x = torch.randn(2, 20, tokens, D, generator=gen(1), device="cuda").bfloat16()
        at = [slice(0, 6), slice(6, 8), slice(12, 18), slice(18, 20)]
    pos = i32([list(range(5, 5 + tokens)), list(range(70, 70 + tokens))])
    q, k, qo, ko = (x[:, s] for s in at)
    want = x.clone()
    a, b = r.apply(q, k, pos, torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k))
    want[:, at[2]], want[:, at[3]] = a, b
    r.apply(q, k, pos, qo, ko)
    assert torch.equal(x, want)
    want[:, at[0]], want[:, at[1]] = a, b
    r.apply(q, k, pos)
    assert torch.equal(x, want)
    with pytest.raises(B.TQError):   # the last query head is the keys' first
        r.apply(q, x[:, 5:7] if layout != "alternating" else x[:, 15:17], pos)
