"""Refusals of the long-context operators (include/tq.h), all decided on the host: nothing is
launched, so these run without a GPU."""
import pytest
import torch

from kv_cache_quantization_gb300 import _binding as B
from kv_cache_quantization_gb300 import api

OK16, OK256 = 1 << 12, 1 << 12      # plausible addresses, 16- and 256-byte aligned


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from kv_cache_quantization_gb300 import build
        build.build()
    return B.load()


def desc(batch=2, hq=28, hkv=4, d=128, cap=4096, mx=4096, tail=0, q=B.TQ_BF16, out=B.TQ_BF16):
    return B.tq_attn_desc(batch, hq, hkv, d, cap, mx, tail, 0.0, q, out)


BAD = [
    (desc(d=64), B.TQ_ERR_UNSUPPORTED),
    (desc(batch=-1), B.TQ_ERR_INVALID_ARG),
    (desc(hkv=5), B.TQ_ERR_INVALID_ARG),
    (desc(hkv=0), B.TQ_ERR_INVALID_ARG),
    (desc(hq=36), B.TQ_ERR_UNSUPPORTED),          # nine query heads per KV head
    (desc(cap=1000, mx=1000), B.TQ_ERR_INVALID_ARG),
    (desc(mx=8192), B.TQ_ERR_INVALID_ARG),
    (desc(mx=-1), B.TQ_ERR_INVALID_ARG),
    (desc(q=7), B.TQ_ERR_UNSUPPORTED),
]


def pages(**k):
    import ctypes
    p = B.tq_pages(**{**dict(block_table=OK16, max_pages=16, page_tokens=256, num_pages=99), **k})
    return ctypes.pointer(p)


BAD_PAGES = [dict(block_table=0), dict(block_table=OK16 + 2), dict(max_pages=15), dict(page_tokens=100),
             dict(page_tokens=0), dict(num_pages=0)]


def key(idx=OK16, sgn=OK16, xn=OK16, rn=OK16, p=None):
    return B.tq_prod_cache(idx, sgn, xn, rn, p)


def value(idx=OK16, xn=OK16, p=None):
    return B.tq_mse_cache(idx, xn, p)


# ------------------------------------------------------------------ descriptors

@pytest.mark.parametrize("d,status", BAD)
def test_bad_descriptors(d, status):
    assert B.tq_block_select_workspace_bytes(d) == 0
    assert B.tq_sparse_workspace_bytes(d, 16) == 0
    assert B.tq_prefix_workspace_bytes(d, 1024) == 0
    assert B.tq_block_select(d, OK16, B.tq_block_cache(OK16), OK16, 1, 1, 16, OK16, OK256, 1 << 40,
                             None) == status
    assert B.tq_sparse_attention(d, 1, 1, OK16, key(), value(), OK16, OK16, 16, OK16, OK256, 1 << 40,
                                 None) == status
    assert B.tq_prefix_attention(d, 1, 1, OK16, key(), value(), 1024, 1024, OK16, key(), value(),
                                 OK16, OK16, OK256, 1 << 40, None) == status


def test_attention_outputs_are_16_bit():
    d = desc(out=B.TQ_F32)
    assert B.tq_sparse_workspace_bytes(d, 16) == 0 and B.tq_prefix_workspace_bytes(d, 64) == 0
    assert B.tq_sparse_attention(d, 1, 1, OK16, key(), value(), OK16, OK16, 16, OK16, OK256, 1 << 40,
                                 None) == B.TQ_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        api.PrefixPlan(1, 4, 4, 64, 64, 64, 64, out_dtype=torch.float32, device="cpu")
    assert B.tq_sparse_workspace_bytes(desc(tail=8), 16) == 0      # no FP16 tail here


def test_limits_of_size():
    big = desc(cap=1 << 30, mx=1 << 30)
    assert B.tq_prefix_workspace_bytes(big, 1 << 20) > 0
    assert B.tq_prefix_workspace_bytes(desc(cap=(1 << 30) + 64, mx=(1 << 30) + 1), 0) == 0
    assert B.tq_prefix_workspace_bytes(desc(), (1 << 30) + 1) == 0
    assert B.tq_prefix_workspace_bytes(desc(batch=1 << 20), 0) == 0       # 28 · 2^20 query rows
    assert B.tq_block_select_workspace_bytes(desc(batch=1 << 15)) == 0    # 2^17 rows of blocks
    assert B.tq_block_select_workspace_bytes(big) == 0
    assert B.tq_sparse_workspace_bytes(desc(), (1 << 24) + 1) == 0


def test_workspace_sizes_grow_with_the_call():
    assert 0 < B.tq_sparse_workspace_bytes(desc(batch=1), 16) < B.tq_sparse_workspace_bytes(desc(batch=64), 16)
    assert B.tq_prefix_workspace_bytes(desc(), 0) > 0              # an empty prefix is allowed
    assert B.tq_prefix_workspace_bytes(desc(), -1) == 0
    assert B.tq_sparse_workspace_bytes(desc(), 0) == 0
    assert B.tq_block_select_workspace_bytes(desc(mx=0)) > 0
    assert B.tq_block_select_workspace_bytes(None or desc(batch=0)) > 0


# ------------------------------------------------------------------ bounds

def bounds(x=OK16, dtype=B.TQ_BF16, batch=1, heads=2, tokens=10, sb=2560, sh=1280, st=128, pos=None,
           count=None, blocks=None, cap=4096):
    return B.tq_block_bounds(x, dtype, batch, heads, tokens, sb, sh, st, pos, count,
                             blocks or B.tq_block_cache(OK16), cap, None)


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(x=OK16 + 1), dict(batch=-1), dict(heads=0), dict(tokens=-1), dict(sb=-1), dict(sh=-1),
    dict(st=-1), dict(cap=0), dict(cap=100), dict(blocks=B.tq_block_cache(0)),
    dict(blocks=B.tq_block_cache(OK16 + 8)),
])
def test_bounds_refusals(kw):
    assert bounds(**kw) == B.TQ_ERR_INVALID_ARG


def test_bounds_types_and_nothing_to_do():
    assert bounds(dtype=5) == B.TQ_ERR_UNSUPPORTED
    assert bounds(batch=0) == B.TQ_OK and bounds(tokens=0) == B.TQ_OK


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_bad_pages(kw):
    p = pages(**kw)
    d = desc()
    assert bounds(blocks=B.tq_block_cache(OK16, p)) == B.TQ_ERR_INVALID_ARG
    assert B.tq_block_select(d, OK16, B.tq_block_cache(OK16, p), OK16, 1, 1, 16, OK16, OK256, 1 << 40,
                             None) == B.TQ_ERR_INVALID_ARG
    for k, v in ((key(p=p), value()), (key(), value(p=p))):
        assert B.tq_sparse_attention(d, 1, 1, OK16, k, v, OK16, OK16, 16, OK16, OK256, 1 << 40,
                                     None) == B.TQ_ERR_INVALID_ARG
        assert B.tq_prefix_attention(d, 1, 1, OK16, key(), value(), 1024, 1024, OK16, k, v, OK16, OK16,
                                     OK256, 1 << 40, None) == B.TQ_ERR_INVALID_ARG
        assert B.tq_prefix_attention(d, 1, 1, OK16, k, v, 4096, 1024, OK16, key(), value(), OK16, OK16,
                                     OK256, 1 << 40, None) == B.TQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("kw", [
    dict(q=0), dict(blocks=0), dict(blocks=OK16 + 4), dict(lens=0), dict(out=0), dict(ws=0),
    dict(ws=OK256 + 16), dict(size=64), dict(first=-1), dict(last=-1), dict(keep=0), dict(first=9, last=8),
])
def test_select_refusals(kw):
    a = {**dict(q=OK16, blocks=OK16, lens=OK16, first=1, last=1, keep=16, out=OK16, ws=OK256, size=1 << 40), **kw}
    assert B.tq_block_select(desc(), a["q"], B.tq_block_cache(a["blocks"]), a["lens"], a["first"],
                             a["last"], a["keep"], a["out"], a["ws"], a["size"],
                             None) == B.TQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("k,v", [(key(idx=0), value()), (key(sgn=0), value()), (key(xn=0), value()),
                                 (key(rn=0), value()), (key(), value(idx=0)), (key(), value(xn=0)),
                                 (key(idx=OK16 + 8), value()), (key(), value(xn=OK16 + 4))])
def test_cache_refusals(k, v):
    d = desc()
    assert B.tq_sparse_attention(d, 1, 1, OK16, k, v, OK16, OK16, 16, OK16, OK256, 1 << 40,
                                 None) == B.TQ_ERR_INVALID_ARG
    for pk, pv, ok, ov in ((k, v, key(), value()), (key(), value(), k, v)):
        assert B.tq_prefix_attention(d, 1, 1, OK16, pk, pv, 1024, 1024, OK16, ok, ov, OK16, OK16, OK256,
                                     1 << 40, None) == B.TQ_ERR_INVALID_ARG


def test_attention_refusals():
    d = desc()
    assert B.tq_sparse_attention(d, None, None, OK16, key(), value(), OK16, OK16, 16, OK16, OK256,
                                 1 << 40, None) == B.TQ_ERR_INVALID_ARG              # no codecs
    assert B.tq_sparse_attention(d, 1, 1, OK16, key(), value(), OK16, 0, 16, OK16, OK256, 1 << 40,
                                 None) == B.TQ_ERR_INVALID_ARG                       # no list
    assert B.tq_sparse_attention(d, 1, 1, OK16, key(), value(), OK16, OK16, 0, OK16, OK256, 1 << 40,
                                 None) == B.TQ_ERR_INVALID_ARG
    for cap, mx, length in ((1000, 1000, OK16), (0, 0, OK16), (1024, 2048, OK16), (1024, 1024, 0)):
        assert B.tq_prefix_attention(d, 1, 1, OK16, key(), value(), cap, mx, length, key(), value(), OK16,
                                     OK16, OK256, 1 << 40, None) == B.TQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ the Python layer

def test_block_bounds_object():
    b = api.BlockBounds.empty(2, 3, 100, device="cpu")
    assert b.bounds.shape == (2, 3, 2, 2, 128) and b.capacity == 128
    b.expect(2, 3, 128)
    for rows, heads, slots in ((3, 3, 128), (2, 2, 128), (2, 3, 64)):
        with pytest.raises(ValueError):
            b.expect(rows, heads, slots)
    t = torch.zeros(2, 5, dtype=torch.int32)
    p = api.BlockBounds.empty_paged(api.Pages(t, 192, 7), 3, device="cpu")
    assert p.bounds.shape == (7, 3, 3, 2, 128) and p.capacity == 960
    p.expect(2, 3, 960)
    with pytest.raises(ValueError):
        p.expect(3, 3, 960)
    with pytest.raises(ValueError):
        api.BlockBounds.empty_paged(api.Pages(t, 100, 7), 3, device="cpu")
    with pytest.raises(ValueError):
        api.BlockBounds(b.bounds.float()).expect(2, 3, 128)


def test_cache_shapes():
    class Codec:
        def __init__(self, bits, index_bits):
            self.bits, self.index_bits = bits, index_bits

    k, v = api.ProdCache.empty(2, 3, 128, 4, device="cpu"), api.MSECache.empty(2, 3, 128, 2, device="cpu")
    api._expect_caches(k, v, 2, 3, 128, Codec(4, 3), Codec(2, 2), "cache")
    for rows, heads, slots, kb, vb in ((3, 3, 128, 3, 2), (2, 4, 128, 3, 2), (2, 3, 192, 3, 2), (2, 3, 128, 2, 2),
                                       (2, 3, 128, 3, 3)):
        with pytest.raises(ValueError):
            api._expect_caches(k, v, rows, heads, slots, Codec(kb + 1, kb), Codec(vb, vb), "cache")


def test_plans_refuse():
    with pytest.raises(ValueError):
        api.SparsePlan(1, 4, 4, 640, 640, 4, first_blocks=3, last_blocks=2, device="cpu")
    with pytest.raises(ValueError):
        api.SparsePlan(1, 4, 3, 640, 640, 4, device="cpu")
    with pytest.raises(ValueError):
        api.PrefixPlan(1, 4, 4, 64, 64, 64, 128, device="cpu")      # prefix longer than its cache
