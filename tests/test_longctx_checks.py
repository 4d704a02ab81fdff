"""What the Python layer of the long-context operators refuses before anything is launched, on
tensors of the host (and on stand-ins that say they lie on a GPU)."""
import dataclasses

import pytest
import torch

from kv_cache_quantization_gb300 import api


class Codec:
    def __init__(self, bits, index_bits):
        self.bits, self.index_bits = bits, index_bits


KC = Codec(3, 2)


def pair(vbits, pages=None):
    if pages is None:
        return (api.ProdCache.empty(2, 3, 128, 3, device="cpu"),
                api.MSECache.empty(2, 3, 128, vbits, device="cpu"))
    return (api.ProdCache.empty_paged(pages, 3, 3, device="cpu"),
            api.MSECache.empty_paged(pages, 3, vbits, device="cpu"))


def expect(k, v):
    api._expect_caches(k, v, 2, 3, 128, KC, Codec(v.bits, v.bits), "cache")


class OnGpu:
    """An array's description with another device."""

    def __init__(self, t, device):
        self.shape, self.dtype, self.device, self._t, self._d = t.shape, t.dtype, f"cuda:{device}", t, device

    def is_contiguous(self):
        return self._t.is_contiguous()

    def get_device(self):
        return self._d


def spoilt(t):
    """Arrays that must not stand in t's place: another capacity, heads, type, or strides."""
    slot = {5: 3, 4: 2, 3: 2}[t.dim()]
    short = list(t.shape)
    short[slot] //= 2
    yield torch.zeros(short, dtype=t.dtype)
    heads = list(t.shape)
    heads[1] -= 1
    yield torch.zeros(heads, dtype=t.dtype)
    yield t.to(torch.int32)
    yield torch.zeros([*t.shape[:-1], 2 * t.shape[-1]], dtype=t.dtype)[..., ::2]
    yield torch.zeros([*t.shape, 1], dtype=t.dtype)


@pytest.mark.parametrize("vbits", [1, 2, 3, 4])
@pytest.mark.parametrize("paged", [False, True])
def test_every_array_of_the_caches_is_checked(paged, vbits):
    pages = api.Pages(torch.zeros(2, 2, dtype=torch.int32), 64, 5) if paged else None
    k, v = pair(vbits, pages)
    expect(k, v)
    for cache in (k, v):
        for f in ("idx", "sgn", "xnorm", "rnorm") if cache is k else ("idx", "xnorm"):
            for bad in spoilt(getattr(cache, f)):
                other = dataclasses.replace(cache, **{f: bad})
                with pytest.raises(ValueError):
                    expect(*((other, v) if cache is k else (k, other)))


@pytest.mark.parametrize("field", ["sgn", "xnorm", "rnorm", "values", "value norms", "key table", "value table"])
def test_arrays_on_another_device(field):
    """Every array and block table lies on the device of the key codes."""
    def at(t, device):
        return OnGpu(t, device)

    def table(device):
        p = api.Pages(torch.zeros(2, 2, dtype=torch.int32), 64, 5)
        p.block_table = at(p.block_table, device)
        return p

    def build(other):
        d = {f: 1 if f == other else 0 for f in
             ("sgn", "xnorm", "rnorm", "values", "value norms", "key table", "value table")}
        k, v = pair(2, api.Pages(torch.zeros(2, 2, dtype=torch.int32), 64, 5))
        return (api.ProdCache(at(k.idx, 0), at(k.sgn, d["sgn"]), at(k.xnorm, d["xnorm"]), at(k.rnorm, d["rnorm"]),
                              table(d["key table"])),
                api.MSECache(at(v.idx, d["values"]), at(v.xnorm, d["value norms"]), 2, table(d["value table"])))

    expect(*build(None))
    with pytest.raises(ValueError):
        expect(*build(field))


def test_bounds_with_a_table_on_another_device():
    t = torch.zeros(2, 5, dtype=torch.int32)
    b = api.BlockBounds.empty_paged(api.Pages(t, 192, 7), 3, device="cpu")
    b.expect(2, 3, 960)
    b.pages.block_table = OnGpu(t, 0)
    with pytest.raises(ValueError):
        b.expect(2, 3, 960)


def test_a_replaced_array_is_checked_again():
    k, v = pair(2)
    expect(k, v)
    good = k.sgn
    k.sgn = good[:, :, :64].contiguous()
    with pytest.raises(ValueError):
        expect(k, v)
    k.sgn = good
    expect(k, v)
    v.bits = 1
    with pytest.raises(ValueError):
        expect(k, v)
