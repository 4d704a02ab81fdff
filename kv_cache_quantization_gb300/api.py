"""PyTorch-facing convenience layer over the C ABI.

PyTorch only owns memory and streams here: caches and workspaces are torch tensors whose
addresses are handed to libtq.so; every step of quantisation and attention runs in the
library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional

import numpy as np
import torch

from . import _binding as B

HEAD_DIM = B.TQ_HEAD_DIM

_DT = {torch.float32: B.TQ_F32, torch.float16: B.TQ_F16, torch.bfloat16: B.TQ_BF16}


def tq_dtype(dt: torch.dtype) -> int:
    if dt not in _DT:
        raise TypeError(f"unsupported dtype {dt}")
    return _DT[dt]


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ host constants

def lloyd_max_codebook(index_bits: int, d: int = HEAD_DIM) -> np.ndarray:
    """Ascending Lloyd-Max levels for the sphere-coordinate law (library host code)."""
    out = np.zeros(1 << index_bits, dtype=np.float64)
    B.check(B.tq_lloyd_max_codebook(d, index_bits, out.ctypes.data), "tq_lloyd_max_codebook")
    return out


def rotation_from_gaussian(g: np.ndarray) -> np.ndarray:
    """Π = sign-fixed Q of G = QR (library host code)."""
    g = np.ascontiguousarray(g, dtype=np.float64)
    d = g.shape[0]
    out = np.zeros((d, d), dtype=np.float64)
    B.check(B.tq_rotation_from_gaussian(d, g.ctypes.data, out.ctypes.data),
            "tq_rotation_from_gaussian")
    return out


def layer_constants(layer: int = 0, d: int = HEAD_DIM):
    """(Π, S) of a layer from the per-layer Gaussians (seeds 42 + 7ℓ and 43 + 7ℓ)."""
    from .synth import gaussian_matrix, layer_seeds
    sp, ss = layer_seeds(layer)
    return rotation_from_gaussian(gaussian_matrix(sp, d)), gaussian_matrix(ss, d)


# ------------------------------------------------------------------ codec

class Codec:
    """Owns a tq_codec (device copies of Π, Πᵀ, Sᵀ, M and the codebook)."""

    def __init__(self, kind: int, bits: int, pi: np.ndarray, s: Optional[np.ndarray] = None,
                 centroids: Optional[np.ndarray] = None):
        self.kind = kind
        self.bits = bits
        self.index_bits = bits - 1 if kind == B.TQ_PROD else bits
        if centroids is None:
            centroids = lloyd_max_codebook(self.index_bits)
        self.pi = np.ascontiguousarray(pi, dtype=np.float64)
        self.s = None if s is None else np.ascontiguousarray(s, dtype=np.float64)
        self.centroids = np.ascontiguousarray(centroids, dtype=np.float64)
        h = ctypes.c_void_p()
        B.check(B.tq_codec_create(HEAD_DIM, kind, bits, self.pi.ctypes.data,
                                  0 if self.s is None else self.s.ctypes.data,
                                  self.centroids.ctypes.data, h), "tq_codec_create")
        self.handle = h

    @classmethod
    def prod(cls, bits: int, layer: int = 0) -> "Codec":
        pi, s = layer_constants(layer)
        return cls(B.TQ_PROD, bits, pi, s)

    @classmethod
    def mse(cls, bits: int, layer: int = 0) -> "Codec":
        pi, _ = layer_constants(layer)
        return cls(B.TQ_MSE, bits, pi)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            B.tq_codec_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ caches

def _cap(capacity: int) -> int:
    a = B.TQ_CAPACITY_ALIGN
    return (capacity + a - 1) // a * a


@dataclasses.dataclass
class Pages:
    """A block table over a page pool (include/tq.h, tq_pages): token t of sequence b lives in
    slot t % page_tokens of page block_table[b, t // page_tokens]."""
    block_table: torch.Tensor   # int32 [batch, max_pages], on the device
    page_tokens: int
    num_pages: int

    def __post_init__(self):
        if self.block_table.dtype != torch.int32 or self.block_table.dim() != 2:
            raise ValueError("block_table must be int32 [batch, max_pages]")
        self.block_table = self.block_table.contiguous()
        self._c = B.tq_pages(self.block_table.data_ptr(), self.block_table.shape[1],
                             self.page_tokens, self.num_pages)
        self._p = ctypes.pointer(self._c)

    @property
    def max_pages(self):
        return self.block_table.shape[1]

    @property
    def capacity(self):
        """Slots per sequence."""
        return self.max_pages * self.page_tokens

    def c(self):
        return self._p


def _pages_ptr(pages):
    return None if pages is None else pages.c()


def _holds(t: torch.Tensor, shape, dtype, device):
    return t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == device


class _Arrays:
    """What the key and value caches share: their layout, (sequences or pages, heads, slots, index
    bits, device), found out from all arrays at the first call that asks and again after one was
    replaced.  (The calls of long contexts ask; an array is not to be resized in place.)"""

    _layout = None

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_layout":
            object.__setattr__(self, "_layout", None)

    def layout(self):
        """Refuses arrays that are not codes and norms of one layout (include/tq.h) on one device."""
        n, d = self.xnorm.shape, self.xnorm.get_device()
        if len(n) != 3 or not _holds(self.xnorm, n, torch.float32, d) or not self._codes(n, d):
            got = ", ".join(f"{f} {t.dtype} {list(t.shape)} on {t.device}"
                            for f, t in vars(self).items() if hasattr(t, "dtype"))
            raise ValueError(f"expected contiguous uint8 codes and float32 norms of one layout on one device, "
                             f"got {got}")
        self._layout = (*n, self._bits(), d)
        return self._layout


@dataclasses.dataclass
class ProdCache(_Arrays):
    """Packed key cache [batch][heads][capacity] (layout of include/tq.h); with `pages` the
    arrays are a page pool [num_pages][heads][page_tokens] addressed through a block table."""
    idx: torch.Tensor      # uint8 [B, H, b-1, cap, 16]
    sgn: torch.Tensor      # uint8 [B, H, cap, 16]
    xnorm: torch.Tensor    # float32 [B, H, cap]
    rnorm: torch.Tensor    # float32 [B, H, cap]
    pages: Optional[Pages] = None

    @classmethod
    def empty(cls, batch, heads, capacity, bits, device="cuda"):
        cap = _cap(capacity)
        return cls(torch.zeros(batch, heads, bits - 1, cap, 16, dtype=torch.uint8, device=device),
                   torch.zeros(batch, heads, cap, 16, dtype=torch.uint8, device=device),
                   torch.zeros(batch, heads, cap, dtype=torch.float32, device=device),
                   torch.zeros(batch, heads, cap, dtype=torch.float32, device=device))

    @classmethod
    def empty_paged(cls, pages: Pages, heads, bits, device="cuda"):
        """A zeroed page pool of pages.num_pages pages for the block table `pages`."""
        c = cls.empty(pages.num_pages, heads, pages.page_tokens, bits, device)
        if c.capacity != pages.page_tokens:
            raise ValueError("page_tokens must be a multiple of TQ_CAPACITY_ALIGN")
        c.pages = pages
        return c

    def _bits(self):
        return self.idx.shape[2]

    def _codes(self, n, d):
        b = self.idx.shape[2] if len(self.idx.shape) == 5 else 0
        return (_holds(self.rnorm, n, torch.float32, d) and _holds(self.sgn, (*n, 16), torch.uint8, d) and
                _holds(self.idx, (n[0], n[1], b, n[2], 16), torch.uint8, d))

    @property
    def capacity(self):
        return self.pages.capacity if self.pages is not None else self.sgn.shape[2]

    def c(self):
        return B.tq_prod_cache(self.idx.data_ptr(), self.sgn.data_ptr(), self.xnorm.data_ptr(),
                               self.rnorm.data_ptr(), _pages_ptr(self.pages))

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (self.idx, self.sgn, self.xnorm, self.rnorm))


@dataclasses.dataclass
class MSECache(_Arrays):
    """Packed value cache [batch][heads][capacity]: bit planes, or nibbles for 4 bits; with
    `pages` a page pool as for ProdCache."""
    idx: torch.Tensor      # uint8 [B, H, bits, cap, 16] or [B, H, cap, 64]
    xnorm: torch.Tensor    # float32 [B, H, cap]
    bits: int
    pages: Optional[Pages] = None

    @classmethod
    def empty(cls, batch, heads, capacity, bits, device="cuda"):
        cap = _cap(capacity)
        if bits == 4:
            idx = torch.zeros(batch, heads, cap, 64, dtype=torch.uint8, device=device)
        else:
            idx = torch.zeros(batch, heads, bits, cap, 16, dtype=torch.uint8, device=device)
        return cls(idx, torch.zeros(batch, heads, cap, dtype=torch.float32, device=device), bits)

    @classmethod
    def empty_paged(cls, pages: Pages, heads, bits, device="cuda"):
        """A zeroed page pool of pages.num_pages pages for the block table `pages`."""
        c = cls.empty(pages.num_pages, heads, pages.page_tokens, bits, device)
        if c.xnorm.shape[2] != pages.page_tokens:
            raise ValueError("page_tokens must be a multiple of TQ_CAPACITY_ALIGN")
        c.pages = pages
        return c

    def _bits(self):
        return self.bits

    def _codes(self, n, d):
        return _holds(self.idx, (*n, 64) if self.bits == 4 else (n[0], n[1], self.bits, n[2], 16), torch.uint8, d)

    @property
    def capacity(self):
        return self.pages.capacity if self.pages is not None else self.xnorm.shape[2]

    def c(self):
        return B.tq_mse_cache(self.idx.data_ptr(), self.xnorm.data_ptr(), _pages_ptr(self.pages))

    def nbytes(self):
        return self.idx.numel() + self.xnorm.numel() * 4


# ------------------------------------------------------------------ calls

def _x_args(x: torch.Tensor):
    if x.dim() != 4 or x.shape[-1] != HEAD_DIM or x.stride(-1) != 1:
        raise ValueError("x must be [batch, heads, tokens, 128] with contiguous last dim")
    return *x.shape[:3], *x.stride()[:3]


def quantize_prod(codec: Codec, x: torch.Tensor, cache: ProdCache, pos=None, count=None,
                  stream=None):
    bsz, h, t, sb, sh, st = _x_args(x)
    B.check(B.tq_quantize_prod(codec.handle, x, tq_dtype(x.dtype), bsz, h, t, sb, sh, st, pos,
                               count, cache.c(), cache.capacity, _stream(stream)),
            "tq_quantize_prod")


def quantize_mse(codec: Codec, x: torch.Tensor, cache: MSECache, pos=None, count=None,
                 stream=None):
    bsz, h, t, sb, sh, st = _x_args(x)
    B.check(B.tq_quantize_mse(codec.handle, x, tq_dtype(x.dtype), bsz, h, t, sb, sh, st, pos,
                              count, cache.c(), cache.capacity, _stream(stream)),
            "tq_quantize_mse")


def prod_scores(codec: Codec, q: torch.Tensor, keys: ProdCache, n: int, out=None, stream=None):
    """[nq, n] raw estimator scores of fp32 queries q [nq, 128] against keys[0, 0, :n]."""
    q = q.contiguous()
    if out is None:
        out = torch.empty(q.shape[0], n, dtype=torch.float32, device=q.device)
    B.check(B.tq_prod_scores(codec.handle, q, q.shape[0], q.stride(0), keys.c(), keys.capacity,
                             n, out, out.stride(0), _stream(stream)), "tq_prod_scores")
    return out


def attention_quality(codec: Codec, q: torch.Tensor, k: torch.Tensor, keys: ProdCache, n: int,
                      softmax_scale=None, stream=None):
    """(KL [nq], top-1 position over exact keys [nq], over compressed keys [nq]) for fp32
    queries q [nq, 128] against the exact keys k [n, 128] and their codes keys[0, 0, :n]."""
    q = q.contiguous()
    k = k.contiguous()
    nq = q.shape[0]
    scratch = torch.empty(B.tq_attention_quality_scratch_bytes(nq, n), dtype=torch.uint8,
                          device=q.device)
    kl = torch.empty(nq, dtype=torch.float32, device=q.device)
    te = torch.empty(nq, dtype=torch.int32, device=q.device)
    tc = torch.empty(nq, dtype=torch.int32, device=q.device)
    B.check(B.tq_attention_quality(codec.handle, q, nq, k, tq_dtype(k.dtype), keys.c(),
                                   keys.capacity, n, softmax_scale or 0.0, scratch,
                                   scratch.numel(), kl, te, tc, _stream(stream)),
            "tq_attention_quality")
    return kl, te, tc


class DecodePlan:
    """A decode-attention configuration with its workspace (allocated once, reused)."""

    def __init__(self, batch, q_heads, kv_heads, capacity, max_seq_len, q_dtype=torch.bfloat16,
                 out_dtype=torch.float32, tail_capacity=0, softmax_scale=None, device="cuda"):
        self.desc = B.tq_attn_desc(batch, q_heads, kv_heads, HEAD_DIM, _cap(capacity),
                                   max_seq_len, tail_capacity,
                                   softmax_scale if softmax_scale else 0.0,
                                   tq_dtype(q_dtype), tq_dtype(out_dtype))
        nbytes = B.tq_decode_workspace_bytes(self.desc)
        if nbytes == 0:
            raise ValueError("invalid decode-attention configuration")
        # caller-owned scratch; the library clears what must start at zero on every call
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.out_dtype = out_dtype
        self.shape = (batch, q_heads, HEAD_DIM)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.out_dtype, device=device)

    def run(self, kc: Codec, vc: Codec, q, k: ProdCache, v: MSECache, seq_lens, out, stream=None):
        B.check(B.tq_decode_attention(self.desc, kc.handle, vc.handle, q, k.c(), v.c(), seq_lens,
                                      out, self.workspace, self.workspace.numel(),
                                      _stream(stream)), "tq_decode_attention")
        return out

    def step(self, kc: Codec, vc: Codec, q, k_new, v_new, k: ProdCache, v: MSECache, pos, out,
             lens_out=None, stream=None):
        """Appends k_new, v_new [batch, kv_heads, 128] at pos[b] and attends pos[b] + 1 tokens."""
        if k_new.dtype != v_new.dtype or not (k_new.is_contiguous() and v_new.is_contiguous()):
            raise ValueError("k_new and v_new must be contiguous and of one dtype")
        B.check(B.tq_decode_step(self.desc, kc.handle, vc.handle, q, k_new, v_new,
                                 tq_dtype(k_new.dtype), k.c(), v.c(), pos, lens_out, out,
                                 self.workspace, self.workspace.numel(), _stream(stream)),
                "tq_decode_step")
        return out

    def run_asym(self, vc: Codec, q, k_f16, v: MSECache, seq_lens, k_tail, v_tail, tail_lens,
                 out, stream=None):
        B.check(B.tq_decode_attention_asym(self.desc, vc.handle, q, k_f16, v.c(), seq_lens,
                                           k_tail, v_tail, tail_lens, out, self.workspace,
                                           self.workspace.numel(), _stream(stream)),
                "tq_decode_attention_asym")
        return out


class PrefillPlan:
    """Attention of chunks of n_queries queries per sequence over a compressed cache
    (tq_prefill_attention), with its workspace."""

    def __init__(self, batch, n_queries, q_heads, kv_heads, capacity, max_seq_len, causal=True,
                 q_dtype=torch.bfloat16, out_dtype=torch.float32, device="cuda"):
        self.desc = B.tq_attn_desc(batch, q_heads, kv_heads, HEAD_DIM, _cap(capacity), max_seq_len,
                                   0, 0.0, tq_dtype(q_dtype), tq_dtype(out_dtype))
        self.n_queries = n_queries
        self.causal = 1 if causal else 0
        nbytes = B.tq_prefill_workspace_bytes(self.desc, n_queries)
        if nbytes == 0:
            raise ValueError("invalid prefill-attention configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.out_dtype = out_dtype
        self.shape = (batch, n_queries, q_heads, HEAD_DIM)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.out_dtype, device=device)

    def run(self, kc: Codec, vc: Codec, q, k: ProdCache, v: MSECache, seq_lens, out, stream=None):
        B.check(B.tq_prefill_attention(self.desc, self.n_queries, self.causal, kc.handle, vc.handle,
                                       q, k.c(), v.c(), seq_lens, out, self.workspace,
                                       self.workspace.numel(), _stream(stream)),
                "tq_prefill_attention")
        return out


# ------------------------------------------------------------------ long contexts

# These calls run once per layer and step and mostly in less time than a careful wrapper takes, so
# their checks read each property once and the library is called with plain integers.

def _device(*tensors):
    """The current device, which the library works on: tensors of another one are refused."""
    d = torch._C._cuda_getDevice()
    for t in tensors:
        if t.get_device() != d:
            raise ValueError(f"expected tensors on the current device cuda:{d}, got one on {t.device}")
    return d


def _on(stream, device):
    """Handle of the stream: the device's current one by default."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _expect(t: torch.Tensor, shape, dtype, name):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, "
                         f"got {t.dtype} {list(t.shape)}")


def _fits(layout, pages, rows, heads, slots):
    """Whether arrays of a layout hold `rows` sequences of `slots` slots."""
    if layout[1] != heads:
        return False
    if pages is None:
        return layout[0] >= rows and layout[2] == slots
    return (layout[0] >= pages.num_pages and layout[2] == pages.page_tokens and
            pages.capacity == slots and pages.block_table.shape[0] >= rows and
            pages.block_table.get_device() == layout[4])


def _expect_caches(k: "ProdCache", v: "MSECache", rows, heads, slots, kc, vc, name):
    """A pair of caches (or pools) for `rows` sequences of `slots` slots: every array of each."""
    kl, vl = k._layout or k.layout(), v._layout or v.layout()
    if not (_fits(kl, k.pages, rows, heads, slots) and _fits(vl, v.pages, rows, heads, slots)) or kl[4] != vl[4]:
        raise ValueError(f"{name}: expected {rows} sequences or a block table for them, {heads} heads and "
                         f"{slots} slots on one device, got keys {list(k.xnorm.shape)} on {k.xnorm.device} and "
                         f"values {list(v.xnorm.shape)} on {v.xnorm.device}")
    if kl[3] != kc.index_bits or vl[3] != vc.bits:
        raise ValueError(f"{name}: the caches hold codes of other widths than the codecs'")


@dataclasses.dataclass
class BlockBounds:
    """Per-block bounds of a cache's keys (include/tq.h, tq_block_cache): lower and upper bounds
    of the 128 channels over each block of 64 tokens; with `pages` a pool as for ProdCache."""
    bounds: torch.Tensor   # bfloat16 [B, H, cap / 64, 2, 128]
    pages: Optional[Pages] = None

    @classmethod
    def empty(cls, batch, heads, capacity, device="cuda"):
        return cls(torch.zeros(batch, heads, _cap(capacity) // B.TQ_BLOCK_TOKENS, 2, HEAD_DIM,
                               dtype=torch.bfloat16, device=device))

    @classmethod
    def empty_paged(cls, pages: Pages, heads, device="cuda"):
        if pages.page_tokens % B.TQ_CAPACITY_ALIGN:
            raise ValueError("page_tokens must be a multiple of TQ_CAPACITY_ALIGN")
        b = cls.empty(pages.num_pages, heads, pages.page_tokens, device)
        b.pages = pages
        return b

    @property
    def capacity(self):
        return self.pages.capacity if self.pages is not None \
            else self.bounds.shape[2] * B.TQ_BLOCK_TOKENS

    def c(self):
        return B.tq_block_cache(self.bounds.data_ptr(), _pages_ptr(self.pages))

    def expect(self, rows, heads, slots):
        """Refuses bounds that are not those of `rows` sequences of `slots` slots."""
        t, p = self.bounds, self.pages
        n = slots if p is None else p.page_tokens
        s = t.shape
        if s != (s[0], heads, n // B.TQ_BLOCK_TOKENS, 2, HEAD_DIM) or t.dtype != torch.bfloat16 or \
                not t.is_contiguous() or s[0] < (rows if p is None else p.num_pages) or \
                p is not None and (p.capacity != slots or p.block_table.shape[0] < rows or
                                   p.block_table.get_device() != t.get_device()):
            raise ValueError(f"bounds: expected {rows} sequences or a block table for them, {heads} heads "
                             f"and {slots} slots, got {t.dtype} {list(s)}")


def block_bounds(x: torch.Tensor, blocks: BlockBounds, pos=None, count=None, stream=None):
    """Folds keys x [batch, heads, tokens, 128] into their blocks' bounds, at the cache positions
    pos[b].. (0) and count[b] tokens each (all): the arguments of quantize_prod."""
    bsz, h, t, sb, sh, stride_t = _x_args(x)
    slots = blocks.capacity
    blocks.expect(bsz, h, slots)
    d = _device(x, blocks.bounds)
    at = n = None
    if pos is not None:
        _expect(pos, (bsz,), torch.int32, "pos")
        _device(pos)
        at = pos.data_ptr()
    if count is not None:
        _expect(count, (bsz,), torch.int32, "count")
        _device(count)
        n = count.data_ptr()
    st = B.load().tq_block_bounds(x.data_ptr(), tq_dtype(x.dtype), bsz, h, t, sb, sh, stride_t, at, n,
                                  blocks.c(), slots, _on(stream, d))
    if st:
        B.check(st, "tq_block_bounds")


class SparsePlan:
    """Block-sparse decode attention: which blocks a query attends (tq_block_select) and attention
    over them (tq_sparse_attention), with the workspace of both (allocated once, reused; calls of
    a plan are to be serialised on one stream).  Of each sequence at most max_blocks blocks of 64
    tokens are attended, the first first_blocks and the last last_blocks always."""

    def __init__(self, batch, q_heads, kv_heads, capacity, max_seq_len, max_blocks,
                 first_blocks=1, last_blocks=2, q_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                 softmax_scale=None, device="cuda"):
        self.desc = B.tq_attn_desc(batch, q_heads, kv_heads, HEAD_DIM, _cap(capacity),
                                   max_seq_len, 0, softmax_scale if softmax_scale else 0.0,
                                   tq_dtype(q_dtype), tq_dtype(out_dtype))
        sizes = (B.tq_block_select_workspace_bytes(self.desc),
                 B.tq_sparse_workspace_bytes(self.desc, max_blocks))
        if 0 in sizes or first_blocks < 0 or last_blocks < 0 or \
                first_blocks + last_blocks > max_blocks:
            raise ValueError("invalid sparse-attention configuration")
        self.nbytes = max(sizes)
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.rows, self.list_shape = (batch,), (batch, kv_heads, max_blocks)
        self.max_blocks, self.first_blocks, self.last_blocks = max_blocks, first_blocks, last_blocks
        self.batch, self.kv_heads, self.capacity = batch, kv_heads, _cap(capacity)
        self.q_dtype, self.out_dtype = q_dtype, out_dtype
        self.shape = (batch, q_heads, HEAD_DIM)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.out_dtype, device=device)

    def new_list(self, device="cuda"):
        return torch.empty(self.list_shape, dtype=torch.int32, device=device)

    def _check_select(self, q, blocks, seq_lens, out):
        _expect(q, self.shape, self.q_dtype, "q")
        _expect(seq_lens, self.rows, torch.int32, "seq_lens")
        _expect(out, self.list_shape, torch.int32, "out")
        blocks.expect(self.batch, self.kv_heads, self.capacity)

    def _select(self, q, blocks, seq_lens, out, stream):
        st = B.load().tq_block_select(self.desc, q.data_ptr(), blocks.c(), seq_lens.data_ptr(),
                                      self.first_blocks, self.last_blocks, self.max_blocks,
                                      out.data_ptr(), self.workspace.data_ptr(), self.nbytes, stream)
        if st:
            B.check(st, "tq_block_select")
        return out

    def select(self, q, blocks: BlockBounds, seq_lens, out, stream=None):
        """The blocks of each (sequence, KV head) that q [batch, q_heads, 128] attends, ascending,
        −1 behind them, into out [batch, kv_heads, max_blocks] int32."""
        d = _device(q, blocks.bounds, seq_lens, out, self.workspace)
        self._check_select(q, blocks, seq_lens, out)
        return self._select(q, blocks, seq_lens, out, _on(stream, d))

    def _check_run(self, kc, vc, q, k, v, seq_lens, block_list, out):
        _expect(q, self.shape, self.q_dtype, "q")
        _expect(seq_lens, self.rows, torch.int32, "seq_lens")
        _expect(block_list, self.list_shape, torch.int32, "block_list")
        _expect(out, self.shape, self.out_dtype, "out")
        _expect_caches(k, v, self.batch, self.kv_heads, self.capacity, kc, vc, "cache")

    def _run(self, kc, vc, q, k, v, seq_lens, block_list, out, stream):
        st = B.load().tq_sparse_attention(self.desc, kc.handle, vc.handle, q.data_ptr(), k.c(), v.c(),
                                          seq_lens.data_ptr(), block_list.data_ptr(),
                                          self.max_blocks, out.data_ptr(),
                                          self.workspace.data_ptr(), self.nbytes, stream)
        if st:
            B.check(st, "tq_sparse_attention")
        return out

    def run(self, kc: Codec, vc: Codec, q, k: ProdCache, v: MSECache, seq_lens, block_list, out,
            stream=None):
        """Attention of q over the listed blocks of the cache, into out [batch, q_heads, 128]."""
        d = _device(q, k.idx, v.idx, seq_lens, block_list, out, self.workspace)
        self._check_run(kc, vc, q, k, v, seq_lens, block_list, out)
        return self._run(kc, vc, q, k, v, seq_lens, block_list, out, _on(stream, d))

    def step(self, kc: Codec, vc: Codec, q, k_new, v_new, k: ProdCache, v: MSECache,
             blocks: BlockBounds, pos, seq_lens, block_list, out, stream=None):
        """One decode step: appends k_new, v_new [batch, kv_heads, 128] at pos[b] (codes and
        bounds), selects blocks and attends them.  seq_lens holds pos + 1.  All arguments are
        checked before anything is written."""
        d = _device(q, k_new, v_new, k.idx, v.idx, blocks.bounds, pos, seq_lens, block_list, out, self.workspace)
        for x, name in ((k_new, "k_new"), (v_new, "v_new")):
            if x.shape != (self.batch, self.kv_heads, HEAD_DIM) or x.dtype not in _DT:
                raise ValueError(f"{name} must be [{self.batch}, {self.kv_heads}, {HEAD_DIM}] of float32, "
                                 f"float16 or bfloat16, got {x.dtype} {list(x.shape)}")
            size = x.element_size()
            if x.stride(2) != 1 or (x.data_ptr() | x.stride(0) * size | x.stride(1) * size) % 16:
                raise ValueError(f"{name} must have contiguous vectors that begin at multiples of 16 bytes")
        if kc.kind != B.TQ_PROD or vc.kind != B.TQ_MSE:
            raise ValueError("expected a codec of keys (TQ_PROD) and one of values (TQ_MSE)")
        _expect(pos, self.rows, torch.int32, "pos")
        self._check_select(q, blocks, seq_lens, block_list)
        self._check_run(kc, vc, q, k, v, seq_lens, block_list, out)
        stream = _on(stream, d)
        k_new, v_new = k_new.unsqueeze(2), v_new.unsqueeze(2)
        quantize_prod(kc, k_new, k, pos=pos, stream=stream)
        quantize_mse(vc, v_new, v, pos=pos, stream=stream)
        block_bounds(k_new, blocks, pos=pos, stream=stream)
        self._select(q, blocks, seq_lens, block_list, stream)
        return self._run(kc, vc, q, k, v, seq_lens, block_list, out, stream)


class PrefixPlan:
    """Decode attention of a batch whose sequences share a prefix (tq_prefix_attention), with its
    workspace (allocated once, reused; calls of a plan are to be serialised on one stream)."""

    def __init__(self, batch, q_heads, kv_heads, capacity, max_seq_len, prefix_capacity,
                 prefix_max_len, q_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                 softmax_scale=None, device="cuda"):
        self.desc = B.tq_attn_desc(batch, q_heads, kv_heads, HEAD_DIM, _cap(capacity),
                                   max_seq_len, 0, softmax_scale if softmax_scale else 0.0,
                                   tq_dtype(q_dtype), tq_dtype(out_dtype))
        nbytes = B.tq_prefix_workspace_bytes(self.desc, prefix_max_len)
        if nbytes == 0 or prefix_max_len > _cap(prefix_capacity):
            raise ValueError("invalid prefix-attention configuration")
        self.nbytes = nbytes
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.rows = (batch,)
        self.batch, self.kv_heads, self.capacity = batch, kv_heads, _cap(capacity)
        self.prefix_capacity, self.prefix_max_len = _cap(prefix_capacity), prefix_max_len
        self.q_dtype, self.out_dtype = q_dtype, out_dtype
        self.shape = (batch, q_heads, HEAD_DIM)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.out_dtype, device=device)

    def run(self, kc: Codec, vc: Codec, q, prefix_k: ProdCache, prefix_v: MSECache, prefix_len,
            k: ProdCache, v: MSECache, seq_lens, out, stream=None):
        """Attention of q [batch, q_heads, 128] over the prefix's prefix_len (int32 [1]) tokens and
        each sequence's own seq_lens[b] tokens."""
        d = _device(q, prefix_k.idx, prefix_v.idx, prefix_len, k.idx, v.idx, seq_lens, out,
                    self.workspace)
        _expect(q, self.shape, self.q_dtype, "q")
        _expect(prefix_len, (1,), torch.int32, "prefix_len")
        _expect(seq_lens, self.rows, torch.int32, "seq_lens")
        _expect(out, self.shape, self.out_dtype, "out")
        _expect_caches(prefix_k, prefix_v, 1, self.kv_heads, self.prefix_capacity, kc, vc, "prefix")
        _expect_caches(k, v, self.batch, self.kv_heads, self.capacity, kc, vc, "cache")
        st = B.load().tq_prefix_attention(self.desc, kc.handle, vc.handle, q.data_ptr(),
                                          prefix_k.c(), prefix_v.c(), self.prefix_capacity,
                                          self.prefix_max_len, prefix_len.data_ptr(), k.c(), v.c(),
                                          seq_lens.data_ptr(), out.data_ptr(),
                                          self.workspace.data_ptr(), self.nbytes, _on(stream, d))
        if st:
            B.check(st, "tq_prefix_attention")
        return out


# ------------------------------------------------------------------ rotary positions

class Rotary:
    """Rotary positions (include/tq.h, tq_rotary): angles position · f_i on pairs of the first
    rotary_dim coordinates, neighbouring ones (interleaved) or halves.  Frequencies are
    base^(−2i/rotary_dim), divided by `factor` for longer contexts, all of them or, with
    original_len, by parts (tq_rotary_frequencies); or an array of rotary_dim / 2 of the caller's."""

    def __init__(self, rotary_dim=HEAD_DIM, base=10000.0, interleaved=False, factor=1.0, original_len=0,
                 low_turns=1.0, high_turns=32.0, magnitude=1.0, frequencies=None):
        if frequencies is None:
            frequencies = np.zeros(HEAD_DIM // 2, dtype=np.float64)
            B.check(B.tq_rotary_frequencies(rotary_dim, base, factor, original_len, low_turns, high_turns,
                                            frequencies.ctypes.data), "tq_rotary_frequencies")
            frequencies = frequencies[:rotary_dim // 2]
        self.frequencies = np.ascontiguousarray(frequencies, dtype=np.float64)
        if self.frequencies.shape != (rotary_dim // 2,):
            raise ValueError(f"expected {rotary_dim // 2} frequencies, got {list(self.frequencies.shape)}")
        self.rotary_dim, self.interleaved, self.magnitude = rotary_dim, bool(interleaved), float(magnitude)
        self._c = B.tq_rotary()
        B.check(B.tq_rotary_init(self._c, rotary_dim, int(self.interleaved), self.frequencies,
                                 self.magnitude), "tq_rotary_init")

    @staticmethod
    def _io(x, y, name, batch, tokens, dtype):
        sx, sy, shape = x.stride(), y.stride(), x.shape
        if len(shape) != 4 or shape[0] != batch or shape[2] != tokens or shape[3] != HEAD_DIM or x.dtype != dtype or \
                y.shape != shape or y.dtype != dtype or sx[3] != 1 or sy[3] != 1:
            raise ValueError(f"{name} must be [{batch}, heads, {tokens}, {HEAD_DIM}] of {dtype} with contiguous "
                             f"last dim, and its output the same, got {x.dtype} {list(shape)} and {y.dtype} "
                             f"{list(y.shape)}")
        return B.tq_rotary_io(x.data_ptr(), y.data_ptr(), shape[1], sx[0], sx[1], sx[2], sy[0], sy[1], sy[2])

    def apply(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """Turns q and k [batch, heads, tokens, 128] (any strides, k may be None) by their positions,
        int32 [batch, tokens], in one launch; into q_out and k_out, memory apart from the inputs, or in
        place.  Returns both."""
        if q_out is None:
            q_out = q
        batch, tokens = positions.shape
        ps, dtype = positions.stride(), q.dtype
        if positions.dtype != torch.int32 or (tokens > 1 and ps[1] != 1):
            raise ValueError("positions must be int32 [batch, tokens] with contiguous rows")
        io_k = None
        if k is None:
            d = _device(q, positions, q_out)
        else:
            if k_out is None:
                k_out = k
            d = _device(q, k, positions, q_out, k_out)
            io_k = self._io(k, k_out, "k", batch, tokens, dtype)
        st = B.load().tq_rotary_apply(self._c, tq_dtype(dtype), batch, tokens, positions.data_ptr(), ps[0],
                                      self._io(q, q_out, "q", batch, tokens, dtype), io_k, _on(stream, d))
        if st:
            B.check(st, "tq_rotary_apply")
        return q_out, k_out


# ------------------------------------------------------------------ prompts on exact keys

class PromptPlan:
    """Attention of packed sequences over their exact keys and values (tq_prompt_attention), with its
    workspace (allocated once, reused; calls of a plan are to be serialised on one stream).  total_q
    and total_k are the rows of q and of k and v, which may hold more than the sequences; max_k_len is
    about the keys of the longest sequence and splits the work."""

    def __init__(self, batch, q_heads, kv_heads, total_q, total_k, max_k_len, causal=True, dtype=torch.bfloat16,
                 softmax_scale=None, device="cuda"):
        self.desc = B.tq_prompt_desc(batch, q_heads, kv_heads, HEAD_DIM, total_q, total_k, max_k_len, int(bool(causal)),
                                     softmax_scale if softmax_scale else 0.0, tq_dtype(dtype))
        self.nbytes = B.tq_prompt_workspace_bytes(self.desc)
        if self.nbytes == 0:
            raise ValueError("invalid prompt-attention configuration")
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.dtype, self.shape, self.k_shape = dtype, (total_q, q_heads, HEAD_DIM), (total_k, kv_heads, HEAD_DIM)
        self.starts = (batch + 1,)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.dtype, device=device)

    def run(self, q, k, v, q_starts, k_starts, out, stream=None):
        """Attention of q [total_q, q_heads, 128] over k and v [total_k, kv_heads, 128] (views with any
        strides of multiples of 8 elements), into out [total_q, q_heads, 128], q itself or memory apart from
        the inputs; q_starts and k_starts, int32 [batch + 1], are where each sequence's rows begin (the
        same for whole prompts)."""
        d = _device(q, k, v, q_starts, k_starts, out, self.workspace)
        sq, sk, sv = q.stride(), k.stride(), v.stride()
        for t, s, shape, name in ((q, sq, self.shape, "q"), (k, sk, self.k_shape, "k"), (v, sv, self.k_shape, "v")):
            if t.shape != shape or t.dtype != self.dtype or s[2] != 1:
                raise ValueError(f"{name} must be {self.dtype} {list(shape)} with contiguous last dim, "
                                 f"got {t.dtype} {list(t.shape)}")
        _expect(q_starts, self.starts, torch.int32, "q_starts")
        _expect(k_starts, self.starts, torch.int32, "k_starts")
        _expect(out, self.shape, self.dtype, "out")
        st = B.load().tq_prompt_attention(self.desc, q.data_ptr(), sq[0], sq[1], k.data_ptr(), sk[0], sk[1], v.data_ptr(),
                                          sv[0], sv[1], q_starts.data_ptr(), k_starts.data_ptr(), out.data_ptr(),
                                          self.workspace.data_ptr(), self.nbytes, _on(stream, d))
        if st:
            B.check(st, "tq_prompt_attention")
        return out


# ------------------------------------------------------------------ drafted tokens

class TreePlan:
    """Attention of drafted tokens over the compressed cache (tq_tree_attention), with its workspace
    (allocated once, reused; calls of a plan are to be serialised on one stream).  The drafted
    tokens' keys and values are in the cache behind the history; max_seq_len bounds a history and
    its drafted tokens."""

    def __init__(self, batch, n_nodes, q_heads, kv_heads, capacity, max_seq_len, q_dtype=torch.bfloat16,
                 out_dtype=torch.bfloat16, softmax_scale=None, device="cuda"):
        self.desc = B.tq_attn_desc(batch, q_heads, kv_heads, HEAD_DIM, _cap(capacity),
                                   max_seq_len, 0, softmax_scale if softmax_scale else 0.0,
                                   tq_dtype(q_dtype), tq_dtype(out_dtype))
        self.nbytes = B.tq_tree_workspace_bytes(self.desc, n_nodes)
        if self.nbytes == 0:
            raise ValueError("invalid tree-attention configuration")
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.batch, self.n_nodes, self.kv_heads, self.capacity = batch, n_nodes, kv_heads, _cap(capacity)
        self.q_dtype, self.out_dtype = q_dtype, out_dtype
        self.rows, self.shape = (batch,), (batch, n_nodes, q_heads, HEAD_DIM)

    def new_out(self, device="cuda"):
        return torch.empty(self.shape, dtype=self.out_dtype, device=device)

    def run(self, kc: Codec, vc: Codec, q, k: ProdCache, v: MSECache, seq_lens, tree, out, stream=None):
        """Attention of q [batch, n_nodes, q_heads, 128] over each sequence's seq_lens[b] tokens and the
        drafted tokens that tree, int64 [batch, n_nodes] ([1, n_nodes]: one for all sequences), names:
        bit j of a node's number is drafted token j, token seq_lens[b] + j of the cache."""
        d = _device(q, k.idx, v.idx, seq_lens, tree, out, self.workspace)
        _expect(q, self.shape, self.q_dtype, "q")
        _expect(seq_lens, self.rows, torch.int32, "seq_lens")
        shared = tree.shape[0] == 1
        _expect(tree, (1 if shared else self.batch, self.n_nodes), torch.int64, "tree")
        _expect(out, self.shape, self.out_dtype, "out")
        _expect_caches(k, v, self.batch, self.kv_heads, self.capacity, kc, vc, "cache")
        st = B.load().tq_tree_attention(self.desc, self.n_nodes, kc.handle, vc.handle, q.data_ptr(), k.c(), v.c(),
                                        seq_lens.data_ptr(), tree.data_ptr(), 0 if shared else self.n_nodes,
                                        out.data_ptr(), self.workspace.data_ptr(), self.nbytes, _on(stream, d))
        if st:
            B.check(st, "tq_tree_attention")
        return out


def keep_tokens(k: ProdCache, v: MSECache, pos, keep, stream=None):
    """Keeps tokens of those behind pos[b] (int32 [batch]): for each entry j ≥ 0 of keep, int32 [batch,
    at most 64], the codes of token pos[b] + j become those of token pos[b] + i, i the entry's index
    (include/tq.h, tq_keep_tokens)."""
    kl, vl, slots = k._layout or k.layout(), v._layout or v.layout(), k.capacity
    n = keep.shape
    if len(n) != 2:
        raise ValueError("keep must be int32 [batch, tokens]")
    batch, heads = n[0], kl[1]
    if not (_fits(kl, k.pages, batch, heads, slots) and _fits(vl, v.pages, batch, heads, slots)) or kl[4] != vl[4]:
        raise ValueError(f"expected caches of {batch} sequences or block tables for them, of the same heads and "
                         f"slots on one device, got keys {list(k.xnorm.shape)} and values {list(v.xnorm.shape)}")
    _expect(pos, (batch,), torch.int32, "pos")
    _expect(keep, n, torch.int32, "keep")
    d = _device(k.idx, pos, keep)
    st = B.load().tq_keep_tokens(k.c(), kl[3] + 1, v.c(), vl[3], batch, heads, slots, pos.data_ptr(),
                                 keep.data_ptr(), n[1], _on(stream, d))
    if st:
        B.check(st, "tq_keep_tokens")


def copy_pages(src, dst, k: Optional[ProdCache] = None, v: Optional[MSECache] = None,
               blocks: Optional[BlockBounds] = None, stream=None):
    """Copies page src[i] to page dst[i] (int32 [n], −1: passed over) of a pool in every array given: its
    keys, values and block bounds (include/tq.h, tq_copy_pages).  Of a flat cache the sequences are
    the pages."""
    pools, kc, vc, bc, kbits, vbits = [], None, None, None, 0, 0      # (pages, heads, slots, device) of each
    if k is not None:
        pages, heads, slots, bits, at = k._layout or k.layout()
        pools.append((pages, heads, slots, at))
        kc, kbits = k.c(), bits + 1
    if v is not None:
        pages, heads, slots, vbits, at = v._layout or v.layout()
        pools.append((pages, heads, slots, at))
        vc = v.c()
    if blocks is not None:
        t = blocks.bounds
        s = t.shape
        if len(s) != 5 or s[3] != 2 or s[4] != HEAD_DIM or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"bounds must be contiguous bfloat16 [pages, heads, blocks, 2, 128], got {t.dtype} {list(s)}")
        pools.append((s[0], s[1], s[2] * B.TQ_BLOCK_TOKENS, t.get_device()))
        bc = blocks.c()
    if not pools or any(p != pools[0] for p in pools):
        raise ValueError("expected keys, values or bounds of pools of one shape on one device, got "
                         + (", ".join(str(list(p[:3])) for p in pools) or "none"))
    pages, heads, slots, at = pools[0]
    n = src.shape
    if len(n) != 1:
        raise ValueError("src must be int32 [n]")
    _expect(src, n, torch.int32, "src")
    _expect(dst, n, torch.int32, "dst")
    d = _device(src, dst)
    if at != d:
        raise ValueError(f"expected a pool on the current device cuda:{d}")
    st = B.load().tq_copy_pages(kc, kbits, vc, vbits, bc, heads, pages, slots, src.data_ptr(), dst.data_ptr(), n[0],
                                _on(stream, d))
    if st:
        B.check(st, "tq_copy_pages")


class TailStore:
    """A cache in the asymmetric layout: a compressed part (FP16 keys, MSE-coded values) and an
    FP16 tail of the most recent tokens that compacts into the compressed part when it fills
    (tq_store_append); read with DecodePlan.run_asym."""

    def __init__(self, vc: Codec, batch, kv_heads, capacity, tail_capacity=256, device="cuda"):
        cap = _cap(capacity)
        self.vc = vc
        self.batch, self.kv_heads, self.capacity, self.tail_capacity = batch, kv_heads, cap, tail_capacity
        self.k_f16 = torch.zeros(batch, kv_heads, cap, HEAD_DIM, dtype=torch.float16, device=device)
        self.v = MSECache.empty(batch, kv_heads, cap, vc.bits, device=device)
        self.k_tail = torch.zeros(batch, kv_heads, tail_capacity, HEAD_DIM, dtype=torch.float16,
                                  device=device)
        self.v_tail = torch.zeros_like(self.k_tail)
        self.comp_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.tail_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.workspace = torch.empty(max(B.tq_store_workspace_bytes(batch), 256), dtype=torch.uint8,
                                     device=device)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        """k_new, v_new: [batch, kv_heads, 128] contiguous, one dtype."""
        B.check(B.tq_store_append(self.vc.handle, self.batch, self.kv_heads, k_new, v_new,
                                  tq_dtype(k_new.dtype), self.k_f16, self.v.c(), self.capacity,
                                  self.k_tail, self.v_tail, self.tail_capacity, self.comp_lens,
                                  self.tail_lens, self.workspace, self.workspace.numel(),
                                  _stream(stream)), "tq_store_append")

    def plan(self, q_heads, q_dtype=torch.bfloat16, out_dtype=torch.float32, device="cuda"):
        return DecodePlan(self.batch, q_heads, self.kv_heads, self.capacity, self.capacity, q_dtype,
                          out_dtype, tail_capacity=self.tail_capacity, device=device)

    def decode(self, plan: "DecodePlan", q, out, stream=None):
        return plan.run_asym(self.vc, q, self.k_f16, self.v, self.comp_lens, self.k_tail,
                             self.v_tail, self.tail_lens, out, stream=stream)


def device_status():
    """(status, flags) of the device status word (synchronises the device)."""
    return B.tq_device_status()
