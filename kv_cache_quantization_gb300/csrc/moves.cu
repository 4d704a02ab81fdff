// Moving codes inside a cache: whole pages of a pool (tq_copy_pages: forks of sequences, a pool put
// in order) and single tokens (tq_keep_tokens: the accepted ones of the tokens drafted behind a
// sequence move to the front of them).
#include <algorithm>

#include "tq_internal.h"

TQ_DEFINE_FLAGS(tq_take_flags_moves)

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---------------------------------------------------------------- pages
// A page is one contiguous span of each array.  The spans are cut into pieces of kPiece vectors of
// 16 bytes, and a CTA copies every `ways`-th piece of a page, kFlight loads in flight a thread.
constexpr int kArrays = 7, kCopyThreads = 256, kFlight = 4, kPiece = kCopyThreads * kFlight;

struct CopyArgs {
  uint4* base[kArrays];
  uint32_t vecs[kArrays];        // 16-byte vectors of a page
  int pieces[kArrays + 1];       // pieces before each array's
  int arrays, ways, n, num_pages;
  const int* src;
  const int* dst;
};

// Bound by the copy's bytes: 2048 pages of 256 tokens and 8 heads (3-bit keys, 2-bit values, bounds) take
// 130 us, 6.5 TB/s; 8 pages 2.4 us, a launch.  The scan of all pairs for one that this one's destination collides
// with runs while the first loads are in flight.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  const int i = blockIdx.x / a.ways, tid = threadIdx.x;
  const long long src = a.src[i], dst = a.dst[i];
  if (src < 0 || dst < 0) {
    // −1 is passed over; anything else is a bad page
    if ((src < -1 || dst < -1) && blockIdx.x % a.ways == 0 && tid == 0) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
    return;
  }
  bool ok = src < a.num_pages && dst < a.num_pages;
  if (ok && src == dst) return;
  bool first = true;
  for (int piece = blockIdx.x % a.ways; piece < a.pieces[a.arrays]; piece += a.ways) {
    uint4 v[kFlight];
    int k = 0;
    while (k + 1 < a.arrays && piece >= a.pieces[k + 1]) ++k;
    const uint32_t at = (uint32_t)(piece - a.pieces[k]) * kPiece + tid;
    if (ok) {
      const uint4* from = a.base[k] + src * a.vecs[k];
#pragma unroll
      for (int f = 0; f < kFlight; ++f)
        if (at + f * kCopyThreads < a.vecs[k]) v[f] = from[at + f * kCopyThreads];
    }
    if (first) {
      // the pair is left out if its destination is another one's source or destination
      bool clash = !ok;
      if (ok)
        for (int j = tid; j < a.n; j += kCopyThreads) {
          const int s = a.src[j], d = a.dst[j];
          clash |= j != i && s >= 0 && d >= 0 && s != d && (s == dst || d == dst);
        }
      ok = !__syncthreads_or(clash);
      if (!ok && blockIdx.x % a.ways == 0 && tid == 0) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
      if (!ok) return;
      first = false;
    }
    uint4* to = a.base[k] + dst * a.vecs[k];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (at + f * kCopyThreads < a.vecs[k]) to[at + f * kCopyThreads] = v[f];
  }
}

// Long lists.  Above, each of n CTAs looks at all n pairs, which is most of the time from some thousand small
// pages on.  Here two CTAs an SM hold up to kManyPairs pairs each, their destinations in a hash table, so that
// a CTA looks at the list once for all of them; then its warps take its pages' pieces of kWarpPiece vectors in
// turn: 65536 pages of 6 KB (64 tokens of one head, 3-bit keys, 2-bit values) 222 us, 3.5 TB/s.
constexpr int kManyThreads = 512, kManyPairs = 256, kSlots = 1024, kWarpPiece = 32 * kFlight;

__global__ void __launch_bounds__(kManyThreads, 2) copy_many_pages_kernel(const __grid_constant__ CopyArgs a, int per_cta) {
  __shared__ int src[kManyPairs], dst[kManyPairs], slot[kSlots], left_out[kManyPairs];
  const int tid = threadIdx.x, i0 = blockIdx.x * per_cta, pairs = min(per_cta, a.n - i0);
  for (int i = tid; i < kSlots; i += kManyThreads) slot[i] = 0;
  auto first_slot = [](int page) { return (int)(((uint32_t)page * 2654435761u) >> 22); };      // (spreads runs of pages)
  bool bad = false, mine = false;
  if (tid < pairs) {
    const int s = a.src[i0 + tid], d = a.dst[i0 + tid];
    src[tid] = s;
    dst[tid] = d;
    if (s < 0 || d < 0) bad = s < -1 || d < -1;
    else bad = s >= a.num_pages || d >= a.num_pages;
    mine = s >= 0 && d >= 0 && !bad && s != d;
    left_out[tid] = !mine;
  }
  __syncthreads();
  if (mine)
    for (int h = first_slot(dst[tid]);; h = (h + 1) % kSlots) {      // (at most a quarter of the slots are taken)
      const int there = atomicCAS(&slot[h], 0, tid + 1);
      if (there == 0) break;
      if (dst[there - 1] == dst[tid]) {
        left_out[there - 1] = left_out[tid] = 2;
        break;
      }
    }
  __syncthreads();
  auto find = [&](int page) {       // the pair here that has this destination, or −1
    for (int h = first_slot(page);; h = (h + 1) % kSlots) {
      const int k = slot[h] - 1;
      if (k < 0 || dst[k] == page) return k;
    }
  };
#pragma unroll 4
  for (int j = tid; j < a.n; j += kManyThreads) {
    const int s = a.src[j], d = a.dst[j];
    if (s < 0 || d < 0 || s == d) continue;
    const int ks = find(s), kd = find(d);
    if (ks >= 0) left_out[ks] = 2;
    if (kd >= 0 && i0 + kd != j) left_out[kd] = 2;
  }
  __syncthreads();
  bad = bad || (mine && left_out[tid] == 2);
  if (bad) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
  uint32_t before[kArrays + 1] = {};        // vectors before each array's
#pragma unroll
  for (int k = 0; k < kArrays; ++k) before[k + 1] = before[k] + (k < a.arrays ? a.vecs[k] : 0u);
  const uint32_t total = before[kArrays], pieces = (total + kWarpPiece - 1) / kWarpPiece;
  uint32_t piece = tid >> 5;
  for (int i = 0;; piece += kManyThreads / 32) {
    while (piece >= pieces) {
      piece -= pieces;
      ++i;
    }
    if (i >= pairs) break;
    if (left_out[i]) continue;
    const long long from = src[i], to = dst[i];
    uint4 v[kFlight];
    uint4* at[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const uint32_t e = piece * kWarpPiece + f * 32 + (tid & 31);
      at[f] = nullptr;
      if (e >= total) continue;
      int k = 0;
      uint32_t x = e;
#pragma unroll
      for (int m = 1; m < kArrays; ++m)
        if (e >= before[m] && m < a.arrays) {
          k = m;
          x = e - before[m];
        }
      at[f] = a.base[k] + to * a.vecs[k] + x;
      v[f] = a.base[k][from * a.vecs[k] + x];
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (at[f]) *at[f] = v[f];
  }
}

// ---------------------------------------------------------------- tokens
// A CTA moves the tokens of one (sequence, head): all are read before any is written, so a list may
// be in any order.  An item is 16 bytes of a token's codes or one of its norms; a block has as many
// threads as items up to kKeepThreads (short lists with 256 threads a block: 10.2 us for 6.4, 512
// sequences of 8 heads and 16 entries).
constexpr int kKeepThreads = 256, kMaxItems = 12;         // 4 + 1 + 4 vectors, 3 norms
constexpr int kPerThread = TQ_TREE_NODES * kMaxItems / kKeepThreads;

struct KeepArgs {
  uint8_t* kidx;
  uint8_t* ksgn;
  float* kxn;
  float* krn;
  uint8_t* vidx;
  float* vxn;
  tq_rowmap kmap, vmap;
  int kslots, vslots;
  int kplanes, vparts, nibbles;      // key index planes, 16-byte parts of a value
  int heads, capacity, max_keep;
  const int* pos;
  const int* keep;
};

// Address of item j of the token in slot ks of row kr (values: vs of vr).
__device__ __forceinline__ char* item_at(const KeepArgs& a, int j, long long kr, int ks, long long vr, int vs) {
  if (j < a.kplanes) return reinterpret_cast<char*>(a.kidx) + ((kr * a.kplanes + j) * a.kslots + ks) * 16;
  if (j == a.kplanes) return reinterpret_cast<char*>(a.ksgn) + (kr * a.kslots + ks) * 16;
  j -= a.kplanes + 1;
  if (j < a.vparts)
    return reinterpret_cast<char*>(a.vidx) + (a.nibbles ? (vr * a.vslots + vs) * 64 + j * 16
                                                        : ((vr * a.vparts + j) * a.vslots + vs) * 16);
  j -= a.vparts;
  return reinterpret_cast<char*>(j == 0 ? a.kxn + kr * a.kslots + ks
                                 : j == 1 ? a.krn + kr * a.kslots + ks : a.vxn + vr * a.vslots + vs);
}

// Bound by latency: list, block table, codes, one after the other, and the launch (32 sequences of 4
// heads and 5 entries: 3.0 us; 512 of 8 heads and 16: 6.4 us).
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const __grid_constant__ KeepArgs a) {
  const int h = blockIdx.x % a.heads, b = blockIdx.x / a.heads;
  const int per = a.kplanes + 1 + a.vparts + 3, wide = per - 3;
  const long long pos = a.pos[b];
  const int* keep = a.keep + (long long)b * a.max_keep;
  uint4 v[kPerThread];
  char* to[kPerThread];
#pragma unroll
  for (int n = 0; n < kPerThread; ++n) {
    const int x = threadIdx.x + n * blockDim.x, i = x / per, j = x % per;
    to[n] = nullptr;
    const int from = i < a.max_keep ? keep[i] : -1;
    if (from < 0) continue;
    if (pos < 0 || pos + i >= a.capacity || pos + from >= a.capacity) {
      if (h == 0 && j == 0) atomicOr(&g_tq_flags, TQ_FLAG_POS_OVERFLOW);
      continue;
    }
    if (from == i) continue;
    long long kr[2], vr[2];
    int ks[2], vs[2];
    bool ok = true;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = (int)pos + (e ? i : from);
      ok &= tq_map_slot(a.kmap, a.heads, b, h, t, kr[e], ks[e]);
      ok &= tq_map_slot(a.vmap, a.heads, b, h, t, vr[e], vs[e]);
    }
    if (!ok) {
      if (h == 0 && j == 0) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
      continue;
    }
    const char* src = item_at(a, j, kr[0], ks[0], vr[0], vs[0]);
    to[n] = item_at(a, j, kr[1], ks[1], vr[1], vs[1]);
    if (j < wide) v[n] = *reinterpret_cast<const uint4*>(src);
    else v[n].x = *reinterpret_cast<const uint32_t*>(src);
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kPerThread; ++n) {
    const int j = (threadIdx.x + n * blockDim.x) % per;
    if (!to[n]) continue;
    if (j < wide) *reinterpret_cast<uint4*>(to[n]) = v[n];
    else *reinterpret_cast<uint32_t*>(to[n]) = v[n].x;
  }
}

}  // namespace

extern "C" tq_status tq_copy_pages(const tq_prod_cache* k, int32_t key_bits, const tq_mse_cache* v,
                                   int32_t value_bits, const tq_block_cache* blocks, int32_t heads,
                                   int32_t num_pages, int32_t page_tokens, const int32_t* src,
                                   const int32_t* dst, int32_t n, tq_stream_t stream_) {
  if (heads <= 0 || num_pages <= 0 || n < 0) return TQ_ERR_INVALID_ARG;
  if (page_tokens <= 0 || page_tokens % TQ_CAPACITY_ALIGN) return TQ_ERR_INVALID_ARG;
  if (k && (key_bits < 2 || key_bits > 5)) return TQ_ERR_UNSUPPORTED;
  if (v && (value_bits < 1 || value_bits > 4)) return TQ_ERR_UNSUPPORTED;
  if (n > TQ_MAX_PAIRS || (long long)heads * page_tokens > (1 << 26)) return TQ_ERR_UNSUPPORTED;
  CopyArgs a{};
  bool bad = n && (!src || !dst);
  bad = bad || reinterpret_cast<uintptr_t>(src) % 4 || reinterpret_cast<uintptr_t>(dst) % 4;
  auto add = [&](void* p, long long bytes_per_token) {
    bad = bad || !p || !aligned16(p);
    a.base[a.arrays] = static_cast<uint4*>(p);
    a.vecs[a.arrays] = (uint32_t)((long long)heads * page_tokens * bytes_per_token / 16);
    a.pieces[a.arrays + 1] = a.pieces[a.arrays] + (int)((a.vecs[a.arrays] + kPiece - 1) / kPiece);
    ++a.arrays;
  };
  if (k) {
    add(k->idx, (key_bits - 1) * 16);
    add(k->sgn, 16);
    add(k->xnorm, 4);
    add(k->rnorm, 4);
  }
  if (v) {
    add(v->idx, value_bits * 16);
    add(v->xnorm, 4);
  }
  if (blocks) add(blocks->bounds, 2 * TQ_D * 2 / TQ_BLOCK_TOKENS);
  if (bad || !a.arrays) return TQ_ERR_INVALID_ARG;
  if (n == 0) return TQ_OK;
  a.n = n;
  a.num_pages = num_pages;
  a.src = src;
  a.dst = dst;
  // Which kernel: a CTA of the first reads a list of 8n bytes for a page, which the copy hides (4096 pages of 47
  // KB 66 us and 74, 16384 of 188 KB 918 and 994) until the list is twice as long as the page (16384 pages of 47
  // KB 261 us and 269, 32768 of 94 KB 1117 and 996, 4096 of 12 KB 35 and 19, 65536 of 6 KB 2359 and 222).
  long long page = 0;
  for (int i = 0; i < a.arrays; ++i) page += a.vecs[i] * 16LL;
  if (4LL * n > page) {
    const int most = std::max(2 * tq_num_sms(), (n + kManyPairs - 1) / kManyPairs), per_cta = (n + most - 1) / most;
    copy_many_pages_kernel<<<(unsigned)((n + per_cta - 1) / per_cta), kManyThreads, 0, reinterpret_cast<cudaStream_t>(stream_)>>>(
        a, per_cta);
    return tq_cuda_status(cudaGetLastError());
  }
  // CTAs that share a page: as many as give each SM about eight, up to one for each piece
  const int want = std::max(tq_num_sms(), 1) * 8;
  a.ways = std::min(a.pieces[a.arrays], std::max(1, (want + n - 1) / n));
  const long long grid = (long long)n * a.ways;
  copy_pages_kernel<<<(unsigned)grid, kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream_)>>>(a);
  return tq_cuda_status(cudaGetLastError());
}

extern "C" tq_status tq_keep_tokens(tq_prod_cache k, int32_t key_bits, tq_mse_cache v,
                                    int32_t value_bits, int32_t batch, int32_t heads,
                                    int32_t capacity, const int32_t* pos, const int32_t* keep,
                                    int32_t max_keep, tq_stream_t stream_) {
  if (batch < 0 || heads <= 0 || max_keep < 0) return TQ_ERR_INVALID_ARG;
  if (capacity <= 0 || capacity % TQ_CAPACITY_ALIGN) return TQ_ERR_INVALID_ARG;
  if (key_bits < 2 || key_bits > 5 || value_bits < 1 || value_bits > 4) return TQ_ERR_UNSUPPORTED;
  if (max_keep > TQ_TREE_NODES || (long long)batch * heads > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  if (!k.idx || !k.sgn || !k.xnorm || !k.rnorm || !v.idx || !v.xnorm) return TQ_ERR_INVALID_ARG;
  if (batch && max_keep && (!pos || !keep)) return TQ_ERR_INVALID_ARG;
  if (!aligned16(k.idx) || !aligned16(k.sgn) || !aligned16(k.xnorm) || !aligned16(k.rnorm) ||
      !aligned16(v.idx) || !aligned16(v.xnorm))
    return TQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(keep) % 4) return TQ_ERR_INVALID_ARG;
  KeepArgs a{};
  tq_status st = tq_rowmap_of(k.pages, capacity, &a.kmap);
  if (st == TQ_OK) st = tq_rowmap_of(v.pages, capacity, &a.vmap);
  if (st != TQ_OK) return st;
  if (batch == 0 || max_keep == 0) return TQ_OK;
  a.kidx = k.idx; a.ksgn = k.sgn; a.kxn = k.xnorm; a.krn = k.rnorm;
  a.vidx = v.idx; a.vxn = v.xnorm;
  a.kslots = tq_row_slots(a.kmap, capacity);
  a.vslots = tq_row_slots(a.vmap, capacity);
  a.kplanes = key_bits - 1;
  a.vparts = value_bits;
  a.nibbles = value_bits == 4;
  a.heads = heads;
  a.capacity = capacity;
  a.max_keep = max_keep;
  a.pos = pos;
  a.keep = keep;
  const int items = max_keep * (a.kplanes + 1 + a.vparts + 3);
  const int threads = std::min(kKeepThreads, (items + 31) / 32 * 32);      // (more items: three a thread at most)
  keep_tokens_kernel<<<(unsigned)(batch * heads), threads, 0,
                       reinterpret_cast<cudaStream_t>(stream_)>>>(a);
  return tq_cuda_status(cudaGetLastError());
}
