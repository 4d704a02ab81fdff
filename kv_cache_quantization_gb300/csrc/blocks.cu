// Which parts of a long cache a decode query should read: bounds of the keys of each 64-token
// block, kept beside the cache as the keys are written (tq_block_bounds), and the selection of
// blocks by an upper bound of the query's products with their keys (tq_block_select).
//
// Mathematics.  With lo_j ≤ k_j ≤ hi_j for every key k of a block,
//   ⟨q, k⟩ = Σ_j q_j k_j ≤ Σ_j max(q_j lo_j, q_j hi_j) = ⟨min(q, 0), lo⟩ + ⟨max(q, 0), hi⟩,
// one product of length 256 with the block's bounds.  The bounds are bf16, rounded outward, so
// the inequality survives the rounding; minima and maxima do not depend on an order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "tc_ptx.h"
#include "tq_internal.h"

TQ_DEFINE_FLAGS(tq_take_flags_blocks)

namespace {

constexpr int kBlock = TQ_BLOCK_TOKENS;
constexpr int kRow = 2 * TQ_D;          // bf16 values per block: 128 lower, 128 upper bounds

// ---------------------------------------------------------------- bounds
struct BoundsArgs {
  const void* x;
  int batch, heads, tokens;
  long long sb, sh, st;
  const int* pos;
  const int* count;
  __nv_bfloat16* bounds;
  tq_rowmap map;
  int capacity;
  int nt;                  // blocks that a chunk of `tokens` tokens can touch
  long long units;         // batch · heads · nt
};

// bf16 bits of the nearest number not above (up = false) or not below (up = true) x
__device__ __forceinline__ uint32_t outward(float x, bool up) {
  const uint32_t u = __float_as_uint(x);
  const bool away = (u & 0xffffu) && (up ? !(u >> 31) : (u >> 31));
  return (u + (away ? 0x10000u : 0u)) >> 16;
}

// Lane's view of the rows of one block: 16 bytes of a row per load (8 values of 16 bits and two
// rows a warp, or 4 values of 32 bits and one row).
template <typename T>
struct Rows {
  static constexpr int kPer = 16 / sizeof(T);        // values per lane
  static constexpr int kLanes = TQ_D / kPer;         // lanes per row
  static constexpr int kStep = 32 / kLanes;          // rows per load
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// One warp per (sequence, head, block): it reads the chunk's rows that fall in the block, 8
// loads of 512 bytes in flight, and owns the block's bounds, so there is nothing atomic.
// Bound by reading the keys: 8 × 262144 bf16 keys take 89.7 us, 6.2 TB/s (98.8 us with 16 loads
// in flight and 95.3 us with 32: their registers cost more warps than they feed).  kVec: rows are
// 16-byte aligned.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsArgs a) {
  using R = Rows<T>;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= a.units) return;
  const int i = (int)(unit % a.nt);
  const int h = (int)(unit / a.nt % a.heads), b = (int)(unit / a.nt / a.heads);
  const long long pos = a.pos ? a.pos[b] : 0;
  long long n = a.count ? min(max(a.count[b], 0), a.tokens) : a.tokens;
  if (n > 0 && (pos < 0 || pos + n > a.capacity)) {
    if (i == 0 && h == 0 && lane == 0) atomicOr(&g_tq_flags, TQ_FLAG_POS_OVERFLOW);
    if (pos < 0) return;
    n = min(n, (long long)a.capacity - pos);
  }
  const long long blk = pos / kBlock + i;
  const long long first = max(blk * kBlock - pos, 0LL);               // the chunk's tokens in
  const long long last = min((blk + 1) * kBlock - pos, n);            // this block
  if (first >= last) return;
  long long row;
  int slot;
  if (!tq_map_slot(a.map, a.heads, b, h, (int)(blk * kBlock), row, slot)) {
    if (lane == 0) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
    return;
  }
  const T* x = static_cast<const T*>(a.x) + b * a.sb + h * a.sh + (lane % R::kLanes) * R::kPer;
  float lo[R::kPer], hi[R::kPer];
#pragma unroll
  for (int j = 0; j < R::kPer; ++j) {
    lo[j] = INFINITY;
    hi[j] = -INFINITY;
  }
  constexpr int kFlight = 8;
  for (long long t0 = first; t0 < last; t0 += kFlight * R::kStep) {
    alignas(16) T v[kFlight][R::kPer];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      // rows past the end repeat the last one
      const long long t = min(t0 + k * R::kStep + lane / R::kLanes, last - 1);
      if (kVec) {
        *reinterpret_cast<uint4*>(v[k]) = __ldg(reinterpret_cast<const uint4*>(x + t * a.st));
      } else {
#pragma unroll
        for (int j = 0; j < R::kPer; ++j) v[k][j] = x[t * a.st + j];
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int j = 0; j < R::kPer; ++j) {
        const float f = to_float(v[k][j]);
        lo[j] = fminf(lo[j], f);
        hi[j] = fmaxf(hi[j], f);
      }
  }
#pragma unroll
  for (int j = 0; j < R::kPer; ++j)
#pragma unroll
    for (int o = R::kLanes; o < 32; o *= 2) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
    }
  const int slots = tq_row_slots(a.map, a.capacity);
  uint16_t* dst = reinterpret_cast<uint16_t*>(a.bounds) +
                  (row * (slots / kBlock) + slot / kBlock) * kRow + (lane % R::kLanes) * R::kPer;
  // a block that this chunk does not begin goes on: fold its bounds in
  const bool goes_on = blk * kBlock < pos;
  if (lane < R::kLanes) {
#pragma unroll
    for (int j = 0; j < R::kPer; j += 2) {
      uint32_t l[2], u[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] = outward(lo[j + e], false);
        u[e] = outward(hi[j + e], true);
        if (goes_on) {
          l[e] = __float_as_uint(fminf(__uint_as_float(l[e] << 16),
                                       __uint_as_float((uint32_t)dst[j + e] << 16))) >> 16;
          u[e] = __float_as_uint(fmaxf(__uint_as_float(u[e] << 16),
                                       __uint_as_float((uint32_t)dst[TQ_D + j + e] << 16))) >> 16;
        }
      }
      *reinterpret_cast<uint32_t*>(dst + j) = l[0] | l[1] << 16;
      *reinterpret_cast<uint32_t*>(dst + TQ_D + j) = u[0] | u[1] << 16;
    }
  }
}

// ---------------------------------------------------------------- selection
struct SelectArgs {
  const void* q;
  int q_dtype;
  const __nv_bfloat16* bounds;
  tq_rowmap map;
  int capacity, max_len;
  const int* seq_lens;
  int Hkv, G;
  int nb;                 // blocks of max_len tokens (row stride of the workspace arrays)
  int rounds, chunks;     // rounds of kRound blocks per CTA of the scoring kernel, CTAs per row
  int first, last, keep;
  float* score;           // [B·Hkv][nb]
  float* err;             // [B·Hkv][chunks] bounds of Σ|terms| of a chunk's blocks
  unsigned long long* exact;   // [B·Hkv][nb] ordered 64-bit scores of the blocks in doubt
  int* doubt;             // [B·Hkv][nb] their numbers
  int* list;              // [B·Hkv][keep]
};

constexpr int kPerWarp = 4;      // blocks per warp and round of the scoring kernel
constexpr int kRound = 8 * kPerWarp;

__device__ __forceinline__ float load_elem(const void* base, int dtype, long long i) {
  if (dtype == TQ_F32) return static_cast<const float*>(base)[i];
  const uint16_t u = static_cast<const uint16_t*>(base)[i];
  if (dtype == TQ_BF16) return __uint_as_float((uint32_t)u << 16);
  return __half2float(__ushort_as_half(u));
}

// Pointer to the 256 bounds of block blk; null where its page is bad.
__device__ __forceinline__ const __nv_bfloat16* bounds_at(const SelectArgs& a, int b, int h, int blk) {
  long long row;
  int slot;
  if (!tq_map_slot(a.map, a.Hkv, b, h, blk * kBlock, row, slot)) return nullptr;
  return a.bounds + (row * (tq_row_slots(a.map, a.capacity) / kBlock) + slot / kBlock) * kRow;
}

__device__ __forceinline__ int blocks_of(const SelectArgs& a, int b) {
  return (min(max(a.seq_lens[b], 0), a.max_len) + kBlock - 1) / kBlock;
}

// The larger of two numbers ≥ 0, NaN if either is one.
__device__ __forceinline__ float larger_or_nan(float a, float b) { return a != a || b <= a ? a : b; }

// Sums over the 32 lanes of each of N values a lane: N/2 + N/4 + ... shuffles instead of 5·N.
// Lane l ends with the sum of value l / (32 / N) (N ≤ 32, a power of two) in v[0].
template <int N, typename T>
__device__ __forceinline__ void lane_sums(T (&v)[N], int lane) {
#pragma unroll
  for (int o = 16, n = N; o; o >>= 1) {
    if (n > 1) {
      // the upper lanes take the upper half of the values
      n /= 2;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const T mine = lane & o ? v[i + n] : v[i], other = lane & o ? v[i] : v[i + n];
          v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

// Scores in 32 bits of the blocks of one (sequence, KV head): the largest over the group's
// query heads.  A warp takes four blocks with one 512-byte load each (the next four in flight),
// lanes 0–15 the lower and lanes 16–31 the upper bounds, against the negative and the positive
// parts of the query rows in shared memory, four heads at a time (16 sums share their
// shuffles).  The loop over heads is kept rolled: most calls are short, and then fetching the
// instructions costs more than issuing them (unrolled over eight heads this kernel took 8.5 us
// for 4 × 512 blocks).  Bound by the latency of two dependent loads for short rows, by issuing
// about 12 instructions per block and head for long ones.
//
// Beside the scores goes a bound of Σ|terms|, from which the selection takes how far a score may
// be off.  An infinite bound of a channel times the 0 of queries of the other sign is NaN here, in
// the score (which is then too low) and in the bound of Σ|terms|, which stays NaN: the selection
// then trusts no 32-bit score of the row.  The 64-bit scores use one bound a channel, by the sign.
__global__ void __launch_bounds__(256) block_score_kernel(const SelectArgs a) {
  __shared__ float4 s_q[TQ_MAX_GROUP + 1][2][32];   // [head][first or second four][lane]; last: max |.|
  __shared__ float s_err[8];
  const int row = blockIdx.y, b = row / a.Hkv, h = row % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int len = a.seq_lens[b];
  const int heads = (a.G + 3) / 4 * 4;          // absent heads repeat head 0: the maximum is the same
  for (int i = threadIdx.x; i < heads * TQ_D; i += 256) {
    const int g = i / TQ_D, c = i % TQ_D;
    const float v = load_elem(a.q, a.q_dtype, ((long long)row * a.G + (g < a.G ? g : 0)) * TQ_D + c);
    float* at = reinterpret_cast<float*>(&s_q[g][(c >> 2) & 1][c >> 3]) + (c & 3);
    at[0] = v > 0.f ? 0.f : v;         // lanes 0–15 (NaN goes to both)
    at[16 * 4] = v < 0.f ? 0.f : v;    // lanes 16–31
  }
  if (len > a.max_len && blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    atomicOr(&g_tq_flags, TQ_FLAG_LEN_OVERFLOW);
  const int nblk = (min(max(len, 0), a.max_len) + kBlock - 1) / kBlock;
  const int first = blockIdx.x * a.rounds * kRound, end = min(first + a.rounds * kRound, nblk);
  if (nblk <= a.keep || first >= end) return;   // nothing to choose, or nothing here
  auto fetch = [&](int begin, uint4 (&x)[kPerWarp], uint32_t& in) {
    // (plain loads, the kernel before may have written tables and bounds; all of one kind first, so
    // that they are in flight together)
    const __nv_bfloat16* p[kPerWarp];
    in = 0;
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
      p[i] = begin + i < end ? bounds_at(a, b, h, begin + i) : nullptr;
      if (p[i]) in |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i)
      x[i] = p[i] ? reinterpret_cast<const uint4*>(p[i])[lane] : make_uint4(0, 0, 0, 0);
    if (lane == 0 && __popc(in) < min(end - begin, kPerWarp)) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
  };
  uint4 next[kPerWarp];
  uint32_t next_in;
  int begin = first + warp * kPerWarp;
  fetch(begin, next, next_in);
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * TQ_D; i += 256) {
    float m = 0.f;
    for (int g = 0; g < a.G; ++g) m = fmaxf(m, fabsf(reinterpret_cast<const float*>(s_q[g])[i]));
    reinterpret_cast<float*>(s_q[TQ_MAX_GROUP])[i] = m;
  }
  __syncthreads();
  float err = 0.f;
  for (; begin < end; begin += kRound) {
    tq::f32x2 v[kPerWarp][4];
    const uint32_t in = next_in;
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
      const uint32_t w[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[i][j] = tq::pack2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
    if (begin + kRound < end) fetch(begin + kRound, next, next_in);
    {
      const float4 m0 = s_q[TQ_MAX_GROUP][0][lane], m1 = s_q[TQ_MAX_GROUP][1][lane];
      const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
      for (int i = 0; i < kPerWarp; ++i) {
        float e = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = tq::unpack2(v[i][j]);
          e = fmaf(m[2 * j], fabsf(x.x), e);
          e = fmaf(m[2 * j + 1], fabsf(x.y), e);
        }
        err = larger_or_nan(err, e);
      }
    }
    float best = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < heads; g += 4) {
      float t[4 * kPerWarp];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(&s_q[g + k][0][lane]);
        const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(&s_q[g + k][1][lane]);
#pragma unroll
        for (int i = 0; i < kPerWarp; ++i) {
          tq::f32x2 s = tq::mul2(q0.x, v[i][0]);
          s = tq::fma2(q0.y, v[i][1], s);
          s = tq::fma2(q1.x, v[i][2], s);
          s = tq::fma2(q1.y, v[i][3], s);
          const float2 p = tq::unpack2(s);
          t[4 * i + k] = p.x + p.y;
        }
      }
      lane_sums(t, lane);           // lane l: block l / 8, head g + l / 2 % 4
      best = fmaxf(best, t[0]);     // (a NaN head is left out)
    }
    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 4));
    const int i = lane / (32 / kPerWarp);
    if (lane % (32 / kPerWarp) == 0 && begin + i < end)
      a.score[(long long)row * a.nb + begin + i] = (in >> i) & 1u ? best : -INFINITY;
  }
  // Σ over lanes of each lane's largest partial sum: at least every block's Σ|terms|
#pragma unroll
  for (int o = 16; o; o >>= 1) err += __shfl_xor_sync(0xffffffffu, err, o);
  if (lane == 0) s_err[warp] = err;
  __syncthreads();
  if (threadIdx.x == 0) {
    float e = 0.f;
    for (int i = 0; i < 8; ++i) e = larger_or_nan(e, s_err[i]);
    a.err[(long long)row * a.chunks + blockIdx.x] = e;
  }
}

// Integers in the order of the numbers (no NaN reaches them: a maximum leaves it out).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);              // −0 as +0
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = __double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

constexpr int kSelThreads = 1024;

// Sums over the CTA, one barrier each: consecutive sums use the two halves of the scratch in
// turn, so that a thread may write the next one while others read this one.
struct CtaSum {
  int (*scratch)[32];
  int turn;
  __device__ __forceinline__ int operator()(int v) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) scratch[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    const int w = threadIdx.x & 31;
    v = __reduce_add_sync(0xffffffffu, w < (int)(blockDim.x >> 5) ? scratch[turn][w] : 0);
    turn ^= 1;
    return v;
  }
};

// The largest t ≥ start with at least `want` of the keys ≥ t (start has at least that many):
// bit by bit from `bit` down, one count per bit, stopping at a count that is `want` exactly.
// Bits above are those of start.
template <typename K, typename Count>
__device__ __forceinline__ K kth_key(K start, int bit, int want, CtaSum& sum, Count count) {
  K t = start;
  for (; bit >= 0; --bit) {
    const K c = t | ((K)1 << bit);
    const int got = sum(count(c));
    if (got >= want) t = c;
    if (got == want) break;
  }
  return t;
}

// One CTA per (sequence, KV head).  The 32-bit scores are off by at most E each; with v the
// smallest score among the `want` largest, blocks above v + 2E are kept and blocks below v − 2E
// are not, whatever the rounding.  Those between are scored again in 64 bits (the products are
// exact there, the sums have one fixed order) and ranked, ties to the lowest number: the selection
// does not depend on how 32-bit sums round.  The ordered scores stay in registers, kItems a thread
// (kItems = 0: read again from the workspace, for rows of more than 16 · 1024 candidates).  Bound
// by the latency of the counts, one per bit until the kept ones are told apart.
template <int kItems>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const SelectArgs a) {
  extern __shared__ uint32_t s_dyn[];     // keep bits
  __shared__ int s_red[2][32];
  __shared__ uint32_t s_low[32], s_high[32], s_err[32], s_kth[32];
  const int row = blockIdx.x, b = row / a.Hkv, h = row % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int nblk = blocks_of(a, b);
  int* list = a.list + (long long)row * a.keep;
  if (nblk <= a.keep) {
    for (int i = tid; i < a.keep; i += blockDim.x) list[i] = i < nblk ? i : -1;
    return;
  }
  CtaSum sum{s_red, 0};
  const int words = (nblk + 31) / 32;
  uint32_t* bits = s_dyn;
  const int lo = a.first, n = nblk - a.first - a.last;      // candidates lo .. lo + n − 1
  const float* score = a.score + (long long)row * a.nb + lo;
  const int want = a.keep - a.first - a.last;               // < n
  // visits (candidate, ordered score) of this thread
  uint32_t keys[kItems > 0 ? kItems : 1];
  if (kItems > 0) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = tid + k * (int)blockDim.x;
      keys[k] = i < n ? ordered(score[i]) : 0u;     // (0 is below every number's)
    }
  }
  auto each = [&](auto&& f) {
    if (kItems > 0) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = tid + k * (int)blockDim.x;
        if (i < n) f(i, keys[k]);
      }
    } else {
      for (int i = tid; i < n; i += blockDim.x) f(i, ordered(score[i]));
    }
  };
  for (int i = tid; i < words; i += blockDim.x) {
    // the forced blocks of this word: below first, and from tail on
    const int f = a.first - 32 * i, tail = nblk - a.last - 32 * i, past = nblk - 32 * i;
    auto below = [](int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u; };
    bits[i] = below(f) | (below(past) & ~below(tail));
  }
  uint32_t low = ~0u, high = 0u, worst = 0u;
  each([&](int, uint32_t k) {
    low = min(low, k);
    high = max(high, k);
  });
  for (int i = tid; i < (nblk + a.rounds * kRound - 1) / (a.rounds * kRound); i += blockDim.x) {
    const float e = a.err[(long long)row * a.chunks + i];
    worst = max(worst, e != e ? ~0u : __float_as_uint(e));     // NaN above all
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  worst = __reduce_max_sync(0xffffffffu, worst);
  if (lane == 0) {
    s_low[warp] = low;
    s_high[warp] = high;
    s_err[warp] = worst;
  }
  __syncthreads();
  low = __reduce_min_sync(0xffffffffu, lane < nwarps ? s_low[lane] : ~0u);
  high = __reduce_max_sync(0xffffffffu, lane < nwarps ? s_high[lane] : 0u);
  worst = __reduce_max_sync(0xffffffffu, lane < nwarps ? s_err[lane] : 0u);
  // four multiply-adds and six additions on a term's way into the sum, half a step of 32 bits
  // each, and the product's own: 11·2^-24·Σ|terms|; 2^-20 leaves room for the rounding of the
  // bound itself.  Where products are subnormal or vanish, 256 of them are off by at most 2^-150
  // each, in the score and in the bound: 2^-140 covers both
  const float E = worst == ~0u ? INFINITY : fmaf(__uint_as_float(worst), 0x1p-20f, 0x1p-140f);
  if (want > 0) {
    // all keys agree above the highest bit in which low and high differ
    const int top = low == high ? -1 : 31 - __clz((int)(low ^ high));
    const uint32_t start = top < 0 ? low : high & ~((2u << top) - 1u);
    const uint32_t t = kth_key<uint32_t>(start, top, want, sum, [&](uint32_t c) {
      int mine = 0;
      each([&](int, uint32_t k) { mine += k >= c; });
      return mine;
    });
    // v: the smallest key ≥ t
    uint32_t v = ~0u;
    each([&](int, uint32_t k) {
      if (k >= t) v = min(v, k);
    });
    v = __reduce_min_sync(0xffffffffu, v);
    if (lane == 0) s_kth[warp] = v;
    __syncthreads();
    v = __reduce_min_sync(0xffffffffu, lane < nwarps ? s_kth[lane] : ~0u);
    const float vf = unordered(v);
    const float up = vf + 2.f * E, down = vf - 2.f * E;
    // kept whatever the rounding; in doubt (with an infinite E every block is)
    int sure = 0, open = 0;
    each([&](int i, uint32_t k) {
      const float s = unordered(k);
      const bool in = s > up, out = s < down;
      sure += in;
      open += !in && !out;
      if (in) atomicOr(&bits[(lo + i) >> 5], 1u << ((lo + i) & 31));
    });
    sure = sum(sure);
    open = sum(open);
    const int need = want - sure;
    int* doubt = a.doubt + (long long)row * a.nb;
    unsigned long long* exact = a.exact + (long long)row * a.nb;
    if (open <= need) {
      each([&](int i, uint32_t k) {
        const float s = unordered(k);
        if (!(s > up) && !(s < down)) atomicOr(&bits[(lo + i) >> 5], 1u << ((lo + i) & 31));
      });
    } else {
      // the blocks in doubt, in ascending order
      int base = 0;
      for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + tid;
        const float s = i < n ? score[i] : 0.f;
        const bool d = i < n && !(s > up) && !(s < down);
        const uint32_t vote = __ballot_sync(0xffffffffu, d);
        __syncthreads();
        if (lane == 0) s_red[0][warp] = __popc(vote);
        __syncthreads();
        const int c = lane < nwarps ? s_red[0][lane] : 0;
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
        if (d) doubt[base + before + __popc(vote & ((1u << lane) - 1))] = lo + i;
        base += __reduce_add_sync(0xffffffffu, c);
      }
      __syncthreads();
      // a row of zero queries has nothing to score: every term is 0 (Σ|terms| alone may be 0
      // because its products vanish in 32 bits)
      int some = worst != 0u;
      if (worst == 0u) {
        for (int i = tid; i < a.G * TQ_D; i += blockDim.x)
          some |= !(load_elem(a.q, a.q_dtype, (long long)row * a.G * TQ_D + i) == 0.f);
        some = __syncthreads_or(some);
      }
      for (int i = tid; !some && i < open; i += blockDim.x) exact[i] = ordered(0.0);
      for (int i = warp; some && i < open; i += nwarps) {
        // lane l: channels 4l .. 4l + 3 of every head, all loads first
        const __nv_bfloat16* p = bounds_at(a, b, h, doubt[i]);
        double best = -INFINITY;
        if (p) {
          double l[4], u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            l[j] = __bfloat162float(p[4 * lane + j]);
            u[j] = __bfloat162float(p[TQ_D + 4 * lane + j]);
          }
#pragma unroll 1
          for (int g0 = 0; g0 < a.G; g0 += 4) {     // four heads at a time (absent: head 0 again)
            double s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const long long at = ((long long)row * a.G + (g0 + k < a.G ? g0 + k : 0)) * TQ_D + 4 * lane;
              s[k] = 0.0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x = load_elem(a.q, a.q_dtype, at + j);
                s[k] += (double)x * (x < 0.f ? l[j] : u[j]);
              }
            }
            lane_sums(s, lane);
            best = fmax(best, s[0]);      // a NaN head is left out
          }
          best = fmax(best, __shfl_xor_sync(0xffffffffu, best, 16));
          best = fmax(best, __shfl_xor_sync(0xffffffffu, best, 8));
        }
        if (lane == 0) exact[i] = ordered(best);
      }
      __syncthreads();
      if (open <= 32) {
        // few: each lane ranks its block against the others
        if (warp == 0) {
          const unsigned long long k = lane < open ? exact[lane] : 0ull;
          int ahead = 0;
          for (int i = 0; i < open; ++i) {
            const unsigned long long o = __shfl_sync(0xffffffffu, k, i);
            ahead += o > k || (o == k && i < lane);
          }
          if (lane < open && ahead < need) atomicOr(&bits[doubt[lane] >> 5], 1u << (doubt[lane] & 31));
        }
      } else {
      const unsigned long long t64 =
          kth_key<unsigned long long>(0ull, 63, need, sum, [&](unsigned long long c) {
            int mine = 0;
            for (int i = tid; i < open; i += blockDim.x) mine += exact[i] >= c;
            return mine;
          });
      int above = 0;
      for (int i = tid; i < open; i += blockDim.x) above += exact[i] > t64;
      above = sum(above);
      const int left = need - above;    // places for keys equal to t64, in ascending order
      int at = 0;
      for (int i0 = 0; i0 < open; i0 += blockDim.x) {
        const int i = i0 + tid;
        const unsigned long long k = i < open ? exact[i] : 0ull;
        const bool eq = i < open && k == t64;
        const uint32_t vote = __ballot_sync(0xffffffffu, eq);
        __syncthreads();
        if (lane == 0) s_red[0][warp] = __popc(vote);
        __syncthreads();
        const int c = lane < nwarps ? s_red[0][lane] : 0;
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
        const bool in = i < open && (k > t64 || (eq && at + before + __popc(vote & ((1u << lane) - 1)) < left));
        if (in) atomicOr(&bits[doubt[i] >> 5], 1u << (doubt[i] & 31));
        at += __reduce_add_sync(0xffffffffu, c);
      }
      }
    }
  }
  // the kept blocks in ascending order: words of 32 blocks, counted then written
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += blockDim.x) {
    __syncthreads();
    const int w = w0 + tid;
    uint32_t m = w < words ? bits[w] : 0u;
    const int c = __popc(m);
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_red[0][warp] = incl;
    __syncthreads();
    const int ws = lane < nwarps ? s_red[0][lane] : 0;
    int at = base + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0) + incl - c;
    base += __reduce_add_sync(0xffffffffu, ws);
    while (m) {
      list[at++] = 32 * w + __ffs((int)m) - 1;
      m &= m - 1;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
void launch_bounds_t(const BoundsArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  if (vec) block_bounds_kernel<T, true><<<grid, 256, 0, stream>>>(a);
  else block_bounds_kernel<T, false><<<grid, 256, 0, stream>>>(a);
}

cudaLaunchConfig_t config(dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return c;
}

tq_status launch_score(const SelectArgs& a, dim3 grid, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(grid, 256, 0, stream, attr);
  return tq_cuda_status(cudaLaunchKernelEx(&cfg, block_score_kernel, a));
}

tq_status launch_select(const SelectArgs& a, int rows, int nb, cudaStream_t stream) {
  // about four candidates a thread, 16 where that is not enough threads
  const int threads = std::min(kSelThreads, std::max(128, ((nb + 3) / 4 + 31) / 32 * 32));
  auto kern = nb <= 4 * threads ? block_select_kernel<4>
            : nb <= 16 * threads ? block_select_kernel<16> : block_select_kernel<0>;
  const size_t smem = (size_t)(nb + 31) / 32 * sizeof(uint32_t);
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3(rows), threads, smem, stream, attr);
  return tq_cuda_status(cudaLaunchKernelEx(&cfg, kern, a));
}

struct SelPlan {
  int G, nb, rounds, chunks;
  size_t err_off, exact_off, doubt_off, bytes;
};

tq_status select_plan(const tq_attn_desc* d, SelPlan* p) {
  if (!d) return TQ_ERR_INVALID_ARG;
  if (d->head_dim != TQ_HEAD_DIM) return TQ_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->q_heads <= 0 || d->kv_heads <= 0) return TQ_ERR_INVALID_ARG;
  if (d->q_heads % d->kv_heads) return TQ_ERR_INVALID_ARG;
  if (d->q_heads / d->kv_heads > TQ_MAX_GROUP) return TQ_ERR_UNSUPPORTED;
  if (d->capacity <= 0 || d->capacity % TQ_CAPACITY_ALIGN) return TQ_ERR_INVALID_ARG;
  if (d->max_seq_len < 0 || d->max_seq_len > d->capacity) return TQ_ERR_INVALID_ARG;
  if (d->q_dtype != TQ_F32 && d->q_dtype != TQ_F16 && d->q_dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  // rows of the scoring grid, and keep bits of a row in shared memory (1.5 M blocks)
  if ((long long)d->batch * d->kv_heads > 65535 || d->max_seq_len > (1 << 26)) return TQ_ERR_UNSUPPORTED;
  p->G = d->q_heads / d->kv_heads;
  p->nb = std::max((d->max_seq_len + kBlock - 1) / kBlock, 1);
  const size_t rows = (size_t)d->batch * d->kv_heads;
  // rounds per CTA: about three CTAs per SM; one round where there are fewer.  (Two per SM, what
  // fits at once, took 15.3 for 18.0 us on 8 × 4096 blocks and 19.3 for 16.1 us on 128 ragged rows
  // of 64 to 256, where smaller CTAs even the rows out: calls in a row, in one run; runs of one
  // version differ by up to 2 us, 17.8 to 20.1 and 14.9 to 18.5 us.)
  const long long all = (long long)rows * ((p->nb + kRound - 1) / kRound);
  const long long fit = 3LL * std::max(tq_num_sms(), 1);
  p->rounds = (int)std::max<long long>(1, (all + fit - 1) / fit);
  p->chunks = (p->nb + p->rounds * kRound - 1) / (p->rounds * kRound);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p->err_off = up(rows * p->nb * sizeof(float));
  p->exact_off = p->err_off + up(rows * p->chunks * sizeof(float));
  p->doubt_off = p->exact_off + up(rows * p->nb * sizeof(unsigned long long));
  p->bytes = p->doubt_off + up(rows * p->nb * sizeof(int)) + 256;
  return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_block_bounds(const void* x, tq_dtype x_dtype, int32_t batch, int32_t heads,
                                     int32_t tokens, int64_t stride_b, int64_t stride_h,
                                     int64_t stride_t, const int32_t* pos, const int32_t* count,
                                     tq_block_cache blocks, int32_t capacity, tq_stream_t stream_) {
  if (batch < 0 || heads <= 0 || tokens < 0) return TQ_ERR_INVALID_ARG;
  if (stride_b < 0 || stride_h < 0 || stride_t < 0) return TQ_ERR_INVALID_ARG;
  if (capacity <= 0 || capacity % TQ_CAPACITY_ALIGN) return TQ_ERR_INVALID_ARG;
  if (x_dtype != TQ_F32 && x_dtype != TQ_F16 && x_dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  if (!x || !blocks.bounds || !aligned16(blocks.bounds)) return TQ_ERR_INVALID_ARG;
  const int elem = x_dtype == TQ_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % elem) return TQ_ERR_INVALID_ARG;
  BoundsArgs a{};
  tq_status st = tq_rowmap_of(blocks.pages, capacity, &a.map);
  if (st != TQ_OK) return st;
  if (batch == 0 || tokens == 0) return TQ_OK;
  a.x = x;
  a.batch = batch; a.heads = heads; a.tokens = tokens;
  a.sb = stride_b; a.sh = stride_h; a.st = stride_t;
  a.pos = pos; a.count = count;
  a.bounds = reinterpret_cast<__nv_bfloat16*>(blocks.bounds);
  a.capacity = capacity;
  a.nt = (int)(pos ? (tokens + (kBlock - 2LL)) / kBlock + 1 : (tokens + (kBlock - 1LL)) / kBlock);
  a.units = (long long)batch * heads * a.nt;
  if ((a.units + 7) / 8 > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  const bool vec = aligned16(x) && stride_b * elem % 16 == 0 && stride_h * elem % 16 == 0 &&
                   stride_t * elem % 16 == 0;
  const unsigned grid = (unsigned)((a.units + 7) / 8);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (x_dtype == TQ_F32) launch_bounds_t<float>(a, vec, grid, stream);
  else if (x_dtype == TQ_F16) launch_bounds_t<__half>(a, vec, grid, stream);
  else launch_bounds_t<__nv_bfloat16>(a, vec, grid, stream);
  return tq_cuda_status(cudaGetLastError());
}

extern "C" size_t tq_block_select_workspace_bytes(const tq_attn_desc* desc) {
  SelPlan p;
  return select_plan(desc, &p) == TQ_OK ? p.bytes : 0;
}

extern "C" tq_status tq_block_select(const tq_attn_desc* desc, const void* q, tq_block_cache blocks,
                                     const int32_t* seq_lens, int32_t first_blocks,
                                     int32_t last_blocks, int32_t max_blocks, int32_t* list,
                                     void* workspace, size_t workspace_bytes, tq_stream_t stream_) {
  SelPlan p;
  tq_status st = select_plan(desc, &p);
  if (st != TQ_OK) return st;
  if (first_blocks < 0 || last_blocks < 0 || max_blocks <= 0 || max_blocks > (1 << 24) ||
      (long long)first_blocks + last_blocks > max_blocks)
    return TQ_ERR_INVALID_ARG;
  if (!q || !blocks.bounds || !aligned16(blocks.bounds) || !seq_lens || !list || !workspace)
    return TQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < p.bytes)
    return TQ_ERR_INVALID_ARG;
  SelectArgs a{};
  if ((st = tq_rowmap_of(blocks.pages, desc->capacity, &a.map)) != TQ_OK) return st;
  if (desc->batch == 0) return TQ_OK;
  char* ws = static_cast<char*>(workspace);
  a.q = q; a.q_dtype = desc->q_dtype;
  a.bounds = reinterpret_cast<const __nv_bfloat16*>(blocks.bounds);
  a.capacity = desc->capacity; a.max_len = desc->max_seq_len;
  a.seq_lens = seq_lens;
  a.Hkv = desc->kv_heads; a.G = p.G;
  a.nb = p.nb; a.rounds = p.rounds; a.chunks = p.chunks;
  a.first = first_blocks; a.last = last_blocks; a.keep = max_blocks;
  a.score = reinterpret_cast<float*>(ws);
  a.err = reinterpret_cast<float*>(ws + p.err_off);
  a.exact = reinterpret_cast<unsigned long long*>(ws + p.exact_off);
  a.doubt = reinterpret_cast<int*>(ws + p.doubt_off);
  a.list = list;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int rows = desc->batch * desc->kv_heads;
  if ((st = launch_score(a, dim3(p.chunks, rows), stream)) != TQ_OK) return st;
  return launch_select(a, rows, p.nb, stream);
}
