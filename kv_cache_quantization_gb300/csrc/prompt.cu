// Attention of packed prompts over exact keys and values (tq_prompt_attention), before they are coded.
//
// Mathematics.  Query i of a sequence with nq queries and nk keys attends keys j < lim(i), nk or
// i + nk − nq + 1 where causal:  out_i = Σ_j w_j v_j / Σ_j w_j,  w_j = 2^(scale·log2(e)·q_i·k_j − ref),
// in one pass over the keys with a running reference ref per row.  The reference follows the running
// maximum only when that has grown by 2^8, so the accumulator is hardly ever scaled; weights are at
// most 2^8 in bf16, and at most 2^15 in fp16, whose reference lies 2^7 below the maximum so that a
// long tail of small weights stays above what fp16 holds (2^-32 of the largest).
//
// A CTA has two streams of 128 query rows × tiles of 128 keys (one stream with two score buffers and half
// the rows would read K and V twice as often: shared memory does not hold that rate).  The rows are `tokens` tokens × the
// query heads of one KV head (a group of 7: 18 tokens, 126 rows), so that a tile of keys is read
// once for the group and the causal border crosses few tiles.  With more rows than one stream holds,
// the streams are two blocks of rows over the same keys; otherwise they are the same rows over
// alternating tiles of keys, added up at the end.
//   1 loader thread   TMA tiles of K and V (32 KB each, 128-byte swizzle) into a ring of 5
//   2 issuer warps    S = Q·Kᵀ (128 × 128 × 128) and O += P·V (P in TMEM over the scores it came from)
//                     of a stream each, so that one's softmax runs beside the other one's products
//   8 softmax warps   a thread per row and stream: scores to weights, back to TMEM
//   1 guard warp      tiles of V that some row does not attend in full: rows past the sequence are
//                     zeroed, and infinite or NaN values past the first row's border are taken out
//                     (a weight of 0 would not hide them); rows that do attend those get them back
//                     at the end
// Where the rows are too few to fill the GPU the keys are split over CTAs, whose records (ref, Σw, O)
// prompt_merge_kernel joins.
//
// Measured: 32768 causal tokens of 28/4 bf16 heads 4.49 ms (1713 TFLOP/s, 90% of a large library
// product's rate; 4.95 ms, 1556 TFLOP/s, in runs of seconds under the power limit), 8192 × 8192 without
// a mask 583 us (1651); one token each of 32 sequences behind 8192
// keys of 8 heads 175 us (6.1 TB/s of keys and values); one token behind 128 keys 6.0 us.  What bounds long
// prompts is the chain of a tile (weights 500 cycles and more, their hand-over, 1024 of products, S back:
// about 2700 for both streams, where the products take 2048), then the shared memory that S = Q·Kᵀ reads:
// without any softmax the two issuers reach 2056 TFLOP/s.
//
// Roundings: P to the inputs' type (half a step of it relative to each weight, as V itself is held),
// the output once.  Scores, references, sums and accumulators are 32 bits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "tc_ptx.h"
#include "tq_internal.h"

TQ_DEFINE_FLAGS(tq_take_flags_prompt)

namespace {

using tq::mbar_arrive;
using tq::s32;
using tq::tc_after;
using tq::tc_before;

constexpr int kTile = 128;              // query rows of a stream, keys of a tile
constexpr int kStages = 5;
constexpr int kTileBytes = kTile * TQ_D * 2, kHalfBytes = kTileBytes / 2;   // halves: 64 channels
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kIssueWarp = 9, kGuardWarp = 11;      // (an issuer per stream)
// named barriers
constexpr int kBarSoftmax = 1, kBarTurn = 2;      // + stream
constexpr int kRecFloats = 132;         // O[128], ref, Σw, padding
constexpr int kMaxGuarded = 4;          // tiles that the borders of a CTA's rows can cross: at most 3
constexpr int kSCol = 0, kOCol = 256;   // TMEM columns: scores (weights over them) and O of both streams

struct PromptArgs {
  const int* q_starts;
  const int* k_starts;
  int batch, total_q, total_k;
  int G, Hq, causal;
  int tokens;               // of a stream's rows
  int per_cta;              // tokens of a CTA: `tokens` or twice that
  int tiles, splits;        // CTAs along the queries, along the keys
  float scale;              // softmax_scale · log2(e)
  void* out;                // [total_q][Hq][128]
  float* rec;               // [splits][total_q · Hq][kRecFloats]
  const uint16_t* v;        // for values that the guard took out
  long long v_t, v_h;
};

struct alignas(1024) Smem {
  unsigned char q[2][kTileBytes];
  unsigned char kv[kStages][kTileBytes];
  uint64_t full[kStages], empty[kStages];
  uint64_t gfull[kMaxGuarded];    // V of a guarded tile has arrived (`full`: it may be used)
  uint64_t qfull, gdone, sfull[2], pfull[2][2], odone[2][2], drain;     // [stream][part of a tile]
  uint32_t tmem;
  int poison;               // the guard took values out
};

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity) {
  return __all_sync(0xffffffffu, tq::mbar_wait(bar, parity));
}
// Bounded wait of one thread in short suspensions (2 us at most each; 10^6 of them take between 20 ms
// and 2 s).  It wakes sooner than one long suspension and is little code.
__device__ __forceinline__ bool poll(uint64_t* bar, unsigned parity) {
#pragma unroll 1
  for (int i = 0; i < 1000000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(s32(bar)), "r"(parity), "r"(2000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 consecutive TMEM columns of the thread's lane.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// One box of a tensor map: 64 channels of (heads, tokens) from (channel, head, token).
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int channel, int head, int token,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(s32(dst)), "l"(map), "r"(channel), "r"(head), "r"(token), "r"(s32(bar))
      : "memory");
}
// Shared-memory matrix descriptor with 128-byte swizzle.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return tq::smem_desc(saddr, lbo, sbo) | (2ull << 61);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool kBf16>
__device__ __forceinline__ float widen(uint16_t u) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)u << 16);
  return __half2float(__ushort_as_half(u));
}
// The top bit of each half of a pair that is infinite or NaN (its exponent is all ones).
template <bool kBf16>
__device__ __forceinline__ uint32_t special2(uint32_t u) {
  constexpr uint32_t m = kBf16 ? 0x7f807f80u : 0x7c007c00u, one = kBf16 ? 0x00800080u : 0x04000400u;
  return ((u & m) + one) & 0x80008000u;
}

// Weights of 64 scores with a reference, packed; returns their sum.  Without a reference: of any
// size (the caller takes them again).
template <bool kBf16>
__device__ __forceinline__ float weights(const float (&x)[64], tq::f32x2 scale2, float ref, uint32_t (&p)[32]) {
  const float off = ref == -INFINITY ? 0.f : -ref;
  const tq::f32x2 off2 = tq::pack2(off, off);
  tq::f32x2 l0 = tq::pack2(0.f, 0.f), l1 = l0;
#pragma unroll
  for (int k = 0; k < 64; k += 4) {
    const float2 u = tq::unpack2(tq::fma2(tq::pack2(x[k], x[k + 1]), scale2, off2));
    const float2 v = tq::unpack2(tq::fma2(tq::pack2(x[k + 2], x[k + 3]), scale2, off2));
    const float w0 = ex2(u.x), w1 = ex2(u.y), w2 = ex2(v.x), w3 = ex2(v.y);
    l0 = tq::add2(l0, tq::pack2(w0, w1));
    l1 = tq::add2(l1, tq::pack2(w2, w3));
    p[k / 2] = pack<kBf16>(w0, w1);
    p[k / 2 + 1] = pack<kBf16>(w2, w3);
  }
  const float2 l = tq::unpack2(tq::add2(l0, l1));
  return l.x + l.y;
}

// What a CTA works on.
struct Work {
  int h;                    // KV head
  int q0, k0, nq, nk;       // the sequence's first query and key, its numbers of them
  int tok0, ntok;           // its tokens here
  int split;
  int j0, n;                // tiles of keys: first, number (of the stream with most)
  int n0;                   // tiles of stream 0
  bool pair;                // streams are two blocks of rows
  int free_to;              // keys before this one are attended by every row here

  __device__ __forceinline__ int limit(const PromptArgs& a, int token) const {
    return a.causal ? min(max(token + nk - nq + 1, 0), nk) : nk;
  }
};

// Tiles [first, first + count) of a stream, every `step`-th of the CTA's.
struct Stream {
  int count, step, tile0, tok0;
};
__device__ __forceinline__ Stream stream_of(const PromptArgs& a, const Work& w, int s) {
  if (w.pair) return Stream{s ? w.n : w.n0, 1, w.j0, w.tok0 + s * a.tokens};
  return Stream{s ? w.n / 2 : (w.n + 1) / 2, 2, w.j0 + s, w.tok0};
}

template <bool kBf16>
__device__ __forceinline__ void put32(const PromptArgs& a, long long row, const float (&o)[32], float inv, int c) {
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * TQ_D + c);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    dst[i] = make_uint4(pack<kBf16>(o[8 * i] * inv, o[8 * i + 1] * inv), pack<kBf16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                        pack<kBf16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack<kBf16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
}

// The softmax of one stream's tiles: a thread per row, 64 scores at a time.
//
// Weights are taken with the reference as it is, and their sum tells whether that was right: a sum of
// at most 2^8 (fp16: 2^15) has no weight above.  Only where a row's sum is larger, or where a row
// has no reference yet, is the maximum looked for, the reference moved there and O scaled.  So there
// is no pass for the maximum in the chain from S to P (350 of 3000 cycles a tile).  Weights are handed
// over 64 at a time, so that their products begin while the other 64 are made.  (Two threads a row, 32
// scores at a time in rolled loops, with the maximum first: 621 us for 608, 8192 × 8192.)
template <bool kBf16>
__device__ __forceinline__ bool softmax_stream(const PromptArgs& a, Smem& sm, const Work& w, int s, int warp4, int lane,
                                               float& ref, float& sum) {
  constexpr float kLift = kBf16 ? 0.f : 7.f, kMost = kBf16 ? 256.f : 32768.f;   // 2^8 above the reference's maximum
  const Stream st = stream_of(a, w, s);
  const int r = 32 * warp4 + lane, token = st.tok0 + r / a.G;
  const bool there = token < w.tok0 + w.ntok && r < a.tokens * a.G;
  const int lim = there ? w.limit(a, token) : 0;
  const uint32_t lanes = (uint32_t)(32 * warp4) << 16;
  const uint32_t scol = lanes + kSCol + 128 * s, ocol = lanes + kOCol + 128 * s;
  const tq::f32x2 scale2 = tq::pack2(a.scale, a.scale);
  bool ok = true;
  ref = there ? -INFINITY : 0.f;      // in the units of the exponent (rows that are not used need none)
  sum = 0.f;
#pragma unroll 1
  for (int i = 0; i < st.count; ++i) {
    const int at = (st.tile0 + i * st.step) * kTile;
    ok = ok && warp_wait(&sm.sfull[s], i & 1);
    if (!ok) break;
    tc_after();
    if (at + kTile > w.free_to) {
      const int n = lim - at;                // scores that the row attends
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        float x[16];
        tmem_load16(scol + c, reinterpret_cast<uint32_t*>(x));
        tq::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c + k >= n) x[k] = -INFINITY;
        tq::tmem_st_32x32b_x16(scol + c, reinterpret_cast<uint32_t*>(x));
      }
      tq::tmem_wait_st();
    }
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      float x[64];
      uint32_t p[32];
      __syncwarp();       // (lane 0 arrived alone)
      tq::tmem_ld_32x32b_x32(scol + 64 * part, reinterpret_cast<uint32_t*>(x));
      tq::tmem_ld_32x32b_x32(scol + 64 * part + 32, reinterpret_cast<uint32_t*>(x) + 32);
      tq::tmem_wait_ld();
      float l = weights<kBf16>(x, scale2, ref, p);
      const bool bad = there && (!(l <= kMost) || ref == -INFINITY);
      if (__any_sync(0xffffffffu, bad)) {
        float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = max3(m[k], x[c + k], x[c + 4 + k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], x[60 + k]);
        const float top = max3(m[0], m[1], fmaxf(m[2], m[3])) * a.scale - kLift;
        const float next = bad && top > ref ? top : ref;
        if (i > 0 || part > 0) {
          ok = warp_wait(&sm.odone[s][part ^ 1], (part ? i : i - 1) & 1);      // (of the part before)
          if (!ok) break;
          tc_after();
          const float corr = ref == -INFINITY ? 0.f : ex2(ref - next);
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            tmem_load16(ocol + c, o);
            tq::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
            tq::tmem_st_32x32b_x16(ocol + c, o);
          }
          sum *= corr;
        }
        ref = next;
        l = weights<kBf16>(x, scale2, ref, p);
      }
      tq::tmem_st_32x32b_x32(scol + 32 * part, p);
      sum += l;
      tq::tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pfull[s][part]);
    }
    if (!ok) break;
  }
  if (st.count > 0) ok = ok && warp_wait(&sm.odone[s][1], (st.count - 1) & 1);
  return ok;
}

// Four records (reference, Σw; O) joined to a running one.  A record with a sum of 0 attends nothing; a
// NaN sum has no reference and stays.
__device__ __forceinline__ void join4(const float2 (&ml)[4], const float4 (&x)[4], float& m, float& l, float4& o) {
  float top = m;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
  const float mine = m == -INFINITY ? 1.f : ex2(m - top);
  l *= mine;
  o.x *= mine; o.y *= mine; o.z *= mine; o.w *= mine;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (ml[k].y == 0.f) continue;
    const float f = ml[k].x == -INFINITY ? 1.f : ex2(ml[k].x - top);
    l = fmaf(ml[k].y, f, l);
    o.x = fmaf(x[k].x, f, o.x);
    o.y = fmaf(x[k].y, f, o.y);
    o.z = fmaf(x[k].z, f, o.z);
    o.w = fmaf(x[k].w, f, o.w);
  }
  m = top;
}

// A channel's values that the guard took out of n keys (v: the first one's, `stride` elements apart),
// given back to a row that attends them: O and so the row become what they are, infinite or NaN.
// Rare and slow.
template <bool kBf16>
__device__ __noinline__ float give_back(const uint16_t* v, long long stride, int n, float o) {
  for (int j = 0; j < n; ++j)
    if (special2<kBf16>(v[j * stride])) o += widen<kBf16>(v[j * stride]);
  return o;
}

// Where K (value = 0) and V (1) of a tile lie.  Pairs share a ring of kStages stages that holds K and
// V of tiles 0, 1, ... in turn; alternating streams have a stage each for their K and their V.  Who
// waits for a stage waits for every use of it, so that a phase's parity says which one is meant.
struct Place {
  int stage;
  unsigned phase;
};
__device__ __forceinline__ Place place(const Work& w, int t, int value) {
  if (w.pair) return Place{(2 * t + value) % kStages, (unsigned)((2 * t + value) / kStages) & 1};
  return Place{2 * (t & 1) + value, (unsigned)(t >> 1) & 1};
}

// The products of one stream: S = Q·Kᵀ of its first tile, then O += P·V of each with S of the next.
//
// An issuer a stream, because around the products of a tile an issuer has 400 cycles and more of
// waits and commits, in which the tensor pipe stood still with one issuer for both (without any
// softmax 1560 TFLOP/s for 8192 × 8192 bf16; 2056 with two).  Pairs issue in turn, a tile's 16
// products each: left alone, both streams' products run at once and then both softmaxes (4250 cycles
// a tile of both, 1850 of them waiting for S).  The stream is a constant, so that TMEM addresses are.
template <bool kBf16, int s>
__device__ __forceinline__ bool issue_stream(Smem& sm, const Work& w) {
  constexpr uint32_t kType = kBf16 ? (1u << 7) | (1u << 10) : 0u;
  constexpr uint32_t kIdescS = tq::idesc_f16(128, 128) | kType;
  constexpr uint32_t kIdescO = kIdescS | (1u << 16);       // B (values) is N-major
  const uint64_t q = swizzled_desc(s32(sm.q[0]), 16, 1024) + (s && w.pair ? kTileBytes >> 4 : 0);
  const uint64_t kdesc = swizzled_desc(s32(sm.kv[0]), 16, 1024);
  const uint64_t vdesc = swizzled_desc(s32(sm.kv[0]), kHalfBytes, 1024);
  const int step = w.pair ? 1 : 2, first = w.pair ? 0 : s;
  const int live = w.pair && !s ? w.n0 : w.n;              // tiles before this one are this stream's too
  bool ok = true;
  auto wait = [&](uint64_t* bar, unsigned parity) { ok = ok && poll(bar, parity); };
  auto agree = [&] { ok = __all_sync(0xffffffffu, ok); };
  if (s == 1 && w.pair) tq::named_arrive(kBarTurn, 64);
  if (first < w.n) wait(&sm.qfull, 0);
  // (a wait that gave up stops the issues, not the turns: both issuers take the same number of them)
  int i = -1;
  for (int t = first - step; t < w.n; t += step, ++i) {
    const Place pv = place(w, max(t, 0), 1), pk = place(w, t + step, 0);
    const bool weigh = i >= 0, score = t + step < w.n;
    const uint64_t v = vdesc + pv.stage * (kTileBytes >> 4), k = kdesc + pk.stage * (kTileBytes >> 4);
    // (the weights come last: the rest is there before them)
    if (weigh) wait(&sm.full[pv.stage], pv.phase);
    if (score) wait(&sm.full[pk.stage], pk.phase);
    __syncwarp();         // (lanes leave their waits one by one; a barrier takes the warp as one)
    if (w.pair) tq::named_sync(kBarTurn + s, 64);
    if (!weigh || t >= live) {
      agree();
    } else {
      // in two parts of 64 keys, as their weights come
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        wait(&sm.pfull[s][part], i & 1);
        agree();
        tc_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
            tq::mma_ts(kOCol + 128 * s, kSCol + 128 * s + 8 * ks, v + ks * (2048 >> 4), kIdescO, ks ? 1u : (uint32_t)(i > 0));
          tq::mma_commit(&sm.odone[s][part]);
        }
      }
    }
    tc_after();
    if (ok && elect_one()) {
      if (weigh) tq::mma_commit(&sm.empty[pv.stage]);
      if (score) {
        if (t + step < live) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const int d = (ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2;
            tq::mma_ss(kSCol + 128 * s, q + d, k + d, kIdescS, ks > 0);
          }
          tq::mma_commit(&sm.sfull[s]);
        }
        tq::mma_commit(&sm.empty[pk.stage]);
      }
    }
    __syncwarp();
    if (w.pair && (s == 0 || score)) tq::named_arrive(kBarTurn + (s ^ 1), 64);
  }
  // whatever was issued has ended before the tensor memory is given back
  if (elect_one()) tq::mma_commit(&sm.drain);
  __syncwarp();
  return tq::mbar_wait(&sm.drain, 0) && ok;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PromptArgs a) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid < 3) {
    const CUtensorMap* map = tid == 0 ? &qmap : tid == 1 ? &kmap : &vmap;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  // What runs before may have written everything that is read from here on; what comes after waits
  // for this kernel's end in the same way.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the CTA's work.  Sequence b's CTAs are numbered from ⌊q_starts[b] / per_cta⌋ + b on, which
  // leaves each enough numbers; the last tokens of a sequence, which attend most, come first
  Work w;
  w.split = blockIdx.x % a.splits;
  const int rest = blockIdx.x / a.splits;
  w.h = rest / a.tiles;
  const int number = a.tiles - 1 - rest % a.tiles;
  auto start = [&](const int* p, int b, int most) { return min(max(p[b], 0), most); };
  if (const long long i = (long long)blockIdx.x * kThreads + tid; i < a.batch) {      // (CTAs are no fewer than sequences)
    const int qa = a.q_starts[i], qb = a.q_starts[i + 1], ka = a.k_starts[i], kb = a.k_starts[i + 1];
    if (qa < 0 || qb < qa || qb > a.total_q || ka < 0 || kb < ka || kb > a.total_k) atomicOr(&g_tq_flags, TQ_FLAG_LEN_OVERFLOW);
  }
  // The last sequence that begins at or before the CTA's number, looked for by all threads: among up to 384
  // at once, else among every `step`-th of the rest, then between two of those.  (Each CTA looking at every
  // sequence took the square of them: 1.8 ms for 16000 single tokens, 49 ms for 100000.)
  int b = -1;
  for (int n = a.batch; n > 0;) {
    const int step = (n + kThreads - 1) / kThreads, i = b + 1 + tid * step;
    const int c = __syncthreads_count(tid * step < n && start(a.q_starts, i, a.total_q) / a.per_cta + i <= number);
    if (c == 0) break;
    b += 1 + (c - 1) * step;
    n = min(step, a.batch - b) - 1;
  }
  if (b < 0) return;        // before the first sequence
  w.q0 = start(a.q_starts, b, a.total_q);
  w.k0 = start(a.k_starts, b, a.total_k);
  w.nq = max(start(a.q_starts, b + 1, a.total_q) - w.q0, 0);
  w.nk = max(start(a.k_starts, b + 1, a.total_k) - w.k0, 0);
  w.tok0 = (number - w.q0 / a.per_cta - b) * a.per_cta;
  w.ntok = min(a.per_cta, w.nq - w.tok0);
  if (w.ntok <= 0 || w.tok0 < 0) return;      // (below 0: starts that do not ascend)
  w.pair = w.ntok > a.tokens;
  w.free_to = w.limit(a, w.tok0);
  const int total = (w.limit(a, w.tok0 + w.ntok - 1) + kTile - 1) / kTile;
  // (2^21 tiles and 2^10 parts at most: 32 bits hold the products)
  w.j0 = (int)((uint32_t)total * w.split / a.splits);
  w.n = (int)((uint32_t)total * (w.split + 1) / a.splits) - w.j0;
  // (pairs: stream 0's tokens come first and attend fewer tiles)
  w.n0 = w.pair ? min(max((w.limit(a, w.tok0 + a.tokens - 1) + kTile - 1) / kTile - w.j0, 0), w.n) : w.n;
  // tiles that some row does not attend in full: the last `guarded` ones
  const int guarded = min(w.n, max(0, w.j0 + w.n - w.free_to / kTile));

  if (warp == kIssueWarp) tq::tmem_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tq::mbar_init(&sm.full[i], 1);
      tq::mbar_init(&sm.empty[i], w.pair ? 2 : 1);
    }
    tq::mbar_init(&sm.qfull, 1);
    tq::mbar_init(&sm.gdone, 1);
    for (int i = 0; i < kMaxGuarded; ++i) tq::mbar_init(&sm.gfull[i], 1);
    for (int i = 0; i < 2; ++i) {
      tq::mbar_init(&sm.sfull[i], 1);
      tq::mbar_init(&sm.pfull[i][0], 4);
      tq::mbar_init(&sm.pfull[i][1], 4);
      tq::mbar_init(&sm.odone[i][0], 1);
      tq::mbar_init(&sm.odone[i][1], 1);
    }
    tq::mbar_init(&sm.drain, 2);
    sm.poison = 0;
    tq::mbar_init_fence();
  }
  tc_before();
  __syncthreads();
  tc_after();
  bool ok = sm.tmem == 0;   // all 512 columns: they begin at address 0
  if (warp < kLoadWarp) {
    // ================================================================ softmax
    const int s = warp >> 2, warp4 = warp & 3, r = 32 * warp4 + lane;
    float ref, sum;
    ok = softmax_stream<kBf16>(a, sm, w, s, warp4, lane, ref, sum) && ok;
    if (guarded) ok = ok && warp_wait(&sm.gdone, 0);
    ok = tq::named_sync_and(kBarSoftmax, 256, ok);
    if (ok) {
      tc_after();
      const bool poison = guarded && *reinterpret_cast<volatile int*>(&sm.poison);
      const Stream st = stream_of(a, w, s);
      const int token = st.tok0 + r / a.G;
      const bool there = r < a.tokens * a.G && token < w.tok0 + w.ntok;
      const long long row = (long long)(w.q0 + token) * a.Hq + w.h * a.G + r % a.G;
      const uint32_t ocol = ((uint32_t)(32 * warp4) << 16) + kOCol + 128 * s;
      // Columns [c0, c1) of the row are this thread's.  Alternating streams hold parts of the same rows:
      // each gives the other one half of its columns (through the ring, which is done with) and keeps
      // the other half.
      int c0 = 0, c1 = 128;
      float mine = 1.f, other = 0.f;       // factors of its own part and the other one's
      float4* given = reinterpret_cast<float4*>(sm.kv[0]) + r;               // [stream][16][row]
      float2* stats = reinterpret_cast<float2*>(sm.kv[2]) + r;               // [stream][row]
      if (!w.pair) {
        if (w.n > 1) {
          c0 = 64 * s;
          c1 = c0 + 64;
          stats[kTile * s] = make_float2(ref, sum);
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            float o[32];
            tq::tmem_ld_32x32b_x32(ocol + (64 - c0) + c, reinterpret_cast<uint32_t*>(o));
            tq::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              given[(16 * s + (c + k) / 4) * kTile] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
          tq::named_sync(kBarSoftmax, 256);
          const float2 rs = stats[kTile * (s ^ 1)];
          const float both = fmaxf(ref, rs.x);
          mine = ref == -INFINITY ? 0.f : ex2(ref - both);
          other = rs.x == -INFINITY ? 0.f : ex2(rs.x - both);
          sum = sum * mine + rs.y * other;     // (a NaN sum stays)
          ref = both;
        } else if (s == 1) {
          c1 = 0;                              // (one tile: stream 0's)
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      float* rec = a.rec + ((long long)w.split * a.total_q * a.Hq + row) * kRecFloats;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        // Rows that are not there skip the body and rows with values given back loop in it, each lane as
        // often as it has to: the warp meets before the load, which takes all of its lanes at once.
        __syncwarp();
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
        if (st.count > 0) {
          tq::tmem_ld_32x32b_x32(ocol + c, reinterpret_cast<uint32_t*>(o));
          tq::tmem_wait_ld();
        }
        if (there) {
          if (!w.pair && w.n > 1) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 x = given[(16 * (s ^ 1) + (c - c0 + k) / 4) * kTile];
              o[k] = fmaf(o[k], mine, x.x * other);
              o[k + 1] = fmaf(o[k + 1], mine, x.y * other);
              o[k + 2] = fmaf(o[k + 2], mine, x.z * other);
              o[k + 3] = fmaf(o[k + 3], mine, x.w * other);
            }
          }
          if (poison) {
            const int first = max(w.free_to, w.j0 * kTile), n = min(w.limit(a, token), (w.j0 + w.n) * kTile) - first;
            const uint16_t* v = a.v + (long long)(w.k0 + first) * a.v_t + w.h * a.v_h + c;
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = give_back<kBf16>(v + k, a.v_t, n, o[k]);
          }
          if (a.splits > 1) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(rec + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          } else {
            put32<kBf16>(a, row, o, inv, c);
          }
        }
      }
      __syncwarp();
      if (there && a.splits > 1 && c0 == 0 && c1) *reinterpret_cast<float2*>(rec + 128) = make_float2(ref, sum);
    }
  } else {
    if (warp == kLoadWarp) {
      // ============================================================== loader
      if (lane == 0 && w.n > 0) {
        int uses[kStages] = {};        // of each stage so far
        auto load = [&](int t, int value) {
          const int st = place(w, t, value).stage, guard = value ? t - (w.n - guarded) : -1;
          if (uses[st] && !(ok = ok && tq::mbar_wait(&sm.empty[st], (uses[st] - 1) & 1))) return;
          ++uses[st];
          uint64_t* bar = guard >= 0 ? &sm.gfull[guard] : &sm.full[st];
          tq::mbar_expect_tx(bar, kTileBytes);
          for (int c = 0; c < 2; ++c)
            tma_load(sm.kv[st] + c * kHalfBytes, value ? &vmap : &kmap, 64 * c, w.h, w.k0 + (w.j0 + t) * kTile, bar);
        };
        const int blocks = w.pair ? 2 : 1, bytes = a.tokens * a.G * 128;
        tq::mbar_expect_tx(&sm.qfull, blocks * 2 * bytes);
        for (int s = 0; s < blocks; ++s)
          for (int c = 0; c < 2; ++c)
            tma_load(sm.q[s] + c * kHalfBytes, &qmap, 64 * c, w.h * a.G, w.q0 + w.tok0 + s * a.tokens, &sm.qfull);
        const int step = w.pair ? 1 : 2;
        for (int t = 0; t < w.n && ok; t += step) {
          load(t, 0);
          if (!w.pair && t + 1 < w.n && ok) load(t + 1, 0);
          if (ok) load(t, 1);
          if (!w.pair && t + 1 < w.n && ok) load(t + 1, 1);
        }
        // copies in flight end before the block does, whatever happened
        // (a guarded tile's `full` follows its copy)
        ok = tq::mbar_wait(&sm.qfull, 0) && ok;
        for (int i = 0; i < kStages; ++i)
          if (uses[i]) ok = tq::mbar_wait(&sm.full[i], (uses[i] - 1) & 1) && ok;
      }
    } else if (warp < kGuardWarp) {
      // ============================================================== issuers
      if (warp == kIssueWarp) ok = issue_stream<kBf16, 0>(sm, w) && ok;
      else ok = issue_stream<kBf16, 1>(sm, w) && ok;
    } else {
      // ============================================================== guard
      for (int g = 0; g < guarded && ok; ++g) {
        const int t = w.n - guarded + g;
        const int st = place(w, t, 1).stage;
        // (the guarded tiles are the last ones: a limit that grows with the tiles before them)
        ok = __all_sync(0xffffffffu, tq::mbar_wait(&sm.gfull[g], 0, 20000000ull + 20000ull * w.n));
        if (!ok) break;
        const int key0 = (w.j0 + t) * kTile;
        for (int i = lane; i < 2 * kTile; i += 32) {         // (row, half of the channels)
          const int j = i & (kTile - 1);
          uint4* row = reinterpret_cast<uint4*>(sm.kv[st] + (i >> 7) * kHalfBytes + j * 128);
          if (key0 + j >= w.nk) {
#pragma unroll
            for (int c = 0; c < 8; ++c) row[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
          } else if (key0 + j >= w.free_to) {
            uint32_t bad = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 x = row[(c + lane) & 7];
              bad |= special2<kBf16>(x.x) | special2<kBf16>(x.y) | special2<kBf16>(x.z) | special2<kBf16>(x.w);
            }
            if (bad) {
              uint32_t* word = reinterpret_cast<uint32_t*>(row);
#pragma unroll 1
              for (int c = 0; c < 32; ++c) {
                const uint32_t x = special2<kBf16>(word[c]);
                word[c] &= ~((x >> 15) * 0xffffu);
              }
              *reinterpret_cast<volatile int*>(&sm.poison) = 1;
            }
          }
        }
        tq::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.full[st]);
          if (g == guarded - 1) mbar_arrive(&sm.gdone);
        }
      }
    }
  }
  if (!ok && lane == 0) atomicOr(&g_tq_flags, TQ_FLAG_TIMEOUT);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kIssueWarp) tq::tmem_dealloc(sm.tmem, 512);
}

// Records of a row joined with their log-sum-exp weights: four warps a row, each every fourth record.
template <bool kBf16>
__global__ void __launch_bounds__(128) prompt_merge_kernel(const PromptArgs a) {
  __shared__ float4 acc[4][32];
  __shared__ float2 part[4];
  const long long rows = (long long)a.total_q * a.Hq, row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // rows of no sequence are left as they are
  if (row / a.Hq < a.q_starts[0] || row / a.Hq >= a.q_starts[a.batch]) return;
  const float* rec = a.rec + row * kRecFloats;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = warp; s0 < a.splits; s0 += 16) {
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* r = rec + (s0 + 4 * k) * rows * kRecFloats;
      if (s0 + 4 * k < a.splits) {
        ml[k] = *reinterpret_cast<const float2*>(r + 128);
        x[k] = *reinterpret_cast<const float4*>(r + 4 * lane);
      }
    }
    join4(ml, x, m, l, o);
  }
  acc[warp][lane] = o;
  if (lane == 0) part[warp] = make_float2(m, l);
  __syncthreads();
  if (warp) return;
  float2 ml[4];
  float4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ml[k] = part[k];
    x[k] = acc[k][lane];
  }
  m = -INFINITY, l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  join4(ml, x, m, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * TQ_D) + lane;
  *dst = make_uint2(pack<kBf16>(o.x * inv, o.y * inv), pack<kBf16>(o.z * inv, o.w * inv));
}

// ---------------------------------------------------------------- host
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Plan {
  int G, tokens, per_cta, tiles, splits;
  size_t bytes;
};

// Parts of the keys of sequences with one block of rows each that make the estimated time least, in
// tiles (1.5 us each where all SMs read).  A part costs its tiles and about 3.5 more for its start and end (5
// us), a record 2 times 528 bytes of the join (of 5 bytes a picosecond).  Parts that all have an SM take
// the time of one; one sequence's are alike and go in waves; those of a batch differ with its lengths,
// which the host does not know (taken: half of the longest to all of it, three quarters of it on average),
// and take an SM's share of the work and half of the longest part.  Within 6% of the best number of parts in
// twelve batches of 2 to 100 sequences, alike or from 1% of the longest on.
int key_parts(long long units, long long tiles, long long rows, long long sms, bool alike) {
  constexpr double kPart = 3.5, kRecord = 2 * 528 / 7.5e6;
  const long long most = std::min(std::max(tiles / 2, 1LL), std::min<long long>(1023, 8 * sms / units + 8));
  double best = 0;
  int parts = 1;
  for (long long s = 1; s <= most; ++s) {
    const long long items = units * s, waves = (items + sms - 1) / sms;
    const double item = (double)((tiles + s - 1) / s) + kPart;
    const double t = (items <= sms || alike ? (double)waves * item
                                            : (double)units * (0.75 * (double)tiles + kPart * (double)s) / (double)sms + item / 2) +
                     (s > 1 ? kRecord * (double)(rows * s) : 0.0);
    if (s == 1 || t < best) {
      best = t;
      parts = (int)s;
    }
  }
  return parts;
}

tq_status make_plan(const tq_prompt_desc* d, Plan* p) {
  if (!d) return TQ_ERR_INVALID_ARG;
  if (d->head_dim != TQ_HEAD_DIM) return TQ_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->q_heads <= 0 || d->kv_heads <= 0 || d->q_heads % d->kv_heads) return TQ_ERR_INVALID_ARG;
  if (d->q_heads / d->kv_heads > TQ_MAX_GROUP) return TQ_ERR_UNSUPPORTED;
  if (d->total_q < 0 || d->total_k < 0 || d->max_k_len < 0) return TQ_ERR_INVALID_ARG;
  if (d->dtype != TQ_F16 && d->dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  if (d->total_q > (1 << 28) || d->total_k > (1 << 28) || d->batch > (1 << 20)) return TQ_ERR_UNSUPPORTED;
  p->G = d->q_heads / d->kv_heads;
  p->tokens = kTile / p->G;
  const int n = tq_num_sms();
  const long long sms = n > 0 ? n : 152;
  // CTAs for sequences of about the same length (the lengths lie on the device; the grid is for any).
  const long long each = d->batch ? (d->total_q + d->batch - 1) / d->batch : 0;
  auto ctas = [&](long long per) { return std::max<long long>(1, d->batch * ((each + per - 1) / per) * d->kv_heads); };
  // One block of rows a CTA where each has an SM of its own (its two streams halve the keys' time; a few
  // more CTAs than SMs are the short ones of a causal call), else two: many more would pay for starts
  // and ends twice (28/4 heads: 8 prompts of 100 tokens 11.1 us for 14.8, 1000 tokens behind 8000
  // keys 107 for 136; 700 tokens, 156 CTAs of one block, 14.7 us and 18.1 with two).
  p->per_cta = ctas(p->tokens) * 10 <= sms * 11 ? p->tokens : 2 * p->tokens;
  // Keys split, each part with at least two tiles: with several blocks of rows a sequence so that the CTAs
  // fill the GPU once, else by an estimate, in single blocks (one token of 8 sequences behind 8192 keys, 32
  // units of 64 tiles: 4 parts 31 us, 5 parts 45, 8 parts 35; 8 sequences of 8 heads behind 1600 to 21000 keys:
  // 90 us, unsplit, two parts 106 and 176).
  const long long key_tiles = ((long long)d->max_k_len + kTile - 1) / kTile;
  if (d->batch && each <= p->tokens) {
    p->splits = key_parts((long long)d->batch * d->kv_heads, key_tiles, (long long)d->total_q * d->q_heads, sms, d->batch == 1);
    if (p->splits > 1) p->per_cta = p->tokens;
  } else {
    p->splits = (int)std::max<long long>(1, std::min<long long>(std::min<long long>(sms / ctas(p->per_cta), key_tiles / 2), 1023));
  }
  p->tiles = d->total_q / p->per_cta + d->batch;
  const long long units = (long long)p->tiles * d->kv_heads;
  if (units * p->splits > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  p->bytes = 256;
  if (p->splits > 1) p->bytes += (size_t)p->splits * d->total_q * d->q_heads * kRecFloats * sizeof(float);
  return TQ_OK;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Vectors [tokens][heads][128] in boxes of 64 channels × `box_heads` heads × `box_tokens` tokens.
bool encode(CUtensorMap* map, bool bf16, const void* x, int tokens, int heads, int64_t stride_t, int64_t stride_h,
            int box_heads, int box_tokens) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {TQ_D, (cuuint64_t)heads, (cuuint64_t)std::max(tokens, 1)};
  // (a dimension of one has no stride of its own)
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? stride_h : TQ_D) * 2, (cuuint64_t)(tokens > 1 ? stride_t : TQ_D) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, one[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(x), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Vectors at multiples of 16 bytes, at distances below 2^40 bytes.
bool good(const void* x, int tokens, int heads, int64_t stride_t, int64_t stride_h) {
  if (tokens == 0) return true;
  auto bad = [](int n, int64_t s) { return n > 1 && (s < TQ_D || s % 8 || s >= (1ll << 39)); };
  return x && aligned16(x) && !bad(tokens, stride_t) && !bad(heads, stride_h);
}

template <bool kBf16>
tq_status launch(const CUtensorMap (&maps)[3], const PromptArgs& a, long long grid, cudaStream_t stream) {
  constexpr int smem = (int)sizeof(Smem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static bool configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return TQ_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(prompt_kernel<kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return TQ_ERR_CUDA;
    configured[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prompt_kernel<kBf16>, maps[0], maps[1], maps[2], a) != cudaSuccess) return TQ_ERR_CUDA;
  if (a.splits > 1) {
    cfg.gridDim = dim3((unsigned)((long long)a.total_q * a.Hq));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, prompt_merge_kernel<kBf16>, a) != cudaSuccess) return TQ_ERR_CUDA;
  }
  return tq_cuda_status(cudaGetLastError());
}

}  // namespace

extern "C" size_t tq_prompt_workspace_bytes(const tq_prompt_desc* desc) {
  Plan p;
  return make_plan(desc, &p) == TQ_OK ? p.bytes : 0;
}

extern "C" tq_status tq_prompt_attention(const tq_prompt_desc* d, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                                         const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v,
                                         int64_t v_stride_t, int64_t v_stride_h, const int32_t* q_starts,
                                         const int32_t* k_starts, void* out, void* workspace, size_t workspace_bytes,
                                         tq_stream_t stream) {
  Plan p;
  tq_status st = make_plan(d, &p);
  if (st != TQ_OK) return st;
  if (d->batch == 0 || d->total_q == 0) return TQ_OK;
  if (!good(q, d->total_q, d->q_heads, q_stride_t, q_stride_h) || !good(k, d->total_k, d->kv_heads, k_stride_t, k_stride_h) ||
      !good(v, d->total_k, d->kv_heads, v_stride_t, v_stride_h))
    return TQ_ERR_INVALID_ARG;
  if (!q_starts || !k_starts || !out || !aligned16(out) || reinterpret_cast<uintptr_t>(q_starts) % 4 ||
      reinterpret_cast<uintptr_t>(k_starts) % 4)
    return TQ_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < p.bytes) return TQ_ERR_INVALID_ARG;
  // A CTA writes rows while others read keys, values and their own queries; its own queries it has read by then.
  const tq_vectors o{out, {1, 1, 1}, {}, (long long)d->total_q * d->q_heads * TQ_D * 2};
  auto over = [&](const void* x, int tokens, int heads, int64_t stride_t, int64_t stride_h) {
    return tq_vectors_meet(o, tq_vectors{x, {tokens, heads, 1}, {stride_t * 2, stride_h * 2, 0}, TQ_D * 2});
  };
  const bool in_place = q == out && (d->total_q == 1 || q_stride_t == (int64_t)d->q_heads * TQ_D) && (d->q_heads == 1 || q_stride_h == TQ_D);
  if (over(k, d->total_k, d->kv_heads, k_stride_t, k_stride_h) || over(v, d->total_k, d->kv_heads, v_stride_t, v_stride_h) ||
      (!in_place && over(q, d->total_q, d->q_heads, q_stride_t, q_stride_h)))
    return TQ_ERR_INVALID_ARG;
  const bool bf16 = d->dtype == TQ_BF16;
  CUtensorMap maps[3];
  // (without keys nothing is loaded; the maps need some address all the same, and no strides)
  const int kv_heads = d->total_k ? d->kv_heads : 1;
  if (!encode(&maps[0], bf16, q, d->total_q, d->q_heads, q_stride_t, q_stride_h, p.G, p.tokens) ||
      !encode(&maps[1], bf16, d->total_k ? k : q, d->total_k, kv_heads, k_stride_t, k_stride_h, 1, kTile) ||
      !encode(&maps[2], bf16, d->total_k ? v : q, d->total_k, kv_heads, v_stride_t, v_stride_h, 1, kTile))
    return TQ_ERR_CUDA;
  PromptArgs a{};
  a.q_starts = q_starts;
  a.k_starts = k_starts;
  a.batch = d->batch;
  a.total_q = d->total_q;
  a.total_k = d->total_k;
  a.G = p.G;
  a.Hq = d->q_heads;
  a.causal = d->causal != 0;
  a.tokens = p.tokens;
  a.per_cta = p.per_cta;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.scale = (d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / sqrtf((float)TQ_D)) * 1.4426950408889634f;
  a.out = out;
  a.rec = static_cast<float*>(workspace);
  a.v = static_cast<const uint16_t*>(v);
  a.v_t = v_stride_t;
  a.v_h = v_stride_h;
  const long long grid = (long long)p.tiles * d->kv_heads * p.splits;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return bf16 ? launch<true>(maps, a, grid, s) : launch<false>(maps, a, grid, s);
}
