// Rotary positions of queries and keys, before they are attended or coded (tq_rotary_apply).
//
// Mathematics.  Pair i of a vector at position p turns by θ = p·f_i and is scaled by m:
//   y_a = m·(a·cos θ − b·sin θ),   y_b = m·(a·sin θ + b·cos θ).
// f_i/2π is held as a fraction of 2^64 (turns per position), so that p·f_i is one 64-bit
// multiplication whose overflow drops whole turns: the angle is as good at position 2^31 as at 1.  It
// is cut to 32 bits (2^-31 turns in all) and the nearest quarter turn is taken out in integers; what is
// left, at most an eighth of a turn, is rounded to the 24 bits of a float, by at most 2^-28 turns.
// Together less than 2^-25 radians, which is below what rounding the vectors to 32 bits takes.
// Products and sums are 32 bits, rounded once to the output's type.
//
// Bound by reading and writing the vectors: 131072 tokens of 32/8 fp16 heads take 402 us, 6.68 TB/s, the
// copy rate; a step's 32 tokens of 28/4 heads 3.5 us, a launch.  A warp takes four heads of a token at a
// time, eight lanes a vector and 16 coordinates (8 pairs) a lane, and keeps its lanes' sines and
// cosines while it goes through the token's heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tq_internal.h"

namespace {

struct Side {
  const char* x;
  char* y;
  long long xb, xh, xt, yb, yh, yt;   // strides in bytes
};

struct RotaryArgs {
  tq_rotary r;
  Side q, k;
  int q_heads, heads;       // heads: of both
  int tokens;
  long long rows;           // batch · tokens
  const int* positions;
  long long pos_b;
  int ways;                 // warps that share a token's heads
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

// cos and sin (times m) of pair i at a position.
__device__ __forceinline__ void angle(const tq_rotary& r, int i, int position, float& c, float& s) {
  const uint64_t turns = (uint64_t)(int64_t)position * r.turns[i];
  const uint32_t u = (uint32_t)(turns >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  float s0, c0;
  sincospif((float)(int32_t)(u - (quarter << 30)) * 0x1p-31f, &s0, &c0);   // half turns, |·| ≤ 1/4
  const float a = quarter & 1 ? s0 : c0, b = quarter & 1 ? c0 : s0;
  c = (quarter + 1) & 2 ? -a : a;
  s = quarter & 2 ? -b : b;
  c *= r.magnitude;
  s *= r.magnitude;
}

__device__ __forceinline__ void turn(float a, float b, float c, float s, float& ya, float& yb) {
  ya = fmaf(a, c, -b * s);
  yb = fmaf(a, s, b * c);
}

// Two 16-bit numbers of a word.  (Rounded two at a time: one bf16 number at a time, 40000 tokens of 40 heads
// took 161 us for 131.)
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// kPer = 16 bytes of T.  Lane l of a vector's eight holds pairs 8l..8l + 7 of the turned
// coordinates: neighbouring ones are the 16 coordinates from 16l, halves are 8 from 8l and the 8
// that lie rotary_dim/2 behind; lanes past the turned coordinates copy 16 of the others.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int kPer = 16 / (int)sizeof(T), kVecs = 8 / kPer;      // 16-byte loads of 8 coordinates
  constexpr int kFlight = sizeof(T) == 4 ? 2 : 4;                  // heads in flight a lane
  const int lane = threadIdx.x & 31, unit = lane & 7;
  const long long warp = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long row = warp / a.ways;
  if (row >= a.rows) return;
  const int h0 = (int)(warp % a.ways) * 4 + (lane >> 3), step = a.ways * 4;
  const int b = (int)(row / a.tokens), t = (int)(row % a.tokens);
  const int units = (a.r.rotary_dim + 15) / 16;
  const bool turned = unit < units;
  const int first = turned && !kInterleaved ? 8 * unit : 16 * unit;
  const int second = turned && !kInterleaved ? a.r.rotary_dim / 2 + 8 * unit : 16 * unit + 8;
  const int position = a.positions[b * a.pos_b + t];
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
    if (turned && (!kInterleaved || 16 * unit + 2 * i < a.r.rotary_dim)) angle(a.r, 8 * unit + i, position, c[i], s[i]);
  }
  for (int h = h0; h < a.heads; h += kFlight * step) {
    uint4 v[kFlight][2][kVecs];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int hf = h + f * step;
      if (hf >= a.heads) break;
      const bool key = hf >= a.q_heads;
      const Side& x = key ? a.k : a.q;
      if (!turned && x.x == x.y) continue;      // in place: nothing to copy
      const char* p = x.x + b * x.xb + (hf - (key ? a.q_heads : 0)) * x.xh + t * x.xt;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        v[f][0][i] = reinterpret_cast<const uint4*>(p + first * sizeof(T))[i];
        v[f][1][i] = reinterpret_cast<const uint4*>(p + second * sizeof(T))[i];
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int hf = h + f * step;
      if (hf >= a.heads) break;
      const bool key = hf >= a.q_heads;
      const Side& x = key ? a.k : a.q;
      if (!turned && x.x == x.y) continue;
      char* p = x.y + b * x.yb + (hf - (key ? a.q_heads : 0)) * x.yh + t * x.yt;
      if (turned) {
        uint32_t* wa = reinterpret_cast<uint32_t*>(v[f][0]);
        uint32_t* wb = reinterpret_cast<uint32_t*>(v[f][1]);
        float ya[2], yb[2];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (kInterleaved && 16 * unit + 2 * i >= a.r.rotary_dim) continue;       // (copied as it is)
            uint32_t* ea = kInterleaved ? (i < 4 ? wa : wb) + 2 * (i & 3) : wa + i;
            uint32_t* eb = kInterleaved ? ea + 1 : wb + i;
            turn(__uint_as_float(*ea), __uint_as_float(*eb), c[i], s[i], ya[0], yb[0]);
            *ea = __float_as_uint(ya[0]);
            *eb = __float_as_uint(yb[0]);
          }
        } else if constexpr (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (16 * unit + 2 * i >= a.r.rotary_dim) continue;
            uint32_t* w = (i < 4 ? wa : wb) + (i & 3);
            const float2 x = widen2<T>(*w);
            turn(x.x, x.y, c[i], s[i], ya[0], yb[0]);
            *w = narrow2<T>(ya[0], yb[0]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 xa = widen2<T>(wa[i]), xb = widen2<T>(wb[i]);
            turn(xa.x, xb.x, c[2 * i], s[2 * i], ya[0], yb[0]);
            turn(xa.y, xb.y, c[2 * i + 1], s[2 * i + 1], ya[1], yb[1]);
            wa[i] = narrow2<T>(ya[0], ya[1]);
            wb[i] = narrow2<T>(yb[0], yb[1]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        reinterpret_cast<uint4*>(p + first * sizeof(T))[i] = v[f][0][i];
        reinterpret_cast<uint4*>(p + second * sizeof(T))[i] = v[f][1][i];
      }
    }
  }
}

// Any even rotary_dim, any strides: lanes take pairs (of coordinates that are copied, behind the turned
// ones) i and i + 32 of a vector, a warp's loads of four heads in flight
// together (34 × 1060 tokens of 40/8 fp32 heads, 98 coordinates: 273 us, 6.5 TB/s; one head at a time 621).
template <typename T>
__global__ void __launch_bounds__(256) rotary_any_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int kFlight = 4;
  const int lane = threadIdx.x & 31;
  const long long warp = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long row = warp / a.ways;
  if (row >= a.rows) return;
  const int b = (int)(row / a.tokens), t = (int)(row % a.tokens);
  const int position = a.positions[b * a.pos_b + t], half = a.r.rotary_dim / 2;
  bool turned[2];
  float c[2], s[2];
  int at[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    turned[j] = i < half;
    c[j] = 1.f;
    s[j] = 0.f;
    if (turned[j]) angle(a.r, i, position, c[j], s[j]);
    at[j][0] = turned[j] && !a.r.interleaved ? i : 2 * i;
    at[j][1] = turned[j] && !a.r.interleaved ? i + half : 2 * i + 1;
  }
  for (int h = (int)(warp % a.ways); h < a.heads; h += kFlight * a.ways) {
    T v[kFlight][2][2];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int hf = h + f * a.ways;
      if (hf >= a.heads) break;
      const bool key = hf >= a.q_heads;
      const Side& x = key ? a.k : a.q;
      const T* p = reinterpret_cast<const T*>(x.x + b * x.xb + (hf - (key ? a.q_heads : 0)) * x.xh + t * x.xt);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!turned[j] && x.x == x.y) continue;      // in place: nothing to copy
        v[f][j][0] = p[at[j][0]];
        v[f][j][1] = p[at[j][1]];
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int hf = h + f * a.ways;
      if (hf >= a.heads) break;
      const bool key = hf >= a.q_heads;
      const Side& x = key ? a.k : a.q;
      T* y = reinterpret_cast<T*>(x.y + b * x.yb + (hf - (key ? a.q_heads : 0)) * x.yh + t * x.yt);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!turned[j] && x.x == x.y) continue;
        if (turned[j]) {
          float ya, yb;
          turn(to_float<T>(v[f][j][0]), to_float<T>(v[f][j][1]), c[j], s[j], ya, yb);
          v[f][j][0] = from_float<T>(ya);
          v[f][j][1] = from_float<T>(yb);
        }
        y[at[j][0]] = v[f][j][0];
        y[at[j][1]] = v[f][j][1];
      }
    }
  }
}

tq_vectors inputs(const Side& s, int batch, int heads, int tokens, int elem) {
  return tq_vectors{s.x, {batch, heads, tokens}, {s.xb, s.xh, s.xt}, TQ_D * elem};
}
tq_vectors outputs(const Side& s, int batch, int heads, int tokens, int elem) {
  return tq_vectors{s.y, {batch, heads, tokens}, {s.yb, s.yh, s.yt}, TQ_D * elem};
}

// One side of a call in bytes; false for a bad one: among others an output whose vectors overlap each
// other (no dimension may lie inside another one's step) or the input without being the input.
bool side_of(const tq_rotary_io* io, int batch, int tokens, int elem, Side* s, bool* vec) {
  *s = Side{};
  if (!io || io->heads == 0) return true;
  if (io->heads < 0 || !io->x || !io->y) return false;
  const int64_t strides[6] = {io->x_stride_b, io->x_stride_h, io->x_stride_t,
                              io->y_stride_b, io->y_stride_h, io->y_stride_t};
  uintptr_t low = reinterpret_cast<uintptr_t>(io->x) | reinterpret_cast<uintptr_t>(io->y);
  if (low % elem) return false;
  for (int64_t x : strides) {
    if (x < 0) return false;
    low |= (uintptr_t)(x * elem);
  }
  const int64_t n[3] = {batch, io->heads, tokens};
  int64_t y_span = TQ_D;                      // elements from the first to behind the last
  bool same = io->x == io->y;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return strides[3 + a] < strides[3 + b]; });
  for (int d : order) {
    if (n[d] == 1) continue;
    if (strides[3 + d] < y_span) return false;
    same = same && strides[d] == strides[3 + d];
    y_span += (n[d] - 1) * strides[3 + d];
  }
  *vec = *vec && low % 16 == 0;
  *s = Side{static_cast<const char*>(io->x), static_cast<char*>(io->y), strides[0] * elem, strides[1] * elem,
            strides[2] * elem, strides[3] * elem, strides[4] * elem, strides[5] * elem};
  return same || !tq_vectors_meet(inputs(*s, batch, io->heads, tokens, elem), outputs(*s, batch, io->heads, tokens, elem));
}

template <typename T>
void launch(const RotaryArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  if (!vec) rotary_any_kernel<T><<<grid, 256, 0, stream>>>(a);
  else if (a.r.interleaved) rotary_kernel<T, true><<<grid, 256, 0, stream>>>(a);
  else rotary_kernel<T, false><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

extern "C" tq_status tq_rotary_frequencies(int32_t rotary_dim, double base, double factor,
                                           int32_t original_len, double low_turns,
                                           double high_turns, double* frequencies) {
  if (rotary_dim < 2 || rotary_dim > TQ_HEAD_DIM || rotary_dim % 2 || !frequencies) return TQ_ERR_INVALID_ARG;
  if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) || original_len < 0)
    return TQ_ERR_INVALID_ARG;
  if (original_len && (!(low_turns >= 0) || !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return TQ_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586477;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double share = 0;            // of the frequency that stays
    if (original_len) {
      const double turns = original_len * f / two_pi;
      share = std::min(1.0, std::max(0.0, (turns - low_turns) / (high_turns - low_turns)));
    }
    frequencies[i] = share * f + (1 - share) * (f / factor);
  }
  return TQ_OK;
}

extern "C" tq_status tq_rotary_init(tq_rotary* r, int32_t rotary_dim, int32_t interleaved,
                                    const double* frequencies, double magnitude) {
  if (!r || !frequencies || rotary_dim < 2 || rotary_dim > TQ_HEAD_DIM || rotary_dim % 2)
    return TQ_ERR_INVALID_ARG;
  if (!std::isfinite(magnitude) || !std::isfinite((float)magnitude)) return TQ_ERR_INVALID_ARG;
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(frequencies[i]) || std::fabs(frequencies[i]) > 1e6) return TQ_ERR_INVALID_ARG;
  *r = tq_rotary{};
  r->rotary_dim = rotary_dim;
  r->interleaved = interleaved != 0;
  r->magnitude = (float)magnitude;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    // f/2π as the exact product with 1/2π in two parts (106 bits), whole turns dropped
    const double f = std::fabs(frequencies[i]), hi = f * 0x1.45f306dc9c883p-3;
    const double lo = std::fma(f, 0x1.45f306dc9c883p-3, -hi) + f * -0x1.6b01ec5417056p-57;
    const double frac = hi - std::floor(hi);
    const uint64_t turns = (uint64_t)std::ldexp(frac, 64) + (uint64_t)(int64_t)std::ldexp(lo, 64);
    r->turns[i] = frequencies[i] < 0 ? 0 - turns : turns;
  }
  return TQ_OK;
}

extern "C" tq_status tq_rotary_apply(const tq_rotary* r, tq_dtype dtype, int32_t batch,
                                     int32_t tokens, const int32_t* positions,
                                     int64_t pos_stride_b, const tq_rotary_io* q,
                                     const tq_rotary_io* k, tq_stream_t stream_) {
  if (!r || r->rotary_dim < 2 || r->rotary_dim > TQ_HEAD_DIM || r->rotary_dim % 2) return TQ_ERR_INVALID_ARG;
  if (dtype != TQ_F32 && dtype != TQ_F16 && dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  if (batch < 0 || tokens < 0 || pos_stride_b < 0) return TQ_ERR_INVALID_ARG;
  if (!batch || !tokens) return TQ_OK;
  if (!positions || reinterpret_cast<uintptr_t>(positions) % 4) return TQ_ERR_INVALID_ARG;
  RotaryArgs a{};
  bool vec = r->interleaved || r->rotary_dim % 16 == 0;
  const int elem = dtype == TQ_F32 ? 4 : 2;
  if (!side_of(q, batch, tokens, elem, &a.q, &vec) || !side_of(k, batch, tokens, elem, &a.k, &vec)) return TQ_ERR_INVALID_ARG;
  // one side's output over the other side's vectors: warps would read what others write
  if (a.q.x && a.k.x) {
    const tq_vectors qx = inputs(a.q, batch, q->heads, tokens, elem), qy = outputs(a.q, batch, q->heads, tokens, elem);
    const tq_vectors kx = inputs(a.k, batch, k->heads, tokens, elem), ky = outputs(a.k, batch, k->heads, tokens, elem);
    if (tq_vectors_meet(qy, ky) || tq_vectors_meet(qx, ky) || tq_vectors_meet(qy, kx)) return TQ_ERR_INVALID_ARG;
  }
  const long long qh = q ? q->heads : 0, heads = qh + (k ? k->heads : 0);
  if (heads > (1 << 20)) return TQ_ERR_UNSUPPORTED;
  a.rows = (long long)batch * tokens;
  if (heads == 0) return TQ_OK;
  a.r = *r;
  a.q_heads = (int)qh;
  a.heads = (int)heads;
  a.tokens = tokens;
  a.positions = positions;
  a.pos_b = pos_stride_b;
  // Warps a token: one while the tokens alone fill the GPU (each computes its angles once for all
  // heads), more where they do not, up to one for each four heads (one, where lanes take pairs).
  const int most = (int)(vec ? (heads + 3) / 4 : heads);
  const long long want = (long long)std::max(tq_num_sms(), 1) * 32;
  a.ways = (int)std::min<long long>(most, std::max<long long>(1, (want + a.rows - 1) / a.rows));
  const long long grid = (a.rows * a.ways + 7) / 8;
  if (grid > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype == TQ_F32) launch<float>(a, vec, (unsigned)grid, stream);
  else if (dtype == TQ_F16) launch<__half>(a, vec, (unsigned)grid, stream);
  else launch<__nv_bfloat16>(a, vec, (unsigned)grid, stream);
  return tq_cuda_status(cudaGetLastError());
}
