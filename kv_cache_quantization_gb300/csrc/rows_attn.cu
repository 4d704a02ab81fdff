// Decode attention of many query rows over one token stream of the compressed cache: over a
// prefix that a whole batch shares (tq_prefix_attention), over the blocks that a selection
// kept of each sequence (tq_sparse_attention), and of the tokens drafted behind a sequence over its
// history and each other (tq_tree_attention, which rows_tree.cu compiles from this file).
//
// Mathematics.  With y = Π q, z = S q and a token's code (i, s, ‖x‖, ‖r‖), the estimator of
// ⟨q, k⟩ (QJL deep-dive §五) is
//   ‖x‖·( ⟨y, c[i]⟩ + ρ·⟨z, s⟩ ),   ρ = ‖r‖/‖x‖·√(π/2)/d,
// one product of length 256 of the row [y, z] with the token's operand [c[i], ±ρ].  A value is
// ‖v‖·Πᵀc[j], so the output row is Πᵀ·Σ_t p_t‖v_t‖c[j_t] / Σ_t p_t.  The weights of the value
// product are w_t = 2^(e_t − m) with e_t = score + log2‖v_t‖ and m a reference kLift below the
// running maximum of e (not of the score) or up to kGrow lower: they are at most 2^(kGrow + kLift) =
// 2^15 whatever the norms, so fp16 holds them; the denominator is Σ w_t/‖v_t‖ in 32 bits.  kLift
// uses what fp16 has above: a weight is held to 2^-32 of the largest (without it to 2^-25, and the numerator lost a
// tail of many small weights that the denominator kept: 65535 of 2^-25.1 behind one of 1 moved a
// row by 2.1e-3 of its norm).
//
// One CTA works on one item: up to 128 query rows × a run of 128-token tiles.
//   12 expander warps turn the codes of a tile into fp16 operands in shared memory, four for
//                     the key levels, four for the signs and norms, four for the value levels
//                     (a byte permute looks four levels up at a time; codes of the next tile
//                     are in flight in registers meanwhile),
//   1 issuer warp     D = [y, z]·[c, ±ρ]ᵀ (128 × 128 × 256, rows in TMEM as the A operand) and
//                     O += W·V (128 × 128 × 128, W in TMEM over the scores it came from),
//   8 softmax warps   one thread per (row, half of the tile's tokens).
// D has two buffers, so tile t + 1 is scored while tile t's softmax runs.  (One more warp of the
// issuer's warpgroup could request codes ahead into L2: it made every case 5 to 15% slower, the
// expanders' loads one tile ahead are early enough.)
// The items' (m, l, O) records are merged, and rotated back once per row, by rows_merge_kernel.
//
// Why the rows are the M dimension: the expansion of a token, which is most of the work, is then
// shared by up to 128 rows, and a row's softmax is one thread's.  Few rows waste MMA rows, not
// time: with 32 rows a tile takes about 3,000 cycles, with 112 about 4,000, where the MMAs alone
// take 1,536.  No unit is near its peak: with 32 rows issue is at 58%, the integer pipe at 52, the
// tensor pipe at 50 and shared memory at 52%, with 112 rows at 50, 40, 27 and less; the first stall
// is a wait for memory or TMEM (long scoreboard).  So a tile's time is the chain of hand-overs from
// expansion (about 13 instructions for eight level coordinates, 8 for eight signs) to product to
// softmax (about 9 a score, through TMEM and back), with units that are half busy.  Instruction
// fetch shows wherever code is long, which is why the roles' loops are kept rolled.  Measured: a
// prefix of 262144 tokens for 8 sequences of 32/8 heads 184 us (281 TFLOP/s, 1.07 TB/s), of 65536
// for 64 of 28/4 heads 171 us (531 TFLOP/s), of 32768 for 32 60 us; 32 blocks of each of 32
// sequences 46 us.  (With 4-bit values the warps of the signs could expand a quarter of them: 167 us
// for the 64 sequences, 47 us for the blocks; not done.)
//
// Roundings to 16 bits: the rotated query and sketch, ρ, the levels (scaled so that fp16 holds
// them best, to 8e-5 with 16 levels, 2e-5 with 8 and 2e-6 with 4) and the weights, each off by at
// most half a step of fp16 (2^-11 relative); together 0.7 to 1.4e-3 of a row's norm, below the
// output's own 2^-8 a value in bf16.  fp16 outputs (2^-11 a value) would show them: for those (kFine)
// query, sketch, ρ and weights are pairs of fp16 numbers (about 2^-21; the levels stay single), for
// 56 instead of 24 matrix instructions a tile, and the second halves of query and sketch take the
// place of the second D: 97 us for the 32 sequences, 395 for the 8, 289 for the 64, 69 for the
// blocks.  Scores, maxima, sums and accumulators are 32 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <climits>

#include "tc_ptx.h"
#include "tq_internal.h"

#ifdef TQ_ROWS_TREE
TQ_DEFINE_FLAGS(tq_take_flags_tree)
#else
TQ_DEFINE_FLAGS(tq_take_flags_rows)
#endif

namespace {

using tq::mbar_arrive;
using tq::s32;
using tq::tc_after;
using tq::tc_before;

#ifdef TQ_ROWS_TREE
constexpr bool kTree = true;
#else
constexpr bool kTree = false;
#endif
constexpr int kTile = 128;              // tokens per tile, and query rows per item
// 8 softmax warps, 3 × 4 expander warps, and a warpgroup that holds the issuer warp alone
constexpr int kKeyWarp = 8, kSignWarp = 12, kValueWarp = 16, kIssueWarp = 20;
constexpr int kThreads = 768;
// Registers per thread: 80 at launch, 61,440 of the block, split by what each role spills least
// with: softmax 80, expanders 88, issuer 56 (256·80 + 384·88 + 128·56 = 61,440), or with pairs of
// operands 96, 72 and 72 (256·96 + 384·72 + 128·72 = 61,440).
constexpr int kRegsLaunch = 80;
template <bool kFine>
struct Regs {
  static constexpr bool kWide = kFine || kTree;      // (trees hold 32 scores a thread)
  static constexpr int softmax = kWide ? 96 : 80, expand = kWide ? 72 : 88, issue = kWide ? 72 : 56;
};
constexpr int kRecFloats = 132;         // acc[128], m, l, padding
constexpr int kLBO = 2048;              // bytes between 8-position chunks of an operand image
constexpr int kKBytes = 32 * kLBO;      // key operand: 128 tokens × 256 positions, fp16
constexpr int kVBytes = 16 * kLBO;
constexpr int kQCol = 0, kDCol = 128, kOCol = 384;   // TMEM columns
constexpr int kQLowCol = 256;           // (fine: the second halves of y and z, over the second D)
constexpr int kFacSlots = 4;
constexpr float kAlpha = 64.f, kBeta = 4.f;   // scales of y and z in the fp16 row operand
constexpr float kLift = 7.f;            // the reference is taken 2^7 below the maximum
constexpr float kGrow = 8.f;            // and follows it when it has grown by 2^8
constexpr float kTiny = 8.6736174e-19f; // 2^-60: smaller value norms count as zero
constexpr float kQjl = 1.2533141373155003f / 128.f;   // √(π/2)/d

// fp16 levels as byte tables for a byte permute: levels 0–7 in lo[0..1], hi[0..1], 8–15 behind.
struct LevelBytes {
  uint32_t lo[4], hi[4];
};

struct CacheSide {
  const uint8_t* kidx;
  const uint8_t* ksgn;
  const float* kxn;
  const float* krn;
  const uint8_t* vidx;
  const float* vxn;
  tq_rowmap kmap, vmap;
  int kslots, vslots;       // slots of a row: the capacity (flat) or the page's
  int same_map;             // keys and values lie alike
};

struct RowsArgs {
  CacheSide own, pre;
  const int* seq_lens;
  const int* pre_len;
  const int* list;          // [B][Hkv][max_blocks] block numbers, or null
  int max_blocks;
  int max_len, max_pre;     // bounds of the lengths that the split is made for
  int B, Hq, Hkv, G;
  int row_tiles, pre_splits, own_splits;
  LevelBytes kt, vt;
  float rho_scale;          // ρ's scale in the key operand
  const uint4* qop;         // [B·Hq][256] fp16 row operands
  const float* qf;          // [B·Hq] factor of the products
  float* rec;               // [pre_splits + own_splits][B·Hq][kRecFloats]
#ifdef TQ_ROWS_TREE
  // Trees: rows are [B][nodes][Hq]; every item is of one sequence, row_tiles items a (sequence, KV
  // head) and split, own_splits splits.
  const unsigned long long* tree;   // [B][nodes], rows tree_b apart: drafted tokens that a node attends
  long long tree_b;
  int nodes;
  const int* order;         // the sequences, the longest first, from the kernel before (nullptr: as they are)
#endif
};

struct alignas(1024) Smem {
  unsigned char k[2][kKBytes];
  unsigned char v[2][kVBytes];
  float fac[kFacSlots][3][kTile];    // ‖x‖, log2‖v‖, 1/‖v‖ of a tile's tokens
  float tmax[2][2][kTile];           // [tile parity][half of the tokens][row]
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ffull[kFacSlots];
  uint64_t qfull, drain;
  uint32_t tmem;
  int tiles;
};

__device__ __forceinline__ float load_elem(const void* base, int dtype, long long i) {
  if (dtype == TQ_F32) return static_cast<const float*>(base)[i];
  const uint16_t u = static_cast<const uint16_t*>(base)[i];
  if (dtype == TQ_BF16) return __uint_as_float((uint32_t)u << 16);
  return __half2float(__ushort_as_half(u));
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Bounded wait of a whole warp: false for all lanes once any gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity) {
  return __all_sync(0xffffffffu, tq::mbar_wait(bar, parity));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// N consecutive TMEM columns of the thread's lane.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t* r) {
  if constexpr (N == 32) {
    tq::tmem_ld_32x32b_x32(at, r);
  } else {
    static_assert(N == 16, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at));
  }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t* v) {
  if constexpr (N == 32) {
    tq::tmem_st_32x32b_x32(at, v);
  } else if constexpr (N == 16) {
    tq::tmem_st_32x32b_x16(at, v);
  } else {
    static_assert(N == 8, "columns");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                 "r"(v[7])
                 : "memory");
  }
}
constexpr __host__ __device__ uint32_t shr(uint32_t x, int n) { return n >= 0 ? x >> n : x << -n; }

// Coordinate of operand position p.  Planes: chunk 4w + r of eight positions holds bits
// r, r + 4, ..., r + 28 of word w (one AND spreads them over eight nibbles).  Signs: chunk
// 4w + c holds the bit pairs (j, j + 16), j = 4c..4c + 3 (one AND leaves both at the sign bits
// of an fp16 pair).  Nibble codes keep their order.
__host__ __device__ constexpr int plane_coord(int p) {
  return (p & ~31) + 4 * (p & 7) + ((p >> 3) & 3);
}
__host__ __device__ constexpr int sign_coord(int p) {
  return (p & ~31) + 4 * ((p >> 3) & 3) + ((p & 7) >> 1) + 16 * (p & 1);
}

// The position of a coordinate: the inverses of these.
__host__ __device__ constexpr int plane_position(int j) { return (j & ~31) + ((j >> 2) & 7) + 8 * (j & 3); }
__host__ __device__ constexpr int sign_position(int j) {
  return (j & ~31) + ((j >> 4) & 1) + 2 * (j & 3) + 8 * ((j >> 2) & 3);
}

// Eight fp16 levels of eight 3-bit indices (one per nibble of s; with 16 levels `top` holds the
// fourth bit, 8 | bit per nibble: a permute in sign-replicating mode makes it a byte mask).
template <bool k16>
__device__ __forceinline__ uint4 levels8(const LevelBytes& t, uint32_t s, uint32_t top) {
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sh = h ? s >> 16 : s;
    uint32_t lo = prmt(t.lo[0], t.lo[1], sh), hi = prmt(t.hi[0], t.hi[1], sh);
    if (k16) {
      const uint32_t m = prmt(0x8000u, 0u, h ? top >> 16 : top);
      lo = (lo & ~m) | (prmt(t.lo[2], t.lo[3], sh) & m);
      hi = (hi & ~m) | (prmt(t.hi[2], t.hi[3], sh) & m);
    }
    w[2 * h] = prmt(lo, hi, 0x5140u);
    w[2 * h + 1] = prmt(lo, hi, 0x7362u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Chunk r of a word of NB planes.
template <int NB>
__device__ __forceinline__ uint4 plane_chunk(const LevelBytes& t, const uint32_t (&w)[NB], int r) {
  uint32_t s = shr(w[0], r) & 0x11111111u, top = 0;
  if (NB >= 2) s |= shr(w[NB >= 2 ? 1 : 0], r - 1) & 0x22222222u;
  if (NB >= 3) s |= shr(w[NB >= 3 ? 2 : 0], r - 2) & 0x44444444u;
  if (NB >= 4) top = (shr(w[NB >= 4 ? 3 : 0], r) & 0x11111111u) | 0x88888888u;
  return levels8<NB == 4>(t, s, top);
}

// The tokens that an item attends.
struct Item {
  int t0, tiles, len, nblk, b, h;
  const int* list;
};

// Where the 32 tokens of a warp lie in a cache's arrays: all in one 64-token block, so the row
// (and the page) is the warp's.  Slots past the sequence's length but in its last block are in
// the cache: they are read, and masked where it matters.  A cursor walks an item's tiles; in a
// run of tokens it only adds 128 and looks the table up where a page ends.
struct Spot {
  bool some;      // at least the first token is attended
  int token0;
  long long row;
  int slot;
};

template <bool kList>
struct Cursor {
  const RowsArgs& a;
  const tq_rowmap& map;
  const Item& it;
  int first;          // the warp's first token in a tile
  bool flag;          // this thread reports bad pages
  int t, token0, page, slot, row;

  __device__ __forceinline__ Cursor(const RowsArgs& a_, const tq_rowmap& m, const Item& i, int f, bool fl)
      : a(a_), map(m), it(i), first(f), flag(fl), t(0), page(0), row(0) {
    if (!kList) {
      token0 = slot = it.t0 * kTile + first;
      if (map.table) {
        page = token0 / map.page_tokens;
        slot = token0 - page * map.page_tokens;
        row = -1;
      }
    }
  }
  __device__ __forceinline__ Spot next() {
    Spot s{false, -1, 0, 0};
    if (kList) {
      const int at = 2 * (it.t0 + t++) + (first >> 6);
      const int blk = at < a.max_blocks ? __ldg(it.list + at) : -1;
      if (blk >= 0 && blk < it.nblk) s.token0 = blk * 64 + (first & 63);
      s.some = s.token0 >= 0 && s.token0 < it.len;
      if (s.some) s.some = tq_map_slot(map, a.Hkv, it.b, it.h, s.token0, s.row, s.slot);
      else return s;
    } else {
      s.token0 = token0;
      s.some = token0 < it.len;
      token0 += kTile;
      if (!s.some) return s;
      if (!map.table) {
        s.row = (long long)it.b * a.Hkv + it.h;
        s.slot = slot;
      } else {
        while (slot >= map.page_tokens) {
          slot -= map.page_tokens;
          ++page;
          row = -1;
        }
        if (row < 0) {
          row = __ldg(map.table + (long long)it.b * map.max_pages + page);
          if (row < 0 || row >= map.num_pages) row = map.num_pages;   // bad until the page ends
        }
        s.some = row < map.num_pages;
        s.row = (long long)row * a.Hkv + it.h;
        s.slot = slot;
      }
      slot += kTile;
    }
    if (!s.some && flag) atomicOr(&g_tq_flags, TQ_FLAG_PAGE);
    return s;
  }
};

// Loads of the next tile's codes: volatile, so that they are issued here and not where the values
// are used, a tile later (the compiler may sink a plain read-only load that far).
__device__ __forceinline__ uint4 load_early(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}
__device__ __forceinline__ float load_early(const float* p) {
  float x;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}

__device__ __forceinline__ uint32_t word(const uint4& x, int w) {
  return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w;
}

// NB planes of 16 bytes of one token.  Offsets within a row stay below 2^32 bytes (the host
// checks).  Where the warp has no token the registers keep what they hold: any code is a finite
// operand.
template <int NB>
__device__ __forceinline__ void load_planes(const uint8_t* base, const Spot& s, int slots, int lane,
                                            uint4 (&o)[NB]) {
  if (!s.some) return;
  const uint8_t* row = base + s.row * ((long long)NB * slots * 16);
#pragma unroll
  for (int p = 0; p < NB; ++p)
    o[p] = load_early(reinterpret_cast<const uint4*>(row + ((uint32_t)(p * slots + s.slot + lane) * 16u)));
}

// Level chunks 0–15 of a token from its NB planes (c is used up).  The loop over words is kept
// rolled, as the other expanders' are: the roles' code has to fit the instruction caches of an SM
// side by side.
template <int NB>
__device__ __forceinline__ void put_planes(const LevelBytes& t, uint4 (&c)[NB], unsigned char* dst) {
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    uint32_t x[NB];
#pragma unroll
    for (int p = 0; p < NB; ++p) {
      x[p] = c[p].x;
      c[p].x = c[p].y;
      c[p].y = c[p].z;
      c[p].z = c[p].w;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<uint4*>(dst + r * kLBO) = plane_chunk<NB>(t, x, r);
    dst += 4 * kLBO;
  }
}

// Hands a tile's operand part over: generic writes before the tensor core's reads.
__device__ __forceinline__ void hand_over(uint64_t* bar, int lane) {
  tq::fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The three kinds of expander warps.  Each returns false once a wait gave up.
template <int IB, bool kFine, bool kList>
__device__ __forceinline__ bool expand_keys(const RowsArgs& a, const CacheSide& side, Smem& sm,
                                            const Item& it, int first, int lane) {
  constexpr int kBufs = kFine ? 1 : 2;
  const int off = (first >> 3) * 128 + (lane >> 3) * 128 + (lane & 7) * 16;
  uint4 next[IB] = {};
  Cursor<kList> cur(a, side.kmap, it, first, lane == 0);
  load_planes<IB>(side.kidx, cur.next(), side.kslots, lane, next);
  for (int t = 0; t < it.tiles; ++t) {
    uint4 c[IB];
#pragma unroll
    for (int p = 0; p < IB; ++p) c[p] = next[p];
    if (t + 1 < it.tiles) load_planes<IB>(side.kidx, cur.next(), side.kslots, lane, next);
    const int st = t % kBufs;
    if (t >= kBufs && !warp_wait(&sm.kempty[st], (t / kBufs - 1) & 1)) return false;
    put_planes<IB>(a.kt, c, sm.k[st] + off);
    hand_over(&sm.kfull[st], lane);
  }
  return true;
}

template <bool kFine, bool kList>
__device__ __forceinline__ bool expand_signs(const RowsArgs& a, const CacheSide& side, Smem& sm,
                                             const Item& it, int first, int lane) {
  constexpr int kBufs = kFine ? 1 : 2;
  const int off = (first >> 3) * 128 + (lane >> 3) * 128 + (lane & 7) * 16;
  struct Raw {
    uint4 s;
    float xn, rn, vn;
    bool ok;
  };
  Cursor<kList> kcur(a, side.kmap, it, first, false), vcur(a, side.vmap, it, first, false);
  auto load = [&](Raw& o) {
    const Spot k = kcur.next();
    Spot v = k;
    if (!side.same_map) v = vcur.next();
    const bool some = k.some && v.some;
    o.ok = some && k.token0 + lane < it.len;
    if (!some) return;
    const long long at = k.row * side.kslots + k.slot + lane;
    o.s = load_early(reinterpret_cast<const uint4*>(side.ksgn) + at);
    o.xn = load_early(side.kxn + at);
    o.rn = load_early(side.krn + at);
    o.vn = load_early(side.vxn + v.row * side.vslots + v.slot + lane);
  };
  Raw next{};
  load(next);
  for (int t = 0; t < it.tiles; ++t) {
    const Raw c = next;
    if (t + 1 < it.tiles) load(next);
    const int st = t % kBufs, fs = t % kFacSlots;
    // the factors' slot is free: tile t − 4 was weighed before tile t − 2 was scored (kempty)
    if (t >= kBufs && !warp_wait(&sm.kempty[st], (t / kBufs - 1) & 1)) return false;
    const bool some = c.vn >= kTiny;
    sm.fac[fs][0][first + lane] = c.ok ? c.xn : 0.f;
    sm.fac[fs][1][first + lane] = !c.ok ? -INFINITY : some ? __log2f(c.vn) : c.vn < kTiny ? -60.f : c.vn;
    sm.fac[fs][2][first + lane] = !c.ok ? 0.f : some ? __fdividef(1.f, c.vn) : 1.152921504606847e18f;   // 2^60
    // ρ ≤ 1 or so for codes of any key (‖r‖ is the norm of a quantisation residual); a zero key
    // has both norms 0
    const float rho = c.ok && c.xn > 0.f ? __fdividef(c.rn, c.xn) * a.rho_scale : 0.f;
    const __half2 r2 = __float2half2_rn(rho);
    uint32_t neg = *reinterpret_cast<const uint32_t*>(&r2) ^ 0x80008000u;
    unsigned char* dst = sm.k[st] + 16 * kLBO + off;
    uint4 sg = c.s;
    // fine: ρ as two fp16 numbers, the second's 16 chunks behind the first's
#pragma unroll 1
    for (int w = 0; w < (kFine ? 8 : 4); ++w) {
      if (kFine && w == 4) {
        const __half2 l2 = __float2half2_rn(rho - __low2float(r2));
        neg = *reinterpret_cast<const uint32_t*>(&l2) ^ 0x80008000u;
        sg = c.s;
      }
      const uint32_t x = sg.x;
      sg.x = sg.y;
      sg.y = sg.z;
      sg.z = sg.w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 o;
        o.x = (shr(x, 4 * q + 0 - 15) & 0x80008000u) ^ neg;
        o.y = (shr(x, 4 * q + 1 - 15) & 0x80008000u) ^ neg;
        o.z = (shr(x, 4 * q + 2 - 15) & 0x80008000u) ^ neg;
        o.w = (shr(x, 4 * q + 3 - 15) & 0x80008000u) ^ neg;
        *reinterpret_cast<uint4*>(dst + q * kLBO) = o;
      }
      dst += 4 * kLBO;
    }
    hand_over(&sm.kfull[st], lane);
    if (lane == 0) mbar_arrive(&sm.ffull[fs]);
  }
  return true;
}

template <int VB, bool kList>
__device__ __forceinline__ bool expand_values(const RowsArgs& a, const CacheSide& side, Smem& sm,
                                              const Item& it, int first, int lane) {
  constexpr int kRegs = VB == 4 ? 4 : VB;
  const int off = (first >> 3) * 128 + (lane >> 3) * 128 + (lane & 7) * 16;
  uint4 next[kRegs] = {};
  float next_vn = 0.f;
  Cursor<kList> cur(a, side.vmap, it, first, lane == 0 && !side.same_map);
  auto load = [&]() {
    const Spot s = cur.next();
    if (s.some) next_vn = load_early(side.vxn + s.row * side.vslots + s.slot + lane);
    if constexpr (VB == 4) {
      if (!s.some) return;
      const uint4* p = reinterpret_cast<const uint4*>(side.vidx + s.row * ((long long)side.vslots * 64) +
                                                      (uint32_t)(s.slot + lane) * 64u);
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i] = load_early(p + i);
    } else {
      load_planes<VB>(side.vidx, s, side.vslots, lane, next);
    }
  };
  load();
  for (int t = 0; t < it.tiles; ++t) {
    uint4 c[kRegs];
#pragma unroll
    for (int p = 0; p < kRegs; ++p) c[p] = next[p];
    // a zero vector adds nothing, whatever its code (a norm that is NaN or past the length has
    // no weight to meet it)
    const bool some = next_vn >= kTiny;
    if (t + 1 < it.tiles) load();
    LevelBytes tb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tb.lo[i] = some ? a.vt.lo[i] : 0u;
      tb.hi[i] = some ? a.vt.hi[i] : 0u;
    }
    const int st = t & 1;
    if (t >= 2 && !warp_wait(&sm.vempty[st], ((t >> 1) - 1) & 1)) return false;
    unsigned char* dst = sm.v[st] + off;
    if constexpr (VB == 4) {
#pragma unroll 1
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = word(c[0], k);
          *reinterpret_cast<uint4*>(dst + k * kLBO) =
              levels8<true>(tb, x & 0x77777777u, ((x >> 3) & 0x11111111u) | 0x88888888u);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) c[k] = c[k + 1];
        dst += 4 * kLBO;
      }
    } else {
      put_planes<VB>(tb, c, dst);
    }
    hand_over(&sm.vfull[st], lane);
  }
  return true;
}

template <int IB, int VB, bool kFine, bool kList>
__device__ __forceinline__ bool expand(const RowsArgs& a, const CacheSide& side, Smem& sm,
                                       const Item& it, int warp, int lane) {
  const int first = 32 * (warp & 3);
  if (warp < kSignWarp) return expand_keys<IB, kFine, kList>(a, side, sm, it, first, lane);
  if (warp < kValueWarp) return expand_signs<kFine, kList>(a, side, sm, it, first, lane);
  return expand_values<VB, kList>(a, side, sm, it, first, lane);
}

// Valid length of a sequence: clamped to what the call was sized for, flagged if longer.
__device__ __forceinline__ int clamp_len(int len, int most) {
  if (len > most) {
    atomicOr(&g_tq_flags, TQ_FLAG_LEN_OVERFLOW);
    return most;
  }
  return len < 0 ? 0 : len;
}

#ifdef TQ_ROWS_TREE
// Which drafted tokens a row attends: token t is the item's token j0 + t of them, the ones before them
// (the history) are all attended, and those past the length have no weight anyway.
struct RowMask {
  unsigned long long seen;
  int j0;

  // Bit i: whether the row attends token t + i, i < 16.
  __device__ __forceinline__ uint32_t at(int t) const {
    const int j = j0 + t;
    if (j <= -16) return 0xffffu;
    if (j < 0) return (uint32_t)(seen << -j) | ((1u << -j) - 1u);
    return j < TQ_TREE_NODES ? (uint32_t)(seen >> j) : 0u;
  }
};
#endif

// What a softmax thread ends with.
struct Stats {
  float m, l;
  bool ok;
};

#ifdef TQ_ROWS_TREE

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The softmax of every tile by 8 warps: thread (lane group wl, half hf) of TMEM lane 32·wl + lane, rows
// in one, two or four lane groups (reps) as below.  A thread's scores go kN at a time, 32 where it has
// as many, so that an item of at most 64 rows keeps them in registers between the passes and one of
// 128 rows goes twice: a pass waits for TMEM and shared memory once for each.
template <bool kFine, int kN>
__device__ __forceinline__ Stats softmax_tiles(Smem& sm, int tiles, int reps, int wl, int hf, int lane,
                                               float f, const RowMask& mask) {
  const int rep = wl / (4 / reps), groups = 4 / reps;       // groups of 16 tokens per thread
  const int group0 = (2 * rep + hf) * groups;
  const uint32_t lane_base = (uint32_t)(32 * wl) << 16;
  const int r = 32 * wl + lane;
  const tq::f32x2 f2 = tq::pack2(f, f);
  Stats z{-INFINITY, 0.f, true};
  bool ok = true;
  auto wait = [&](uint64_t* bar, unsigned parity) { return ok = ok && warp_wait(bar, parity); };
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    const int buf = kFine ? 0 : t & 1;
    wait(&sm.ffull[t % kFacSlots], (t / kFacSlots) & 1);
    wait(&sm.sfull[buf], (kFine ? t : t >> 1) & 1);
    tc_after();
    const uint32_t dcol = lane_base + kDCol + 128 * buf + 16 * group0;
    const float* fx = sm.fac[t % kFacSlots][0] + 16 * group0;
    float mt = -INFINITY;
    uint32_t d[kN];      // the last scores stay here, the others go back to TMEM
#pragma unroll 1
    for (int c = 0;; c += kN) {
      tmem_load<kN>(dcol + c, d);
      tq::tmem_wait_ld();
      float* e = reinterpret_cast<float*>(d);
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 xn = *reinterpret_cast<const float4*>(fx + c + i);
        const float4 lv = *reinterpret_cast<const float4*>(fx + kTile + c + i);
        const float2 x = tq::unpack2(tq::fma2(tq::mul2(tq::pack2(e[i], e[i + 1]), f2),
                                              tq::pack2(xn.x, xn.y), tq::pack2(lv.x, lv.y)));
        const float2 y = tq::unpack2(tq::fma2(tq::mul2(tq::pack2(e[i + 2], e[i + 3]), f2),
                                              tq::pack2(xn.z, xn.w), tq::pack2(lv.z, lv.w)));
        e[i] = x.x; e[i + 1] = x.y; e[i + 2] = y.x; e[i + 3] = y.y;
      }
      // (uniform: the same tokens for all rows of an item)
      const int token = t * kTile + 16 * group0 + c;
      if (mask.j0 + token > -kN) {
#pragma unroll
        for (int g = 0; g < kN; g += 16) {
          const uint32_t seen = mask.at(token + g);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (!(seen >> k & 1u)) e[g + k] = -INFINITY;
        }
      }
      float m0 = e[0], m1 = e[1];
#pragma unroll
      for (int k = 2; k < kN - 2; k += 4) {
        m0 = max3(m0, e[k], e[k + 2]);
        m1 = max3(m1, e[k + 1], e[k + 3]);
      }
      mt = max3(mt, max3(m0, e[kN - 2], m1), e[kN - 1]);
      if (c + kN >= 16 * groups) break;
      tmem_store<kN>(dcol + c, d);
    }
    sm.tmax[t & 1][hf][r] = mt;
    // A wait that gave up ends both halves' loops here, together (neither then waits for the
    // other)
    if (!tq::named_sync_and(1 + wl, 64, ok)) {
      z.ok = false;
      return z;
    }
    mt = fmaxf(mt, sm.tmax[t & 1][hf ^ 1][r]);
    const float m_new = mt - z.m > kGrow + kLift ? mt - kLift : z.m;
    if (t > 0 && __any_sync(0xffffffffu, m_new != z.m)) {
      // as below: O follows the reference, once O += W(t − 1)·V(t − 1) is done
      wait(&sm.vempty[(t - 1) & 1], ((t - 1) >> 1) & 1);
      tc_after();
      const float corr = z.m == -INFINITY ? 0.f : ex2(z.m - m_new);
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        uint32_t o[16];
        const uint32_t at = lane_base + kOCol + 64 * hf + c;
        tmem_load<16>(at, o);
        tq::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
        tmem_store<16>(at, o);
      }
      z.l *= corr;
    }
    z.m = m_new;
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const tq::f32x2 ref2 = tq::pack2(-ref, -ref);
    tq::f32x2 l2 = tq::pack2(0.f, 0.f), l3 = l2;
    tq::tmem_wait_st();
#pragma unroll 1
    for (int c = 16 * groups - kN;; c -= kN) {
#pragma unroll
      for (int g = 0; g < kN; g += 16) {
        uint32_t w[kFine ? 16 : 8];      // fine: then what the rounding left
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 iv = *reinterpret_cast<const float4*>(fx + 2 * kTile + c + g + i);
          const float* e = reinterpret_cast<const float*>(d) + g + i;
          const float2 x = tq::unpack2(tq::add2(tq::pack2(e[0], e[1]), ref2));
          const float2 y = tq::unpack2(tq::add2(tq::pack2(e[2], e[3]), ref2));
          const float w0 = ex2(x.x), w1 = ex2(x.y), w2 = ex2(y.x), w3 = ex2(y.y);
          l2 = tq::fma2(tq::pack2(w0, w1), tq::pack2(iv.x, iv.y), l2);
          l3 = tq::fma2(tq::pack2(w2, w3), tq::pack2(iv.z, iv.w), l3);
          const __half2 p0 = __floats2half2_rn(w0, w1), p1 = __floats2half2_rn(w2, w3);
          w[i / 2] = *reinterpret_cast<const uint32_t*>(&p0);
          w[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&p1);
          if constexpr (kFine) {
            const float2 h0 = __half22float2(p0), h1 = __half22float2(p1);
            const __half2 r0 = __floats2half2_rn(w0 - h0.x, w1 - h0.y);
            const __half2 r1 = __floats2half2_rn(w2 - h1.x, w3 - h1.y);
            w[8 + i / 2] = *reinterpret_cast<const uint32_t*>(&r0);
            w[8 + i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&r1);
          }
        }
        tmem_store<kFine ? 16 : 8>(dcol + c + g, w);
      }
      if (c == 0) break;
      tmem_load<kN>(dcol + c - kN, d);
      tq::tmem_wait_ld();
    }
    const float2 lp = tq::unpack2(tq::add2(l2, l3));
    z.l += lp.x + lp.y;
    if (reps > 1) {
      // the other replicas' groups, every other one by each half
      const uint32_t none[kFine ? 16 : 8] = {};
#pragma unroll 1
      for (int g = hf; g < 8; g += 2)
        if (g / (2 * groups) != rep) tmem_store<kFine ? 16 : 8>(lane_base + kDCol + 128 * buf + 16 * g, none);
    }
    tq::tmem_wait_st();
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.pfull[buf]);
  }
  wait(&sm.vempty[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);
  z.ok = ok;
  return z;
}

#else

// The softmax of every tile by 8 warps: thread (lane group wl, half hf) of TMEM lane 32·wl + lane.
// An item of at most 32 (64) rows holds each row in 4 (2) lane groups, the `reps` replicas of a
// row taking a quarter (half) of a tile's tokens each, so that a thread has 16 (32) scores
// instead of 64: with few rows a tile's time is this chain's.  Weights of the tokens that a
// replica leaves to the others are 0, and its O and l are those of its tokens.
//
// Both passes over a thread's scores go 16 at a time in a rolled loop, with the scores in TMEM
// between them: the roles' code has to fit the instruction caches of an SM side by side
// (unrolled, this loop alone took a third of the time of 112 rows).  The weights of a group of
// 16 tokens are stored over the first half of its scores, which no other thread reads.
template <bool kFine>
__device__ __forceinline__ Stats softmax_tiles(Smem& sm, int tiles, int reps, int wl, int hf, int lane,
                                               float f) {
  const int rep = wl / (4 / reps), groups = 4 / reps;       // groups of 16 tokens per thread
  const int group0 = (2 * rep + hf) * groups;
  const uint32_t lane_base = (uint32_t)(32 * wl) << 16;
  const int r = 32 * wl + lane;
  const tq::f32x2 f2 = tq::pack2(f, f);
  Stats z{-INFINITY, 0.f, true};
  bool ok = true;
  auto wait = [&](uint64_t* bar, unsigned parity) { return ok = ok && warp_wait(bar, parity); };
  for (int t = 0; t < tiles; ++t) {
    const int buf = kFine ? 0 : t & 1;
    wait(&sm.ffull[t % kFacSlots], (t / kFacSlots) & 1);
    wait(&sm.sfull[buf], (kFine ? t : t >> 1) & 1);
    tc_after();
    const uint32_t dcol = lane_base + kDCol + 128 * buf + 16 * group0;
    const float* fx = sm.fac[t % kFacSlots][0] + 16 * group0;
    float mt = -INFINITY;
    uint32_t d[16];      // the last group's scores stay here, the others go back to TMEM
#pragma unroll 1
    for (int c = 0;; c += 16) {
      tmem_load<16>(dcol + c, d);
      tq::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 xn = *reinterpret_cast<const float4*>(fx + c + i);
        const float4 lv = *reinterpret_cast<const float4*>(fx + kTile + c + i);
        float* e = reinterpret_cast<float*>(d) + i;
        const float2 x = tq::unpack2(tq::fma2(tq::mul2(tq::pack2(e[0], e[1]), f2),
                                              tq::pack2(xn.x, xn.y), tq::pack2(lv.x, lv.y)));
        const float2 y = tq::unpack2(tq::fma2(tq::mul2(tq::pack2(e[2], e[3]), f2),
                                              tq::pack2(xn.z, xn.w), tq::pack2(lv.z, lv.w)));
        e[0] = x.x; e[1] = x.y; e[2] = y.x; e[3] = y.y;
        mt = fmaxf(mt, fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y)));
      }
      if (c + 16 >= 16 * groups) break;
      tmem_store<16>(dcol + c, d);
    }
    sm.tmax[t & 1][hf][r] = mt;
    // A wait that gave up ends both halves' loops here, together (neither then waits for the
    // other)
    if (!tq::named_sync_and(1 + wl, 64, ok)) {
      z.ok = false;
      return z;
    }
    mt = fmaxf(mt, sm.tmax[t & 1][hf ^ 1][r]);
    // the reference, kLift below the maximum it was taken from (differences of near numbers are
    // exact, so that a weight stays below 2^(kLift + kGrow) however large the scores are)
    const float m_new = mt - z.m > kGrow + kLift ? mt - kLift : z.m;
    if (t > 0 && __any_sync(0xffffffffu, m_new != z.m)) {
      // O (this half of its columns) follows the reference, once O += W(t − 1)·V(t − 1) is
      // done (vempty).  Its barrier is that of every other tile: the phase before, tile t − 3's,
      // ended before tile t was scored, so the parity says which tile is meant
      wait(&sm.vempty[(t - 1) & 1], ((t - 1) >> 1) & 1);
      tc_after();
      const float corr = z.m == -INFINITY ? 0.f : ex2(z.m - m_new);
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        uint32_t o[16];
        const uint32_t at = lane_base + kOCol + 64 * hf + c;
        tmem_load<16>(at, o);
        tq::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
        tmem_store<16>(at, o);
      }
      z.l *= corr;
    }
    z.m = m_new;
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const tq::f32x2 ref2 = tq::pack2(-ref, -ref);
    tq::f32x2 l2 = tq::pack2(0.f, 0.f);
    if (groups > 1) tq::tmem_wait_st();
#pragma unroll 1
    for (int c = 16 * groups - 16;; c -= 16) {
      uint32_t w[kFine ? 16 : 8];      // fine: then what the rounding left
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 iv = *reinterpret_cast<const float4*>(fx + 2 * kTile + c + i);
        const float* e = reinterpret_cast<const float*>(d) + i;
        const float2 x = tq::unpack2(tq::add2(tq::pack2(e[0], e[1]), ref2));
        const float2 y = tq::unpack2(tq::add2(tq::pack2(e[2], e[3]), ref2));
        const float w0 = ex2(x.x), w1 = ex2(x.y), w2 = ex2(y.x), w3 = ex2(y.y);
        l2 = tq::fma2(tq::pack2(w0, w1), tq::pack2(iv.x, iv.y), l2);
        l2 = tq::fma2(tq::pack2(w2, w3), tq::pack2(iv.z, iv.w), l2);
        const __half2 p0 = __floats2half2_rn(w0, w1), p1 = __floats2half2_rn(w2, w3);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&p0);
        w[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&p1);
        if constexpr (kFine) {
          const float2 h0 = __half22float2(p0), h1 = __half22float2(p1);
          const __half2 r0 = __floats2half2_rn(w0 - h0.x, w1 - h0.y);
          const __half2 r1 = __floats2half2_rn(w2 - h1.x, w3 - h1.y);
          w[8 + i / 2] = *reinterpret_cast<const uint32_t*>(&r0);
          w[8 + i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&r1);
        }
      }
      tmem_store<kFine ? 16 : 8>(dcol + c, w);
      if (c == 0) break;
      tmem_load<16>(dcol + c - 16, d);
      tq::tmem_wait_ld();
    }
    const float2 lp = tq::unpack2(l2);
    z.l += lp.x + lp.y;
    if (reps > 1) {
      // the other replicas' groups, every other one by each half
      const uint32_t none[kFine ? 16 : 8] = {};
#pragma unroll 1
      for (int g = hf; g < 8; g += 2)
        if (g / (2 * groups) != rep) tmem_store<kFine ? 16 : 8>(lane_base + kDCol + 128 * buf + 16 * g, none);
    }
    tq::tmem_wait_st();
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.pfull[buf]);
    // tile t + 2 is scored after both halves have arrived here: until then this tile's tmax and
    // factors may still be read (tile t + 1 may be scored already)
  }
  wait(&sm.vempty[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);
  z.ok = ok;
  return z;
}

#endif

#ifdef TQ_ROWS_TREE
// An item's row operands into TMEM (halves hf of a row's positions, all reads in flight at once) and its
// record out of it.  Functions of their own, so that the registers they take are not the loops'.
template <bool kFine>
__device__ __noinline__ void tree_rows_in(const uint4* row, bool there, uint32_t lane_base, int hf) {
#pragma unroll 1
  for (int c = 0; c < (kFine ? 2 : 1); ++c) {
    uint32_t q[64];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint4 x = there ? row[32 * c + 16 * hf + i] : make_uint4(0, 0, 0, 0);
      q[4 * i] = x.x; q[4 * i + 1] = x.y; q[4 * i + 2] = x.z; q[4 * i + 3] = x.w;
    }
    const uint32_t at = lane_base + (c ? kQLowCol : kQCol) + 64 * hf;
    __syncwarp();         // (lanes without a row read nothing)
    tmem_store<32>(at, q);
    tmem_store<32>(at + 32, q + 32);
  }
  tq::tmem_wait_st();
}

__device__ __noinline__ void tree_record(float* part, float* recs, int nodes_row0, int G, int Hq, int rows, int reps,
                                         int wl, int hf, int lane, float m_mine, float l_mine) {
  // lanes' parts through shared memory [128 lanes][kRecFloats] (the operands are done with)
  float* mine = part + (32 * wl + lane) * kRecFloats;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float o[32];
    tmem_load<32>(((uint32_t)(32 * wl) << 16) + kOCol + 64 * hf + 32 * c, reinterpret_cast<uint32_t*>(o));
    tq::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(mine + 64 * hf + 32 * c + 4 * i) =
          make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
  *reinterpret_cast<float2*>(mine + 128 + 2 * hf) = make_float2(m_mine, l_mine);      // (one reference for both halves)
  tq::named_sync(5, 256);
  // replicas of a row added up with their log-sum-exp weights, four rows of a warp side by side
  const int per = kTile / reps;
  for (int row0 = wl + 4 * hf; row0 < rows; row0 += 32) {
    const float* p[4];
    float m[4], l[4] = {};
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = part + min(row0 + 8 * i, rows - 1) * kRecFloats;
      m[i] = -INFINITY;
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = 0; k < reps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], p[i][k * per * kRecFloats + 128]);
    for (int k = 0; k < reps; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 st = *reinterpret_cast<const float4*>(p[i] + k * per * kRecFloats + 128);   // m, l of both halves
        const float w = st.x == -INFINITY ? 0.f : ex2(st.x - m[i]);
        const float4 x = *reinterpret_cast<const float4*>(p[i] + k * per * kRecFloats + 4 * lane);
        acc[i].x = fmaf(w, x.x, acc[i].x);
        acc[i].y = fmaf(w, x.y, acc[i].y);
        acc[i].z = fmaf(w, x.z, acc[i].z);
        acc[i].w = fmaf(w, x.w, acc[i].w);
        l[i] = fmaf(w, st.y + st.w, l[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row0 + 8 * i >= rows) break;
      const int nr = nodes_row0 + row0 + 8 * i;
      float* rec = recs + ((long long)(nr / G) * Hq + nr % G) * kRecFloats;
      *reinterpret_cast<float4*>(rec + 4 * lane) = acc[i];
      if (lane == 0) *reinterpret_cast<float2*>(rec + 128) = make_float2(m[i], l[i]);
    }
  }
}
#endif

// Lengths, lists, block tables and codes are read before this kernel's wait: it starts only when all
// of rows_prep_kernel is past its own wait, so whatever ran before that has ended and been flushed.
template <int IB, int VB, bool kFine>
__global__ void __launch_bounds__(kThreads, 1) rows_attn_kernel(const __grid_constant__ RowsArgs a) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  using R = Regs<kFine>;
  static_assert(256 * R::softmax + 384 * R::expand + 128 * R::issue <= kThreads * kRegsLaunch, "register split");

  // ---- the item: prefix items first (they are the long ones)
  int item = blockIdx.x;
  const int npre = kTree ? 0 : a.pre_splits * a.Hkv * a.row_tiles;
  const bool pre = item < npre;
  int split, h, b = 0, rt = 0;
  if (pre) {
    rt = item % a.row_tiles;
    h = item / a.row_tiles % a.Hkv;
    split = item / (a.row_tiles * a.Hkv);
  } else {
#ifdef TQ_ROWS_TREE
    // one sequence's items side by side (by split first: 233 for 228 us in 32 sequences of 4096 to 16384)
    rt = item % a.row_tiles;
    split = item / a.row_tiles % a.own_splits;
    h = item / (a.row_tiles * a.own_splits) % a.Hkv;
    b = item / (a.row_tiles * a.own_splits * a.Hkv);
    if (a.order) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      b = min(max(*static_cast<const volatile int*>(a.order + b), 0), a.B - 1);
    }
#else
    item -= npre;
    h = item % a.Hkv;
    b = item / a.Hkv % a.B;
    split = item / (a.Hkv * a.B);
#endif
  }
#ifdef TQ_ROWS_TREE
  const int rows = min(kTile, a.nodes * a.G - rt * kTile);
  const int hist = clamp_len(a.seq_lens[b], a.max_len - a.nodes), len = hist + a.nodes;
  const long long nrows = (long long)a.B * a.nodes * a.Hq;
#else
  const int rows = pre ? min(kTile, a.B * a.G - rt * kTile) : a.G;
  const int len = pre ? clamp_len(*a.pre_len, a.max_pre) : clamp_len(a.seq_lens[b], a.max_len);
  const long long nrows = (long long)a.B * a.Hq;
#endif
  const int splits = pre ? a.pre_splits : a.own_splits;
  const int* list = a.list ? a.list + ((long long)b * a.Hkv + h) * a.max_blocks : nullptr;
  const int nblk = (len + 63) / 64;
  const int total = list ? (a.max_blocks + 1) / 2 : (len + kTile - 1) / kTile;
  const int t0 = (int)((long long)total * split / splits);
  int tiles = (int)((long long)total * (split + 1) / splits) - t0;
  if (list) {
    // leave out the tiles behind the last block of this run that is there
    if (tid == 0) sm.tiles = 0;
    __syncthreads();
    int last = 0;
    for (int i = tid; i < 2 * tiles; i += kThreads) {
      const int at = 2 * t0 + i;
      const int blk = at < a.max_blocks ? list[at] : -1;
      if (blk >= 0 && blk < nblk) last = i / 2 + 1;
    }
    if (last) atomicMax(&sm.tiles, last);
    __syncthreads();
    tiles = sm.tiles;
  }
  const int rec_split = pre ? split : a.pre_splits + split;
  auto qrow_of = [&](int r) -> long long {   // query row (b·Hq + head) of item row r
#ifdef TQ_ROWS_TREE
    const int nr = rt * kTile + r;
    return ((long long)b * a.nodes + nr / a.G) * a.Hq + h * a.G + nr % a.G;
#endif
    if (!pre) return (long long)b * a.Hq + h * a.G + r;
    const int rr = rt * kTile + r;
    return (long long)(rr / a.G) * a.Hq + h * a.G + rr % a.G;
  };
  if (tiles <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < rows) {
      float* rec = a.rec + (rec_split * nrows + qrow_of(tid)) * kRecFloats;
      rec[128] = -INFINITY;
      rec[129] = 0.f;
    }
    return;
  }
  const int reps = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;   // lane groups that hold a row

  if (warp == kIssueWarp) tq::tmem_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tq::mbar_init(&sm.kfull[i], 8);
      tq::mbar_init(&sm.vfull[i], 4);
      tq::mbar_init(&sm.kempty[i], 1);
      tq::mbar_init(&sm.vempty[i], 1);
      tq::mbar_init(&sm.sfull[i], 1);
      tq::mbar_init(&sm.pfull[i], 8);
    }
    for (int i = 0; i < kFacSlots; ++i) tq::mbar_init(&sm.ffull[i], 4);
    tq::mbar_init(&sm.qfull, 8);
    tq::mbar_init(&sm.drain, 1);
    tq::mbar_init_fence();
  }
  tc_before();
  __syncthreads();
  tc_after();
  // all 512 columns were asked for, so they begin at address 0: addresses are constants
  bool ok = sm.tmem == 0;   // false once a bounded wait gave up: every role then leaves its loop
  auto wait = [&](uint64_t* bar, unsigned parity) {
    return ok = ok && warp_wait(bar, parity);
  };

  if (warp < kKeyWarp) {
    // ================================================================ softmax
    if (R::kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::softmax));
    const int wl = warp & 3, hf = warp >> 2;
    const int per = kTile / reps;              // rows per replica
    const int r = (32 * wl + lane) & (per - 1);
    const uint32_t lane_base = (uint32_t)(32 * wl) << 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long qr = r < rows ? qrow_of(r) : 0;
    // (plain loads: the kernel before writes the operands while this one runs, so they must not go
    // through the read-only path, which the wait does not order)
    const float f = r < rows ? a.qf[qr] : 0.f;
#ifdef TQ_ROWS_TREE
    tree_rows_in<kFine>(a.qop + qr * (kFine ? 64 : 32), r < rows, lane_base, hf);
#else
    // (fine: the row's second 512 bytes are what the first ones' rounding left)
#pragma unroll 1
    for (int c = 0; c < (kFine ? 4 : 2); ++c) {
      uint32_t q[32];
      const uint4* src = a.qop + qr * (kFine ? 64 : 32) + 32 * (c >> 1) + 16 * hf + 8 * (c & 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = r < rows ? src[i] : make_uint4(0, 0, 0, 0);
        q[4 * i] = x.x; q[4 * i + 1] = x.y; q[4 * i + 2] = x.z; q[4 * i + 3] = x.w;
      }
      tmem_store<32>(lane_base + (c >> 1 ? kQLowCol : kQCol) + 64 * hf + 32 * (c & 1), q);
    }
    tq::tmem_wait_st();
#endif
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.qfull);
#ifdef TQ_ROWS_TREE
    RowMask mask{0, t0 * kTile - hist};
    if (r < rows) mask.seen = a.tree[b * a.tree_b + (rt * kTile + r) / a.G];
    const Stats z = reps < 4 ? softmax_tiles<kFine, 32>(sm, tiles, reps, wl, hf, lane, f, mask)
                             : softmax_tiles<kFine, 16>(sm, tiles, reps, wl, hf, lane, f, mask);
#else
    const Stats z = softmax_tiles<kFine>(sm, tiles, reps, wl, hf, lane, f);
#endif
    // ---- the item's record: lanes' parts through shared memory (the operands are done with),
    // replicas of a row added up with their log-sum-exp weights
    ok = ok && tq::named_sync_and(5, 256, z.ok);
    if (ok) {
      tc_after();
#ifdef TQ_ROWS_TREE
      float* recs = a.rec + (rec_split * nrows + (long long)b * a.nodes * a.Hq + h * a.G) * kRecFloats;
      tree_record(reinterpret_cast<float*>(sm.k[0]), recs, rt * kTile, a.G, a.Hq, rows, reps, wl, hf, lane, z.m, z.l);
#else
      float* part = reinterpret_cast<float*>(sm.k[0]);      // [128 lanes][kRecFloats]
      float* mine = part + (32 * wl + lane) * kRecFloats;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float o[32];
        tmem_load<32>(lane_base + kOCol + 64 * hf + 32 * c, reinterpret_cast<uint32_t*>(o));
        tq::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(mine + 64 * hf + 32 * c + 4 * i) =
              make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      mine[128 + 2 * hf] = z.m;       // both halves have the same reference
      mine[129 + 2 * hf] = z.l;
      tq::named_sync(5, 256);
      for (int row = warp; row < rows; row += 8) {
        float* rec = a.rec + (rec_split * nrows + qrow_of(row)) * kRecFloats;
        float m = -INFINITY;
        for (int k = 0; k < reps; ++k) m = fmaxf(m, part[(k * per + row) * kRecFloats + 128]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        for (int k = 0; k < reps; ++k) {
          const float* p = part + (k * per + row) * kRecFloats;
          const float w = p[128] == -INFINITY ? 0.f : ex2(p[128] - m);
          const float4 x = *reinterpret_cast<const float4*>(p + 4 * lane);
          acc.x = fmaf(w, x.x, acc.x);
          acc.y = fmaf(w, x.y, acc.y);
          acc.z = fmaf(w, x.z, acc.z);
          acc.w = fmaf(w, x.w, acc.w);
          l = fmaf(w, p[129] + p[131], l);
        }
        *reinterpret_cast<float4*>(rec + 4 * lane) = acc;
        if (lane == 0) *reinterpret_cast<float2*>(rec + 128) = make_float2(m, l);
      }
#endif
    }
  } else if (warp < kIssueWarp) {
    // ================================================================ expanders
    if (R::kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::expand));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::expand));
    const Item it{t0, tiles, len, nblk, b, h, list};
    if (pre) ok = expand<IB, VB, kFine, false>(a, a.pre, sm, it, warp, lane);
    else if (list) ok = expand<IB, VB, kFine, true>(a, a.own, sm, it, warp, lane);
    else ok = expand<IB, VB, kFine, false>(a, a.own, sm, it, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::issue));
    // ================================================================ MMA issuer
    if (warp == kIssueWarp) {
    constexpr uint32_t kIdescS = tq::idesc_f16(128, 128);
    constexpr uint32_t kIdescO = kIdescS | (1u << 16);   // B (values) is N-major
    // Operands are uniform values (one base descriptor each, constant steps), so that an issue
    // is one instruction and the queue of the tensor core does not run dry.
    const uint64_t kdesc = tq::smem_desc(s32(sm.k[0]), kLBO, 128);
    const uint64_t vdesc = tq::smem_desc(s32(sm.v[0]), 128, kLBO);
    constexpr int kBufs = kFine ? 1 : 2;
    auto weigh = [&](int t) {   // O += W(t)·V(t)
      const int st = t & 1, buf = t % kBufs;
      if (!wait(&sm.vfull[st], (t >> 1) & 1) || !wait(&sm.pfull[buf], (t / kBufs) & 1)) return;
      tc_after();
      if (elect_one()) {
        const uint64_t v = vdesc + st * (kVBytes >> 4);
        const uint32_t w = kDCol + 128 * buf;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tq::mma_ts(kOCol, w + 16 * ks, v + ks * (256 >> 4), kIdescO, t > 0 || ks > 0);
        if (kFine) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tq::mma_ts(kOCol, w + 16 * ks + 8, v + ks * (256 >> 4), kIdescO, 1u);
        }
        tq::mma_commit(&sm.vempty[st]);
      }
      __syncwarp();
    };
    wait(&sm.qfull, 0);
    for (int t = 0; t < tiles && ok; ++t) {
      const int st = t % kBufs;
      if (!wait(&sm.kfull[st], (t / kBufs) & 1)) break;
      tc_after();
      if (elect_one()) {
        const uint64_t k = kdesc + st * (kKBytes >> 4);
        const uint32_t d = kDCol + 128 * st;
#pragma unroll
        for (int ks = 0; ks < 16; ++ks)
          tq::mma_ts(d, kQCol + 8 * ks, k + ks * (2 * kLBO >> 4), kIdescS, ks > 0);
        if (kFine) {   // the rests of y and z, and z with the rest of ρ
#pragma unroll
          for (int ks = 0; ks < 16; ++ks)
            tq::mma_ts(d, kQLowCol + 8 * ks, k + ks * (2 * kLBO >> 4), kIdescS, 1u);
#pragma unroll
          for (int ks = 8; ks < 16; ++ks)
            tq::mma_ts(d, kQCol + 8 * ks, k + (ks + 8) * (2 * kLBO >> 4), kIdescS, 1u);
        }
        tq::mma_commit(&sm.sfull[st]);
        tq::mma_commit(&sm.kempty[st]);
      }
      __syncwarp();
      if (kFine) weigh(t);
      else if (t > 0) weigh(t - 1);
    }
    if (!kFine && ok) weigh(tiles - 1);
    // whatever was issued has ended before the tensor memory is given back
    if (elect_one()) tq::mma_commit(&sm.drain);
    __syncwarp();
    if (!tq::mbar_wait(&sm.drain, 0)) ok = false;
    }
  }
  if (!ok && lane == 0) atomicOr(&g_tq_flags, TQ_FLAG_TIMEOUT);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kIssueWarp) tq::tmem_dealloc(sm.tmem, 512);
}

// ---------------------------------------------------------------- row operands
// y = Π q and z = S q of kRows query rows per CTA, in the operand's order, scaled by a power of
// two of the row so that fp16 holds them.  1024 threads: 256 outputs × 4 quarters of k.
constexpr int kPrepThreads = 1024;
template <int kRows>
__global__ void __launch_bounds__(kPrepThreads)
rows_prep_kernel(const void* q, int q_dtype, int nrows, int fine, const float* __restrict__ piT,
                 const float* __restrict__ sT, float factor, __half* qop, float* qf) {
  __shared__ float qs[kRows][TQ_D];
  __shared__ float part[4][kRows][256];
  __shared__ float scale[kRows];
  const int tid = threadIdx.x, row0 = blockIdx.x * kRows;
  const int p = tid & 255, kq = tid >> 8;
  // position p < 128: y at plane_coord(p); else z at sign_coord(p − 128)
  const float* mat = (p < 128 ? piT + plane_coord(p) : sT + sign_coord(p - 128)) + 32 * kq * TQ_D;
  float w[32];   // the codec's matrices do not depend on the launch before
#pragma unroll
  for (int k = 0; k < 32; ++k) w[k] = __ldg(mat + k * TQ_D);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // not before the wait: rows_attn_kernel reads lengths and codes before it waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i < kRows * TQ_D; i += kPrepThreads) {
    const int r = i / TQ_D;
    qs[r][i % TQ_D] = row0 + r < nrows ? load_elem(q, q_dtype, (long long)row0 * TQ_D + i) : 0.f;
  }
  __syncthreads();
  if (tid < 32 * kRows) {
    const int r = tid >> 5, lane = tid & 31;
    float m = 0.f;
    for (int j = lane; j < TQ_D; j += 32) m = fmaxf(m, fabsf(qs[r][j]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) {
      // ‖q‖ ≤ √128·max|q_j| < 2^(e + 4) with max|q_j| < 2^e
      int e = 0;
      if (m > 0.f && m < INFINITY) frexpf(m, &e);
      e = min(max(e + 4, -110), 120);
      scale[r] = ldexpf(1.f, -e);
      if (row0 + r < nrows) qf[row0 + r] = ldexpf(factor, e);
    }
  }
#pragma unroll 1      // (rolled: short kernels wait for their instructions)
  for (int r = 0; r < kRows; ++r) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&qs[r][32 * kq + k]);
      s = fmaf(w[k], x.x, s);
      s = fmaf(w[k + 1], x.y, s);
      s = fmaf(w[k + 2], x.z, s);
      s = fmaf(w[k + 3], x.w, s);
    }
    part[kq][r][p] = s;
  }
  __syncthreads();
  for (int i = tid; i < kRows * 256; i += kPrepThreads) {
    const int r = i >> 8, c = i & 255;
    if (row0 + r >= nrows) continue;
    const float s = (part[0][r][c] + part[1][r][c]) + (part[2][r][c] + part[3][r][c]);
    const float x = s * scale[r] * (c < 128 ? kAlpha : kBeta);
    const __half h = __float2half_rn(x);
    __half* row = qop + (long long)(row0 + r) * (fine ? 512 : 256) + c;
    row[0] = h;
    if (fine) row[256] = __float2half_rn(x - __half2float(h));
  }
}

// ---------------------------------------------------------------- merge
// Rows' records added up with their log-sum-exp weights, then out = Πᵀ·acc / l.  kRows rows per
// CTA of 16 warps: a warp per (row, share of its records), eight 512-byte reads in flight; then
// 128 columns × 4 quarters of k, the rows sharing the reads of Π.  Bound by the latency of three
// dependent steps (statistics, records, Π) and, for many rows, by reading the records from L2.
constexpr int kMergeThreads = 512;
constexpr int kMaxRecs = 512;           // records of a row (make_plan keeps to it)
template <int kRows>
__global__ void __launch_bounds__(kMergeThreads)
rows_merge_kernel(const float* rec, int nrec, int nrows, const float* __restrict__ pi, int nibbles,
                  float unscale, void* out, int out_dtype) {
  constexpr int kShares = 16 / kRows;
  __shared__ float acc[16][TQ_D];
  __shared__ float sum[kRows][TQ_D];
  __shared__ float weight[kRows][kMaxRecs];
  __shared__ float total[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = tid & 127, kq = tid >> 7, row0 = blockIdx.x * kRows;
  float w[32];   // Π does not depend on the launch before
#pragma unroll
  for (int k = 0; k < 32; ++k) w[k] = __ldg(pi + (32 * kq + k) * TQ_D + j);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long stride = (long long)nrows * kRecFloats;
  if (warp < kRows) {
    const int row = min(row0 + warp, nrows - 1);
    const float* p = rec + (long long)row * kRecFloats + 128;
    float m = -INFINITY;
    for (int s = lane; s < nrec; s += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(p + s * stride);
      // an empty record weighs nothing; a NaN sum (a NaN query) makes the row NaN
      weight[warp][s] = ml.y != ml.y ? ml.y : ml.y != 0.f ? ml.x : -INFINITY;
      if (ml.y != 0.f) m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int s = lane; s < nrec; s += 32) {
      const float ls = p[s * stride + 1], ms = weight[warp][s];
      const float ws = ms == -INFINITY ? 0.f : ex2(ms - m);
      weight[warp][s] = ws;
      if (ws != 0.f) l = fmaf(ls, ws, l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) total[warp] = l;
  }
  __syncthreads();
  {
    const int r = warp / kShares, share = warp % kShares;
    const float* p = rec + (long long)min(row0 + r, nrows - 1) * kRecFloats + 4 * lane;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = share; i0 < nrec; i0 += 8 * kShares) {
      float4 x[8];
      float ws[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * kShares;
        ws[k] = i < nrec ? weight[r][i] : 0.f;
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ws[k] != 0.f) x[k] = *reinterpret_cast<const float4*>(p + i * stride);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s.x = fmaf(x[k].x, ws[k], s.x);
        s.y = fmaf(x[k].y, ws[k], s.y);
        s.z = fmaf(x[k].z, ws[k], s.z);
        s.w = fmaf(x[k].w, ws[k], s.w);
      }
    }
    *reinterpret_cast<float4*>(&acc[warp][4 * lane]) = s;
  }
  __syncthreads();
  for (int i = tid; i < kRows * TQ_D; i += kMergeThreads) {
    const int r = i >> 7, c = i & 127;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kShares; ++k) s += acc[r * kShares + k][c];
    // the value operand's order of coordinates
    sum[r][nibbles ? c : plane_coord(c)] = s;
  }
  __syncthreads();
  float (*prod)[kRows][TQ_D] = reinterpret_cast<float (*)[kRows][TQ_D]>(acc);   // 4 quarters
#pragma unroll 1
  for (int r = 0; r < kRows; ++r) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&sum[r][32 * kq + k]);
      s = fmaf(w[k], x.x, s);
      s = fmaf(w[k + 1], x.y, s);
      s = fmaf(w[k + 2], x.z, s);
      s = fmaf(w[k + 3], x.w, s);
    }
    prod[kq][r][j] = s;
  }
  __syncthreads();
  for (int i = tid; i < kRows * TQ_D; i += kMergeThreads) {
    const int r = i >> 7, c = i & 127;
    if (row0 + r >= nrows) continue;
    const float l = total[r];
    const float s = (prod[0][r][c] + prod[1][r][c]) + (prod[2][r][c] + prod[3][r][c]);
    const float o = l == 0.f ? 0.f : s * unscale / l;
    const long long at = (long long)(row0 + r) * TQ_D + c;
    if (out_dtype == TQ_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(o);
    else static_cast<__half*>(out)[at] = __float2half_rn(o);
  }
}

#ifdef TQ_ROWS_TREE
// ---------------------------------------------------------------- many rows
// Trees have 16 and 64 times the rows of a decode step, and the two kernels above then take as long as
// the attention itself (7168 rows: 28 and 30 us; these take 20 and 16): a CTA reads its matrix for 4 or 8 rows, and its
// threads get 16 bytes from shared memory for every four products.  These keep a matrix in the
// registers of 256 threads, several columns a thread, for as many rows as there are (8 at a time), and
// take the sums of the first kernel in the same order.
constexpr int kManyThreads = 256, kManyRows = 8;

__global__ void __launch_bounds__(kManyThreads, 1)
rows_prep_many_kernel(const void* q, int q_dtype, int nrows, int fine, const float* __restrict__ piT,
                      const float* __restrict__ sT, float factor, __half* qop, float* qf, const int* seq_lens, int batch,
                      int* order) {
  __shared__ float qs[kManyRows][TQ_D];
  __shared__ float part[4][kManyRows][256];
  __shared__ float scale[kManyRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = tid & 63, kq = tid >> 6;
  float w[4][32];   // coordinates p and p + 64 of y and of z, a quarter of k (matrices of the codec's)
  int at[4];        // and their positions in the operand
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const int c = p + 64 * (o & 1);
    at[o] = o < 2 ? plane_position(c) : 128 + sign_position(c);
    const float* mat = (o < 2 ? piT : sT) + 32 * kq * TQ_D + c;
#pragma unroll
    for (int k = 0; k < 32; ++k) w[o][k] = __ldg(mat + k * TQ_D);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // not before the wait: rows_attn_kernel reads lengths and codes before it waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Ranks of the sequences by length, the lower number of equal ones first: the attention takes long items
  // first, so that its last ones are short (16 drafted tokens of 20 sequences of 100 to 30000: 300 us for
  // 344, 8 of 32 of 4096 to 16384: 206 for 215; both with the best splits).  Batches of at most kMostOrdered.
  for (int b = order ? blockIdx.x : batch; b < batch; b += gridDim.x) {
    const int len = seq_lens[b];
    int rank = 0;
    for (int i = 0; i < batch; i += kManyThreads) {
      const int other = i + tid < batch ? seq_lens[i + tid] : INT_MIN;
      rank += __syncthreads_count(i + tid < batch && (other > len || (other == len && i + tid < b)));
    }
    if (tid == 0) order[rank] = b;
  }
  const int step = gridDim.x * kManyRows;
  float next[kManyRows * TQ_D / kManyThreads];     // the next rows' queries are in flight meanwhile
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kManyRows * TQ_D / kManyThreads; ++i) {
      const int e = tid + i * kManyThreads;
      next[i] = row0 + e / TQ_D < nrows ? load_elem(q, q_dtype, (long long)row0 * TQ_D + e) : 0.f;
    }
  };
  load(blockIdx.x * kManyRows);
  for (int row0 = blockIdx.x * kManyRows; row0 < nrows; row0 += step) {
#pragma unroll
    for (int i = 0; i < kManyRows * TQ_D / kManyThreads; ++i) (&qs[0][0])[tid + i * kManyThreads] = next[i];
    __syncthreads();
    load(row0 + step < nrows ? row0 + step : row0);
    {
      const int r = warp;
      float m = 0.f;
      for (int j = lane; j < TQ_D; j += 32) m = fmaxf(m, fabsf(qs[r][j]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) {
        // as above, from the exponent's bits (those of a subnormal m are below −110 anyway)
        int e = 0;
        if (m > 0.f && m < INFINITY) e = (int)(__float_as_uint(m) >> 23) - 126;
        e = min(max(e + 4, -110), 120);
        scale[r] = __uint_as_float((uint32_t)(127 - e) << 23);
        if (row0 + r < nrows) qf[row0 + r] = factor * __uint_as_float((uint32_t)(127 + e) << 23);
      }
    }
#pragma unroll 1
    for (int r = 0; r < kManyRows; ++r) {
      float s[4] = {};
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&qs[r][32 * kq + k]);
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          s[o] = fmaf(w[o][k], x.x, s[o]);
          s[o] = fmaf(w[o][k + 1], x.y, s[o]);
          s[o] = fmaf(w[o][k + 2], x.z, s[o]);
          s[o] = fmaf(w[o][k + 3], x.w, s[o]);
        }
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) part[kq][r][at[o]] = s[o];
    }
    __syncthreads();
    // two neighbouring positions a thread, half of the rows each
    const int c = 2 * (tid & 127);
#pragma unroll
    for (int r = tid >> 7; r < kManyRows; r += 2) {
      if (row0 + r >= nrows) break;
      const float2 a = *reinterpret_cast<const float2*>(&part[0][r][c]), b = *reinterpret_cast<const float2*>(&part[1][r][c]);
      const float2 d = *reinterpret_cast<const float2*>(&part[2][r][c]), e = *reinterpret_cast<const float2*>(&part[3][r][c]);
      const float by = c < 128 ? kAlpha : kBeta;
      const float x = ((a.x + b.x) + (d.x + e.x)) * scale[r] * by, y = ((a.y + b.y) + (d.y + e.y)) * scale[r] * by;
      const __half2 h = __floats2half2_rn(x, y);
      __half2* row = reinterpret_cast<__half2*>(qop + (long long)(row0 + r) * (fine ? 512 : 256) + c);
      row[0] = h;
      if (fine) row[128] = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kManyThreads, 2)
rows_merge_many_kernel(const float* rec, int nrec, int nrows, const float* __restrict__ pi, int nibbles,
                       float unscale, void* out, int out_dtype) {
  __shared__ float sum[kManyRows][TQ_D];
  __shared__ float prod[4][kManyRows][TQ_D];
  __shared__ float total[kManyRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = tid & 63, kq = tid >> 6;
  float w[2][32];   // columns j and j + 64 of Π, a quarter of k
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int k = 0; k < 32; ++k) w[o][k] = __ldg(pi + (32 * kq + k) * TQ_D + j + 64 * o);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long stride = (long long)nrows * kRecFloats;
  for (int row0 = blockIdx.x * kManyRows; row0 < nrows; row0 += gridDim.x * kManyRows) {
    // a warp per row: the records' statistics and eight of their vectors are in flight together; 32
    // records at a time, joined to a running sum
    const float* p = rec + (long long)min(row0 + warp, nrows - 1) * kRecFloats;
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < nrec; s0 += 32) {
      const float2 ml = s0 + lane < nrec ? *reinterpret_cast<const float2*>(p + (s0 + lane) * stride + 128)
                                         : make_float2(-INFINITY, 0.f);
      float4 x[8];
      auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = s0 + i0 + k < nrec ? *reinterpret_cast<const float4*>(p + (s0 + i0 + k) * stride + 4 * lane)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      };
      load(0);
      // an empty record weighs nothing (its vector is not written); a NaN sum (a NaN query) makes the row NaN
      float top = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, m);
      const float mine = m == -INFINITY ? 1.f : ex2(m - top);      // (no record so far: sums of 0, or NaN)
      l *= mine;
      a.x *= mine; a.y *= mine; a.z *= mine; a.w *= mine;
      m = top;
      const float ws = ml.y != ml.y ? ml.y : ml.y == 0.f ? 0.f : ex2(ml.x - m);
      float sum_l = ws == 0.f ? 0.f : ml.y * ws;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum_l += __shfl_xor_sync(0xffffffffu, sum_l, o);
      l += sum_l;
      const int n = min(nrec - s0, 32);
      for (int i0 = 0; i0 < n; i0 += 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = __shfl_sync(0xffffffffu, ws, (i0 + k) & 31);
          if (i0 + k >= n || f == 0.f) continue;
          a.x = fmaf(x[k].x, f, a.x);
          a.y = fmaf(x[k].y, f, a.y);
          a.z = fmaf(x[k].z, f, a.z);
          a.w = fmaf(x[k].w, f, a.w);
        }
        if (i0 + 8 < n) load(i0 + 8);
      }
    }
    if (lane == 0) total[warp] = l;
    const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[warp][nibbles ? 4 * lane + k : plane_coord(4 * lane + k)] = v[k];
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < kManyRows; ++r) {
      float s[2] = {};
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&sum[r][32 * kq + k]);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          s[o] = fmaf(w[o][k], x.x, s[o]);
          s[o] = fmaf(w[o][k + 1], x.y, s[o]);
          s[o] = fmaf(w[o][k + 2], x.z, s[o]);
          s[o] = fmaf(w[o][k + 3], x.w, s[o]);
        }
      }
      prod[kq][r][j] = s[0];
      prod[kq][r][j + 64] = s[1];
    }
    __syncthreads();
#pragma unroll
    for (int i = tid; i < kManyRows * TQ_D / 2; i += kManyThreads) {
      const int r = i >> 6, c = 2 * (i & 63);
      if (row0 + r >= nrows) continue;
      const float inv = total[r] == 0.f ? 0.f : unscale / total[r];
      const float x = ((prod[0][r][c] + prod[1][r][c]) + (prod[2][r][c] + prod[3][r][c])) * inv;
      const float y = ((prod[0][r][c + 1] + prod[1][r][c + 1]) + (prod[2][r][c + 1] + prod[3][r][c + 1])) * inv;
      const long long at = (long long)(row0 + r) * TQ_D + c;
      if (out_dtype == TQ_BF16) *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + at) = __floats2bfloat162_rn(x, y);
      else *reinterpret_cast<__half2*>(static_cast<__half*>(out) + at) = __floats2half2_rn(x, y);
    }
    __syncthreads();
  }
}
#endif

// ---------------------------------------------------------------- host
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Plan {
  int G, rows, row_tiles, pre_splits, own_splits;
  int fine;        // fp16 outputs: operands as pairs of fp16
  size_t qf_off, rec_off, order_off, bytes;
};

#ifndef TQ_ROWS_TREE
// Time of a grid of n1 items of c1 tiles each and then n2 items of c2, taken in order by `sms` SMs
// that each work on one (in tiles).
double makespan(long long n1, double c1, long long n2, double c2, long long sms) {
  const long long rest = n1 % sms;            // items of the last, partial wave of the first kind
  const double start = (double)(n1 / sms) * c1;
  const double until = rest ? start + c1 : start;
  // second-kind items that the other SMs take meanwhile, then all of them
  const long long beside = rest ? (sms - rest) * (long long)(c1 / c2) : 0;
  if (n2 <= beside) return until;
  return until + (double)((n2 - beside + sms - 1) / sms) * c2;
}

// Splits that make the estimated time least (find_splits).  An item costs its tiles, those of few
// rows less (measured: 3,000 cycles with 32 rows, 4,000 with 112), and about two tiles of start
// and end.  Against 3 tiles and one cost: 62.3 for 66.4 us (prefix of 32768, 32 sequences) and 176
// for 191 us (65536, 64 sequences); 5 tiles: 70.1 and 176 us; others the same.
constexpr double kFixed = 2.0, kFewRows = 0.75;
// The arguments that the splits follow from, and what they came to.
struct Splits {
  long long pu, pre, ou, own, sms;
  bool few;          // at most 64 query rows in an item of the prefix
  int sp, so;
};

// The numbers of items that `tiles` are split into, ascending: tiles per item grow by steps of an
// eighth.
constexpr int kMaxWays = 192;
int split_ways(long long tiles, int* ways) {
  int n = 0, begin = kMaxWays;
  for (long long l = 1;; l += std::max<long long>(1, l / 8)) {
    const long long s = (tiles + l - 1) / l;
    if (l >= tiles || s <= kMaxRecs) {
      const int w = l >= tiles ? 1 : (int)s;
      if (begin == kMaxWays || ways[begin] != w) ways[--begin] = w;
    }
    if (l >= tiles) break;
  }
  for (; begin < kMaxWays; ++begin) ways[n++] = ways[begin];
  return n;
}

// The search of all pairs, without those that a lower bound of the time rules out (every SM busy all
// the time): 0.1 to 0.4 us of host time a call, 4 us for 65536 and 8192 tiles (all pairs: ten times
// that).
void find_splits(Splits* x) {
  int pw[kMaxWays] = {0}, ow[kMaxWays];
  const int np = x->pre > 0 ? split_ways(x->pre, pw) : 1;
  const int no = split_ways(std::max<long long>(x->own, 1), ow);
  const double tile = x->few ? kFewRows : 1.0, sms = (double)x->sms;
  double best = 0;
  for (int i = 0; i < np; ++i) {
    const long long sp = pw[i];
    const double cp = sp ? tile * (double)((x->pre + sp - 1) / sp) + kFixed : 0;
    const double pre_least = (double)x->pu * (tile * (double)x->pre + kFixed * (double)sp);
    for (int j = 0; j < no; ++j) {
      const long long so = ow[j];
      if (sp + so > kMaxRecs) break;
      // more records cost the merge: about a tile's time for 64 of them
      const double merge = (double)(sp + so) / 64;
      const double own_least = (double)x->ou * (kFewRows * (double)x->own + kFixed * (double)so);
      if (x->so && (pre_least + own_least) * (1 - 1e-9) > (best - merge) * sms) {
        if (!j) return;      // more items take longer still
        break;
      }
      const double co = kFewRows * (double)((x->own + so - 1) / so) + kFixed;
      if (x->so && std::max(cp, co) + merge > best) continue;
      const double t = makespan(x->pu * sp, cp, x->ou * so, co, x->sms) + merge;
      if (!x->so || t <= best) {      // (equal times: more items)
        best = t;
        x->sp = (int)sp;
        x->so = (int)so;
      }
    }
  }
}

#endif

tq_status check_desc(const tq_attn_desc* d, long long pre_tiles, long long own_tiles) {
  if (!d) return TQ_ERR_INVALID_ARG;
  if (d->head_dim != TQ_HEAD_DIM) return TQ_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->q_heads <= 0 || d->kv_heads <= 0) return TQ_ERR_INVALID_ARG;
  if (d->q_heads % d->kv_heads) return TQ_ERR_INVALID_ARG;
  if (d->q_heads / d->kv_heads > TQ_MAX_GROUP) return TQ_ERR_UNSUPPORTED;
  if (d->capacity <= 0 || d->capacity % TQ_CAPACITY_ALIGN) return TQ_ERR_INVALID_ARG;
  if (d->max_seq_len < 0 || d->max_seq_len > d->capacity) return TQ_ERR_INVALID_ARG;
  if (d->tail_capacity != 0) return TQ_ERR_INVALID_ARG;
  if (d->q_dtype != TQ_F32 && d->q_dtype != TQ_F16 && d->q_dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  if (d->out_dtype != TQ_F16 && d->out_dtype != TQ_BF16) return TQ_ERR_UNSUPPORTED;
  if ((long long)d->batch * d->q_heads > (1 << 24)) return TQ_ERR_UNSUPPORTED;
  if (std::max(pre_tiles, own_tiles) > (1 << 23)) return TQ_ERR_UNSUPPORTED;   // 2^30 tokens: 32-bit token numbers
  return TQ_OK;
}

// Where things lie in the workspace.
void lay_out(const tq_attn_desc* d, Plan* p) {
  p->fine = d->out_dtype == TQ_F16;
  p->order_off = 0;
  p->qf_off = (size_t)p->rows * (p->fine ? 1024 : 512);
  p->rec_off = (p->qf_off + (size_t)p->rows * sizeof(float) + 255) / 256 * 256;
  p->bytes = p->rec_off + (size_t)(p->pre_splits + p->own_splits) * p->rows * kRecFloats * sizeof(float);
}

#ifndef TQ_ROWS_TREE
tq_status make_plan(const tq_attn_desc* d, long long pre_tiles, long long own_tiles, Plan* p) {
  const tq_status st = check_desc(d, pre_tiles, own_tiles);
  if (st != TQ_OK) return st;
  p->G = d->q_heads / d->kv_heads;
  p->rows = d->batch * d->q_heads;
  p->row_tiles = (int)(((long long)d->batch * p->G + kTile - 1) / kTile);
  const int n = tq_num_sms();
  const long long sms = n > 0 ? n : 152;
  const long long pu = (long long)p->row_tiles * d->kv_heads, ou = (long long)d->batch * d->kv_heads;
  Splits want{pu, pre_tiles, ou, own_tiles, sms, (long long)d->batch * p->G <= kTile / 2, 0, 0};
  find_splits(&want);
  p->pre_splits = want.sp;
  p->own_splits = want.so;
  if (pu * p->pre_splits + ou * p->own_splits > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  lay_out(d, p);
  return TQ_OK;
}
#endif

LevelBytes level_bytes(const tq_codec* c) {
  LevelBytes t{};
  for (int i = 0; i < 16; ++i) {
    const __half h = __float2half_rn(i < c->levels ? c->lut_scale * c->centroids[i] : 0.f);
    const uint16_t u = __half_raw(h).x;
    t.lo[i / 4] |= (uint32_t)(u & 255u) << (8 * (i % 4));
    t.hi[i / 4] |= (uint32_t)(u >> 8) << (8 * (i % 4));
  }
  return t;
}

tq_status cache_side(const tq_prod_cache& k, const tq_mse_cache& v, int capacity, CacheSide* s) {
  if (!k.idx || !k.sgn || !k.xnorm || !k.rnorm || !v.idx || !v.xnorm) return TQ_ERR_INVALID_ARG;
  if (!aligned16(k.idx) || !aligned16(k.sgn) || !aligned16(k.xnorm) || !aligned16(k.rnorm) ||
      !aligned16(v.idx) || !aligned16(v.xnorm))
    return TQ_ERR_INVALID_ARG;
  s->kidx = k.idx; s->ksgn = k.sgn; s->kxn = k.xnorm; s->krn = k.rnorm;
  s->vidx = v.idx; s->vxn = v.xnorm;
  tq_status st = tq_rowmap_of(k.pages, capacity, &s->kmap);
  if (st == TQ_OK) st = tq_rowmap_of(v.pages, capacity, &s->vmap);
  if (st != TQ_OK) return st;
  s->kslots = tq_row_slots(s->kmap, capacity);
  s->vslots = tq_row_slots(s->vmap, capacity);
  s->same_map = s->kmap.table == s->vmap.table && s->kmap.max_pages == s->vmap.max_pages &&
                s->kmap.page_tokens == s->vmap.page_tokens && s->kmap.num_pages == s->vmap.num_pages;
  if (s->kslots > (1 << 26) || s->vslots > (1 << 26)) return TQ_ERR_UNSUPPORTED;   // 32-bit offsets
  return TQ_OK;
}

cudaLaunchConfig_t config(unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return c;
}

template <int IB, int VB, bool kFine>
tq_status launch_attn(const RowsArgs& a, unsigned items, cudaStream_t stream) {
  constexpr int smem = (int)sizeof(Smem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static bool configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return TQ_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(rows_attn_kernel<IB, VB, kFine>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return TQ_ERR_CUDA;
    // the warpgroups' shares add up to what the block is launched with: more would wait forever
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, rows_attn_kernel<IB, VB, kFine>) != cudaSuccess) return TQ_ERR_CUDA;
    if (fa.numRegs != kRegsLaunch) return TQ_ERR_UNSUPPORTED;
    configured[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(items, kThreads, smem, stream, attr);
  return tq_cuda_status(cudaLaunchKernelEx(&cfg, rows_attn_kernel<IB, VB, kFine>, a));
}

template <int IB, bool kFine>
tq_status launch_v(const RowsArgs& a, int vbits, unsigned items, cudaStream_t stream) {
  switch (vbits) {
    case 1: return launch_attn<IB, 1, kFine>(a, items, stream);
    case 2: return launch_attn<IB, 2, kFine>(a, items, stream);
    case 3: return launch_attn<IB, 3, kFine>(a, items, stream);
    case 4: return launch_attn<IB, 4, kFine>(a, items, stream);
  }
  return TQ_ERR_UNSUPPORTED;
}

template <int IB>
tq_status launch_k(const RowsArgs& a, int vbits, bool fine, unsigned items, cudaStream_t stream) {
  return fine ? launch_v<IB, true>(a, vbits, items, stream) : launch_v<IB, false>(a, vbits, items, stream);
}

// Rows per CTA of the two kernels around: the fewest (1, 2, 4, most) that keep about one CTA per SM.
int rows_per_cta(int rows, int most) {
  const int sms = std::max(tq_num_sms(), 1);
  for (int r = 1; r < most; r *= 2)
    if ((rows + r - 1) / r <= sms) return r;
  return most;
}

#ifdef TQ_ROWS_TREE
// Rows from which on the kernels for many are faster.
int many_rows() { return 8 * std::max(tq_num_sms(), 1); }

// Sequences up to which they are ranked: ranking costs their square, and an item is a small part of what an SM
// has of larger batches (2 drafted tokens of 8 heads; 2048 sequences, 11 of them of 4096 tokens and the others
// of up to 512: 286 us ranked, 311 not; 8192 of up to 1024 tokens: 1350 and 1220).
constexpr int kMostOrdered = 2048;
#endif

tq_status launch_prep(const void* q, int q_dtype, int rows, int fine, const tq_codec* kc, float factor,
                      void* qop, float* qf, const int* seq_lens, int batch, int* order, cudaStream_t stream) {
#ifdef TQ_ROWS_TREE
  if (rows > many_rows()) {
    const int grid = std::min((rows + kManyRows - 1) / kManyRows, std::max(tq_num_sms(), 1));
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(grid, kManyThreads, 0, stream, attr);
    return tq_cuda_status(cudaLaunchKernelEx(&cfg, rows_prep_many_kernel, q, q_dtype, rows, fine, (const float*)kc->d_piT,
                                             (const float*)kc->d_sT, factor, static_cast<__half*>(qop), qf, seq_lens, batch, order));
  }
#endif
  const int rp = rows_per_cta(rows, 8);
  auto kern = rp == 1 ? rows_prep_kernel<1> : rp == 2 ? rows_prep_kernel<2>
            : rp == 4 ? rows_prep_kernel<4> : rows_prep_kernel<8>;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config((rows + rp - 1) / rp, kPrepThreads, 0, stream, attr);
  return tq_cuda_status(cudaLaunchKernelEx(&cfg, kern, q, q_dtype, rows, fine, (const float*)kc->d_piT,
                                           (const float*)kc->d_sT, factor,
                                           static_cast<__half*>(qop), qf));
}

tq_status launch_merge(const float* rec, int nrec, int rows, const tq_codec* vc, void* out,
                       int out_dtype, cudaStream_t stream) {
#ifdef TQ_ROWS_TREE
  if (rows > many_rows()) {
    const int grid = std::min((rows + kManyRows - 1) / kManyRows, 2 * std::max(tq_num_sms(), 1));
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(grid, kManyThreads, 0, stream, attr);
    return tq_cuda_status(cudaLaunchKernelEx(&cfg, rows_merge_many_kernel, rec, nrec, rows, (const float*)vc->d_pi,
                                             vc->ibits == 4 ? 1 : 0, 1.f / vc->lut_scale, out, out_dtype));
  }
#endif
  const int rp = rows_per_cta(rows, 4);
  auto kern = rp == 1 ? rows_merge_kernel<1> : rp == 2 ? rows_merge_kernel<2> : rows_merge_kernel<4>;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config((rows + rp - 1) / rp, kMergeThreads, 0, stream, attr);
  return tq_cuda_status(cudaLaunchKernelEx(&cfg, kern, rec, nrec, rows, (const float*)vc->d_pi,
                                           vc->ibits == 4 ? 1 : 0, 1.f / vc->lut_scale, out,
                                           out_dtype));
}

tq_status run(const tq_attn_desc* d, const Plan& p, const tq_codec* kc, const tq_codec* vc,
              const void* q, RowsArgs& a, void* out, void* workspace, size_t workspace_bytes,
              tq_stream_t stream_) {
  tq_status st;
  if ((st = tq_check_codec(kc, TQ_PROD)) != TQ_OK) return st;
  if ((st = tq_check_codec(vc, TQ_MSE)) != TQ_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  if (kc->device != dev || vc->device != dev) return TQ_ERR_INVALID_ARG;
  if (!q || !a.seq_lens || !out || !workspace) return TQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < p.bytes)
    return TQ_ERR_INVALID_ARG;
  if (d->batch == 0) return TQ_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  const float scale = d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / sqrtf((float)TQ_D);
  a.B = d->batch; a.Hq = d->q_heads; a.Hkv = d->kv_heads; a.G = p.G;
  a.max_len = d->max_seq_len;
  a.row_tiles = p.row_tiles; a.pre_splits = p.pre_splits; a.own_splits = p.own_splits;
  a.kt = level_bytes(kc);
  a.vt = level_bytes(vc);
  a.rho_scale = kAlpha / kBeta * kc->lut_scale * kQjl;
  a.qop = reinterpret_cast<const uint4*>(ws);
  a.qf = reinterpret_cast<const float*>(ws + p.qf_off);
  a.rec = reinterpret_cast<float*>(ws + p.rec_off);
#ifdef TQ_ROWS_TREE
  a.order = p.order_off ? reinterpret_cast<const int*>(ws + p.order_off) : nullptr;
#endif
  const float factor = scale * 1.4426950408889634f / (kAlpha * kc->lut_scale);
  st = launch_prep(q, d->q_dtype, p.rows, p.fine, kc, factor, ws, reinterpret_cast<float*>(ws + p.qf_off),
                   a.seq_lens, a.B, p.order_off ? reinterpret_cast<int*>(ws + p.order_off) : nullptr, stream);
  if (st != TQ_OK) return st;
  const unsigned items = (unsigned)((long long)p.pre_splits * a.Hkv * p.row_tiles +
                                    (long long)p.own_splits * a.Hkv * a.B * (kTree ? p.row_tiles : 1));
  switch (kc->ibits) {
    case 1: st = launch_k<1>(a, vc->ibits, p.fine, items, stream); break;
    case 2: st = launch_k<2>(a, vc->ibits, p.fine, items, stream); break;
    case 3: st = launch_k<3>(a, vc->ibits, p.fine, items, stream); break;
    case 4: st = launch_k<4>(a, vc->ibits, p.fine, items, stream); break;
    default: st = TQ_ERR_UNSUPPORTED;
  }
  if (st != TQ_OK) return st;
  return launch_merge(a.rec, p.pre_splits + p.own_splits, p.rows, vc, out, d->out_dtype, stream);
}

long long tiles_of(long long tokens) { return (tokens + kTile - 1) / kTile; }

#ifdef TQ_ROWS_TREE

// Splits of a sequence's tiles that make the estimated time least, in tiles.  An item costs its tiles
// and about three more for its start and end (8 us; a tile 2.4 us with 56 rows, 3.1 with 112), and a
// record 2 times 528 bytes of the merge (of 5 bytes a picosecond, a tile 2.4 us).  Items that all have an
// SM take the time of one; one sequence's items are alike and go in waves; those of a batch differ with
// its lengths, which the host does not know (taken: half of the longest to all of it, three quarters of
// it on average), and take an SM's share of the work and a part of the longest item, a quarter where the
// long ones come first.  Within 7% of the best number of splits in seven batches of 16 to 256 sequences of
// which the shortest are 2% to 98% of the longest.
int tree_splits(long long units, long long tiles, long long rows, long long sms, bool alike, bool ordered) {
  constexpr double kItem = 3.0, kRecord = 2 * 528 / 12e6;
  const double tail = ordered ? 0.25 : 0.5;
  const long long most = std::min(std::max(tiles, 1LL), std::min<long long>(kMaxRecs, 8 * sms / std::max(units, 1LL) + 8));
  double best = 0;
  int splits = 1;
  for (long long s = 1; s <= most; ++s) {
    const long long items = units * s, waves = (items + sms - 1) / sms;
    const double item = (double)((tiles + s - 1) / s) + kItem;
    const double t = (items <= sms || alike ? (double)waves * item
                                            : (double)units * (0.75 * (double)tiles + kItem * (double)s) / (double)sms + tail * item) +
                     kRecord * (double)(rows * s);
    if (s == 1 || t < best) {
      best = t;
      splits = (int)s;
    }
  }
  return splits;
}

tq_status plan_tree(const tq_attn_desc* d, int nodes, Plan* p) {
  if (!d || nodes <= 0) return TQ_ERR_INVALID_ARG;
  const long long tiles = tiles_of(d->max_seq_len);
  const tq_status st = check_desc(d, 0, tiles);
  if (st != TQ_OK) return st;
  if (nodes > TQ_TREE_NODES || (long long)d->batch * d->q_heads * nodes > (1 << 24)) return TQ_ERR_UNSUPPORTED;
  if (d->max_seq_len < nodes) return TQ_ERR_INVALID_ARG;
  p->G = d->q_heads / d->kv_heads;
  p->rows = d->batch * d->q_heads * nodes;
  p->row_tiles = (nodes * p->G + kTile - 1) / kTile;
  const int n = tq_num_sms();
  const long long units = (long long)d->batch * d->kv_heads * p->row_tiles;
  p->pre_splits = 0;
  // (rows_prep_many_kernel writes the order)
  const bool ordered = p->rows > many_rows() && d->batch > 1 && d->batch <= kMostOrdered;
  p->own_splits = tree_splits(units, tiles, p->rows, n > 0 ? n : 152, d->batch == 1, ordered);
  if (units * p->own_splits > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  lay_out(d, p);
  if (ordered && units * p->own_splits > (n > 0 ? n : 152)) {
    p->order_off = p->bytes;
    p->bytes += (size_t)d->batch * sizeof(int);
  }
  return TQ_OK;
}

}  // namespace

extern "C" size_t tq_tree_workspace_bytes(const tq_attn_desc* desc, int32_t n_nodes) {
  Plan p;
  return plan_tree(desc, n_nodes, &p) == TQ_OK ? p.bytes : 0;
}

extern "C" tq_status tq_tree_attention(const tq_attn_desc* desc, int32_t n_nodes, const tq_codec* kc,
                                       const tq_codec* vc, const void* q, tq_prod_cache k,
                                       tq_mse_cache v, const int32_t* seq_lens, const uint64_t* tree,
                                       int64_t tree_stride_b, void* out, void* workspace,
                                       size_t workspace_bytes, tq_stream_t stream) {
  Plan p;
  tq_status st = plan_tree(desc, n_nodes, &p);
  if (st != TQ_OK) return st;
  RowsArgs a{};
  if (!tree || reinterpret_cast<uintptr_t>(tree) % 8 || tree_stride_b < 0) return TQ_ERR_INVALID_ARG;
  if (!aligned16(out)) return TQ_ERR_INVALID_ARG;
  if ((st = cache_side(k, v, desc->capacity, &a.own)) != TQ_OK) return st;
  a.seq_lens = seq_lens;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.tree_b = tree_stride_b;
  a.nodes = n_nodes;
  return run(desc, p, kc, vc, q, a, out, workspace, workspace_bytes, stream);
}

#else

tq_status plan_sparse(const tq_attn_desc* d, int max_blocks, Plan* p) {
  if (max_blocks <= 0 || max_blocks > (1 << 24)) return TQ_ERR_INVALID_ARG;
  return make_plan(d, 0, (max_blocks + 1) / 2, p);
}

tq_status plan_prefix(const tq_attn_desc* d, int prefix_max_len, Plan* p) {
  if (!d || prefix_max_len < 0) return TQ_ERR_INVALID_ARG;
  return make_plan(d, tiles_of(prefix_max_len), tiles_of(d->max_seq_len), p);
}

}  // namespace

extern "C" size_t tq_sparse_workspace_bytes(const tq_attn_desc* desc, int32_t max_blocks) {
  Plan p;
  return plan_sparse(desc, max_blocks, &p) == TQ_OK ? p.bytes : 0;
}

extern "C" tq_status tq_sparse_attention(const tq_attn_desc* desc, const tq_codec* kc,
                                         const tq_codec* vc, const void* q, tq_prod_cache k,
                                         tq_mse_cache v, const int32_t* seq_lens,
                                         const int32_t* blocks, int32_t max_blocks, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         tq_stream_t stream) {
  Plan p;
  tq_status st = plan_sparse(desc, max_blocks, &p);
  if (st != TQ_OK) return st;
  RowsArgs a{};
  if (!blocks) return TQ_ERR_INVALID_ARG;
  if ((st = cache_side(k, v, desc->capacity, &a.own)) != TQ_OK) return st;
  a.seq_lens = seq_lens;
  a.list = blocks;
  a.max_blocks = max_blocks;
  return run(desc, p, kc, vc, q, a, out, workspace, workspace_bytes, stream);
}

extern "C" size_t tq_prefix_workspace_bytes(const tq_attn_desc* desc, int32_t prefix_max_len) {
  Plan p;
  return plan_prefix(desc, prefix_max_len, &p) == TQ_OK ? p.bytes : 0;
}

extern "C" tq_status tq_prefix_attention(const tq_attn_desc* desc, const tq_codec* kc,
                                         const tq_codec* vc, const void* q,
                                         tq_prod_cache prefix_k, tq_mse_cache prefix_v,
                                         int32_t prefix_capacity, int32_t prefix_max_len,
                                         const int32_t* prefix_len, tq_prod_cache k,
                                         tq_mse_cache v, const int32_t* seq_lens, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         tq_stream_t stream) {
  Plan p;
  tq_status st = plan_prefix(desc, prefix_max_len, &p);
  if (st != TQ_OK) return st;
  if (prefix_capacity <= 0 || prefix_capacity % TQ_CAPACITY_ALIGN || prefix_max_len > prefix_capacity)
    return TQ_ERR_INVALID_ARG;
  RowsArgs a{};
  if (!prefix_len) return TQ_ERR_INVALID_ARG;
  if ((st = cache_side(prefix_k, prefix_v, prefix_capacity, &a.pre)) != TQ_OK) return st;
  if ((st = cache_side(k, v, desc->capacity, &a.own)) != TQ_OK) return st;
  a.seq_lens = seq_lens;
  a.pre_len = prefix_len;
  a.max_pre = prefix_max_len;
  return run(desc, p, kc, vc, q, a, out, workspace, workspace_bytes, stream);
}

#endif
