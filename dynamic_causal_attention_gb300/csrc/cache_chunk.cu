// cache_chunk.cu — the hybrid layer over the paged 8-bit cache for many query
// rows: prompts in pieces, drafts of many tokens, wide groups of heads.  Same
// mathematics as cache_attn.cu; here both products run on tcgen05 with fp32
// accumulators in TMEM.
//
// A unit is (slot, class, row pair): a class is the dynamic or the frozen
// query heads of one K/V head; its rows are r = t * heads + index (dynamic: the
// last key that a unit sees is then as early as can be) or r = index * n_new + t
// (frozen: each head begins a unit of its own, whose rows share alpha and read
// rho side by side).  A unit takes 256 of them as two tiles of 128, against the
// keys up to the last position among them in tiles of 128.  Splitting a group by
// kind keeps every warp uniform and spares frozen rows the Q K product.  All
// tiles of all units are cut into shares of equal cost, one for each CTA (one per
// SM); a unit that is cut is joined as in cache_attn.cu.
//
// Warp roles (512 threads; registers move to the softmax):
//   warps 0-3, 4-7   the softmax of row tile 0 and 1: one row per thread.  They
//                    also stage Q and write the results.
//   warps 8-11       turn V's e4m3 codes into f16 tiles in shared memory.
//   warps 12, 14     issue the products of row tile 0 and 1 (one lane each); 12
//                    allocates TMEM.
//   warp 13          looks up pages, fetches K and V codes by TMA (a page that is
//                    missing reads as zeros) and writes the scales of each tile.
//
// K needs no conversion: Q K^T runs on 8-bit operands at twice f16's rate, K as e4m3
// and the row of q as a sum of parts, each the rounded rest of the ones before.  Two
// do for most rows: scaled by a power of two to a largest component of 224 to 448,
// the first is e4m3 and leaves at most 4 of a bf16 value's 8 bits (and no more than 8
// units of its last place), the second e5m2, whose 3 bits hold that.  This is exact for
// components down to 2^-6, where e4m3 becomes subnormal: 2^-13 of the row's largest;
// below, they are off by at most 2^-14, 2^-21 of it.  A row tile with an infinity, or
// with a row of more than two such components, takes three e5m2 parts of rows scaled to
// a largest component of 2^14 to 2^15.8: they leave 5, 2 and no bits, exact down to
// 2^-23 of the largest, below off by 2^-31 of it.  (Of 128 normal components, 0.013 lie
// below 2^-6: in a call of 256 row tiles more than two of one row hardly ever do.  The
// call below takes 15% longer if all have three parts.  Two e4m3 parts are exact down
// to 2^-10: beside a component 1000 times the others they left logits off by 2^-7.)  V
// is turned into f16 (exact): splitting the 256 x 128 weights of a tile in its place
// would take six times the arithmetic of converting V's 128 x d_h codes.
//
// TMEM: S of the two row tiles (128 columns each), then their O.  A tile's
// keys are taken in two halves of 64: S, softmax and P V of one half run while
// the other half's do, and P, as packed f16, overwrites the first columns of
// its own half of S, so the next S of a half waits only for the product that
// reads that half's P.  What a tile of keys costs is the chain S, softmax, P V
// and its hand-offs, about 4300 cycles for 256 rows at d_h = 128, against some
// 1800 of the tensor cores' time; 2 x 2000 rows of 16 heads against 8192 keys take
// 265 us, 48% of the measured burst rate of products, and with 4 frozen heads,
// whose weights are 32 loads of two from the window for each half a tile, 271 us
// (41%; with all heads frozen 287, of which 8 for the single stage of V's codes that
// Q's third part leaves room for).
#include <cuda.h>
#include <cuda_bf16.h>
#include <float.h>
#include <math_constants.h>

#include "attn_common.cuh"
#include "cache_common.cuh"
#include "host_common.h"

namespace saf {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 256;     // query rows of a unit
constexpr int kTile = 128;     // keys of a tile
constexpr int kThreads = 512;
// registers of a thread after the split: 2 * 176 + 80 + 80 = 4 * 128
constexpr int kRegsSoftmax = 176, kRegsConvert = 80, kRegsIssue = 80;
// parts that a joining thread has in flight: with 4, 64 registers and 8 blocks of
// an SM, 152 units of 2 to 4 parts take 17 us, with 8 and half the blocks 34
constexpr int kJoinAhead = 4;
constexpr int kStatusCtas = 64;  // status words of the CTAs, behind the call's

enum : int {
  kSiteQ = 64, kSiteK, kSiteV, kSiteP, kSiteO, kSiteS, kSiteMeta, kSiteKFree, kSiteVFree,
  kSiteRaw, kSiteRawFree, kSiteBegin
};

// Instruction descriptor with f16 operands and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A chain of products into one accumulator from one statement: k-step after
// k-step with the descriptors advanced by adds.  One issuing thread then gets a
// product through in about 75 cycles in place of about 160.
#define SAF_HEAD                                                                \
  "{\n\t.reg .pred f, t, e;\n\t.reg .b64 a, b;\n\t.reg .b32 p, q, u, v;\n\t"  \
  "setp.ne.b32 t, 0, 0;\n\tmov.pred f, t;\n\tnot.pred t, f;\n\tsetp.ne.b32 e, %5, 0;\n\t"
#define SAF_PART(AT)                                                                   \
  "mov.b64 a, %1;\n\tmov.b64 b, %2;\n\tmov.b64 {p, u}, a;\n\tmov.b64 {q, v}, b;\n\t" \
  "add.u32 p, p, " AT ";\n\tmov.b64 a, {p, u};\n\t"
#define SAF_MMA8(IDESC, ACC) \
  "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, " IDESC ", " ACC ";\n\t"
#define SAF_MORE(IDESC)                                                                         \
  "add.u32 p, p, 2;\n\tadd.u32 q, q, 2;\n\tmov.b64 a, {p, u};\n\tmov.b64 b, {q, v};\n\t" SAF_MMA8( \
      IDESC, "t")
#define SAF_REST1(IDESC) ""
#define SAF_REST2(IDESC) SAF_MORE(IDESC)
#define SAF_REST4(IDESC) SAF_MORE(IDESC) SAF_MORE(IDESC) SAF_MORE(IDESC)

// S = q0 K^T + q1 K^T: N steps of 32 codes each, the parts STEP apart
template <int N, int STEP>
__device__ __forceinline__ void issue_codes(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc0,
                                            uint32_t idesc1, uint32_t lead) {
  static_assert(N == 1 || N == 2 || N == 4, "");
#define SAF_PARTS(REST) \
  SAF_HEAD SAF_PART("0") SAF_MMA8("%3", "f") REST("%3") SAF_PART("%4") SAF_MMA8("%6", "t") REST("%6") "}"
#define SAF_ARGS \
  ::"r"(d), "l"(q), "l"(k), "r"(idesc0), "n"(STEP), "r"(lead), "r"(idesc1) : "memory"
  if constexpr (N == 1)
    asm volatile(SAF_PARTS(SAF_REST1) SAF_ARGS);
  else if constexpr (N == 2)
    asm volatile(SAF_PARTS(SAF_REST2) SAF_ARGS);
  else
    asm volatile(SAF_PARTS(SAF_REST4) SAF_ARGS);
#undef SAF_PARTS
#undef SAF_ARGS
}
// S += q2 K^T, for rows of Q that need a third part.  A call, so that what follows the
// first two lies right behind them: issued under a predicate in their chain the third
// costs 8% where it is not needed.
template <int N, int STEP>
__device__ __noinline__ void issue_third(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc,
                                         uint32_t lead) {
#define SAF_PARTS(REST) SAF_HEAD SAF_PART("%4") SAF_MMA8("%3", "t") REST("%3") "}"
#define SAF_ARGS ::"r"(d), "l"(q), "l"(k), "r"(idesc), "n"(2 * STEP), "r"(lead) : "memory"
  if constexpr (N == 1)
    asm volatile(SAF_PARTS(SAF_REST1) SAF_ARGS);
  else if constexpr (N == 2)
    asm volatile(SAF_PARTS(SAF_REST2) SAF_ARGS);
  else
    asm volatile(SAF_PARTS(SAF_REST4) SAF_ARGS);
#undef SAF_PARTS
#undef SAF_ARGS
}
#undef SAF_HEAD
#undef SAF_PART
#undef SAF_MMA8
#undef SAF_MORE
#undef SAF_REST1
#undef SAF_REST2
#undef SAF_REST4
// O (+)= P V for 64 keys: 4 steps of 16, P in TMEM (8 columns a step), V's
// descriptor advanced by STEP.
template <int STEP>
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc,
                                         uint32_t accumulate, uint32_t lead) {
#define SAF_MMA "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, "
#define SAF_NEXT "add.u32 a, a, 8;\n\tadd.u32 q, q, %5;\n\tmov.b64 b, {q, v};\n\t"
  asm volatile(
      "{\n\t.reg .pred f, t, e;\n\t.reg .b64 b;\n\t.reg .b32 a, q, v;\n\tsetp.ne.b32 f, %4, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\tmov.b32 a, %1;\n\t"
      "mov.b64 b, %2;\n\tmov.b64 {q, v}, b;\n\t" SAF_MMA "f;\n\t" SAF_NEXT SAF_MMA "t;\n\t"
      SAF_NEXT SAF_MMA "t;\n\t" SAF_NEXT SAF_MMA "t;\n\t}" ::"r"(d),
      "r"(p), "l"(v), "r"(idesc), "r"(accumulate), "n"(STEP), "r"(lead)
      : "memory");
#undef SAF_MMA
#undef SAF_NEXT
}

// ... with e4m3 or e5m2 A and e4m3 B (K-major both).
__host__ __device__ constexpr uint32_t idesc_codes(int M, int N, uint32_t e5m2) {
  return (1u << 4) | (e5m2 << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The rows of a class fall into units of up to 256; a frozen head shares none.
__device__ __forceinline__ int pairs_of(const Rows& r, int gk, bool ice) {
  if (ice) return (r.n_new + kRows - 1) / kRows * gk;
  return (int)(((long long)r.n_new * gk + kRows - 1) / kRows);
}
struct UnitRows {
  int first, n;  // rows [first, first + n) of the class
};
__device__ __forceinline__ UnitRows unit_rows(const Rows& r, int pair, int gk, bool ice) {
  UnitRows u;
  if (ice) {
    const int per = (r.n_new + kRows - 1) / kRows, idx = pair / per;
    const int at = (pair - idx * per) * kRows;
    u.first = idx * r.n_new + at;
    u.n = min(kRows, r.n_new - at);
  } else {
    u.first = pair * kRows;
    u.n = min(kRows, r.n_new * gk - u.first);
  }
  return u;
}
// The tokens [lo, hi) of a unit's rows.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span pair_span(const Rows& r, int pair, int gk, bool ice) {
  const UnitRows u = unit_rows(r, pair, gk, ice);
  Span s;
  if (ice) {
    s.lo = u.first % r.n_new;
    s.hi = s.lo + u.n;
  } else {
    s.lo = u.first / gk;
    s.hi = (u.first + u.n - 1) / gk + 1;
  }
  return s;
}
__device__ __forceinline__ int pair_extent(const Rows& r, int pair, int gk, bool ice) {
  const int e = r.base + pair_span(r, pair, gk, ice).hi;
  return e < 0 ? 0 : (e < r.cap ? e : r.cap);
}
__device__ __forceinline__ int pair_tiles(const Rows& r, int pair, int gk, bool ice) {
  const int n = (pair_extent(r, pair, gk, ice) + kTile - 1) / kTile;
  return n < 1 ? 1 : n;  // rows that see nothing are written too
}
// Row `rr` of a class as (token, index of the head).
__device__ __forceinline__ void row_of(const Rows& r, int rr, int gk, bool ice, int& t, int& idx) {
  if (ice) {
    idx = rr / r.n_new;
    t = rr - idx * r.n_new;
  } else {
    t = rr / gk;
    idx = rr - t * gk;
  }
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// What a share counts, in eighths of a tile of dynamic rows (its two row tiles
// full): the tiles of keys, and behind them the unit's own cost: Q, the first tile
// without company, the results.  Measured with equal units, microseconds:
//                          d_h = 128     64      32
//   tile, dynamic             2.26      1.80    1.57     (one row tile 2.02 1.63 1.47)
//   tile, frozen              2.33      2.31    2.14     (one row tile 2.13 1.73 1.58)
//   unit, dynamic, frozen     11, 8.7   6.3, 4.4   4.5, 3.3
// With tiles alone counted, 2 x 2000 rows of 16 heads, 4 of them frozen, against
// 8192 keys took 5% longer (the average SM was idle for a tenth of them), 12 x 76
// rows of 128 heads against 388 keys 34%.  (At d_h = 128 the frozen tile counts 9
// and units a little less than alone; with 8 for both kinds of tile that call takes
// 5% longer.)
struct Costs {
  int tile[2][2];  // [frozen][both row tiles]
  int unit[2];     // [frozen]
};
__device__ __forceinline__ constexpr Costs costs_of(int d) {
  return d == 128  ? Costs{{{7, 8}, {8, 9}}, {34, 28}}
         : d == 64 ? Costs{{{7, 8}, {8, 11}}, {28, 20}}
                   : Costs{{{7, 8}, {8, 11}}, {23, 17}};
}
constexpr int kMaxTileCost = 11;

// Walks the units in order: slots, then groups of classes (equal width and
// kind), row pairs, classes.  seek() and the sums are taken by whole warps.
template <int D>
struct Walk {
  const CacheChunk& p;
  Rows rows;
  int b, group, pair, cls, ut, each;  // the unit's tiles and what one costs
  __device__ __forceinline__ explicit Walk(const CacheChunk& q) : p(q) {}
  __device__ __forceinline__ int gk() const { return p.group_width[group]; }
  __device__ __forceinline__ bool ice() const { return p.group_static[group]; }
  __device__ __forceinline__ int classes(int g) const {
    return p.group_first[g + 1] - p.group_first[g];
  }
  static __device__ __forceinline__ int tile_cost(const Rows& r, int pair, int gk, bool ice) {
    constexpr Costs k = costs_of(D);
    const bool both = unit_rows(r, pair, gk, ice).n > 128;
    return ice ? (both ? k.tile[1][1] : k.tile[1][0]) : (both ? k.tile[0][1] : k.tile[0][0]);
  }
  static __device__ __forceinline__ int unit_cost(bool ice) {
    constexpr Costs k = costs_of(D);
    return ice ? k.unit[1] : k.unit[0];
  }
  __device__ __forceinline__ long long cost() const {
    return (long long)ut * each + unit_cost(ice());
  }
  // the tiles of the unit that begin before `upto` > 0, counted from its start
  __device__ __forceinline__ int tiles_before(long long upto) const {
    return upto >= (long long)ut * each ? ut : ((int)upto + each - 1) / each;
  }
  __device__ long long slot_cost(int slot) const {
    const Rows r = slot_rows(p.a.c, slot);
    const int lane = threadIdx.x & 31;
    long long sum = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      long long mine = 0;
      const int w = p.group_width[g], n = pairs_of(r, w, p.group_static[g]);
      for (int i = lane; i < n; i += 32)
        mine += (long long)pair_tiles(r, i, w, p.group_static[g]) *
                    tile_cost(r, i, w, p.group_static[g]) +
                unit_cost(p.group_static[g]);
      sum += mine * classes(g);
    }
    return warp_sum(sum);
  }
  // To the unit at `at` of slot `slot`; returns how far that is from its start.
  __device__ long long seek(int slot, long long at) {
    const int lane = threadIdx.x & 31;
    b = slot;
    rows = slot_rows(p.a.c, b);
    for (group = 0;; ++group) {
      const int n = pairs_of(rows, gk(), ice()), n_cls = classes(group);
      for (pair = 0; pair < n; pair += 32) {
        const int i = pair + lane;
        const int mine = i < n ? pair_tiles(rows, i, gk(), ice()) : 0;
        const int one = i < n ? tile_cost(rows, i, gk(), ice()) : 0;
        long long upto = i < n ? ((long long)mine * one + unit_cost(ice())) * n_cls : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(~0u, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned over = __ballot_sync(~0u, at < upto);
        if (over) {
          const int l = __ffs(over) - 1;
          pair += l;
          ut = __shfl_sync(~0u, mine, l);
          each = __shfl_sync(~0u, one, l);
          at -= __shfl_sync(~0u, upto, l) - cost() * n_cls;
          cls = p.group_first[group] + (int)(at / cost());
          return at % cost();
        }
        at -= __shfl_sync(~0u, upto, 31);
      }
    }
  }
  // among all that the slots could have
  __device__ int number() const {
    return b * p.slot_units + p.group_unit[group] + pair * classes(group) + cls -
           p.group_first[group];
  }
  __device__ void next() {
    if (++cls == p.group_first[group + 1]) {
      if (++pair >= pairs_of(rows, gk(), ice())) {
        pair = 0;
        if (++group == p.n_groups) {
          do {
            rows = slot_rows(p.a.c, ++b);
          } while (rows.n_new == 0);
          group = 0;
        }
      }
      cls = p.group_first[group];
      ut = pair_tiles(rows, pair, gk(), ice());
      each = tile_cost(rows, pair, gk(), ice());
    }
  }
};

template <bool V>
struct Const {
  static constexpr bool value = V;
};

struct Share {
  long long size, begin, end, in_slot;
  int b;
};
// Every CTA finds its share, the tiles that begin in [begin, end): each warp sums a
// run of slots, the sums of the warps before give where a run begins, and the warp
// whose run holds the share's beginning walks it.
template <int D>
__device__ Share find_share(const CacheChunk& p, long long* scan /* [warps + 2] */) {
  const Walk<D> w(p);
  constexpr int kN = kThreads / 32;
  const int warp = threadIdx.x >> 5, n_seqs = p.a.c.n_seqs;
  const int per = (n_seqs + kN - 1) / kN;
  const int b0 = min(warp * per, n_seqs), b1 = min(b0 + per, n_seqs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += w.slot_cost(b);
  scan[warp] = sum;
  __syncthreads();
  long long total = 0, mine = 0;
  for (int i = 0; i < kN; ++i) {
    if (i == warp) mine = total;
    total += scan[i];
  }
  Share s;
  // at least a tile: every CTA that a unit passes then has one of its tiles
  s.size = max((total + gridDim.x - 1) / gridDim.x, (long long)kMaxTileCost);
  s.begin = min(s.size * blockIdx.x, total);
  s.end = min(s.begin + s.size, total);
  if (s.begin < s.end && mine <= s.begin && s.begin < mine + sum) {
    long long at = mine;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long t = w.slot_cost(b);
      if (s.begin < at + t) break;
      at += t;
    }
    scan[kN] = b;
    scan[kN + 1] = s.begin - at;
  }
  __syncthreads();
  s.b = (int)scan[kN];
  s.in_slot = scan[kN + 1];
  return s;
}

template <int D>
struct Smem {
  static constexpr int CODES = kTile * D;     // e4m3
  static constexpr int TILE = 2 * CODES;      // f16
  static constexpr int QTILE = 3 * CODES;     // Q's three parts
  // stages of K codes and of V codes.  V's is free again as soon as its codes lie in
  // registers (two stages are no faster); tile n's scales and pattern, written behind
  // that, then find those of tile n - 4 read: the codes of n - 1 are read when n - 2
  // has been converted, which waits for the products of n - 4
  static constexpr int KST = D == 128 ? 2 : 3, RST = 1;
  static constexpr int OFF_Q = 0;             // two row tiles
  static constexpr int OFF_V = 2 * QTILE;     // two stages of f16 V
  static constexpr int OFF_K = OFF_V + 2 * TILE;
  static constexpr int OFF_R = OFF_K + KST * CODES;
  static constexpr int OFF_META = OFF_R + RST * CODES;  // 4 tiles x 8 groups of 16 keys x 16 bytes
  // frozen rows: 128 alphas and the 384 rhos of a tile, times log2(e), and the rhos
  // again from the second one on, 16 banks further, so that rows of either parity
  // read two at a time; for 4 tiles
  static constexpr int WIN0 = 128, WIN1 = WIN0 + 384 + 16;  // in floats
  static constexpr int PAT = (WIN1 + 384) * 4;
  static constexpr int OFF_PAT = OFF_META + 4 * 8 * 16;
  static constexpr int OFF_SCAN = OFF_PAT + 4 * PAT;
  static constexpr int OFF_BAR = OFF_SCAN + (kThreads / 32 + 4) * 8;
  static constexpr int NBAR = 2 + 2 * KST + 2 * RST + 4 + 4 + 4 + 4 + 4 + 2 + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 48;
  static constexpr int ALLOC = BYTES + 1024;  // slack to align the base to 1024 B
  static_assert(ALLOC <= 232448, "shared memory budget exceeded");
};

// Byte offset of 16-byte chunk ch of row r of a [128 x D] tile of codes: rows
// of D bytes, swizzled over D bytes.
template <int D>
__device__ __forceinline__ uint32_t code_at(uint32_t r, uint32_t ch) {
  if (D == 128) return r * 128 + ((ch ^ (r & 7)) << 4);
  if (D == 64) return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
  return r * 32 + ((ch ^ ((r >> 2) & 1)) << 4);
}

// The first 16 of w to 64 contiguous bytes.
__device__ __forceinline__ void st_global_words16(void* to, const uint32_t (&w)[32], bool wide) {
  uint4* p = reinterpret_cast<uint4*>(to);
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i / 4),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                   "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
    } else {
      p[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      p[i / 4 + 1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    }
}

// Byte offset of 16-byte unit u of row r of a [128 x D] f16 tile.
template <int D>
__device__ __forceinline__ uint32_t unit_at(uint32_t r, uint32_t u) {
  if (D == 32) return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
  return (u >> 3) * 16384u + sw128_offset(r, u & 7);
}

// A warp fetches 32 rows of Q of a unit of dynamic heads, from row r0 of row tile
// g, side by side (kL lanes to a row): 8 components lie where 16 codes of hi or lo
// will, an even piece in hi's place and an odd one in lo's.
template <int D>
__device__ __forceinline__ void fetch_q(const CacheChunk& p, const Walk<D>& w, const UnitRows& unit,
                                        int g, int r0, uint32_t stage) {
  constexpr int kL = D / 8, kR = 32 / kL;
  const int lane = threadIdx.x & 31;
  int mine = -1;
  if (g * 128 + r0 + lane < unit.n) {
    int t, idx;
    row_of(w.rows, unit.first + g * 128 + r0 + lane, w.gk(), false, t, idx);
    mine = (int)((size_t)p.order[p.cls_first[w.cls] + idx] * p.a.c.n_q + t);
  }
  const uint16_t* slot_q = p.a.Q + (size_t)w.b * p.a.c.H * p.a.c.n_q * D;
#pragma unroll 2
  for (int i = 0; i < 32; i += kR) {
    const int rl = i + lane / kL, u = lane % kL;
    const int src = __shfl_sync(~0u, mine, rl);
    cp_async16(stage + (u & 1) * (kTile * D) + code_at<D>(r0 + rl, u >> 1),
               slot_q + (size_t)(unsigned)max(src, 0) * D + u * 8, src >= 0 ? 16 : 0);
  }
  cp_async_commit();
}

// The lowest n bits (none for n < 1, all from 32 on), and 16 for each of 2 bits.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n < 1 ? 0u : ~0u >> (n < 32 ? 32 - n : 0);
}
__device__ __forceinline__ uint32_t spread16(uint32_t x) {
  return (x & 1 ? 0xffffu : 0u) | (x & 2 ? 0xffff0000u : 0u);
}

// Whether `x` holds in one of the 128 threads that share named barrier `id`.
__device__ __forceinline__ bool any_of_128(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// The threads of row tile g turn its rows of Q into codes, where they lie, row r each:
// two parts or, if a row asks for it, three (see the top).  Returns the factor of the
// row's logits.  The arithmetic is in f16, which loses nothing here: a part is the
// rounded rest of the ones before, and what f16 rounds off (2^-25) is far below the
// least step of e5m2 (2^-16).
template <int D>
__device__ __noinline__ float q_codes(uint32_t stage, uint32_t r, int g, int* three_parts) {
  constexpr int kCodes = Smem<D>::CODES;
  auto load = [&](int u, uint32_t(&y)[8]) {
    lds_words(*reinterpret_cast<uint32_t(*)[4]>(y), stage + code_at<D>(r, u));
    lds_words(*reinterpret_cast<uint32_t(*)[4]>(y + 4), stage + kCodes + code_at<D>(r, u));
  };
  __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll 2
  for (int u = 0; u < D / 16; ++u) {
    uint32_t y[8];
    load(u, y);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&y[k])));
  }
  const float amax = fmaxf(__low2float(top2), __high2float(top2));
  const bool inf = amax == CUDART_INF_F;  // e4m3 has none
  const int bits = __float_as_int(amax);
  // amax 2^-e in (224, 448]
  int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  // components that e4m3 holds as a subnormal number: the first part keeps less of
  // them than 4 bits, and the second may round the rest
  int small = 0;
  const __nv_bfloat162 limit = __float2bfloat162_rn(pow2f(max(-126, min(120, e) - 6)));
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll 2
  for (int u = 0; u < D / 16; ++u) {
    uint32_t y[8];
    load(u, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 x = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&y[k]));
      small += __popc(__hlt2_mask(x, limit) & __hgt2_mask(x, zero));
    }
  }
  const bool three = any_of_128(1 + g, inf || small > 2 * 16);  // 16 bits for each
  if (r == 0) *three_parts = three;
  e = amax > 0.f ? max(-126, three ? min(113, e - 7) : min(120, e)) : 0;
  const float down = pow2f(-e);
  auto convert = [&](auto kind) {
    constexpr int kParts = decltype(kind)::value ? 3 : 2;
#pragma unroll 2
    for (int u = 0; u < D / 16; ++u) {
      uint32_t y[8], parts[kParts][4];
      load(u, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t codes[kParts][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t v = y[2 * k + j];
          uint32_t rest = pack_f16x2(__uint_as_float(v << 16) * down,
                                     __uint_as_float(v & 0xffff0000u) * down);
#pragma unroll
          for (int n = 0; n < kParts; ++n) {
            const bool e4m3 = kParts == 2 && n == 0;
            uint32_t code = e4m3 ? f16x2_e4m3x2(rest) : f16x2_e5m2x2(rest);
            const uint32_t f = e4m3 ? e4m3x2_f16x2((uint16_t)code) : e5m2x2_f16x2(code);
            const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&rest),
                                      *reinterpret_cast<const __half2*>(&f));
            rest = *reinterpret_cast<const uint32_t*>(&x);
            if (kParts == 3 && n == 0 && inf) {  // saturated infinities: their code, no rest
              if ((rest & 0x7fffu) == 0x7c00u) {
                code = (code & 0xff00u) | (rest >> 8 & 0xffu);
                rest &= 0xffff0000u;
              }
              if ((rest & 0x7fff0000u) == 0x7c000000u) {
                code = (code & 0xffu) | (rest >> 16 & 0xff00u);
                rest &= 0xffffu;
              }
            }
            codes[n][j] = code;
          }
        }
#pragma unroll
        for (int n = 0; n < kParts; ++n) parts[n][k] = codes[n][0] | codes[n][1] << 16;
      }
#pragma unroll
      for (int n = 0; n < kParts; ++n)
        st_shared_v4(stage + n * kCodes + code_at<D>(r, u), parts[n][0], parts[n][1],
                     parts[n][2], parts[n][3]);
    }
  };
  if (three)
    convert(Const<true>());
  else
    convert(Const<false>());
  return pow2f(e) * (rsqrtf((float)D) * kLog2e);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CacheChunk p) {
  using G = TileGeom<D>;
  using L = Smem<D>;
  const CacheCall& c = p.a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;          // [2] Q staged (128 arrivals)
  uint64_t* k_full = q_full + 2;          // [KST] codes of K have landed
  uint64_t* k_empty = k_full + L::KST;    // [KST] their products done
  uint64_t* r_full = k_empty + L::KST;    // [RST] codes of V have landed
  uint64_t* r_empty = r_full + L::RST;    // [RST] in registers (128 arrivals)
  uint64_t* v_full = r_empty + L::RST;    // [2] f16 V written (128)
  uint64_t* v_empty = v_full + 2;         // [2] its products done
  uint64_t* m_full = v_empty + 2;         // [4] a tile's scales and pattern (32)
  // of row tile g and half h of a tile, at 2 g + h
  uint64_t* s_full = m_full + 4;          // [4] S done
  uint64_t* p_full = s_full + 4;          // [4] P written, O rescaled (128)
  // P V done: its products, and the issuing thread itself, which has seen
  // v_full: what the converting warps wrote before is then visible
  uint64_t* o_done = p_full + 4;          // [4] (2)
  // the issuer of row tile g has come to a unit in which the tile has rows: its
  // softmax, which waits for nothing in units where it has none, may not run ahead
  // of the ring of scales (a parity tells two neighbouring phases apart only)
  uint64_t* begun = o_done + 4;           // [2] (1)
  uint64_t* drained = begun + 2;           // [2] every product of an issuer done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  // of row tile g: whether its rows of Q are in three parts
  int* three_parts = reinterpret_cast<int*>(smem + L::OFF_MISC + 8);  // [2]
  // of row tile g: the last of its units (counted from 1, at 4 g + count % 4) whose
  // V holds NaN at an edge
  int* nan_seg = reinterpret_cast<int*>(smem + L::OFF_MISC + 16);  // [8]
  const WaitCtl wc{abort_flag, p.a.status + kStatusCtas + blockIdx.x};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(v_full + i, 128);
      mbar_init(v_empty + i, 2);  // both issuers
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_done + i, 2);
    }
    for (int i = 0; i < L::KST; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 2);
    }
    for (int i = 0; i < L::RST; ++i) {
      mbar_init(r_full + i, 1);
      mbar_init(r_empty + i, 128);
    }
    for (int i = 0; i < 4; ++i) mbar_init(m_full + i, 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(begun + i, 1);
      mbar_init(drained + i, 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) nan_seg[i] = 0;
    fence_barrier_init();
    if (!p.by_unit) p.a.join[blockIdx.x] = make_int4(-1, 0, 0, 0);
    *wc.status = 0;
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // the joining kernel may be set up meanwhile; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;");
  const Share sh = find_share<D>(p, reinterpret_cast<long long*>(smem + L::OFF_SCAN));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sQ = smem_u32(smem + L::OFF_Q), sK = smem_u32(smem + L::OFF_K),
                 sV = smem_u32(smem + L::OFF_V), sR = smem_u32(smem + L::OFF_R),
                 sM = smem_u32(smem + L::OFF_META);
  constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S of row tile g at 128 g, O at 256 + 128 g

  Walk<D> w(p);
  int tile = 0;
  long long at = sh.end;  // where the unit begins
  if (sh.begin < sh.end) {
    const long long off = w.seek(sh.b, sh.in_slot);
    at = sh.begin - off;
    if (off > 0) tile = w.tiles_before(off);
    if (tile == w.ut) {  // all its tiles begin in the shares before
      tile = 0;
      at += w.cost();
      if (at < sh.end) w.next();
    }
  }
  if (at < sh.end) {
    if (warp < 8) {
      // ------------------------------------------------------------ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      const int g = warp >> 2, r = threadIdx.x & 127;
      const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_col = trow + kS + g * 128, o_col = trow + kO + g * 128;
      uint32_t n_tile = 0, n_s = 0, n_p = 0;  // tiles of the CTA; S and P of this row tile
      bool first = true;                      // it is the CTA's first
      bool staged = false;                    // the unit's rows of Q are on their way
      uint32_t n_unit = 0;                    // units in which it has rows
      for (;;) {
        const int tile_end = w.tiles_before(sh.end - at);
        const int gk = w.gk(), kv = p.cls_kv[w.cls];
        const bool ice = w.ice();
        const UnitRows unit = unit_rows(w.rows, w.pair, gk, ice);
        if (g * 128 < unit.n) {
          const bool live = g * 128 + r < unit.n;
          int t = 0, idx = 0;
          if (live) row_of(w.rows, unit.first + g * 128 + r, gk, ice, t, idx);
          const int h = p.order[p.cls_first[w.cls] + idx];
          const int pos = live ? w.rows.base + t : -1;
          const int lim_all = min(pos + 1, w.rows.cap);  // keys below it are seen
          const size_t row = ((size_t)w.b * c.H + h) * c.n_q + t;
          const bool warp_live = g * 128 + (warp & 3) * 32 < unit.n;
          float fac = 1.f;
          if (!ice) {
            const uint32_t stage = sQ + g * L::QTILE;
            if (!staged) fetch_q<D>(p, w, unit, g, (warp & 3) * 32, stage);
            staged = false;
            cp_async_wait<0>();
            __syncwarp();
            fac = q_codes<D>(stage, r, g, three_parts + g);
            fence_proxy_async_smem();
            mbar_arrive(q_full + g);
          }
          mbar_wait(begun + g, n_unit++ & 1, wc, kSiteBegin);
          float m = -CUDART_INF_F, l = 0.f;
          auto softmax = [&](auto kind) {
            constexpr bool kIce = decltype(kind)::value;
            for (int i = tile; i < tile_end; ++i) {
              const uint32_t nt = n_tile + (i - tile);
              mbar_wait(m_full + (nt & 3), (nt >> 2) & 1, wc, kSiteMeta);
#pragma unroll 1
              for (int hf = 0; hf < 2; ++hf) {
                const int bar = 2 * g + hf;
                // a half's P V of the tile before is done when its S is: that S was
                // issued after it
                if (!kIce)
                  mbar_wait(s_full + bar, n_s & 1, wc, kSiteS);
                else if (n_p > 0)
                  mbar_wait(o_done + bar, (n_p - 1) & 1, wc, kSiteO);
                __syncwarp();
                tc_fence_after();
                if (warp_live) {
                  const uint32_t meta = sM + (nt & 3) * 128 + 64 * hf;
                  const uint32_t col = s_col + 64 * hf;
                  const int j0 = i * kTile + 64 * hf;
                  const int lim = lim_all - j0;  // columns below it are seen
                  const uint32_t holes = lds_word(meta + 12) >> 4 * hf & 15u;
                  const bool edge = __any_sync(~0u, lim < 64 || holes);
                  // a row of S: 4 groups of 16 keys, each of one page with one scale
                  uint32_t s[4][16];
                  float gm[4];
                  if (!kIce) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld_max_x16(col + 16 * q, s[q], gm[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_wait_ld(s[q]);
                    asm volatile("" : "+f"(gm[0]), "+f"(gm[1]), "+f"(gm[2]), "+f"(gm[3]));
                  } else {
                    // distance of (row, column k): entry (row of the unit) - k + 127 of
                    // the window; entries e - k - 1 and e - k are read together
                    const float* pat =
                        reinterpret_cast<const float*>(smem + L::OFF_PAT + (nt & 3) * L::PAT);
                    const int e = g * 128 + r + 127 - 64 * hf;
                    const float* win = pat + (e & 1 ? L::WIN0 + e - 1 : L::WIN1 + e - 2);
                    pat += 64 * hf;
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                      const float4 x = *reinterpret_cast<const float4*>(pat + k);
                      const float2 w0 = *reinterpret_cast<const float2*>(win - k);
                      const float2 w1 = *reinterpret_cast<const float2*>(win - k - 2);
                      uint32_t* y = s[k / 16] + k % 16;
                      y[0] = __float_as_uint(x.x + w0.y);
                      y[1] = __float_as_uint(x.y + w0.x);
                      y[2] = __float_as_uint(x.z + w1.y);
                      y[3] = __float_as_uint(x.w + w1.x);
                    }
                  }
                  if (edge) {
                    // behind the row, or without a page: such a key weighs nothing, whatever
                    // a q or a pattern that is not finite makes of the zeros read for it
                    const uint32_t seen[2] = {low_bits(lim) & ~spread16(holes),
                                              low_bits(lim - 32) & ~spread16(holes >> 2)};
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                      if (!(seen[k / 32] >> (k % 32) & 1)) s[k / 16][k % 16] = 0xff800000u;
                  }
                  if (edge || kIce) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                      float x = fmax3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]),
                                      __uint_as_float(s[q][2]));
#pragma unroll
                      for (int k = 3; k < 15; k += 2)
                        x = fmax3(x, __uint_as_float(s[q][k]), __uint_as_float(s[q][k + 1]));
                      gm[q] = fmaxf(x, __uint_as_float(s[q][15]));
                    }
                  }
                  float a[4], b[4], inv[4], top = -CUDART_INF_F;
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const float4 mt = lds_f32x4(meta + 16 * q);
                    // never zero: keys that the row does not see are at -inf already, and
                    // 0 * -inf is NaN.  (The largest S, below 2^33, times the least normal
                    // number is nothing beside a logit.)
                    a[q] = kIce ? 1.f : fmaxf(fac * mt.x, FLT_MIN);
                    b[q] = mt.y;
                    inv[q] = mt.z;
                    top = fmaxf(top, fmaf(gm[q], a[q], b[q]));
                  }
                  const bool need = top > m + (kRoom + kLag);
                  if (__any_sync(~0u, need)) {
                    top -= kRoom;
                    const float corr = need ? fast_exp2(m - top) : 1.f;
                    if (need) m = top;
                    l *= corr;
                    if (i > tile || hf) {
                      // the last product into O: the other half's
                      mbar_wait(o_done + (bar ^ 1), (hf ? n_p : n_p - 1) & 1, wc, kSiteO);
                      __syncwarp();
                      tc_fence_after();
#pragma unroll 1
                      for (int q = 0; q < D; q += 16) {
                        uint32_t o[16];
                        tmem_ld_x16(o_col + q, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                          o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
                        tmem_st_x16(o_col + q, o);
                      }
                    }
                  }
                  const float base = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const uint64_t a2 = f2_pack(a[q], a[q]), b2 = f2_pack(b[q] - base, b[q] - base);
                    uint64_t sum = 0;
                    uint32_t pk[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                      float x, y;
                      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[q][k]),
                                               __uint_as_float(s[q][k + 1])),
                                       a2, b2),
                                x, y);
                      x = fast_exp2(x);
                      y = fast_exp2(y);
                      sum = f2_add(sum, f2_pack(x, y));
                      pk[k / 2] = pack_f16x2(x, y);
                    }
                    float x, y;
                    f2_unpack(sum, x, y);
                    l = fmaf(x + y, inv[q], l);
                    tmem_st_x8(col + 8 * q, pk);
                  }
                  tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(p_full + bar);
              }
              if (!kIce) ++n_s;
              ++n_p;
            }
          };
          if (ice)
            softmax(Const<true>());
          else
            softmax(Const<false>());
          // ---- the next unit's rows of Q, now that no product reads this one's: they
          // come while this one ends
          if (at + w.cost() < sh.end) {
            Walk<D> x = w;
            x.next();
            const UnitRows u0 = unit_rows(x.rows, x.pair, x.gk(), x.ice());
            staged = !x.ice() && g * 128 < u0.n;
            if (staged) fetch_q<D>(p, x, u0, g, (warp & 3) * 32, sQ + g * L::QTILE);
          }
          // ---- results
          mbar_wait(o_done + 2 * g, (n_p - 1) & 1, wc, kSiteO);
          mbar_wait(o_done + 2 * g + 1, (n_p - 1) & 1, wc, kSiteO);
          __syncwarp();
          tc_fence_after();
          const bool whole = tile == 0 && tile_end == w.ut;
          if (warp_live && !__any_sync(~0u, *abort_flag)) {
            uint32_t nan[D / 32];
#pragma unroll
            for (int q = 0; q < D / 32; ++q) nan[q] = 0;
            const bool edge_nan = nan_seg[4 * g + (n_unit & 3)] == (int)n_unit;
            if (edge_nan) {
              // V holds NaN at a key of an edge tile: rows that see it take it.  The
              // first such tile holds the first row's position or the last key, which
              // lies before it where the sequence is longer than the page table
              const int lo = min(w.rows.base + pair_span(w.rows, w.pair, gk, ice).lo,
                                 pair_extent(w.rows, w.pair, gk, ice));
              const int first = max(0, lo / kTile * kTile);
              for (int j = max(first, tile * kTile); j < min(lim_all, tile_end * kTile); ++j) {
                const int page = page_at(c, w.b, j >> c.page_shift);
                if (page < 0) continue;
                const uint32_t* v = reinterpret_cast<const uint32_t*>(
                    c.layer + (size_t)page * c.page_stride + c.off_v +
                    (((size_t)kv << c.page_shift) + (j & ((1 << c.page_shift) - 1))) * D);
                for (int q = 0; q < D / 4; ++q)
                  for (int k = 0; k < 4; ++k)
                    if ((v[q] >> (8 * k) & 0x7f) == 0x7f) nan[q / 8] |= 1u << (q % 8 * 4 + k);
              }
            }
            // a row without weight: 0, even if a key that it sees holds NaN (a part's sum
            // goes out as it is: another part may have weight)
            const float inv = whole ? 1.f / l : 1.f;
            const bool none = whole && l == 0.f;
            // partial sums: [D / 4][row][4], so that a warp's stores are contiguous
            const size_t part = (size_t)(2 * blockIdx.x + (first ? 0 : 1)) * kRows;
            const int pr = g * 128 + r;
            // a thread's row goes out in whole sectors where the base allows it: half as
            // many accesses as 16 bytes at a time
            uint16_t* to = p.a.out + row * D;
            const bool wide = (reinterpret_cast<uintptr_t>(p.a.out) & 31) == 0;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld_x32(o_col + 32 * q, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
              if (edge_nan) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (nan[q] >> k & 1) o[k] = 0x7fc00000u;
              }
              if (whole && live) {
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                  o[k / 2] = none ? 0u
                                  : pack_bf16x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1]));
                st_global_words16(to + 32 * q, o, wide);
              } else if (live) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  *reinterpret_cast<uint4*>(p.a.acc + part * D +
                                            ((size_t)(8 * q + k / 4) * kRows + pr) * 4) =
                      make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
              }
            }
            if (live && whole && p.a.lse) p.a.lse[row] = (m + log2f(l)) * kLn2;
            if (live && !whole)
              *reinterpret_cast<float2*>(p.a.ml + (part + pr) * 2) = make_float2(m, l);
          }
        }
        if (threadIdx.x == 0 && tile == 0) {
          // the unit begins here and ends in CTA `last`; only the last that begins
          // here can be cut
          const long long end = at + (long long)(w.ut - 1) * w.each;  // its last tile
          const int last = max((int)blockIdx.x, (int)(end / sh.size));
          p.a.join[p.by_unit ? w.number() : blockIdx.x] =
              make_int4(tile_end < w.ut ? w.b << 8 | w.cls : -1, w.pair, blockIdx.x,
                        last | (first ? 0 : 1 << 30));
        }
        n_tile += tile_end - tile;
        first = false;
        at += w.cost();
        if (at >= sh.end) break;
        tile = 0;
        w.next();
      }
    } else if (warp < 12) {
      // ------------------------------------------------------------ V: codes -> f16
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
      const int tid = threadIdx.x - 256;
      constexpr int kCh = D / 16;              // 16-byte chunks of a row of codes
      constexpr int kN = kTile * kCh / 128;    // chunks of a thread in a tile
      constexpr int kStep = 128 / kCh;         // rows between a thread's chunks
      // a row's upper chunks go with its neighbour's lower ones (d_h = 128), so
      // that the stores of 8 lanes touch every bank
      const int ch = tid % kCh, row0 = (tid / kCh) ^ (D == 128 ? ch >> 2 : 0);
      uint32_t vc = 0;
      int n_unit[2] = {0, 0};
      for (;;) {
        const int tile_end = w.tiles_before(sh.end - at);
        const bool both = unit_rows(w.rows, w.pair, w.gk(), w.ice()).n > 128;
        ++n_unit[0];
        n_unit[1] += both;
        // keys that not every row sees, and what lies behind the last key, may
        // hold NaN: 0 * NaN must not reach the other rows
        const int sure = min(w.rows.base + pair_span(w.rows, w.pair, w.gk(), w.ice()).lo + 1,
                             pair_extent(w.rows, w.pair, w.gk(), w.ice()));
        for (int i = tile; i < tile_end; ++i) {
          const uint32_t rs = vc % L::RST, st = vc & 1;
          mbar_wait(r_full + rs, (vc / L::RST) & 1, wc, kSiteRaw);
          uint4 x[kN];
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const float4 y = lds_f32x4(sR + rs * L::CODES + code_at<D>(row0 + n * kStep, ch));
            x[n] = *reinterpret_cast<const uint4*>(&y);
          }
          mbar_arrive(r_empty + rs);
          mbar_wait(v_empty + st, ((vc >> 1) & 1) ^ 1, wc, kSiteVFree);
          const bool clean = (i + 1) * kTile > sure;
          bool bad = false;
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const uint32_t in[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) e4m3x4_f16x4(in[k], y[2 * k], y[2 * k + 1]);
            if (clean) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __half2 z = *reinterpret_cast<const __half2*>(&y[k]);
                const uint32_t ok = __heq2_mask(z, z);
                bad |= ok != ~0u;
                y[k] &= ok;
              }
            }
            const uint32_t to = sV + st * L::TILE, row = row0 + n * kStep;
            st_shared_v4(to + unit_at<D>(row, 2 * ch), y[0], y[1], y[2], y[3]);
            st_shared_v4(to + unit_at<D>(row, 2 * ch + 1), y[4], y[5], y[6], y[7]);
          }
          if (bad) {
            nan_seg[n_unit[0] & 3] = n_unit[0];
            if (both) nan_seg[4 + (n_unit[1] & 3)] = n_unit[1];
          }
          fence_proxy_async_smem();
          mbar_arrive(v_full + st);
          ++vc;
        }
        at += w.cost();
        if (at >= sh.end) break;
        tile = 0;
        w.next();
      }
    } else {
      // ------------------------------------------------------------ products
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
      // (whole warps, so that descriptors and counters stay in uniform registers)
      const int uwarp = __shfl_sync(~0u, warp, 0);
      if (uwarp == 12 || uwarp == 14) {
        const int g = (uwarp - 12) >> 1;
        const uint32_t lead = lane == 0;
        auto commit = [&](uint64_t* bar) {
          if (lead) mma_commit(bar);
        };
        auto arrive = [&](uint64_t* bar) {
          if (lead) mbar_arrive(bar);
        };
        constexpr uint32_t id_o = idesc_f16(128, D, false, true);
        auto poll = [&](uint64_t* bar, uint32_t parity, const WaitCtl& c, int site) {
          poll_bar(bar, parity, c, site);
          __syncwarp();
        };
        const uint32_t s_col = tmem + kS + g * 128, o_col = tmem + kO + g * 128;
        const uint64_t qt = sdesc(sQ + g * L::QTILE, 16, 8 * D, swizzle_layout_code(D));
        uint32_t kc = 0, vc = 0, n_q = 0, n_p = 0;
        uint32_t id_s = 0;  // of the first part of the unit's rows of Q
        tile = __shfl_sync(~0u, tile, 0);
        for (;;) {
          const int tile_end = __shfl_sync(~0u, w.tiles_before(sh.end - at), 0);
          const bool ice = __shfl_sync(~0u, (int)w.ice(), 0);
          const bool mine = __shfl_sync(~0u, unit_rows(w.rows, w.pair, w.gk(), ice).n, 0) > g * 128;
          // K and V of tile i + 1 are waited for while a product of tile i runs, so
          // that the waits are not part of the row tile's chain
          auto wait_k = [&](uint32_t n) {
            poll(k_full + n % L::KST, (n / L::KST) & 1, wc, kSiteK);
          };
          auto wait_v = [&](uint32_t n) { poll(v_full + (n & 1), (n >> 1) & 1, wc, kSiteV); };
          // S of 64 keys: the tile's first or second half
          auto issue_s = [&](int hf) {
            const uint64_t kt = sdesc(sK + kc % L::KST * L::CODES + hf * 64 * D, 16, 8 * D,
                                      swizzle_layout_code(D));
            constexpr uint32_t id1 = idesc_codes(128, 64, 1);
            issue_codes<D / 32, (L::CODES >> 4)>(s_col + 64 * hf, qt, kt, id_s, id1, lead);
            if (id_s == id1) issue_third<D / 32, (L::CODES >> 4)>(s_col + 64 * hf, qt, kt, id1, lead);
            commit(s_full + 2 * g + hf);
          };
          auto k_done = [&]() {
            if (mine)
              commit(k_empty + kc % L::KST);
            else
              arrive(k_empty + kc % L::KST);
            ++kc;
          };
          if (mine) arrive(begun + g);
          if (!ice) {
            wait_k(kc);
            if (mine) {
              poll(q_full + g, n_q++ & 1, wc, kSiteQ);
              id_s = idesc_codes(128, 64, __shfl_sync(~0u, *(volatile int*)(three_parts + g), 0));
              tc_fence_after();
              issue_s(0);
              issue_s(1);
            }
            k_done();
          }
          wait_v(vc);
          for (int i = tile; i < tile_end; ++i) {
            const bool next = i + 1 < tile_end, more = !ice && next;
            const uint32_t st = vc++ & 1;
            if (mine) {
              const uint64_t vt = G::mnmajor_desc(sV + st * L::TILE, 0);
              constexpr int kVStep = 16 * G::SWZ >> 4;
#pragma unroll 1
              for (int hf = 0; hf < 2; ++hf) {
                const int bar = 2 * g + hf;
                poll(p_full + bar, n_p & 1, wc, kSiteP);
                tc_fence_after();
                issue_pv<kVStep>(o_col, s_col + 64 * hf, vt + 4 * kVStep * hf, id_o,
                                 i > tile || hf, lead);
                commit(o_done + bar);
                arrive(o_done + bar);
                if (hf)
                  commit(v_empty + st);
                else if (next) {
                  wait_v(vc);
                  if (!ice) wait_k(kc);
                }
                // S takes the columns of the P that these products read
                if (more) {
                  poll(o_done + bar, n_p & 1, wc, kSiteO);
                  tc_fence_after();
                  issue_s(hf);
                }
              }
              ++n_p;
            } else {
              arrive(v_empty + st);
              if (next) wait_v(vc);
              if (more) wait_k(kc);
            }
            if (more) k_done();
          }
          at += w.cost();
          if (at >= sh.end) break;
          tile = 0;
          w.next();
        }
        // every product has completed before TMEM is freed
        commit(drained + g);
        mbar_drain(drained + g, 0);
      } else if (warp == 13) {
        // ---------------------------------------------------------- codes and scales
        uint32_t kc = 0, vc = 0;
        const int per = 1 << (c.page_shift - 4);  // groups of 16 keys in a page
        const bool issues = lane < 8 && lane % per == 0;
        for (;;) {
          const int tile_end = w.tiles_before(sh.end - at);
          const int kv = p.cls_kv[w.cls], kh = w.ice() ? -1 : c.k_of[kv];
          const int ext = pair_extent(w.rows, w.pair, w.gk(), w.ice());
          // lane % 8: its group's page, two tiles ahead, and scales, one ahead
          auto look_up = [&](int tl) {
            const int j = tl * kTile + 16 * (lane & 7);
            return tl < tile_end && j < ext ? page_at(c, w.b, j >> c.page_shift) : -1;
          };
          auto scales = [&](int page) {
            if (page < 0) return make_float2(1.f, -1.f);
            const uint8_t* rec = c.layer + (size_t)page * c.page_stride;
            return make_float2(
                kh >= 0 ? __ldg(reinterpret_cast<const float*>(rec + c.off_ks) + kh) : 1.f,
                __ldg(reinterpret_cast<const float*>(rec + c.off_vs) + kv));
          };
          // frozen rows: the lane's 4 alphas and 12 rhos of a tile
          const UnitRows unit = unit_rows(w.rows, w.pair, w.gk(), w.ice());
          const float *al = nullptr, *rh = nullptr;
          int d_lo = 0;  // distance of the window's first entry, plus the tile's first key
          if (w.ice()) {
            int t0, idx;
            row_of(w.rows, unit.first, w.gk(), true, t0, idx);
            const size_t h = (size_t)p.order[p.cls_first[w.cls] + idx] * p.a.T_pat;
            al = p.a.alpha + h;
            rh = p.a.rho + h;
            d_lo = w.rows.base + t0 - 127;
          }
          float pat[16];
          auto fetch_pattern = [&](int tl) {
            if (!w.ice() || tl >= tile_end) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = tl * kTile + lane + 32 * k;
              pat[k] = j < p.a.T_pat ? __ldg(al + j) * kLog2e : -CUDART_INF_F;
            }
#pragma unroll
            for (int k = 0; k < 12; ++k) {
              const int d = d_lo - tl * kTile + lane + 32 * k;
              pat[4 + k] = d >= 0 && d < p.a.T_pat ? __ldg(rh + d) * kLog2e : -CUDART_INF_F;
            }
          };
          int page = look_up(tile), page1 = look_up(tile + 1);
          float2 sc = scales(page);
          fetch_pattern(tile);
          for (int i = tile; i < tile_end; ++i) {
            const int page2 = look_up(i + 2);
            const float2 sc1 = scales(page1);
            if (kh >= 0) {
              const uint32_t st = kc % L::KST;
              mbar_wait(k_empty + st, ((kc / L::KST) & 1) ^ 1, wc, kSiteKFree);
              if (lane == 0) mbar_arrive_expect_tx(k_full + st, L::CODES);
              __syncwarp();
              // each page from a lane of its own: one thread gets a copy through in
              // about 560 cycles only
              if (issues)
                tma_load_4d(smem + L::OFF_K + st * L::CODES + lane * 16 * D, &tm_k, k_full + st,
                            kh, page);
              ++kc;
            }
            const uint32_t st = vc % L::RST;
            mbar_wait(r_empty + st, ((vc / L::RST) & 1) ^ 1, wc, kSiteRawFree);
            const uint32_t holes = __ballot_sync(~0u, page < 0);
            if (lane < 8) {
              // a group without a page: every logit -inf
              const bool there = page >= 0;
              *reinterpret_cast<float4*>(smem + L::OFF_META + (vc & 3) * 128 + lane * 16) =
                  make_float4(sc.x, there ? __log2f(sc.y) : -CUDART_INF_F,
                              there ? __fdividef(1.f, sc.y) : 1.f, __uint_as_float(holes & 255u));
            }
            if (w.ice()) {
              float* to = reinterpret_cast<float*>(smem + L::OFF_PAT + (vc & 3) * L::PAT) + lane;
#pragma unroll
              for (int k = 0; k < 16; ++k) to[32 * k] = pat[k];
#pragma unroll
              for (int k = 0; k < 12; ++k) to[L::WIN1 - 1 + 32 * k] = pat[4 + k];
            }
            mbar_arrive(m_full + (vc & 3));
            fetch_pattern(i + 1);
            if (lane == 0) mbar_arrive_expect_tx(r_full + st, L::CODES);
            __syncwarp();
            if (issues)
              tma_load_4d(smem + L::OFF_R + st * L::CODES + lane * 16 * D, &tm_v, r_full + st, kv,
                          page);
            ++vc;
            page = page1;
            page1 = page2;
            sc = sc1;
          }
          at += w.cost();
          if (at >= sh.end) break;
          tile = 0;
          w.next();
        }
        // every copy has landed before the CTA ends
        for (uint32_t s = 0; s < L::KST; ++s)
          if (kc > s) mbar_drain(k_full + (kc - 1 - s) % L::KST, ((kc - 1 - s) / L::KST) & 1);
        for (uint32_t s = 0; s < L::RST; ++s)
          if (vc > s) mbar_drain(r_full + (vc - 1 - s) % L::RST, ((vc - 1 - s) / L::RST) & 1);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a unit that was cut (see cache_attn.cu); x: the unit or the
// CTA that left it, y: slices of its rows.  One block also gathers the CTAs' status.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8)
    cache_chunk_join_kernel(const __grid_constant__ CacheChunk p, int n_ctas, int split) {
  const CacheCall& c = p.a.c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    __shared__ int worst;
    if (threadIdx.x == 0) worst = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n_ctas; i += kJoinThreads)
      if (p.a.status[kStatusCtas + i]) worst = p.a.status[kStatusCtas + i];
    __syncthreads();
    if (threadIdx.x == 0) p.a.status[0] = worst;
  }
  if (p.by_unit) {  // a unit that the slot has no rows for has no entry
    const int b = blockIdx.x / p.slot_units, at = blockIdx.x - b * p.slot_units;
    int g = 0;
    while (g + 1 < p.n_groups && at >= p.group_unit[g + 1]) ++g;
    const int pair = (at - p.group_unit[g]) / (p.group_first[g + 1] - p.group_first[g]);
    if (pair >= pairs_of(slot_rows(c, b), p.group_width[g], p.group_static[g])) return;
  }
  const int4 u = p.a.join[blockIdx.x];
  if (u.x < 0) return;
  const int b = u.x >> 8, cls = u.x & 255, pair = u.y, cta = u.z, last = u.w & ~(1 << 30);
  const int n = last - cta + 1, first = 2 * cta + (u.w >> 30 & 1);
  const Rows rows = slot_rows(c, b);
  int gk = 0;
  bool ice = false;
  for (int g = 0; g < p.n_groups; ++g)
    if (cls >= p.group_first[g]) {
      gk = p.group_width[g];
      ice = p.group_static[g];
    }
  const UnitRows unit = unit_rows(rows, pair, gk, ice);
  const int per = kJoinThreads / split, s = threadIdx.x / per;
  for (int i0 = blockIdx.y * per; i0 < kRows * (D / 4); i0 += gridDim.y * per) {
    const int i = i0 + threadIdx.x % per, r = i % kRows, d = i / kRows * 4;
    const Part x = join_parts<kJoinAhead>(s, split, n, r < unit.n, [&](int k) {
      const size_t at = (size_t)(k == 0 ? first : 2 * (cta + k)) * kRows;
      const float2 ml = *reinterpret_cast<const float2*>(p.a.ml + (at + r) * 2);
      return Part{ml.x, ml.y,
                  *reinterpret_cast<const float4*>(p.a.acc + at * D +
                                                   ((size_t)(d / 4) * kRows + r) * 4)};
    });
    if (s == 0 && r < unit.n) {
      int t, idx;
      row_of(rows, unit.first + r, gk, ice, t, idx);
      const int h = p.order[p.cls_first[cls] + idx];
      const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
      *reinterpret_cast<uint2*>(p.a.out + row * D + d) = mean4(x.o, x.l);
      if (d == 0 && p.a.lse) p.a.lse[row] = (x.m + log2f(x.l)) * kLn2;
    }
    if (split > 1) __syncthreads();  // the threads' parts are read
  }
}

template <int D>
cudaError_t launch(const CacheChunk& p, int n_sms, cudaStream_t s) {
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(cache_chunk_kernel<D>),
                                       Smem<D>::ALLOC);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  const CacheCall& c = p.a.c;
  CUtensorMap tm_k, tm_v;
  const uint8_t* v = c.layer + c.off_v;
  // without stored K heads its map stands for V's and is never used
  if (!encode_pages(&tm_v, v, D, 1 << c.page_shift, c.H_kv, c.n_pages, c.page_stride) ||
      !encode_pages(&tm_k, c.H_k ? c.layer : v, D, 1 << c.page_shift, c.H_k ? c.H_k : c.H_kv,
                    c.n_pages, c.page_stride))
    return cudaErrorInvalidValue;
  cache_chunk_kernel<D><<<n_sms, kThreads, Smem<D>::ALLOC, s>>>(tm_k, tm_v, p);
  trace_end(s, "cache_chunk");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const long long units = (long long)p.slot_units * c.n_seqs;
  const int split = join_split(n_sms, units);
  cfg.gridDim = dim3(p.by_unit ? (int)units : n_sms,
                     kRows * (D / 4) * split / kJoinThreads / (p.by_unit ? 1 : 2));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  e = cudaLaunchKernelEx(&cfg, cache_chunk_join_kernel<D>, p, n_sms, split);
  trace_end(s, "cache_chunk_join");
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

CacheAttnWs cache_chunk_ws(int d_h, int n_sms) {
  CacheAttnWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~(size_t)255;
    return o;
  };
  w.status = take((kStatusCtas + (size_t)n_sms) * sizeof(int));
  w.join = take((size_t)n_sms * sizeof(int4));
  w.ml = take((size_t)2 * n_sms * kRows * 2 * 4);
  w.acc = take((size_t)2 * n_sms * kRows * d_h * 4);
  w.total = off;
  return w;
}

cudaError_t launch_cache_chunk(const CacheAttn& a, int d_h, int n_sms, cudaStream_t s) {
  CacheChunk p;
  p.a = a;
  const CacheCall& c = a.c;
  // classes: the dynamic and the frozen heads of each K/V head, those of equal
  // width side by side
  int n = 0;
  p.n_groups = 0;
  int width[2][kMaxHeads];
  for (int kv = 0; kv < c.H_kv; ++kv) {
    int at = kv * c.group;
    for (int kind = 0; kind < 2; ++kind) {
      width[kind][kv] = 0;
      for (int h = kv * c.group; h < (kv + 1) * c.group; ++h)
        if ((c.is_static[h] != 0) == (kind == 1)) {
          p.order[at++] = (uint8_t)h;
          ++width[kind][kv];
        }
    }
  }
  for (int w = c.group; w >= 1; --w)
    for (int kind = 0; kind < 2; ++kind) {
      const int before = n;
      for (int kv = 0; kv < c.H_kv; ++kv)
        if (width[kind][kv] == w) {
          p.cls_kv[n] = (uint8_t)kv;
          p.cls_first[n] = (int16_t)(kv * c.group + (kind ? width[0][kv] : 0));
          ++n;
        }
      if (n > before) {
        p.group_width[p.n_groups] = w;
        p.group_static[p.n_groups] = kind;
        p.group_first[p.n_groups++] = before;
      }
    }
  p.group_first[p.n_groups] = n;
  long long units = 0;
  for (int g = 0; g < p.n_groups; ++g) {
    const long long w = p.group_width[g], q = c.n_q;
    p.group_unit[g] = (int)units;
    units += (p.group_static[g] ? (q + kRows - 1) / kRows * w : (q * w + kRows - 1) / kRows) *
             (p.group_first[g + 1] - p.group_first[g]);
  }
  p.slot_units = (int)units;  // no more than rows: below 2^31
  p.by_unit = units * c.n_seqs <= n_sms;
  switch (d_h) {
    case 32: return launch<32>(p, n_sms, s);
    case 64: return launch<64>(p, n_sms, s);
    case 128: return launch<128>(p, n_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace saf
