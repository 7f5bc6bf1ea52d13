// cache_attn.cu — the hybrid layer over the paged 8-bit cache.
//
//   dynamic query head:  x_j = (q . k_j) s_k / sqrt(d)
//   frozen query head:   x_j = alpha(j) + rho(i - j)
//   out = sum_j e^{x_j} s_v v_j / sum_j e^{x_j},   lse = log sum_j e^{x_j}
//
// over the keys j <= i that lie on a page, with codes k_j, v_j and the scales
// s_k, s_v of their block.  The block's V scale joins the exponent: with
// y_j = x_j log2(e) + log2(s_v), the weights of the second product are
// p_j = 2^{y_j - m} under a base m that follows the maximum of the y, and the sum
// of the softmax is sum_j p_j / s_v.  So a weight is rounded to f16 relative to the
// largest contribution to `out`, whatever the scales of the blocks.
//
// This file: few query rows for each slot and K/V head (single tokens and
// short drafts; more rows go to cache_chunk.cu).  Such calls are bound by the
// bytes of the codes, so the kernel is built around keeping many of them in
// flight for few instructions: each warp has a ring of its own in shared
// memory, filled by asynchronous copies several steps ahead (a step is 4 KB:
// 16 keys of K and V at d_h = 128), and waits for nobody else.  Both products
// are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that the keys and
// the columns of V fill the 16 rows of a fragment and the few query rows its 8
// columns.  Which key or which component of d a slot of a fragment stands for
// is free as long as both operands agree; it is chosen so that a lane's slots
// are consecutive bytes, read 16 at a time without bank conflicts.
//
// Both products run in f16 with fp32 sums: f16 holds every e4m3 value; a row
// of q is scaled by a power of two into f16's range, which loses bits only of
// components 2^-28 below the row's largest.
#include <cuda_bf16.h>
#include <math_constants.h>
#include <string.h>

#include "cache_common.cuh"

namespace saf {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;

// ------------------------------------------------------------ work split
// A unit is (slot b, K/V head, row tile): up to 8 NT of the slot's n_new * group
// query rows (row r = t * group + h) against all its keys, in tiles of kTile
// keys.  The row tiles of a head lie side by side, so that their codes come from
// L2 after the first.  All tiles of all units, in that order, are cut into shares,
// one for each CTA, equal when a unit counts kUnitCost tiles more for its
// beginning and end (64 slots of up to 2500 tokens, 32 heads of 8: 39 us; with none
// 31% more, with one 7%, with three 2% less; 48 slots of up to 4096, 12 heads of 4,
// d_h = 64: 18 us, 19%, 3% and 8% more); a unit that is cut leaves partial sums,
// joined by a second kernel in the order of the CTAs.  Nothing depends on timing.  A
// share may be a single tile: what a step costs a CTA without company is the latency
// of its loads (one token against 1000, 16 heads of 4: 7.9 us; with shares of 4 tiles
// and more a third longer).
//
// Where no slot can have more than kWholeTiles tiles, each unit is one CTA's
// instead, without a search for its share and without a second kernel: when that was
// chosen, 7.6 us against 8.2 for 4 units of 4 tiles, 8.8 against 12.3 for 256.  With up
// to kWholeTilesMany it pays only where there are units for half of the SMs: 11.5
// against 8.4 us for 4 units of 8 tiles, 11.8 and 11.4 for 64, 13.1 and 15.6 for 256.
// (What a slot can have is the page table's width; what it has is on the GPU.  12
// heads against 100 tokens: 4.1 us in a table of 128 keys, 6.4 in one of 4096.)
constexpr int kUnitCost = 2;
constexpr int kWholeTiles = 4, kWholeTilesMany = 8;
constexpr int kJoinAhead = 8;    // parts that a joining thread has in flight

template <int D>
struct Geo {
  static constexpr int kGroups = 128 / D;           // of 16 keys in a warp's step: 4 KB of codes
  static constexpr int kStep = 16 * kGroups;        // keys of a step
  static constexpr int kTile = kWarps * kStep;      // keys of a tile
  // ring of a warp: K codes, V codes, then for each group K scale, V scale and
  // the number of keys
  static constexpr int kCodes = kStep * D;
  static constexpr int kMeta = 16 * kGroups;
  static constexpr int kStage = 2 * kCodes + 128;
  static_assert(kMeta <= 64, "half a stage holds V codes and the scales");
};

// Where 16-byte chunk `ch` of key `key` of a group lies.  A fragment's reads
// take keys (n / 2) + 4 (n % 2) for n = lane / 4, or the keys lane % 4 and the
// one 4 behind; either way 8 lanes touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int key, int ch) {
  if (D == 128) {
    const int f = (((key & 3) << 1) | ((key >> 1) & 1)) ^ (key & 4);
    return key * 128 + ((ch ^ f) << 4);
  }
  if (D == 64) {
    const int half = (key & 1) ^ ((key >> 2) & 1);
    return (key >> 1) * 128 + half * 64 + ((ch ^ (((key >> 1) & 1) << 1)) << 4);
  }
  return (key >> 2) * 128 + (((key & 3) ^ (((key >> 2) & 1) << 1)) << 5) + (ch << 4);
}

// The units of a slot, n_new * group rows in row tiles of MR for each K/V head, and
// the tiles of keys that each of them takes.
struct SlotUnits {
  int row_tiles, units, tiles;
};
template <int TILE, int MR>
__device__ __forceinline__ SlotUnits slot_units(const CacheCall& c, const Rows& r) {
  SlotUnits u;
  u.row_tiles = (int)(((long long)r.n_new * c.group + MR - 1) / MR);
  u.units = c.H_kv * u.row_tiles;
  u.tiles = max(1, (r.cap + TILE - 1) / TILE);  // rows that see nothing are written too
  return u;
}
template <int TILE, int MR>
__device__ __forceinline__ long long slot_cost(const CacheCall& c, int b) {
  const SlotUnits u = slot_units<TILE, MR>(c, slot_rows(c, b));
  return (long long)u.units * (u.tiles + kUnitCost);
}

struct Share {
  long long size, begin, end;  // of a CTA: the tiles that begin there
  int b;                       // the slot that holds `begin`, and how far behind its start
  long long in_slot;
};

// Every CTA finds its share: each thread sums a run of slots, a block scan
// gives the runs' beginnings, and the thread whose run holds the share's
// beginning walks it.
template <int TILE, int MR>
__device__ Share find_share(const CacheCall& c, long long* scan /* [kWarps + 2] */) {
  constexpr int n = kWarps * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (c.n_seqs + n - 1) / n;
  const int b0 = min(tid * per, c.n_seqs), b1 = min(b0 + per, c.n_seqs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += slot_cost<TILE, MR>(c, b);
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  long long total = 0, mine = upto - sum;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) mine += scan[i];
    total += scan[i];
  }
  Share s;
  s.size = (total + gridDim.x - 1) / gridDim.x;
  s.begin = min(s.size * blockIdx.x, total);
  s.end = min(s.begin + s.size, total);
  if (s.begin < s.end && mine <= s.begin && s.begin < mine + sum) {
    long long at = mine;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long t = slot_cost<TILE, MR>(c, b);
      if (s.begin < at + t) break;
      at += t;
    }
    scan[kWarps] = b;
    scan[kWarps + 1] = s.begin - at;
  }
  __syncthreads();
  s.b = (int)scan[kWarps];
  s.in_slot = scan[kWarps + 1];
  return s;
}

// CTAs that `tiles` more tiles take in shares of `size`; 32 bits are enough: a
// unit has fewer than 2^27 tiles.
__device__ __forceinline__ int cta_span(int tiles, long long size) {
  const unsigned s = (unsigned)(size < 0x40000000 ? size : 0x40000000);
  return (int)(((unsigned)tiles + s - 1) / s);
}

// The 8 x 8 block of 16-bit values of a warp (lane: row lane / 4, columns
// 2 (lane % 4) and the next), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// CTAs on an SM: as many as the registers allow without spills (8 rows: 166 of 168;
// a fourth CTA's 128 cost 32 x 8192 tokens of 16 heads 162 us for 150, two CTAs 178),
// and stages of a ring: with two it is 203 us, with four 160.
template <int NT>
constexpr int kCtas = NT == 1 ? 3 : 2;
constexpr int kStages = 3;
template <int D, int NT>
constexpr int smem_bytes() {
  const int ring = kWarps * kStages * Geo<D>::kStage, merge = kWarps * 8 * NT * (D + 2) * 4;
  return ring > merge ? ring : merge;
}

template <int D, int NT>  // NT: 8 query rows each
__global__ void __launch_bounds__(kWarps * 32, kCtas<NT>)
    cache_attn_kernel(const __grid_constant__ CacheAttn p, int row_tiles, bool whole_units,
                      bool by_unit) {
  constexpr int kMR = 8 * NT;
  constexpr int kG = Geo<D>::kGroups, kStep = Geo<D>::kStep, kTile = Geo<D>::kTile;
  constexpr int kKS = D / 16;            // steps of 16 along d
  constexpr int kKW = D / 16;            // words of a K row that a lane takes
  constexpr int kVW = D / 32;            // words of a V row that a lane takes
  constexpr int kKL = kKW < 4 ? kKW : 4; // words of one load
  constexpr int kVB = D / 8;             // bytes of a V row that a lane takes
  using G = Geo<D>;
  constexpr int kS = kStages;
  extern __shared__ __align__(128) uint8_t smem[];  // the rings; then the warps' sums
  float* merge = reinterpret_cast<float*>(smem);
  __shared__ long long scan[kWarps + 2];
  const CacheCall& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, cc = lane & 3;
  const int kq = (quad >> 1) + 4 * (quad & 1);  // key of the lane's rows of S^T (and kq + 8)

  // the joining kernel may be set up meanwhile; it waits for this one's end
  if (!whole_units) asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // nothing here waits without end
  const int per_slot = c.H_kv * row_tiles;  // units that a slot can have
  Share sh;
  if (whole_units) {
    sh.b = blockIdx.x / per_slot;
  } else {
    sh = find_share<kTile, kMR>(c, scan);
    if (threadIdx.x == 0 && !by_unit) p.join[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (sh.begin >= sh.end) return;
  }
  int b = sh.b;
  Rows rows = slot_rows(c, b);
  SlotUnits su = slot_units<kTile, kMR>(c, rows);
  int unit = 0, tile = 0;
  long long at;  // where the unit begins
  auto next_unit = [&]() {
    if (++unit < su.units) return;
    unit = 0;
    do {
      rows = slot_rows(c, ++b);
    } while (rows.n_new == 0);
    su = slot_units<kTile, kMR>(c, rows);
  };
  if (whole_units) {
    unit = blockIdx.x - sh.b * per_slot;
    if (unit >= su.units) return;
    tile = 0;
    at = sh.begin = 0;
    sh.end = sh.size = su.tiles;
  } else {
    const int cost = su.tiles + kUnitCost;
    unit = (int)(sh.in_slot / cost);
    tile = (int)(sh.in_slot - (long long)unit * cost);
    at = sh.begin - tile;
    if (tile >= su.tiles) {  // all its tiles begin in the shares before
      tile = 0;
      at += cost;
      if (at >= sh.end) return;
      next_unit();
    }
  }

  for (bool first = true;; first = false) {
    // ---- this segment: tiles [tile, tile_end) of the slot's unit (kv, rows r0 ..)
    const int kv = unit / su.row_tiles, r0 = (unit - kv * su.row_tiles) * kMR;
    const int tile_end = (int)min((long long)su.tiles, sh.end - at);
    const int ext = rows.cap;
    const int n_rows = min(kMR, rows.n_new * c.group - r0);
    const int steps = tile_end - tile;
    const int k_head = c.k_of[kv];
    const bool any_dyn = k_head >= 0;  // a dynamic head in the group
    const int key_w = tile * kTile + warp * kStep;  // first key of this warp's step 0

    // ---- Q: the lane's components 16 c .. 16 c + 15 (and + 64; 8 c .. for d_h = 32)
    // of row 8 nt + quad, on their way while the ring starts
    constexpr int kQW = D >= 64 ? 2 : 1;  // 16-byte words of a block of 64 components
    constexpr int kQB = D == 128 ? 2 : 1;
    uint4 qw[NT][kQB][kQW];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + quad;
      const uint16_t* qrow = nullptr;
      if (r < n_rows && any_dyn) {
        const int t = (r0 + r) / c.group, h = kv * c.group + r0 + r - t * c.group;
        if (!c.is_static[h]) qrow = p.Q + (((size_t)b * c.H + h) * c.n_q + t) * D;
      }
#pragma unroll
      for (int blk = 0; blk < kQB; ++blk)
#pragma unroll
        for (int u = 0; u < kQW; ++u) {
          qw[nt][blk][u] = make_uint4(0, 0, 0, 0);
          if (qrow)
            qw[nt][blk][u] =
                __ldg(reinterpret_cast<const uint4*>(qrow + 64 * blk + 8 * kQW * cc + 8 * u));
        }
    }

    // ---- the ring: pages are looked up 32 groups ahead, one for each lane.
    // Without K a stage is half as long and the ring has twice as many, so that as
    // many bytes are in flight.
    const uint32_t ring = smem_u32(smem) + warp * kS * G::kStage;
    const uint32_t stage = any_dyn ? G::kStage : G::kStage / 2;
    const uint32_t off_v = any_dyn ? G::kCodes : 0, off_m = off_v + G::kCodes;
    const int ahead = any_dyn ? kS - 1 : 2 * kS - 1;  // steps in flight
    const int in_page = (1 << c.page_shift) - 1;
    int pages = -1;
    auto group_key = [&](int s, int g) { return key_w + s * kTile + 16 * g; };
    // what does not change from step to step: the lane's chunks in a stage (the
    // third and fourth of d_h = 128 lie 8 keys = 1024 bytes behind the first two),
    // its places in the record, and where its scale comes from (lane 0: K, 1: V)
    constexpr int kChunks = D / 32;  // of a lane in 16 keys of K or V
    const uint32_t to0 = chunk_at<D>(lane / (D / 16), lane % (D / 16));
    const uint32_t to1 = chunk_at<D>(lane / (D / 16) + 512 / D, lane % (D / 16));
    const uint8_t* lane_v = c.layer + c.off_v + (((size_t)kv << c.page_shift) * D) + lane * 16;
    const uint8_t* lane_k =
        c.layer + (((size_t)(any_dyn ? k_head : 0) << c.page_shift) * D) + lane * 16;
    const uint8_t* lane_m = c.layer + (lane == 0 && any_dyn ? c.off_ks + 4 * (size_t)k_head
                                                            : c.off_vs + 4 * (size_t)kv);
    const uint32_t page_stride = (uint32_t)c.page_stride;  // below 2^32: checked on the host
    auto issue = [&](int s, uint32_t st) {
      if (s < steps) {
        if ((s * kG & 31) == 0) {  // the pages of steps s .. s + 32 / kG - 1
          const int at_s = s + lane / kG, key = group_key(at_s, lane % kG);
          pages = at_s < steps && key < ext ? page_at(c, b, key >> c.page_shift) : -1;
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const int page = __shfl_sync(~0u, pages, (s * kG + g) & 31);
          const int key = group_key(s, g);
          const uint32_t meta = st + off_m + 16 * g;
          if (lane == 2)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(meta + 8),
                         "r"(page < 0 ? 0 : min(16, ext - key))
                         : "memory");
          if (page < 0) continue;
          // the 16 keys of a group are contiguous; those behind the last one lie
          // on the page as well
          const uint64_t rec = (uint64_t)(uint32_t)page * page_stride;
          const uint64_t in_rec = rec + (uint32_t)((key & in_page) * D);
          const uint32_t to = st + g * 16 * D;
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            cp_async16(to + off_v + (i & 1 ? to1 : to0) + (i >> 1) * 1024,
                       lane_v + in_rec + i * 512, 16);
          if (any_dyn) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
              cp_async16(to + (i & 1 ? to1 : to0) + (i >> 1) * 1024, lane_k + in_rec + i * 512, 16);
          }
          if (lane < 2) cp_async4(meta + 4 * lane, lane_m + rec);
        }
      }
      cp_async_commit();
    };
    for (int i = 0; i < ahead; ++i) issue(i, ring + i * stage);

    // ---- the rows of this lane: 8 nt + 2c and the next
    int pos[NT][2], head[NT][2];
    bool ice[NT][2];
    const bool odd_rows = n_rows > 1;  // a single row leaves every lane's second one empty
    unsigned frozen = 0;               // bit 2 nt + i: row i of pair nt is frozen in some lane
    const int pos_lo = rows.base + r0 / c.group;  // the row that sees least
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * cc + i;
        const bool live = r < n_rows;
        const int t = live ? (r0 + r) / c.group : 0, hh = live ? r0 + r - t * c.group : 0;
        head[nt][i] = kv * c.group + hh;
        pos[nt][i] = live ? rows.base + t : -1;
        ice[nt][i] = live && c.is_static[head[nt][i]];
        frozen |= (__any_sync(~0u, ice[nt][i]) ? 1u : 0u) << (2 * nt + i);
      }

    // ---- Q^T fragments
    uint32_t qf[NT][kKS][2];
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[D / 4];
      float amax = 0.f;
#pragma unroll
      for (int blk = 0; blk < kQB; ++blk)
#pragma unroll
        for (int u = 0; u < kQW; ++u) {
          const uint4 w = qw[nt][blk][u];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[8 * (kQW * blk + u) + 2 * v] = __uint_as_float(ww[v] << 16);
            x[8 * (kQW * blk + u) + 2 * v + 1] = __uint_as_float(ww[v] & 0xffff0000u);
          }
        }
#pragma unroll
      for (int v = 0; v < D / 4; ++v) amax = fmaxf(amax, fabsf(x[v]));
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
      // amax * 2^-e in [2^14, 2^15); infinite rows keep their infinities
      int e = (__float_as_int(amax) >> 23) - 127 - 14;
      e = amax > 0.f ? max(-126, min(112, e)) : 0;
      const float down = pow2f(-e);
      const float f = pow2f(e) * (rsqrtf((float)D) * kLog2e);
#pragma unroll
      for (int i = 0; i < 2; ++i)  // of rows 2c, 2c + 1: held by quads 2c, 2c + 1
        fac[nt][i] = __shfl_sync(~0u, f, 4 * (2 * cc + i));
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        qf[nt][s][0] = pack_f16x2(x[4 * s] * down, x[4 * s + 1] * down);
        qf[nt][s][1] = pack_f16x2(x[4 * s + 2] * down, x[4 * s + 3] * down);
      }
    }

    // alpha and rho of the frozen rows for one step, fetched a step ahead.  Keys
    // [lo, lo + len) have both, counted from the lane's first key.
    float pa[NT][2][2 * kG], pr[NT][2][2 * kG];
    const float *al[NT][2], *rh[NT][2];
    int lo[NT][2], len[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int first = key_w + kq, x = pos[nt][i];
        const int j0 = max(0, x - p.T_pat + 1), j1 = min(x + 1, p.T_pat);
        al[nt][i] = p.alpha + (size_t)head[nt][i] * p.T_pat + first;
        rh[nt][i] = p.rho + (size_t)head[nt][i] * p.T_pat + (x - first);
        lo[nt][i] = j0 - first;
        len[nt][i] = ice[nt][i] ? max(0, j1 - j0) : 0;
      }
    auto fetch_pattern = [&](int s) {
      if (frozen == 0 || s >= steps) return;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (frozen >> (2 * nt + i) & 1) {
#pragma unroll
            for (int u = 0; u < 2 * kG; ++u) {
              const int j = s * kTile + 8 * u;  // 16 (u / 2) + 8 (u % 2)
              const bool ok = (unsigned)(j - lo[nt][i]) < (unsigned)len[nt][i];
              pa[nt][i][u] = ok ? __ldg(al[nt][i] + j) : -CUDART_INF_F;
              pr[nt][i][u] = ok ? __ldg(rh[nt][i] - j) : 0.f;
            }
          }
    };
    fetch_pattern(0);

    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[nt][j][u] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = -CUDART_INF_F;
        l[nt][i] = 0.f;
      }
    }
    bool v_nan = false;  // a NaN in V at a key that not every row sees

    uint32_t st = ring, st_next = ring + ahead * stage;  // stages of steps s and s + ahead
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      if (any_dyn)
        cp_async_wait<kS - 2>();
      else
        cp_async_wait<2 * kS - 2>();
      __syncwarp();
      // S^T of the step, [group][row pair][key kq: 2 rows | key kq + 8: 2 rows]
      float sc[kG][NT][4];
      int n[kG];
      float ks[kG], vs[kG];
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const float4 mt = lds_f32x4(st + off_m + 16 * g);
        ks[g] = mt.x;
        vs[g] = mt.y;
        n[g] = __float_as_int(mt.z);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) sc[g][nt][u] = 0.f;
        if (any_dyn && n[g] > 0) {
          uint32_t kw[2][kKW];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kKW / kKL; ++i) {
              uint32_t(&w)[kKL] = *reinterpret_cast<uint32_t(*)[kKL]>(kw[h] + kKL * i);
              const uint32_t a = st + g * 16 * D +
                                 (D == 32 ? chunk_at<D>(kq + 8 * h, cc >> 1) + (cc & 1) * 8
                                          : chunk_at<D>(kq + 8 * h, cc + 4 * i));
              lds_words(w, a);
            }
#pragma unroll
          for (int i = 0; i < kKS; ++i) {
            uint32_t a[4];
            e4m3x4_f16x4(kw[0][i], a[0], a[2]);
            e4m3x4_f16x4(kw[1][i], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(sc[g][nt], a, qf[nt][i][0], qf[nt][i][1]);
          }
        }
      }

      // y = x log2(e) + log2(s_v); keys that a row does not see: -inf
      bool grow = false;
      float inv[kG];
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        if (n[g] == 0) continue;
        const int key0 = group_key(s, g);
        const float lv = fast_log2(vs[g]);
        inv[g] = fast_rcp(vs[g]);
        const bool edge = n[g] < 16 || key0 + 15 > pos_lo;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = u & 1, k = kq + 8 * (u >> 1);
            float& y = sc[g][nt][u];
            if (i == 1 && !odd_rows) {
              y = -CUDART_INF_F;
              continue;
            }
            y = fmaf(y, fac[nt][i] * ks[g], lv);
            if ((frozen >> (2 * nt + i) & 1) && ice[nt][i])
              y = fmaf(pa[nt][i][2 * g + (u >> 1)] + pr[nt][i][2 * g + (u >> 1)], kLog2e, lv);
            if (edge && (k >= n[g] || key0 + k > pos[nt][i])) y = -CUDART_INF_F;
            grow |= y > m[nt][i] + (kRoom + kLag);
          }
      }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int g = 0; g < kG; ++g)
              if (n[g] > 0) top = fmaxf(top, fmaxf(sc[g][nt][i], sc[g][nt][2 + i]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            top = fmaxf(top - kRoom, m[nt][i]);
            const float corr = top == -CUDART_INF_F ? 1.f : fast_exp2(m[nt][i] - top);
            m[nt][i] = top;
            l[nt][i] *= corr;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[nt][j][i] *= corr;
              acc[nt][j][2 + i] *= corr;
            }
          }
      }
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        if (n[g] == 0) continue;
        const bool edge = n[g] < 16 || group_key(s, g) + 15 > pos_lo;
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float base = m[nt][u & 1] == -CUDART_INF_F ? 0.f : m[nt][u & 1];
            w[u] = (u & 1) && !odd_rows ? 0.f : fast_exp2(sc[g][nt][u] - base);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[nt][i] = fmaf(w[i] + w[2 + i], inv[g], l[nt][i]);
            pf[nt][i] = transpose8(pack_f16x2(w[2 * i], w[2 * i + 1]));
          }
        }
        // V^T: a lane's words hold 4 components of one of the keys c, c + 4, c + 8,
        // c + 12; pairs of keys side by side
        uint32_t vw[4][kVW];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          lds_words(vw[u], st + off_v + g * 16 * D +
                               chunk_at<D>(cc + 4 * u, quad * kVB >> 4) + (quad * kVB & 15));
#pragma unroll
        for (int i = 0; i < kVW; ++i) {
          uint32_t f[2][4];  // [keys c, c + 4 | c + 8, c + 12][component of the word]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            e4m3x4_f16x4(__byte_perm(vw[2 * h][i], vw[2 * h + 1][i], 0x5140), f[h][0],
                         f[h][1]);
            e4m3x4_f16x4(__byte_perm(vw[2 * h][i], vw[2 * h + 1][i], 0x7362), f[h][2],
                         f[h][3]);
          }
          if (edge) {  // 0 * NaN would reach rows that do not see the key
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const __half2 x = *reinterpret_cast<const __half2*>(&f[h][u]);
                const uint32_t ok = __heq2_mask(x, x);
                v_nan |= ok != ~0u;
                f[h][u] &= ok;
              }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(acc[nt][2 * i + j], a, pf[nt][0], pf[nt][1]);
          }
        }
      }
      fetch_pattern(s + 1);
      __syncwarp();
      issue(s + ahead, st_next);
      st_next = st;
      st += stage;
      if (st == ring + (ahead + 1) * stage) st = ring;
    }
    cp_async_wait<0>();

    if (__any_sync(~0u, v_nan)) {
      // rows that do see a key whose V holds NaN take it
      for (int s = 0; s < steps; ++s)
        for (int k = 0; k < kStep; ++k) {
          const int j = group_key(s, 0) + k, key0 = j & ~15;
          if (j >= ext || (ext - key0 >= 16 && key0 + 15 <= pos_lo)) continue;
          const int page = page_at(c, b, j >> c.page_shift);
          if (page < 0) continue;
          const uint8_t* v = c.layer + (size_t)page * c.page_stride + c.off_v +
                             (((size_t)kv << c.page_shift) + (j & in_page)) * D + quad * kVB;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < kVB; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (j <= pos[nt][i] && (v[t] & 0x7f) == 0x7f)
                  acc[nt][t / 2][2 * (t & 1) + i] = CUDART_NAN_F;
        }
    }

    __syncthreads();  // every warp has read its ring
    // ---- join the warps: [warp][row][D] sums, then [warp][row][2] of (m, l)
    float* mm = merge + kWarps * kMR * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][i] += __shfl_xor_sync(~0u, l[nt][i], o);
        const int r = 8 * nt + 2 * cc + i;
        if (r < n_rows) {
          float* dst = merge + (warp * kMR + r) * D + quad * kVB;
#pragma unroll
          for (int t = 0; t < kVB; t += 4)
            *reinterpret_cast<float4*>(dst + t) =
                make_float4(acc[nt][t / 2][i], acc[nt][t / 2][2 + i], acc[nt][t / 2 + 1][i],
                            acc[nt][t / 2 + 1][2 + i]);
          if (quad == 0)
            *reinterpret_cast<float2*>(mm + (warp * kMR + r) * 2) =
                make_float2(m[nt][i], l[nt][i]);
        }
      }
    __syncthreads();
    const bool whole = tile == 0 && tile_end == su.tiles;
    const int part = 2 * blockIdx.x + (first ? 0 : 1);
    for (int i = threadIdx.x; i < n_rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float mx = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, mm[(w * kMR + r) * 2]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = mm[(w * kMR + r) * 2];
        const float f = mx == -CUDART_INF_F ? 1.f : fast_exp2(mw - mx);
        sum = fmaf(f, mm[(w * kMR + r) * 2 + 1], sum);
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * kMR + r) * D + d);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
      }
      if (whole) {
        const int t = (r0 + r) / c.group, h = kv * c.group + r0 + r - t * c.group;
        const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
        *reinterpret_cast<uint2*>(p.out + row * D + d) = mean4(o, sum);
        if (d == 0 && p.lse) p.lse[row] = (mx + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.acc + ((size_t)part * kMR + r) * D + d) = o;
        if (d == 0)
          *reinterpret_cast<float2*>(p.ml + ((size_t)part * kMR + r) * 2) = make_float2(mx, sum);
      }
    }
    if (tile == 0 && threadIdx.x == 0 && !whole_units) {
      // the unit begins here and ends in CTA `last`; only the last that begins here
      // can be cut
      const int left = max(0, (int)(at + su.tiles - sh.end));  // tiles behind this CTA's
      const int last = blockIdx.x + cta_span(left, sh.size);
      p.join[by_unit ? b * per_slot + unit : blockIdx.x] =
          make_int4(tile_end < su.tiles ? b : -1, unit, blockIdx.x, last | (first ? 0 : 1 << 30));
    }

    // ---- the next unit
    at += su.tiles + kUnitCost;
    if (at >= sh.end) break;
    __syncthreads();  // the merge buffer is free again
    tile = 0;
    next_unit();
  }
}

// Joins the parts of a unit that was cut; x: the unit, or the CTA that left it
// to its successors; y: slices of its rows.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads)
    cache_join_kernel(const __grid_constant__ CacheAttn p, int row_tiles, bool by_unit,
                      int split) {
  constexpr int kMR = 8 * NT;
  const CacheCall& c = p.c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.join[blockIdx.x];
  if (by_unit) {  // a unit that the slot has no rows for has no entry
    const int per_slot = c.H_kv * row_tiles, slot = blockIdx.x / per_slot;
    const Rows r = slot_rows(c, slot);
    if ((int)blockIdx.x - slot * per_slot >= slot_units<1, kMR>(c, r).units) return;
  }
  if (u.x < 0) return;
  const int b = u.x;
  const Rows rows = slot_rows(c, b);
  const int tiles = slot_units<1, kMR>(c, rows).row_tiles;  // of rows
  const int kv = u.y / tiles, r0 = (u.y - kv * tiles) * kMR;
  const int cta = u.z, last = u.w & ~(1 << 30);
  const int n = last - cta + 1, first = 2 * cta + (u.w >> 30 & 1);
  const int n_rows = min(kMR, rows.n_new * c.group - r0);
  const int per = kJoinThreads / split, s = threadIdx.x / per;
  const int i = blockIdx.y * per + threadIdx.x % per;
  const int r = i / (D / 4), d = i % (D / 4) * 4;
  const Part x = join_parts<kJoinAhead>(s, split, n, r < n_rows, [&](int k) {
    const size_t at = (size_t)(k == 0 ? first : 2 * (cta + k)) * kMR + r;
    const float2 ml = *reinterpret_cast<const float2*>(p.ml + at * 2);
    return Part{ml.x, ml.y, *reinterpret_cast<const float4*>(p.acc + at * D + d)};
  });
  if (s || r >= n_rows) return;
  const int t = (r0 + r) / c.group, h = kv * c.group + r0 + r - t * c.group;
  const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
  *reinterpret_cast<uint2*>(p.out + row * D + d) = mean4(x.o, x.l);
  if (d == 0 && p.lse) p.lse[row] = (x.m + log2f(x.l)) * kLn2;
}

int n_ctas(int nt, int n_sms) { return n_sms * (nt == 1 ? kCtas<1> : kCtas<2>); }

template <int D, int NT>
cudaError_t launch(const CacheAttn& p, int n_sms, cudaStream_t s) {
  const int row_tiles = (int)(((long long)p.c.n_q * p.c.group + 8 * NT - 1) / (8 * NT));
  const long long units = (long long)p.c.n_seqs * p.c.H_kv * row_tiles;
  const long long keys = (long long)p.c.max_pages << p.c.page_shift;
  const int whole_tiles = units >= n_sms / 2 ? kWholeTilesMany : kWholeTiles;
  const bool whole = keys <= whole_tiles * Geo<D>::kTile && units < 1ll << 31;
  const bool by_unit = units <= n_ctas(NT, n_sms);
  const int grid = whole ? (int)units : n_ctas(NT, n_sms);
  cudaError_t e = set_max_dynamic_smem(
      reinterpret_cast<const void*>(cache_attn_kernel<D, NT>), smem_bytes<D, NT>());
  if (e != cudaSuccess) return e;
  trace_begin(s);
  cache_attn_kernel<D, NT>
      <<<grid, kWarps * 32, smem_bytes<D, NT>(), s>>>(p, row_tiles, whole, by_unit);
  trace_end(s, "cache_attn");
  e = cudaGetLastError();
  if (e != cudaSuccess || whole) return e;
  // launched while the first kernel runs; waits for its end before it reads
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int split = join_split(grid, units);
  cfg.gridDim = dim3(by_unit ? (int)units : grid,
                     (8 * NT * (D / 4) * split + kJoinThreads - 1) / kJoinThreads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  e = cudaLaunchKernelEx(&cfg, cache_join_kernel<D, NT>, p, row_tiles, by_unit, split);
  trace_end(s, "cache_join");
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch(const CacheAttn& p, int n_sms, cudaStream_t s) {
  return p.c.n_q * p.c.group <= 8 ? launch<D, 1>(p, n_sms, s) : launch<D, 2>(p, n_sms, s);
}

}  // namespace

CacheAttnWs cache_attn_ws(int d_h, int n_sms) {
  CacheAttnWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~(size_t)255;
    return o;
  };
  // the larger of both row counts
  const size_t n1 = (size_t)n_ctas(1, n_sms), n2 = (size_t)n_ctas(2, n_sms);
  const size_t n = n1 > n2 ? n1 : n2, rows = 2 * (n1 * 8 > n2 * 16 ? n1 * 8 : n2 * 16);
  w.status = take(256);
  w.join = take(n * sizeof(int4));
  w.ml = take(rows * 2 * 4);
  w.acc = take(rows * d_h * 4);
  w.total = off;
  return w;
}

cudaError_t launch_cache_attn(const CacheAttn& p, int d_h, int n_sms, cudaStream_t s) {
  switch (d_h) {
    case 32: return launch<32>(p, n_sms, s);
    case 64: return launch<64>(p, n_sms, s);
    case 128: return launch<128>(p, n_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace saf
