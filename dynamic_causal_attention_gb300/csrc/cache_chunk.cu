// cache_chunk.cu — the hybrid layer over the paged 8-bit cache for many query
// rows: prompts in pieces, drafts of many tokens, wide groups of heads.  Same
// mathematics as cache_attn.cu; here both products run on tcgen05 with fp32
// accumulators in TMEM.
//
// A unit is (slot, class, row pair): a class is the dynamic or the frozen
// query heads of one K/V head, its rows are r = t * heads + index, and a unit
// takes 256 of them as two tiles of 128, against the keys up to the last
// position among them in tiles of 128.  Splitting a group by kind keeps every
// warp uniform and spares frozen rows the Q K product.  All tiles of all
// units are cut into equal shares, one for each CTA (one per SM), as in
// cache_attn.cu.
//
// Warp roles (416 threads):
//   warps 0-3, 4-7   the softmax of row tile 0 and 1: one row per thread.  They
//                    also stage Q (scaled into f16) and write the results.
//   warps 8-11       turn e4m3 codes into f16 tiles in shared memory (K: K-major,
//                    V: MN-major, 128-byte swizzle); each thread holds the next
//                    tile's codes in registers while it converts this one.
//   warp 12          allocates TMEM; one lane issues every product.
//
// TMEM: S of the two row tiles (128 columns each), then their O.  P, as packed
// f16, overwrites the first half of its own S, so the next S of a row tile
// waits for the product that reads P; the other row tile's products and
// softmax run meanwhile.  A frozen row writes its logits into S itself.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "attn_common.cuh"
#include "cache_common.cuh"

namespace saf {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 256;     // query rows of a unit
constexpr int kTile = 128;     // keys of a tile
constexpr int kThreads = 416;
constexpr long long kMinTiles = 1;

enum : int { kSiteQ = 64, kSiteK, kSiteV, kSiteP, kSiteO, kSiteS, kSiteMeta, kSiteKFree, kSiteVFree };

// Instruction descriptor with f16 operands and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ int pairs_of(const Rows& r, int gk) {
  return (int)(((long long)r.n_new * gk + kRows - 1) / kRows);
}
__device__ __forceinline__ int pair_extent(const Rows& r, int pair, int gk) {
  int t_hi = (pair * kRows + kRows - 1) / gk + 1;
  if (t_hi > r.n_new) t_hi = r.n_new;
  const int e = r.base + t_hi;
  return e < 0 ? 0 : (e < r.cap ? e : r.cap);
}
__device__ __forceinline__ int pair_tiles(const Rows& r, int pair, int gk) {
  const int n = (pair_extent(r, pair, gk) + kTile - 1) / kTile;
  return n < 1 ? 1 : n;  // rows that see nothing are written too
}

// Walks the units in order: slots, then classes of equal width, row pairs,
// classes.
struct Walk {
  const CacheChunk& p;
  Rows rows;
  int b, group, pair, cls, ut;
  __device__ __forceinline__ explicit Walk(const CacheChunk& q) : p(q) {}
  __device__ __forceinline__ int gk() const { return p.group_width[group]; }
  __device__ long long group_tiles(const Rows& r, int g) const {
    long long sum = 0;
    const int w = p.group_width[g], n = pairs_of(r, w);
    for (int i = 0; i < n; ++i) sum += pair_tiles(r, i, w);
    return sum * (p.group_first[g + 1] - p.group_first[g]);
  }
  __device__ long long slot_tiles(int slot) const {
    const Rows r = slot_rows(p.a.c, slot);
    long long sum = 0;
    for (int g = 0; g < p.n_groups; ++g) sum += group_tiles(r, g);
    return sum;
  }
  // to the unit that holds tile `at` of slot `slot`; returns the tile in it
  __device__ int seek(int slot, long long at) {
    b = slot;
    rows = slot_rows(p.a.c, b);
    group = 0;
    while (group < p.n_groups - 1) {
      const long long n = group_tiles(rows, group);
      if (at < n) break;
      at -= n;
      ++group;
    }
    pair = 0;
    const int n_cls = p.group_first[group + 1] - p.group_first[group];
    ut = pair_tiles(rows, 0, gk());
    while (at >= (long long)ut * n_cls) {
      at -= (long long)ut * n_cls;
      ++pair;
      ut = pair_tiles(rows, pair, gk());
    }
    cls = p.group_first[group] + (int)(at / ut);
    return (int)(at % ut);
  }
  __device__ void next() {
    if (++cls == p.group_first[group + 1]) {
      if (++pair >= pairs_of(rows, gk())) {
        pair = 0;
        if (++group == p.n_groups) {
          do {
            rows = slot_rows(p.a.c, ++b);
          } while (rows.n_new == 0);
          group = 0;
        }
      }
      cls = p.group_first[group];
      ut = pair_tiles(rows, pair, gk());
    }
  }
};

struct Share {
  long long size, begin, end, in_slot;
  int b;
};
// As in cache_attn.cu: a run of slots for each thread, one block scan.
__device__ Share find_share(const CacheChunk& p, long long* scan /* [threads + 4] */) {
  const Walk w(p);
  const int n = blockDim.x, tid = threadIdx.x, n_seqs = p.a.c.n_seqs;
  const int per = (n_seqs + n - 1) / n;
  const int b0 = min(tid * per, n_seqs), b1 = min(b0 + per, n_seqs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += w.slot_tiles(b);
  scan[tid] = sum;
  __syncthreads();
  for (int o = 1; o < n; o <<= 1) {
    const long long x = tid >= o ? scan[tid - o] : 0;
    __syncthreads();
    scan[tid] += x;
    __syncthreads();
  }
  Share s;
  const long long total = scan[n - 1];
  s.size = (total + gridDim.x - 1) / gridDim.x;
  if (s.size < kMinTiles) s.size = kMinTiles;
  s.begin = min(s.size * blockIdx.x, total);
  s.end = min(s.begin + s.size, total);
  const long long mine = scan[tid] - sum;
  if (s.begin < s.end && mine <= s.begin && s.begin < mine + sum) {
    long long at = mine;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long t = w.slot_tiles(b);
      if (s.begin < at + t) break;
      at += t;
    }
    scan[n] = b;
    scan[n + 1] = s.begin - at;
  }
  __syncthreads();
  s.b = (int)scan[n];
  s.in_slot = scan[n + 1];
  return s;
}

template <int D>
struct Smem {
  static constexpr int TILE = kTile * D * 2;  // f16
  static constexpr int OFF_Q = 0;             // two row tiles
  static constexpr int OFF_K = 2 * TILE;      // two stages
  static constexpr int OFF_V = 4 * TILE;      // two stages
  static constexpr int OFF_META = 6 * TILE;   // 4 tiles x 8 groups of 16 keys x 16 bytes
  static constexpr int OFF_SCAN = OFF_META + 4 * 8 * 16;
  static constexpr int OFF_BAR = OFF_SCAN + (kThreads + 4) * 8;
  static constexpr int NBAR = 2 + 4 + 4 + 4 + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 32;
  static constexpr int ALLOC = BYTES + 1024;  // slack to align the base to 1024 B
  static_assert(ALLOC <= 232448, "shared memory budget exceeded");
};

// Byte offset of 16-byte unit u of row r of a [128 x D] f16 tile.
template <int D>
__device__ __forceinline__ uint32_t unit_at(uint32_t r, uint32_t u) {
  if (D == 32) return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
  return (u >> 3) * 16384u + sw128_offset(r, u & 7);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CacheChunk p) {
  using G = TileGeom<D>;
  using L = Smem<D>;
  const CacheCall& c = p.a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;          // [2] Q staged (128 arrivals)
  uint64_t* k_full = q_full + 2;    // [2] stage converted (128)
  uint64_t* k_empty = k_full + 2;   // [2] its products done
  uint64_t* v_full = k_empty + 2;   // [2]
  uint64_t* v_empty = v_full + 2;   // [2]
  uint64_t* m_full = v_empty + 2;   // [4] a tile's scales (128)
  uint64_t* s_full = m_full + 4;    // [2] S of a row tile done
  uint64_t* p_full = s_full + 2;    // [2] P written, O rescaled (128)
  uint64_t* o_done = p_full + 2;    // [2] a tile's P V done
  uint64_t* drained = o_done + 2;   // every product done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  int* nan_seg = reinterpret_cast<int*>(smem + L::OFF_MISC + 16);  // [4]
  const WaitCtl wc{abort_flag, p.a.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(k_full + i, 128);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 128);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(m_full + i, 128);
    mbar_init(drained, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) nan_seg[i] = 0;
    fence_barrier_init();
    p.a.join[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  const Share sh = find_share(p, reinterpret_cast<long long*>(smem + L::OFF_SCAN));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sQ = smem_u32(smem + L::OFF_Q), sK = smem_u32(smem + L::OFF_K),
                 sV = smem_u32(smem + L::OFF_V), sM = smem_u32(smem + L::OFF_META);
  constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S of row tile g at 128 g, O at 256 + 128 g

  if (sh.begin < sh.end) {
    Walk w(p);
    int tile = w.seek(sh.b, sh.in_slot);
    long long at = sh.begin;
    if (warp < 8) {
      // ------------------------------------------------------------ softmax
      const int g = warp >> 2, r = threadIdx.x & 127;
      const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_col = trow + kS + g * 128, o_col = trow + kO + g * 128;
      uint32_t n_tile = 0, n_s = 0, n_p = 0;  // tiles of the CTA; S and P of this row tile
      for (int seg = 0;; ++seg) {
        const int tile_end = (int)min((long long)w.ut, tile + (sh.end - at));
        const int gk = w.gk(), kv = p.cls_kv[w.cls];
        const bool ice = p.cls_static[w.cls];
        const int n_rows = (int)min((long long)kRows,
                                    (long long)w.rows.n_new * gk - (long long)w.pair * kRows);
        if (g * 128 < n_rows) {
          const bool live = g * 128 + r < n_rows;
          const int rr = w.pair * kRows + g * 128 + r;
          const int t = live ? rr / gk : 0;
          const int h = p.order[p.cls_first[w.cls] + (live ? rr - t * gk : 0)];
          const int pos = live ? w.rows.base + t : -1;
          const int lim_all = min(pos + 1, w.rows.cap);  // keys below it are seen
          const size_t row = ((size_t)w.b * c.H + h) * c.n_q + t;
          const bool warp_live = g * 128 + (warp & 3) * 32 < n_rows;
          float fac = 1.f;
          if (!ice) {
            // the row of Q, scaled by a power of two so that its largest
            // component lies in [2^14, 2^15)
            uint4 q[D / 8];
            float amax = 0.f;
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
              q[u] = live ? __ldg(reinterpret_cast<const uint4*>(p.a.Q + row * D) + u)
                          : make_uint4(0, 0, 0, 0);
              const uint32_t x[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
              for (int v = 0; v < 4; ++v)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[v] << 16)),
                                         fabsf(__uint_as_float(x[v] & 0xffff0000u))));
            }
            int e = (__float_as_int(amax) >> 23) - 127 - 14;
            e = amax > 0.f ? max(-126, min(112, e)) : 0;
            const float down = pow2f(-e);
            fac = pow2f(e) * (rsqrtf((float)D) * kLog2e);
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
              const uint32_t x[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
              uint32_t y[4];
#pragma unroll
              for (int v = 0; v < 4; ++v)
                y[v] = pack_f16x2(__uint_as_float(x[v] << 16) * down,
                                  __uint_as_float(x[v] & 0xffff0000u) * down);
              st_shared_v4(sQ + g * L::TILE + unit_at<D>(r, u), y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full + g);
          }
          float m = -CUDART_INF_F, l = 0.f;
          for (int i = tile; i < tile_end; ++i) {
            const uint32_t nt = n_tile + (i - tile);
            mbar_wait(m_full + (nt & 3), (nt >> 2) & 1, wc, kSiteMeta);
            if (!ice) {
              mbar_wait(s_full + g, n_s & 1, wc, kSiteS);
              ++n_s;
            }
            if (n_p > 0) mbar_wait(o_done + g, (n_p - 1) & 1, wc, kSiteO);
            __syncwarp();
            tc_fence_after();
            if (warp_live) {
              const uint32_t meta = sM + (nt & 3) * 128;
              const int j0 = i * kTile;
              const int lim = lim_all - j0;  // columns below it are seen
              const bool edge = __any_sync(~0u, lim < kTile);
              float gm[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t s[32];
                if (!ice) {
                  tmem_ld_x32(s_col + 32 * q, s);
                  tmem_wait_ld(s);
                } else {
                  const float* al = p.a.alpha + (size_t)h * p.a.T_pat + j0 + 32 * q;
                  const float* rh = p.a.rho + (size_t)h * p.a.T_pat + (pos - j0 - 32 * q);
                  // inside the vectors for every column of the warp's rows?
                  const int d0 = pos - j0 - 32 * q;
                  const bool in = j0 + 32 * q + 31 < p.a.T_pat && d0 < p.a.T_pat && d0 >= 31;
                  if (__all_sync(~0u, in)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                      s[k] = __float_as_uint((__ldg(al + k) + __ldg(rh - k)) * kLog2e);
                  } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                      const bool ok = j0 + 32 * q + k < p.a.T_pat && d0 - k >= 0 &&
                                      d0 - k < p.a.T_pat;
                      s[k] = __float_as_uint(
                          ok ? (__ldg(al + k) + __ldg(rh - k)) * kLog2e : -CUDART_INF_F);
                    }
                  }
                  uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(s);
                  uint32_t(&hi)[16] = *reinterpret_cast<uint32_t(*)[16]>(s + 16);
                  tmem_st_x16(s_col + 32 * q, lo);
                  tmem_st_x16(s_col + 32 * q + 16, hi);
                }
                if (edge) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (32 * q + k >= lim) s[k] = 0xff800000u;
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  float x = fmax3(__uint_as_float(s[16 * hh]), __uint_as_float(s[16 * hh + 1]),
                                  __uint_as_float(s[16 * hh + 2]));
#pragma unroll
                  for (int k = 3; k < 15; k += 2)
                    x = fmax3(x, __uint_as_float(s[16 * hh + k]),
                              __uint_as_float(s[16 * hh + k + 1]));
                  gm[2 * q + hh] = fmaxf(x, __uint_as_float(s[16 * hh + 15]));
                }
              }
              float top = -CUDART_INF_F;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 mt = lds_f32x4(meta + 16 * k);
                top = fmaxf(top, fmaf(gm[k], ice ? 1.f : fac * mt.x, mt.y));
              }
              // the maximum moves only when it would grow by more than 2^8:
              // weights up to 2^8 fit f16 as well
              const bool need = top > m + 8.f;
              if (__any_sync(~0u, need)) {
                const float corr = need ? fast_exp2(m - top) : 1.f;
                if (need) m = top;
                l *= corr;
                if (i > tile) {
#pragma unroll 1
                  for (int q = 0; q < D; q += 32) {
                    uint32_t o[32];
                    tmem_ld_x32(o_col + q, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                      o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
                    tmem_st_x16(o_col + q, *reinterpret_cast<uint32_t(*)[16]>(o));
                    tmem_st_x16(o_col + q + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
                  }
                }
              }
              const float base = m == -CUDART_INF_F ? 0.f : m;
              if (ice) tmem_wait_st();
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t s[32], pk[16];
                tmem_ld_x32(s_col + 32 * q, s);
                tmem_wait_ld(s);
                if (edge) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (32 * q + k >= lim) s[k] = 0xff800000u;
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const float4 mt = lds_f32x4(meta + 16 * (2 * q + hh));
                  const float a = ice ? 1.f : fac * mt.x, b = mt.y - base;
                  const uint64_t a2 = f2_pack(a, a), b2 = f2_pack(b, b);
                  uint64_t sum = 0;
#pragma unroll
                  for (int k = 0; k < 16; k += 2) {
                    float x, y;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[16 * hh + k]),
                                             __uint_as_float(s[16 * hh + k + 1])),
                                     a2, b2),
                              x, y);
                    x = fast_exp2(x);
                    y = fast_exp2(y);
                    sum = f2_add(sum, f2_pack(x, y));
                    pk[8 * hh + k / 2] = pack_f16x2(x, y);
                  }
                  float x, y;
                  f2_unpack(sum, x, y);
                  l = fmaf(x + y, mt.z, l);
                }
                tmem_st_x16(s_col + 16 * q, pk);
              }
              tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(p_full + g);
            ++n_p;
          }
          // ---- results
          mbar_wait(o_done + g, (n_p - 1) & 1, wc, kSiteO);
          __syncwarp();
          tc_fence_after();
          const bool whole = tile == 0 && tile_end == w.ut;
          if (warp_live && !__any_sync(~0u, *abort_flag)) {
            uint32_t nan[D / 32];
#pragma unroll
            for (int q = 0; q < D / 32; ++q) nan[q] = 0;
            if (nan_seg[seg & 3] == seg + 1) {
              // V holds NaN at a key of an edge tile: rows that see it take it
              const int first = max(0, (w.rows.base + w.pair * kRows / gk) / kTile * kTile);
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
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            const size_t part =
                ((size_t)(2 * blockIdx.x + (at == sh.begin ? 0 : 1)) * kRows + g * 128 + r);
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld_x32(o_col + 32 * q, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
                if (nan[q] >> k & 1) o[k] = 0x7fc00000u;
              }
              if (live && whole) {
                uint4* dst = reinterpret_cast<uint4*>(p.a.out + row * D + 32 * q);
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                  dst[k / 8] = make_uint4(
                      pack_bf16x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])),
                      pack_bf16x2(__uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])),
                      pack_bf16x2(__uint_as_float(o[k + 4]), __uint_as_float(o[k + 5])),
                      pack_bf16x2(__uint_as_float(o[k + 6]), __uint_as_float(o[k + 7])));
              } else if (live) {
                uint4* dst = reinterpret_cast<uint4*>(p.a.acc + part * D + 32 * q);
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  dst[k / 4] = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
              }
            }
            if (live && whole && p.a.lse) p.a.lse[row] = (m + log2f(l)) * kLn2;
            if (live && !whole)
              *reinterpret_cast<float2*>(p.a.ml + part * 2) = make_float2(m, l);
          }
        }
        if (threadIdx.x == 0 && tile == 0 && tile_end < w.ut) {
          // the unit begins here and ends in CTA `last`
          const int last = (int)((at + w.ut - 1) / sh.size);
          p.a.join[blockIdx.x] =
              make_int4(w.b, w.pair, w.cls, last | (at == sh.begin ? 0 : 1 << 30));
        }
        n_tile += tile_end - tile;
        at += tile_end - tile;
        if (at >= sh.end) break;
        tile = 0;
        w.next();
      }
    } else if (warp < 12) {
      // ------------------------------------------------------------ codes -> f16
      const int tid = threadIdx.x - 256;
      constexpr int kCh = D / 16;              // 16-byte chunks of a row of codes
      constexpr int kN = kTile * kCh / 128;    // chunks of a thread in a tile
      constexpr int kStep = 128 / kCh;         // rows between a thread's chunks
      const int ch = tid % kCh, row0 = tid / kCh;
      uint4 kx[kN], vx[kN];
      float meta_k = 1.f, meta_v = 1.f;  // scales of group tid (tid < 8)
      bool meta_there = false;
      // the tile being fetched, ahead of the one being converted
      Walk f = w;
      int f_tile = tile, f_end = 0;
      long long f_at = at;
      bool f_more = true;
      int f_ext = 0, f_kv = 0, f_kh = -1;
      auto open = [&]() {
        f_end = (int)min((long long)f.ut, f_tile + (sh.end - f_at));
        f_ext = pair_extent(f.rows, f.pair, f.gk());
        f_kv = p.cls_kv[f.cls];
        f_kh = p.cls_static[f.cls] ? -1 : c.k_of[f_kv];
      };
      open();
      auto address = [&](int key, int head, size_t off, bool& ok) {
        const int j = f_tile * kTile + key;
        ok = f_more && j < f_ext;
        const int page = ok ? page_at(c, f.b, j >> c.page_shift) : -1;
        ok = page >= 0;
        return c.layer + (size_t)(ok ? page : 0) * c.page_stride + off +
               (((size_t)head << c.page_shift) + (j & ((1 << c.page_shift) - 1))) * D + 16 * ch;
      };
      auto fetch_k = [&]() {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          bool ok = false;
          const uint8_t* a = nullptr;
          if (f_kh >= 0) a = address(row0 + n * kStep, f_kh, 0, ok);
          kx[n] = ok ? __ldg(reinterpret_cast<const uint4*>(a)) : make_uint4(0, 0, 0, 0);
        }
      };
      auto fetch_v = [&]() {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          bool ok;
          const uint8_t* a = address(row0 + n * kStep, f_kv, c.off_v, ok);
          vx[n] = ok ? __ldg(reinterpret_cast<const uint4*>(a)) : make_uint4(0, 0, 0, 0);
        }
        if (tid < 8) {
          const int j = f_tile * kTile + 16 * tid;
          const int page = f_more && j < f_ext ? page_at(c, f.b, j >> c.page_shift) : -1;
          meta_there = page >= 0;
          if (meta_there) {
            const uint8_t* rec = c.layer + (size_t)page * c.page_stride;
            meta_v = __ldg(reinterpret_cast<const float*>(rec + c.off_vs) + f_kv);
            meta_k = f_kh >= 0 ? __ldg(reinterpret_cast<const float*>(rec + c.off_ks) + f_kh) : 1.f;
          }
        }
      };
      auto fetch_next = [&]() {  // moves on to the next tile of the CTA
        if (++f_tile < f_end) return;
        f_at += f_end - (f_at == sh.begin ? tile : 0);
        if (f_at >= sh.end) {
          f_more = false;
          return;
        }
        f_tile = 0;
        f.next();
        open();
      };
      // one chunk of 16 codes as two units of 8 f16; lanes of the upper half of
      // a row store their second unit first, so that 8 lanes touch every bank
      auto store = [&](uint32_t base, int row, const uint4& x, bool clean, bool& bad) {
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_f16x4(in[i], y[2 * i], y[2 * i + 1]);
        if (clean) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __half2 z = *reinterpret_cast<const __half2*>(&y[i]);
            const uint32_t ok = __heq2_mask(z, z);
            bad |= ok != ~0u;
            y[i] &= ok;
          }
        }
        const bool up = ch * 2 >= kCh;
        const uint32_t a0 = base + unit_at<D>(row, 2 * ch + (up ? 1 : 0));
        const uint32_t a1 = base + unit_at<D>(row, 2 * ch + (up ? 0 : 1));
        st_shared_v4(a0, up ? y[4] : y[0], up ? y[5] : y[1], up ? y[6] : y[2], up ? y[7] : y[3]);
        st_shared_v4(a1, up ? y[0] : y[4], up ? y[1] : y[5], up ? y[2] : y[6], up ? y[3] : y[7]);
      };
      uint32_t kc = 0, vc = 0;
      fetch_k();
      fetch_v();
      for (int seg = 0;; ++seg) {
        const int tile_end = (int)min((long long)w.ut, tile + (sh.end - at));
        const bool ice = p.cls_static[w.cls];
        const int pos_lo = w.rows.base + w.pair * kRows / w.gk();  // the row that sees least
        for (int i = tile; i < tile_end; ++i) {
          bool bad = false;
          fetch_next();
          if (!ice) {
            const int st = kc & 1;
            mbar_wait(k_empty + st, ((kc >> 1) & 1) ^ 1, wc, kSiteKFree);
#pragma unroll
            for (int n = 0; n < kN; ++n)
              store(sK + st * L::TILE, row0 + n * kStep, kx[n], false, bad);
            fetch_k();
            fence_proxy_async_smem();
            mbar_arrive(k_full + st);
            ++kc;
          } else {
            fetch_k();
          }
          const int st = vc & 1;
          mbar_wait(v_empty + st, ((vc >> 1) & 1) ^ 1, wc, kSiteVFree);
          const bool clean = i * kTile + kTile - 1 > pos_lo;  // keys that not every row sees
#pragma unroll
          for (int n = 0; n < kN; ++n)
            store(sV + st * L::TILE, row0 + n * kStep, vx[n], clean, bad);
          if (bad) nan_seg[seg & 3] = seg + 1;
          if (tid < 8) {
            // a group without a page: every logit -inf
            const float lv = meta_there ? __log2f(meta_v) : -CUDART_INF_F;
            *reinterpret_cast<float4*>(smem + L::OFF_META + (vc & 3) * 128 + tid * 16) =
                make_float4(meta_there ? meta_k : 1.f, lv,
                            meta_there ? __fdividef(1.f, meta_v) : 1.f, 0.f);
          }
          mbar_arrive(m_full + (vc & 3));
          fetch_v();
          fence_proxy_async_smem();
          mbar_arrive(v_full + st);
          ++vc;
        }
        at += tile_end - tile;
        if (at >= sh.end) break;
        tile = 0;
        w.next();
      }
    } else if (lane == 0) {
      // ------------------------------------------------------------ products
      constexpr uint32_t id_s = idesc_f16(128, kTile, false, false);
      constexpr uint32_t id_o = idesc_f16(128, D, false, true);
      uint32_t kc = 0, vc = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};
      for (;;) {
        const int tile_end = (int)min((long long)w.ut, tile + (sh.end - at));
        const int gk = w.gk();
        const bool ice = p.cls_static[w.cls];
        const int n_g =
            (long long)w.rows.n_new * gk - (long long)w.pair * kRows > 128 ? 2 : 1;
        auto issue_s = [&](int g) {
          const uint32_t kt = sK + (kc & 1) * L::TILE, qt = sQ + g * L::TILE;
#pragma unroll
          for (int kk = 0; kk < G::KSTEPS; ++kk)
            mma_bf16_ss(tmem + kS + g * 128, G::kmajor_desc(qt, kk), G::kmajor_desc(kt, kk), id_s,
                        kk > 0);
          mma_commit(s_full + g);
        };
        if (!ice) {
          mbar_wait(k_full + (kc & 1), (kc >> 1) & 1, wc, kSiteK);
          for (int g = 0; g < n_g; ++g) {
            mbar_wait(q_full + g, n_q[g] & 1, wc, kSiteQ);
            ++n_q[g];
            tc_fence_after();
            issue_s(g);
          }
          mma_commit(k_empty + (kc & 1));
          ++kc;
        }
        for (int i = tile; i < tile_end; ++i) {
          const bool more = !ice && i + 1 < tile_end;
          mbar_wait(v_full + (vc & 1), (vc >> 1) & 1, wc, kSiteV);
          const uint32_t vt = sV + (vc & 1) * L::TILE;
          for (int g = 0; g < n_g; ++g) {
            mbar_wait(p_full + g, n_p[g] & 1, wc, kSiteP);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_bf16_ts(tmem + kO + g * 128, tmem + kS + g * 128 + 8 * kk,
                          G::mnmajor_desc(vt, kk), id_o, (i > tile || kk > 0));
            mma_commit(o_done + g);
            if (more) {
              if (g == 0) mbar_wait(k_full + (kc & 1), (kc >> 1) & 1, wc, kSiteK);
              // S takes the columns of the P that this product reads
              mbar_wait(o_done + g, n_p[g] & 1, wc, kSiteO);
              tc_fence_after();
              issue_s(g);
            }
            ++n_p[g];
          }
          mma_commit(v_empty + (vc & 1));
          ++vc;
          if (more) {
            mma_commit(k_empty + (kc & 1));
            ++kc;
          }
        }
        at += tile_end - tile;
        if (at >= sh.end) break;
        tile = 0;
        w.next();
      }
      // every product has completed before TMEM is freed
      mma_commit(drained);
      mbar_drain(drained, 0);
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

// Joins the parts of a unit that was cut (see cache_attn.cu); x: the CTA that
// left it, y: slices of its rows.
template <int D>
__global__ void __launch_bounds__(256)
    cache_chunk_join_kernel(const __grid_constant__ CacheChunk p) {
  const CacheCall& c = p.a.c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.a.join[blockIdx.x];
  if (u.x < 0) return;
  const int b = u.x, pair = u.y, cls = u.z, last = u.w & ~(1 << 30);
  const int first = 2 * blockIdx.x + (u.w >> 30 & 1);
  const Rows rows = slot_rows(c, b);
  int gk = 0;
  for (int g = 0; g < p.n_groups; ++g)
    if (cls >= p.group_first[g]) gk = p.group_width[g];
  const int n_rows =
      (int)min((long long)kRows, (long long)rows.n_new * gk - (long long)pair * kRows);
  for (int i = blockIdx.y * 256 + threadIdx.x; i < n_rows * (D / 4); i += gridDim.y * 256) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    auto ml = [&](int part) {
      return *reinterpret_cast<const float2*>(p.a.ml + ((size_t)part * kRows + r) * 2);
    };
    float mx = ml(first).x, sum = 0.f;
    for (int k = blockIdx.x + 1; k <= last; ++k) mx = fmaxf(mx, ml(2 * k).x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = blockIdx.x; k <= last; ++k) {
      const int part = k == (int)blockIdx.x ? first : 2 * k;
      const float2 x = ml(part);
      const float f = mx == -CUDART_INF_F ? 1.f : fast_exp2(x.x - mx);
      sum = fmaf(f, x.y, sum);
      const float4 v =
          *reinterpret_cast<const float4*>(p.a.acc + ((size_t)part * kRows + r) * D + d);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    const int rr = pair * kRows + r, t = rr / gk, h = p.order[p.cls_first[cls] + rr - t * gk];
    const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(p.a.out + row * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (d == 0 && p.a.lse) p.a.lse[row] = (mx + log2f(sum)) * kLn2;
  }
}

template <int D>
cudaError_t launch(const CacheChunk& p, int n_sms, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(p.a.status, 0, sizeof(int), s);
  if (e != cudaSuccess) return e;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(cache_chunk_kernel<D>), Smem<D>::ALLOC);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  cache_chunk_kernel<D><<<n_sms, kThreads, Smem<D>::ALLOC, s>>>(p);
  trace_end(s, "cache_chunk");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_sms, 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  e = cudaLaunchKernelEx(&cfg, cache_chunk_join_kernel<D>, p);
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
  w.status = take(256);
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
  for (int w = c.group; w >= 1; --w) {
    const int before = n;
    for (int kind = 0; kind < 2; ++kind)
      for (int kv = 0; kv < c.H_kv; ++kv)
        if (width[kind][kv] == w) {
          p.cls_kv[n] = (uint8_t)kv;
          p.cls_static[n] = (uint8_t)kind;
          p.cls_first[n] = (int16_t)(kv * c.group + (kind ? width[0][kv] : 0));
          ++n;
        }
    if (n > before) {
      p.group_width[p.n_groups] = w;
      p.group_first[p.n_groups++] = before;
    }
  }
  p.group_first[p.n_groups] = n;
  switch (d_h) {
    case 32: return launch<32>(p, n_sms, s);
    case 64: return launch<64>(p, n_sms, s);
    case 128: return launch<128>(p, n_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace saf
