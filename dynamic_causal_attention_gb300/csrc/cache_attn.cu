// cache_attn.cu — the hybrid layer over the paged 8-bit cache.
//
//   dynamic query head:  x_j = (q . k_j) s_k / sqrt(d)
//   frozen query head:   x_j = alpha(j) + rho(i - j)
//   out = sum_j e^{x_j} s_v v_j / sum_j e^{x_j},   lse = log sum_j e^{x_j}
//
// over the keys j <= i that lie on a page, with codes k_j, v_j and the scales
// s_k, s_v of their block.  The block's V scale joins the exponent: with
// y_j = x_j log2(e) + log2(s_v), the weights of the second product are
// p_j = 2^{y_j - m} under a running maximum m of the y, and the sum of the
// softmax is sum_j p_j / s_v.  So a weight is rounded to f16 relative to the
// largest contribution to `out`, whatever the scales of the blocks.
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

// ------------------------------------------------------------ work split
// A unit is (slot b, row tile, K/V head): rows [16 tile, 16 tile + 16) of the
// slot's n_new * group query rows (row r = t * group + h) against the keys up
// to the last position among them, in tiles of kTile keys.  All tiles of all
// units, in that order, are cut into equal shares, one for each CTA; a unit
// that is cut leaves partial sums, joined by a second kernel in the order of
// the CTAs.  Nothing depends on timing.
constexpr int kMR = 16;      // query rows of a unit
constexpr int kTile = 64;    // keys of a tile: 16 for each warp
constexpr int kWarps = 4;
constexpr int kMinTiles = 4; // least share of a CTA

__device__ __forceinline__ int unit_extent(const Rows& r, int rt, int group) {
  int t_hi = (rt * kMR + kMR - 1) / group + 1;
  if (t_hi > r.n_new) t_hi = r.n_new;
  const int e = r.base + t_hi;
  return e < 0 ? 0 : (e < r.cap ? e : r.cap);
}
__device__ __forceinline__ int unit_tiles(const Rows& r, int rt, int group) {
  const int n = (unit_extent(r, rt, group) + kTile - 1) / kTile;
  return n < 1 ? 1 : n;  // rows that see nothing are written too
}
__device__ __forceinline__ int slot_row_tiles(const Rows& r, int group) {
  return (int)(((long long)r.n_new * group + kMR - 1) / kMR);
}
__device__ __forceinline__ long long slot_tiles(const CacheCall& c, int b) {
  const Rows r = slot_rows(c, b);
  const int n = slot_row_tiles(r, c.group);
  long long sum = 0;
  for (int i = 0; i < n; ++i) sum += unit_tiles(r, i, c.group);
  return sum * c.H_kv;
}

struct Share {
  long long size, begin, end;  // tiles of a CTA
  int b;                       // the slot of tile `begin` and that tile's index in the slot
  long long in_slot;
};

// Every CTA finds its share: each thread sums a run of slots, a block scan
// gives the runs' first tiles, and the thread whose run holds the share's
// first tile walks it.
__device__ Share find_share(const CacheCall& c, long long* scan /* [threads + 4] */) {
  const int n = blockDim.x, tid = threadIdx.x;
  const int per = (c.n_seqs + n - 1) / n;
  const int b0 = min(tid * per, c.n_seqs), b1 = min(b0 + per, c.n_seqs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += slot_tiles(c, b);
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
      const long long t = slot_tiles(c, b);
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

// ------------------------------------------------------------ shared memory
// One step of a warp is 16 keys of one page: K codes, V codes, the two scales
// and the number of keys there.  16-byte chunks are placed so that the reads
// of both products touch every bank once: a product's reads take the keys
// {c, c + 4} and {c + 8, c + 12} for lane % 4 = c.
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

template <int D>
struct Geo {
  static constexpr int kCodes = 16 * D;               // bytes of K or V codes of a step
  static constexpr int kStep = 2 * kCodes + 16;       // + K scale, V scale, key count
  static constexpr int kStages = D == 128 ? 4 : (D == 64 ? 6 : 10);
  static constexpr int kRing = (kStages * kStep + 127) / 128 * 128;
  static constexpr int kMerge = kWarps * kMR * (D + 2) * 4;
  static constexpr int kSmem = kWarps * kRing > kMerge ? kWarps * kRing : kMerge;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, D == 128 ? 3 : 4)
    cache_attn_kernel(const __grid_constant__ CacheAttn p) {
  using G = Geo<D>;
  constexpr int kKS = D / 16;  // steps of 16 along d
  constexpr int kNT = D / 8;   // output tiles of 8 columns
  constexpr int kVB = D / 8;   // bytes of a V row that a lane takes
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scan[kWarps * 32 + 4];
  const CacheCall& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, cc = lane & 3;

  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // nothing here waits without end
  const Share sh = find_share(c, scan);
  if (threadIdx.x == 0) p.join[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (sh.begin >= sh.end) return;

  const uint32_t ring = smem_u32(smem) + warp * G::kRing;
  int b = sh.b;
  Rows rows = slot_rows(c, b);
  int rt = 0;
  long long in_slot = sh.in_slot;
  int ut = unit_tiles(rows, 0, c.group);
  while (in_slot >= (long long)ut * c.H_kv) {
    in_slot -= (long long)ut * c.H_kv;
    ++rt;
    ut = unit_tiles(rows, rt, c.group);
  }
  int kv = (int)(in_slot / ut), tile = (int)(in_slot % ut);
  long long at = sh.begin;

  while (true) {
    // ---- this segment: tiles [tile, tile_end) of unit (b, rt, kv)
    const int tile_end = (int)min((long long)ut, tile + (sh.end - at));
    const int ext = unit_extent(rows, rt, c.group);
    const int n_rows = min(kMR, rows.n_new * c.group - rt * kMR);
    const int steps = tile_end - tile;
    const int k_head = c.k_of[kv];

    // rows of this lane: quad and quad + 8
    int pos[2], head[2];
    bool ice[2];
    const uint16_t* qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rt * kMR + quad + 8 * i;
      const bool live = quad + 8 * i < n_rows;
      const int t = live ? r / c.group : 0, hh = live ? r - t * c.group : 0;
      head[i] = kv * c.group + hh;
      pos[i] = live ? rows.base + t : -1;
      ice[i] = live && c.is_static[head[i]];
      qrow[i] = live && !ice[i] ? p.Q + (((size_t)b * c.H + head[i]) * c.n_q + t) * D : nullptr;
    }
    bool any_dyn = k_head >= 0;  // a dynamic head in the group
    const int pos_lo = rows.base + rt * kMR / c.group;  // the row that sees least

    // ---- Q fragments: lane takes d = 16 c .. 16 c + 15 (and + 64) of its rows
    uint32_t qf[kKS][4];
    float fac[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[D / 4];
      float amax = 0.f;
#pragma unroll
      for (int blk = 0; blk < (D + 63) / 64; ++blk) {
        constexpr int kW = D >= 64 ? 16 : 8;  // d's of a lane in a block
#pragma unroll
        for (int u = 0; u < kW / 8; ++u) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (qrow[i])
            w = __ldg(reinterpret_cast<const uint4*>(qrow[i] + 64 * blk + kW * cc + 8 * u));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[blk * kW + 8 * u + 2 * v] = __uint_as_float(ww[v] << 16);
            x[blk * kW + 8 * u + 2 * v + 1] = __uint_as_float(ww[v] & 0xffff0000u);
          }
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
      fac[i] = pow2f(e) * (rsqrtf((float)D) * kLog2e);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        // the lane's 4 values of step ks: slots 2c, 2c+1 (lo) and 2c+8, 2c+9 (hi)
        const int o = ks * 4;
        qf[ks][i] = pack_f16x2(x[o] * down, x[o + 1] * down);
        qf[ks][2 + i] = pack_f16x2(x[o + 2] * down, x[o + 3] * down);
      }
    }

    // ---- the ring: page numbers are fetched 32 steps ahead by lane
    int pages = -1;
    const int key_w = tile * kTile + warp * 16;  // first key of this warp's step 0
    auto load_pages = [&](int s0) {
      const int key = key_w + (s0 + lane) * kTile;
      pages = key < ext && s0 + lane < steps ? page_at(c, b, key >> c.page_shift) : -1;
    };
    auto issue = [&](int s) {
      if (s < steps) {
        if ((s & 31) == 0) load_pages(s);
        const int page = __shfl_sync(~0u, pages, s & 31);
        const int key0 = key_w + s * kTile;
        const int n = page < 0 ? 0 : min(16, ext - key0);
        const uint32_t st = ring + (s % G::kStages) * G::kStep;
        const uint8_t* rec = c.layer + (size_t)(page < 0 ? 0 : page) * c.page_stride;
        const int slot = key0 & ((1 << c.page_shift) - 1);
        const uint8_t* src_v = rec + c.off_v + (((size_t)kv << c.page_shift) + slot) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int ch = (lane + 32 * i) % (D / 16), key = (lane + 32 * i) / (D / 16);
          cp_async16(st + G::kCodes + chunk_at<D>(key, ch), src_v + key * D + ch * 16,
                     key < n ? 16 : 0);
        }
        if (any_dyn) {
          const uint8_t* src_k = rec + (((size_t)k_head << c.page_shift) + slot) * D;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int ch = (lane + 32 * i) % (D / 16), key = (lane + 32 * i) / (D / 16);
            cp_async16(st + chunk_at<D>(key, ch), src_k + key * D + ch * 16, key < n ? 16 : 0);
          }
        }
        if (lane == 0) {
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + 2 * G::kCodes + 8), "r"(n) : "memory");
          if (n > 0) {
            if (any_dyn)
              cp_async4(st + 2 * G::kCodes, rec + c.off_ks + 4 * (size_t)k_head);
            cp_async4(st + 2 * G::kCodes + 4, rec + c.off_vs + 4 * (size_t)kv);
          }
        }
      }
      cp_async_commit();
    };

    // values of the frozen rows for one step, fetched a step ahead
    float pat[2][4];
    auto fetch_pattern = [&](int s) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (ice[i] && s < steps) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = key_w + s * kTile + cc + 4 * u;  // u: keys c, c+4, c+8, c+12
            const int dist = pos[i] - j;
            float a = -CUDART_INF_F;
            if (dist >= 0 && j < p.T_pat && dist < p.T_pat)
              a = __ldg(p.alpha + (size_t)head[i] * p.T_pat + j) +
                  __ldg(p.rho + (size_t)head[i] * p.T_pat + dist);
            pat[i][u] = a * kLog2e;
          }
        }
    };

    float acc[kNT][4];
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[t][u] = 0.f;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    bool v_nan = false;  // a NaN in V at a key that not every row sees

    __syncwarp();
#pragma unroll
    for (int s = 0; s < G::kStages - 1; ++s) issue(s);
    fetch_pattern(0);
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<G::kStages - 2>();
      __syncwarp();
      const uint32_t st = ring + (s % G::kStages) * G::kStep;
      const int n = __float_as_int(lds_f32(st + 2 * G::kCodes + 8));
      const int key0 = key_w + s * kTile;
      if (n > 0) {
        const float ks = lds_f32(st + 2 * G::kCodes), vs = lds_f32(st + 2 * G::kCodes + 4);
        float sc[2][4];  // [8-key half][row quad: 2 keys | row quad + 8: 2 keys]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 4; ++u) sc[h][u] = 0.f;
        if (any_dyn) {
          const int key = (quad >> 1) + 4 * (quad & 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[kKS];
            if (D == 32) {
              const uint32_t a = st + chunk_at<D>(key + 8 * h, cc >> 1) + (cc & 1) * 8;
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
            } else {
#pragma unroll
              for (int blk = 0; blk < D / 64; ++blk)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * blk]), "=r"(w[4 * blk + 1]), "=r"(w[4 * blk + 2]),
                               "=r"(w[4 * blk + 3])
                             : "r"(st + chunk_at<D>(key + 8 * h, cc + 4 * blk)));
            }
#pragma unroll
            for (int i = 0; i < kKS; ++i) {
              uint32_t b0, b1;
              e4m3x4_f16x4(w[i], b0, b1);
              mma_f16_16816(sc[h], qf[i], b0, b1);
            }
          }
        }
        // y = x log2(e) + log2(s_v); keys that a row does not see: -inf
        const float lv = __log2f(vs), inv = __fdividef(1.f, vs);
        const bool edge = n < 16 || key0 + 15 > pos_lo;
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = fac[i] * ks;
          top[i] = -CUDART_INF_F;
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // keys c + 4 u: half u >> 1, column u & 1
            float& y = sc[u >> 1][2 * i + (u & 1)];
            y = ice[i] ? pat[i][u] + lv : fmaf(y, f, lv);
            if (edge && (cc + 4 * u >= n || key0 + cc + 4 * u > pos[i])) y = -CUDART_INF_F;
            top[i] = fmaxf(top[i], y);
          }
          top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 2));
        }
        if (__any_sync(~0u, top[0] > m[0] || top[1] > m[1])) {
          float corr[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[i], top[i]);
            corr[i] = mn == -CUDART_INF_F ? 1.f : fast_exp2(m[i] - mn);
            m[i] = mn;
            l[i] *= corr[i];
          }
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[t][u] *= corr[u >> 1];
        }
        uint32_t pf[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float base = m[i] == -CUDART_INF_F ? 0.f : m[i];
          float sum = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = fast_exp2(sc[h][2 * i] - base);
            const float p1 = fast_exp2(sc[h][2 * i + 1] - base);
            sum += p0 + p1;
            pf[2 * h + i] = pack_f16x2(p0, p1);
          }
          l[i] = fmaf(sum, inv, l[i]);
        }
        // V: keys c, c + 4 (slots 2c, 2c+1) and c + 8, c + 12 (slots 2c+8, 2c+9)
        uint32_t w[4][(kVB + 3) / 4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t a = st + G::kCodes + chunk_at<D>(cc + 4 * u, quad * kVB >> 4) +
                             (quad * kVB & 15);
          if (D == 128)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[u][0]), "=r"(w[u][1 % (kVB / 4)]), "=r"(w[u][2 % (kVB / 4)]),
                           "=r"(w[u][3 % (kVB / 4)])
                         : "r"(a));
          else if (D == 64)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(w[u][0]), "=r"(w[u][1 % (kVB / 4)])
                         : "r"(a));
          else
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[u][0]) : "r"(a));
        }
#pragma unroll
        for (int i = 0; i < kVB / 4; ++i) {
          uint32_t f[2][4];  // [slots lo, hi][column of the word]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            e4m3x4_f16x4(__byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x5140), f[h][0], f[h][1]);
            e4m3x4_f16x4(__byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x7362), f[h][2], f[h][3]);
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
          for (int u = 0; u < 4; ++u) mma_f16_16816(acc[4 * i + u], pf, f[0][u], f[1][u]);
        }
      }
      fetch_pattern(s + 1);
      __syncwarp();
      issue(s + G::kStages - 1);
    }
    cp_async_wait<0>();

    if (__any_sync(~0u, v_nan)) {
      // rows that do see a key whose V holds NaN take it
      for (int s = 0; s < steps; ++s) {
        const int key0 = key_w + s * kTile;
        for (int k = 0; k < 16; ++k) {
          const int j = key0 + k;
          if (j >= ext || (ext - key0 >= 16 && key0 + 15 <= pos_lo)) continue;
          const int page = page_at(c, b, j >> c.page_shift);
          if (page < 0) continue;
          const uint8_t* v = c.layer + (size_t)page * c.page_stride + c.off_v +
                             (((size_t)kv << c.page_shift) + (j & ((1 << c.page_shift) - 1))) * D;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (j <= pos[u >> 1] && (v[(2 * cc + (u & 1)) * kVB + t] & 0x7f) == 0x7f)
                acc[t][u] = CUDART_NAN_F;
        }
      }
    }

    // ---- join the warps: [warp][row][D] sums, then [warp][row][2] of (m, l)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(~0u, l[i], 1);
      l[i] += __shfl_xor_sync(~0u, l[i], 2);
    }
    __syncthreads();  // every warp has read its ring
    float* mo = reinterpret_cast<float*>(smem);
    float* mm = mo + kWarps * kMR * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = quad + 8 * i;
      if (r < n_rows) {
        float* dst = mo + ((size_t)warp * kMR + r) * D;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          dst[2 * cc * kVB + t] = acc[t][2 * i];
          dst[(2 * cc + 1) * kVB + t] = acc[t][2 * i + 1];
        }
        if (cc == 0) {
          mm[(warp * kMR + r) * 2] = m[i];
          mm[(warp * kMR + r) * 2 + 1] = l[i];
        }
      }
    }
    __syncthreads();
    const bool whole = tile == 0 && tile_end == ut;
    const int part = 2 * blockIdx.x + (at == sh.begin ? 0 : 1);
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
        const float4 x = *reinterpret_cast<const float4*>(mo + ((size_t)w * kMR + r) * D + d);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
      }
      if (whole) {
        const int rr = rt * kMR + r, t = rr / c.group, h = kv * c.group + rr - t * c.group;
        const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: 0
        *reinterpret_cast<uint2*>(p.out + row * D + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d == 0 && p.lse) p.lse[row] = (mx + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.acc + ((size_t)part * kMR + r) * D + d) = o;
        if (d == 0)
          *reinterpret_cast<float2*>(p.ml + ((size_t)part * kMR + r) * 2) = make_float2(mx, sum);
      }
    }
    if (tile == 0 && tile_end < ut && threadIdx.x == 0) {
      // the unit begins here and ends in CTA `last`
      const int last = (int)((at + ut - 1) / sh.size);
      p.join[blockIdx.x] = make_int4(b, rt, kv, last | (at == sh.begin ? 0 : 1 << 30));
    }
    __syncthreads();  // the merge buffer is the ring again

    // ---- the next unit
    at += tile_end - tile;
    if (at >= sh.end) break;
    tile = 0;
    if (++kv == c.H_kv) {
      kv = 0;
      ++rt;
      while (rt >= slot_row_tiles(rows, c.group)) {
        rows = slot_rows(c, ++b);
        rt = 0;
      }
      ut = unit_tiles(rows, rt, c.group);
    }
  }
}

// Joins the parts of a unit that was cut: CTA x takes the unit that CTA x of
// the first kernel left to its successors; y splits the rows.
template <int D>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheAttn p) {
  const CacheCall& c = p.c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.join[blockIdx.x];
  if (u.x < 0) return;
  const int b = u.x, rt = u.y, kv = u.z, last = u.w & ~(1 << 30);
  const int first = 2 * blockIdx.x + (u.w >> 30 & 1);
  const Rows rows = slot_rows(c, b);
  const int n_rows = min(kMR, rows.n_new * c.group - rt * kMR);
  for (int i = blockIdx.y * 128 + threadIdx.x; i < n_rows * (D / 4); i += gridDim.y * 128) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    auto ml = [&](int part) {
      return *reinterpret_cast<const float2*>(p.ml + ((size_t)part * kMR + r) * 2);
    };
    float mx = ml(first).x, sum = 0.f;
    for (int k = blockIdx.x + 1; k <= last; ++k) mx = fmaxf(mx, ml(2 * k).x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = blockIdx.x; k <= last; ++k) {
      const int part = k == (int)blockIdx.x ? first : 2 * k;
      const float2 w = ml(part);
      const float f = mx == -CUDART_INF_F ? 1.f : fast_exp2(w.x - mx);
      sum = fmaf(f, w.y, sum);
      const float4 x =
          *reinterpret_cast<const float4*>(p.acc + ((size_t)part * kMR + r) * D + d);
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
    }
    const int rr = rt * kMR + r, t = rr / c.group, h = kv * c.group + rr - t * c.group;
    const size_t row = ((size_t)b * c.H + h) * c.n_q + t;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(p.out + row * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (d == 0 && p.lse) p.lse[row] = (mx + log2f(sum)) * kLn2;
  }
}

int n_ctas(int d_h, int n_sms) { return n_sms * (d_h == 128 ? 3 : 4); }

template <int D>
cudaError_t launch(const CacheAttn& p, int n_sms, cudaStream_t s) {
  const int grid = n_ctas(D, n_sms);
  cudaError_t e =
      set_max_dynamic_smem(reinterpret_cast<const void*>(cache_attn_kernel<D>), Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  cache_attn_kernel<D><<<grid, kWarps * 32, Geo<D>::kSmem, s>>>(p);
  trace_end(s, "cache_attn");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while the first kernel runs; waits for its end before it reads
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 4);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  e = cudaLaunchKernelEx(&cfg, cache_join_kernel<D>, p);
  trace_end(s, "cache_join");
  return e != cudaSuccess ? e : cudaGetLastError();
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
  const size_t n = (size_t)n_ctas(d_h, n_sms);
  w.status = take(256);
  w.join = take(n * sizeof(int4));
  w.ml = take(2 * n * kMR * 2 * 4);
  w.acc = take(2 * n * kMR * d_h * 4);
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
