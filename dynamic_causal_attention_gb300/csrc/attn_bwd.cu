// attn_bwd.cu — backward of the SAF hybrid layer: dynamic heads, and the
// alpha/rho gradients of frozen heads.
//
// ("When Can Attention Heads Be Statically Defined?", close-reading notes:
// dynamic heads keep the ordinary attention backward; a frozen head's
// attention backward is only dV = P^T dZ, §3.3 / App. D.2 — that part reuses
// the forward's static engine, transposed.  The alpha/rho gradients are an
// extension: the chain rule through Eq. (3).)
//
// bwd_dynamic_kernel (K4): one persistent launch over items (b, h, J), J a
// 128-row key tile, longest first.  Per item K_J and V_J stay in shared
// memory and dK_J, dV_J accumulate in TMEM while the query tiles I = J..nI-1
// stream through:
//     S^T  = K_J Q_I^T,  dP^T = V_J dO_I^T           (tcgen05, fp32 in TMEM)
//     P^T  = exp2(S^T * log2e/sqrt(d) - lse2(i)),   dS^T = P^T * (dP^T - D(i))
//                                                   (compute warps, 1 row/thread)
//     dV_J += P^T dO_I,  dK_J += dS^T Q_I           (tcgen05, A operand in TMEM)
//     dQ_I  = dS K_J                                (tcgen05, dS^T tile in smem
//                                                    read as an MN-major A)
// d_h <= 64: P^T goes, as packed bf16, to spare TMEM columns (dV is a TS MMA)
// and dS^T to one of two swizzled shared-memory tiles (dK and dQ are SS MMAs).
// d_h = 128: TMEM has no spare columns, so P^T and dS^T are written, packed,
// over the S^T columns just read (dV and dK are TS MMAs), dS^T also goes to
// shared memory for dQ, and dQ goes over the dP^T columns.  dQ_I is read from
// TMEM by a second warpgroup and added into an fp32 accumulator (zeroed by the
// pre-pass) with one TMA tensor reduce-add per 32 columns: staged in a tile of
// its own for d_h <= 64, in the step's own Q_I/dO_I stage (once dV and dK have
// read it) for d_h = 128.  A post-pass scales it by 1/sqrt(d) and converts it.
//
// param_grad_kernel (K5): items (h_static, J), handed out in snake order.
// For I = J..nI-1 the batch-summed dP^T(j, i) = sum_b V_b(j) . dO_b(i) is one
// MMA chain with K = B*d; eight compute warps (a 32-row group x a 64-column
// half each) form dl = P(i,j) (dP - sum_b D_b(i)) with P(i,j) rebuilt from the
// static tables and keep the row sums (alpha) in registers.  For the diagonal
// sums (rho) each warp writes its 32 x 32 block of dl to shared memory by
// diagonal, so that lane q adds up diagonals q and q + 32 with vector loads,
// and adds its three distance sums of the tile to global with atomics (no
// barrier across the warps per tile).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_bwd_kernel.cuh"
#include "attn_common.cuh"
#include "attn_kernels.h"
#include "internal.h"

namespace saf {
namespace {

// ============================================================ K5: dalpha/drho
template <int D>
struct PgSmem {
  using G = TileGeom<D>;
  static constexpr int ST = (D == 128) ? 2 : (D == 64 ? 3 : 4);  // (V_b[J], dO_b[I]) pairs
  static constexpr int STAGE = 2 * G::TILE_BYTES;
  static constexpr int AUX = 2048;                     // col values, D sums, r window
  // Per compute warp, its 32 x 32 block of dl laid out by diagonal: row
  // e = k - rr + 32 (k column, rr row of the block), 36 floats a row.
  static constexpr int SKW_ROW = 36;
  static constexpr int SKW = 64 * SKW_ROW * 4;
  static constexpr int OFF_ST = 0;
  static constexpr int OFF_AUX = OFF_ST + ST * STAGE;
  static constexpr int OFF_SKW = OFF_AUX + 2 * AUX;
  static constexpr int OFF_BAR = OFF_SKW + 8 * SKW;
  static constexpr int NBAR = 2 * ST + 4 + 4 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget exceeded");
};

enum : int { kSitePgProd = 201, kSitePgProdAux, kSitePgMma, kSitePgMmaAcc, kSitePgAux, kSitePgAcc };


template <int D>
__global__ void __launch_bounds__(384, 1)
    param_grad_kernel(const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_do, const ParamGradParams p) {
  using G = TileGeom<D>;
  using L = PgSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* st_full = bars;
  uint64_t* st_empty = st_full + L::ST;
  uint64_t* aux_full = st_empty + L::ST;
  uint64_t* aux_empty = aux_full + 2;
  uint64_t* acc_full = aux_empty + 2;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_drained = acc_empty + 2;  // the issuer's products all done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const WaitCtl wc{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::ST; ++s) { mbar_init(st_full + s, 1); mbar_init(st_empty + s, 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(aux_full + s, 1);
      mbar_init(aux_empty + s, 8);  // every compute warp has read the slot
      mbar_init(acc_full + s, 1);
      mbar_init(acc_empty + s, 256);
    }
    mbar_init(mma_drained, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  // Cells of the diagonal blocks that no (row, column) pair maps to are read
  // as zeros, and nothing ever writes them.
  {
    float4* z = reinterpret_cast<float4*>(smem + L::OFF_SKW);
    for (int t = threadIdx.x; t < 8 * L::SKW / 16; t += blockDim.x)
      z[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int H = p.H, T = p.T, B = p.B;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t sc = 0, ac = 0;
      for (int k = 0;; ++k) {
        const int it = snake_item(k, blockIdx.x, gridDim.x);
        if (it >= p.n_items) break;
        const int J = it / p.n_static, hs = it - J * p.n_static, h = p.static_heads[hs];
        for (int I = J; I < p.nI; ++I) {
          const int as = ac & 1;
          mbar_wait(aux_empty + as, ((ac >> 1) & 1) ^ 1, wc, kSitePgProdAux);
          ++ac;
          uint8_t* aux = smem + L::OFF_AUX + as * L::AUX;
          mbar_arrive_expect_tx(aux_full + as, 2048);
          bulk_load(aux, p.row_tab + (size_t)hs * T + I * 128, 512, aux_full + as);
          bulk_load(aux + 512, p.Dsum + (size_t)hs * T + I * 128, 512, aux_full + as);
          bulk_load(aux + 1024, p.r_tab + (size_t)hs * (T + 128) + (I - J) * 128, 1024,
                    aux_full + as);
          for (int b = 0; b < B; ++b) {
            const int s = sc % L::ST;
            mbar_wait(st_empty + s, ((sc / L::ST) & 1) ^ 1, wc, kSitePgProd);
            ++sc;
            uint8_t* st = smem + L::OFF_ST + s * L::STAGE;
            const int row0 = (b * H + h) * T;                          // dO rows
            const int vrow0 = (b * p.H_kv + h / p.group_kv) * T;      // V rows
            mbar_arrive_expect_tx(st_full + s, 2 * G::TILE_BYTES);
            for (int c = 0; c < G::NCHUNK; ++c) {
              tma_load_2d(st + c * G::CHUNK_BYTES, &tm_v, st_full + s, c * G::CHUNK,
                          vrow0 + J * 128);
              tma_load_2d(st + G::TILE_BYTES + c * G::CHUNK_BYTES, &tm_do, st_full + s,
                          c * G::CHUNK, row0 + I * 128);
            }
          }
        }
      }
      for (int s = 0; s < L::ST; ++s)
        if (sc > (uint32_t)s) mbar_drain(st_full + s, ((sc - 1 - s) / L::ST) & 1);
      for (int s = 0; s < 2; ++s)
        if (ac > (uint32_t)s) mbar_drain(aux_full + s, ((ac - 1 - s) >> 1) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id = idesc_bf16(128, 128, false, false);
      uint32_t sc = 0, cc = 0;
      for (int k = 0;; ++k) {
        const int it = snake_item(k, blockIdx.x, gridDim.x);
        if (it >= p.n_items) break;
        const int J = it / p.n_static;
        for (int I = J; I < p.nI; ++I) {
          const int ab = cc & 1;
          mbar_wait(acc_empty + ab, ((cc >> 1) & 1) ^ 1, wc, kSitePgMmaAcc);
          tc_fence_after();
          for (int b = 0; b < B; ++b) {
            const int s = sc % L::ST;
            mbar_wait(st_full + s, (sc / L::ST) & 1, wc, kSitePgMma);
            tc_fence_after();
            const uint32_t sv = smem_u32(smem + L::OFF_ST + s * L::STAGE);
#pragma unroll
            for (int kk = 0; kk < G::KSTEPS; ++kk)
              mma_bf16_ss(tmem + ab * 128, G::kmajor_desc(sv, kk),
                          G::kmajor_desc(sv + G::TILE_BYTES, kk), id, (b > 0 || kk > 0));
            mma_commit(st_empty + s);
            ++sc;
          }
          mma_commit(acc_full + ab);
          ++cc;
        }
      }
      // every product has completed before TMEM is freed (after an abort no
      // later wait guarantees it)
      mma_commit(mma_drained);
      mbar_drain(mma_drained, 0);
    }
  } else if (warp >= 4) {
    // Warp (rg, hf): key rows r = 32 rg + lane of tile J, query columns
    // 64 hf .. 64 hf + 63 of tile I.
    const int rg = warp & 3, hf = (warp - 4) >> 2, w8 = warp - 4;
    const int r = rg * 32 + lane;
    const uint32_t lane_base = (uint32_t)(rg * 32) << 16;
    float* skw = reinterpret_cast<float*>(smem + L::OFF_SKW + w8 * L::SKW);
    // row lane writes block column k to skw[(k - lane + 32) * 36 + lane]
    float* skw_w = skw + (32 - lane) * L::SKW_ROW + lane;
    // lane q sums the block diagonals e = q and e = q + 32
    const float4* skw_lo = reinterpret_cast<const float4*>(skw + lane * L::SKW_ROW);
    const float4* skw_hi = reinterpret_cast<const float4*>(skw + (lane + 32) * L::SKW_ROW);
    const uint64_t m1 = f2_pack(-1.f, -1.f);
    uint32_t ac = 0, cc = 0;
    for (int k = 0;; ++k) {
      const int it = snake_item(k, blockIdx.x, gridDim.x);
      if (it >= p.n_items) break;
      const int J = it / p.n_static, hs = it - J * p.n_static, h = p.static_heads[hs];
      const bool exact = p.mode[hs] != 0;
      const float rowv = p.a_tab[(size_t)hs * T + J * 128 + r];
      const uint64_t row2 = f2_pack(rowv, rowv);
      uint64_t dal2 = 0;
      for (int I = J; I < p.nI; ++I) {
        const int as = ac & 1;
        mbar_wait(aux_full + as, (ac >> 1) & 1, wc, kSitePgAux);
        const float* aux = reinterpret_cast<const float*>(smem + L::OFF_AUX + as * L::AUX);
        const float* colv = aux + 64 * hf;        // 1/Z'(i) or -log2 Z(i)
        const float* dsum = aux + 128 + 64 * hf;  // sum_b D_b(i)
        const float* rwin = aux + 256 + 127 + 64 * hf - r;  // r(i - j), i - j = c - r
        const int ab = cc & 1;
        mbar_wait(acc_full + ab, (cc >> 1) & 1, wc, kSitePgAcc);
        tc_fence_after();
        // diagonal sums of this warp: d = 127 + 64 hf - 32 rg - 32 + 32 m + lane
        float dg0 = 0.f, dg1 = 0.f, dg2 = 0.f;
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t v[32];
          tmem_ld_x32(tmem + lane_base + ab * 128 + 64 * hf + 32 * ch, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int k4 = 0; k4 < 32; k4 += 4) {
            const int c = 32 * ch + k4;
            const float4 cv = *reinterpret_cast<const float4*>(colv + c);
            const float4 ds = *reinterpret_cast<const float4*>(dsum + c);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float w0 = rwin[c + e], w1 = rwin[c + e + 1];
              const uint64_t cv2 = e ? f2_pack(cv.z, cv.w) : f2_pack(cv.x, cv.y);
              const uint64_t ds2 = e ? f2_pack(ds.z, ds.w) : f2_pack(ds.x, ds.y);
              uint64_t p2;
              if (exact) {
                float a0, a1;
                f2_unpack(f2_add(f2_add(f2_pack(w0, w1), cv2), row2), a0, a1);
                p2 = f2_pack(fast_exp2(a0), fast_exp2(a1));
              } else {
                p2 = f2_mul(f2_mul(f2_pack(w0, w1), cv2), row2);
              }
              const uint64_t x2 = f2_fma(ds2, m1, f2_pack(__uint_as_float(v[k4 + e]),
                                                          __uint_as_float(v[k4 + e + 1])));
              const uint64_t dl2 = f2_mul(p2, x2);
              dal2 = f2_add(dal2, dl2);
              float d0, d1;
              f2_unpack(dl2, d0, d1);
              skw_w[(k4 + e) * L::SKW_ROW] = d0;
              skw_w[(k4 + e + 1) * L::SKW_ROW] = d1;
            }
          }
          __syncwarp();
          uint64_t lo_a = 0, lo_b = 0, hi_a = 0, hi_b = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = skw_lo[j];
            const float4 y = skw_hi[j];
            lo_a = f2_add(lo_a, f2_pack(x.x, x.y));
            lo_b = f2_add(lo_b, f2_pack(x.z, x.w));
            hi_a = f2_add(hi_a, f2_pack(y.x, y.y));
            hi_b = f2_add(hi_b, f2_pack(y.z, y.w));
          }
          __syncwarp();
          float t0, t1, t2, t3;
          f2_unpack(f2_add(lo_a, lo_b), t0, t1);
          f2_unpack(f2_add(hi_a, hi_b), t2, t3);
          const float elo = t0 + t1, ehi = t2 + t3;  // block diagonals lane, lane + 32
          if (ch == 0) { dg0 += elo; dg1 += ehi; } else { dg1 += elo; dg2 += ehi; }
        }
        tc_fence_before();
        mbar_arrive(acc_empty + ab);
        ++cc;
        __syncwarp();
        if (lane == 0) mbar_arrive(aux_empty + as);  // this warp has read the table slot
        ++ac;
        // This warp's diagonal sums go straight to drho (no step-wide barrier
        // to combine the eight warps first): lane's sums dg0..dg2 are the
        // block diagonals o = lane, lane + 32, lane + 64, i.e. tile diagonal
        // t = c - r + 127 = o + 95 + 64 hf - 32 rg, global distance
        // (I - J) * 128 - 127 + t.
        const int t0 = lane + 95 + 64 * hf - 32 * rg;
        const int d0 = (I - J) * 128 - 127 + t0;
        const float dgs[3] = {dg0, dg1, dg2};
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          const int delta = d0 + 32 * m;
          if (delta >= 0 && delta < T && dgs[m] != 0.f)
            atomicAdd(&p.drho[(size_t)h * T + delta], dgs[m]);
        }
      }
      float da0, da1;
      f2_unpack(dal2, da0, da1);
      // the two column halves of row r add into a zeroed entry: 0 + a + b is
      // the same in either order
      atomicAdd(&p.dalpha[(size_t)h * T + J * 128 + r], da0 + da1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D>
cudaError_t launch_pg(const ParamGradLaunch& L, cudaStream_t s) {
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(param_grad_kernel<D>),
                                       PgSmem<D>::ALLOC);
  if (e != cudaSuccess) return e;
  if (L.p.n_items == 0) return cudaSuccess;
  const int grid = L.p.n_items < L.num_sms ? L.p.n_items : L.num_sms;
  trace_begin(s);
  param_grad_kernel<D><<<grid, 384, PgSmem<D>::ALLOC, s>>>(L.tm_v, L.tm_do, L.p);
  trace_end(s, "param_grad");
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_dynamic(const BwdLaunch& L, cudaStream_t s) {
  switch (L.d_h) {
    case 32: return launch_dyn<32>(L, s);
    case 64: return launch_dyn<64>(L, s);
    case 128: return launch_dyn<128>(L, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_param_grads(const ParamGradLaunch& L, cudaStream_t s) {
  switch (L.d_h) {
    case 32: return launch_pg<32>(L, s);
    case 64: return launch_pg<64>(L, s);
    case 128: return launch_pg<128>(L, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saf
