// attn_fwd.cu — forward of the SAF hybrid causal attention layer, and the
// static-head engine that the backward reuses for dV.
//
// Method ("When Can Attention Heads Be Statically Defined?", close-reading
// notes): a dynamic head computes softmax_causal(Q K^T / sqrt(d_h)) V (§1); a
// frozen head mixes V with P(i,j) = exp(alpha(j) + rho(i-j)) / Z(i), j <= i
// (Eq. (3)), which the fused kernel rebuilds tile by tile from alpha, rho and
// Z and multiplies by V, without any Q/K work (§3.3, App. D.2, Fig. 2).
//
// Kernels
//   static_prep_kernel  (K1) per static head: the generator tables and
//                       log Z(i).  Because alpha/rho are shared by the batch,
//                       this runs once per head, not once per sequence.
//   hybrid_fwd_kernel   (K2) one persistent launch, one CTA per SM, over a
//                       longest-first list of work items:
//     dynamic item (b, h, I): Q tile I against key tiles J = 0..I; S = Q K^T
//       and O += P V run on tcgen05 with fp32 accumulators in TMEM; online
//       softmax in registers, one query row per thread.
//     static item (h, I, batch group): for J = 0..I a generated tile G[I,J]
//       (bf16, in shared memory) feeds one MMA per sequence of the group, so
//       one generated tile serves the whole batch.
//
// Factored static generator.  With a(j) = exp(alpha(j) - max alpha) and
// r(d) = exp(rho(d) - max rho), P(i,j) = a(j) r(i-j) / Z'(i) where
// Z'(i) = sum_{k<=i} a(k) r(i-k): the shift cancels between numerator and
// Z.  A tile element is then two multiplies, no exponential.  When
// range(alpha) + range(rho) > 80 the products could underflow in fp32, and
// the head falls back to the exact form exp2(alpha2(j) + rho2(i-j) - log2 Z(i)).
//
// Warp roles in K2 (384 threads): warp 0 issues TMA copies, warp 1 issues
// the S = Q K^T MMAs and warp 3 the P V MMAs (one lane each), warp 2 owns the
// TMEM allocation, warps 4..11 are two compute warpgroups (softmax / tile generation / epilogue):
// each tile row belongs to one thread of each, which split its 128 key
// columns and exchange row maxima and sums through shared memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "attn_fwd_kernel.cuh"
#include "attn_kernels.h"
#include "internal.h"

namespace saf {

// ============================================================ K1: static prep
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxFactoredRange = 80.0f;

__device__ __forceinline__ void block_minmax(float& mx, float& mn, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  __syncthreads();
  if (lane == 0) {
    red[warp] = mx;
    red[32 + warp] = mn;
  }
  __syncthreads();
  mx = red[0];
  mn = red[32];
  for (int w = 1; w < nw; ++w) {
    mx = fmaxf(mx, red[w]);
    mn = fminf(mn, red[32 + w]);
  }
}

// grid (T / kPrepRows, n_static), 256 threads (8 warps), dynamic smem 2 * T + 8
// floats.  Each block scans alpha/rho for their finite ranges and picks the
// mode.  Factored heads: the block writes its kPrepRows entries of the tables and,
// block 0, the head's shift max alpha + max rho.  Exact heads: each warp
// also forms log Z of kPrepRows / 8 rows by an online log-sum-exp, its 32 lanes
// splitting the causal sum, merged across lanes in a fixed order.
constexpr int kPrepRows = 128;  // rows of a head per block (T is a multiple of 128)

__global__ void __launch_bounds__(256) static_prep_kernel(StaticPrep p) {
  extern __shared__ float sh[];
  __shared__ float red[64];
  const int T = p.T, hs = blockIdx.y, h = p.heads[hs];
  const int row0 = blockIdx.x * kPrepRows;
  const int nload = row0 + kPrepRows;  // entries 0 .. row0 + kPrepRows - 1 are needed
  float* sa = sh;
  float* sr = sh + T + 8;  // sr[-8 .. -1] = 0: the last stride reads past d = 0
  const float* alpha = p.alpha + (size_t)h * T;
  const float* rho = p.rho + (size_t)h * T;
  // finite max/min of alpha and rho over the whole head (every block agrees)
  float amax = -INFINITY, amin = INFINITY, rmax = -INFINITY, rmin = INFINITY;
  // 16-byte loads, four per thread in flight (T is a multiple of 128)
  const float4* alpha4 = reinterpret_cast<const float4*>(alpha);
  const float4* rho4 = reinterpret_cast<const float4*>(rho);
#pragma unroll 4
  for (int t4 = threadIdx.x; t4 < T / 4; t4 += blockDim.x) {
    const float4 a4 = alpha4[t4], r4 = rho4[t4];
    const float av[4] = {a4.x, a4.y, a4.z, a4.w};
    const float rv[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * t4 + e;
      if (t < nload) {
        sa[t] = av[e];
        sr[t] = rv[e];
      }
      if (isfinite(av[e])) { amax = fmaxf(amax, av[e]); amin = fminf(amin, av[e]); }
      if (isfinite(rv[e])) { rmax = fmaxf(rmax, rv[e]); rmin = fminf(rmin, rv[e]); }
    }
  }
  block_minmax(amax, amin, red);
  block_minmax(rmax, rmin, red);
  const bool all_masked = !(amax > -INFINITY) || !(rmax > -INFINITY);
  const bool exact = !all_masked && ((amax - amin) + (rmax - rmin) > kMaxFactoredRange);
  float* a_tab = p.a_tab + (size_t)hs * T;
  float* r_tab = p.r_tab + (size_t)hs * (T + 128);
  float* row_tab = p.row_tab + (size_t)hs * T;
  float* logZ = p.logZ + (size_t)hs * T;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.mode[hs] = exact ? 1 : 0;
    p.shift[hs] = (exact || all_masked) ? 0.f : amax + rmax;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (!exact) {
    // a = exp(alpha - max), r = exp(rho - max) for this block's kPrepRows entries.
    // Z'(i) is not formed here: the forward sums it from its own tiles and
    // the backward reads it back from the forward's lse.
    __syncthreads();
    for (int t = threadIdx.x; t < kPrepRows; t += blockDim.x) {
      a_tab[row0 + t] = all_masked ? 0.f : expf(sa[row0 + t] - amax);
      r_tab[127 + row0 + t] = all_masked ? 0.f : expf(sr[row0 + t] - rmax);
    }
    if (blockIdx.x == 0 && threadIdx.x < 127) r_tab[threadIdx.x] = 0.f;
    if (blockIdx.x == 0 && threadIdx.x == 127) r_tab[T + 127] = 0.f;
  } else {
    __syncthreads();
    for (int m = 0; m < kPrepRows / 8; ++m) {
      const int i = row0 + warp * (kPrepRows / 8) + m;
      // per-lane online log-sum-exp, then a fixed-order merge across lanes
      float mx = -INFINITY, sm = 0.f;
      for (int k = lane; k <= i; k += 32) {
        const float t = sa[k] + sr[i - k];
        if (t > mx) {
          sm = sm * expf(mx - t) + 1.f;
          mx = t;
        } else if (t > -INFINITY) {
          sm += expf(t - mx);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, mx, o);
        const float so = __shfl_xor_sync(0xffffffffu, sm, o);
        const float mn = fmaxf(mx, mo);
        if (mn > -INFINITY) {
          sm = sm * expf(mx - mn) + so * expf(mo - mn);
          mx = mn;
        }
      }
      if (lane == 0) {
        const float lz = (mx > -INFINITY) ? mx + logf(sm) : -INFINITY;
        logZ[i] = lz;
        row_tab[i] = (mx > -INFINITY) ? -lz * kLog2e : -INFINITY;
      }
    }
    for (int t = threadIdx.x; t < kPrepRows; t += blockDim.x) {
      a_tab[row0 + t] = sa[row0 + t] * kLog2e;
      r_tab[127 + row0 + t] = sr[row0 + t] * kLog2e;
    }
    if (blockIdx.x == 0 && threadIdx.x < 127) r_tab[threadIdx.x] = -INFINITY;
    if (blockIdx.x == 0 && threadIdx.x == 127) r_tab[T + 127] = -INFINITY;
  }
}

__global__ void zero_u32_kernel(uint32_t* dst, size_t n) {
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x)
    dst[i] = 0u;
}

int elementwise_blocks(size_t n) {
  size_t b = (n + 1023) / 1024;
  if (b < 1) b = 1;
  if (b > 4096) b = 4096;
  return (int)b;
}

}  // namespace

cudaError_t launch_static_prep(const StaticPrep& p, cudaStream_t s) {
  if (p.n_static == 0) return cudaSuccess;
  const size_t smem = (2 * (size_t)p.T + 8) * sizeof(float);
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(static_prep_kernel),
                                       160 * 1024);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  static_prep_kernel<<<dim3(p.T / kPrepRows, p.n_static), 256, smem, s>>>(p);
  trace_end(s, "static_prep");
  return cudaGetLastError();
}

cudaError_t launch_zero_u32(void* dst, size_t n_words, cudaStream_t s) {
  trace_begin(s);
  zero_u32_kernel<<<elementwise_blocks(n_words / 4), 256, 0, s>>>(static_cast<uint32_t*>(dst),
                                                                  n_words);
  trace_end(s, "zero");
  return cudaGetLastError();
}

cudaError_t launch_hybrid_fwd(const FwdLaunch& L, cudaStream_t s) {
  switch (L.d_h) {
    case 32: return L.transposed ? launch_fused<32, true>(L, s) : launch_fused<32, false>(L, s);
    case 64: return L.transposed ? launch_fused<64, true>(L, s) : launch_fused<64, false>(L, s);
    case 128:
      return L.transposed ? launch_fused<128, true>(L, s) : launch_fused<128, false>(L, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saf
