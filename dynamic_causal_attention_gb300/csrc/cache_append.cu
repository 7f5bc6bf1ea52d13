// cache_append.cu — new K/V rows into the pages, quantised.
//
// A block is the tokens of one page under one K or V head.  Its scale is the
// least power of two s = 2^e, e >= -64, with 448 s >= |x| for every finite x
// that it holds (448 is e4m3's largest value), and its codes are e4m3(x / s):
// x / s is exact, so a code is rounded once.  When a new token is too large
// for the block's scale, the scale grows and the older codes become
// e4m3(code s_old / s): exact but for codes that sink below e4m3's normal
// range.  A page whose first token is new starts over: what lay there is
// forgotten.  An infinite x is stored as +-448 s, a NaN as NaN; neither counts
// for the scale.
//
// One warp takes one block: it reads its new rows twice (the second time from
// L1 / L2), once for the largest value and once to encode.
#include <cuda_bf16.h>

#include "cache_common.cuh"

namespace saf {
namespace {

constexpr int kWarps = 4;

// 8 consecutive values
__device__ __forceinline__ void load8(const void* base, size_t off, bool f32, float (&x)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    return;
  }
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off));
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(ww[i] << 16);
    x[2 * i + 1] = __uint_as_float(ww[i] & 0xffff0000u);
  }
}

// The exponent of the least scale that holds amax (finite, >= 0).
__device__ __forceinline__ int scale_exponent(float amax) {
  const int bits = __float_as_int(amax);
  // 448 = 1.75 * 2^8: one more when the fraction is above 0.75
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return e < -64 ? -64 : e;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    cache_append_kernel(const __grid_constant__ CacheAppend p) {
  constexpr int kLanes = D / 8;        // lanes of a row
  constexpr int kRows = 32 / kLanes;   // rows that a warp reads at once
  const CacheCall& c = p.c;
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int n_heads = c.H_k + c.H_kv;
  const int head = unit % n_heads, nth = unit / n_heads;  // head: K heads first
  const int b = blockIdx.y;
  const Rows r = slot_rows(c, b);
  const int begin = r.base < 0 ? 0 : r.base;  // rows before position 0 are not kept
  const long long first_col = begin >> c.page_shift;
  const long long lo_page = (first_col + nth) << c.page_shift;
  if (r.n_new == 0 || lo_page >= r.cap) return;
  const int lo = lo_page < begin ? begin : (int)lo_page;          // first new token of the block
  const int hi = min(r.cap, (int)lo_page + (1 << c.page_shift));  // end of its new tokens
  if (lo >= hi) return;
  const int page = page_at(c, b, (int)(first_col + nth));
  if (page < 0) return;  // a hole: nowhere to put them

  const bool is_v = head >= c.H_k;
  const int ph = is_v ? head - c.H_k : head;      // head in the record
  const int kv = is_v ? ph : p.kv_of[ph];         // head of the source
  const void* src = is_v ? p.V : p.K;
  uint8_t* rec = c.layer + (size_t)page * c.page_stride;
  uint8_t* codes = rec + (is_v ? c.off_v : 0) + ((size_t)ph << c.page_shift) * D;
  float* scale_at = reinterpret_cast<float*>(rec + (is_v ? c.off_vs : c.off_ks)) + ph;
  const size_t row0 = ((size_t)b * c.H_kv + kv) * c.n_q;  // source row of t = 0
  const int rl = lane / kLanes, dl = lane % kLanes * 8;

  float amax = 0.f;
  for (int j = lo + rl; j < hi; j += kRows) {
    float x[8];
    load8(src, (row0 + (j - r.base)) * D + dl, p.f32, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(x[i]);
      if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // finite
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  int e = scale_exponent(amax);
  float scale = pow2f(e), inv = pow2f(-e);
  const int n_old = lo - (int)lo_page;
  if (n_old > 0) {
    const float old = *scale_at;
    __syncwarp();  // read by every lane before lane 0 writes it
    if (old >= scale) {
      scale = old;
      inv = 1.f / old;  // exact: an old scale is a power of two
    } else {
      const float f = old * inv;
      for (int i = lane; i < n_old * (D / 4); i += 32) {
        uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
        uint32_t lo2, hi2;
        e4m3x4_f16x4(*w, lo2, hi2);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
        const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
        *w = e4m3x2(a.x * f, a.y * f) | e4m3x2(z.x * f, z.y * f) << 16;
      }
    }
  }
  if (lane == 0) *scale_at = scale;
  for (int j = lo + rl; j < hi; j += kRows) {
    float x[8];
    load8(src, (row0 + (j - r.base)) * D + dl, p.f32, x);
    uint2 w;
    w.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
    w.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
    *reinterpret_cast<uint2*>(codes + (size_t)(j - (int)lo_page) * D + dl) = w;
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppend& p, int d_h, cudaStream_t s) {
  const CacheCall& c = p.c;
  // pages that n_q rows in a row can touch: the first may begin anywhere
  const long long pages = ((long long)c.n_q + (1 << c.page_shift) - 2 >> c.page_shift) + 1;
  const long long units = pages * (c.H_k + c.H_kv);
  const dim3 grid((unsigned)((units + kWarps - 1) / kWarps), (unsigned)c.n_seqs);
  trace_begin(s);
  switch (d_h) {
    case 32: cache_append_kernel<32><<<grid, kWarps * 32, 0, s>>>(p); break;
    case 64: cache_append_kernel<64><<<grid, kWarps * 32, 0, s>>>(p); break;
    case 128: cache_append_kernel<128><<<grid, kWarps * 32, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  trace_end(s, "cache_append");
  return cudaGetLastError();
}

}  // namespace saf
