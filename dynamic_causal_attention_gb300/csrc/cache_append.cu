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
// A call with many rows gives each block a CTA that holds the block's new rows
// in registers between finding the largest value and encoding, so that they are
// read once (4 prompts of 1999 rows, 28 heads, d_h = 128: 17.8 us, 71% of the
// copy rate; from fp32 24.5 us, 86%).  With few
// rows a block has one or two, and one warp takes it and reads them twice, the
// second time from L1.
#include <cuda_bf16.h>

#include "cache_common.cuh"

namespace saf {
namespace {

constexpr int kWarps = 4;
// From kManyRows rows on, a block of more than 256 groups of 8 values has a CTA
// whose threads hold kGroups each.  (Measured, 4 x 1999 rows of 28 heads, d_h =
// 128: blocks of 256 groups 16 us by warps, 21 us by CTAs; of 1024, 20 and 16 us;
// of 2048, 32 and 22 us.  64 x 16 rows of 24 heads: 3.9 and 4.9 us.)
constexpr int kManyRows = 32, kGroups = 4;

// 8 consecutive values as they lie in memory: bf16 or fp32
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void load8(const void* base, size_t off, Raw8<F32>& r) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) +
                                                  off * (F32 ? 4 : 2));
  r.w[0] = __ldg(p);
  if (F32) r.w[F32 ? 1 : 0] = __ldg(p + 1);
}
template <bool F32>
__device__ __forceinline__ void values8(const Raw8<F32>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = r.w[F32 ? i >> 1 : 0];
    if (F32) {
      x[2 * i] = __uint_as_float(i & 1 ? v.z : v.x);
      x[2 * i + 1] = __uint_as_float(i & 1 ? v.w : v.y);
    } else {
      const uint32_t w = i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
      x[2 * i] = __uint_as_float(w << 16);
      x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
}

// The exponent of the least scale that holds amax (finite, >= 0).
__device__ __forceinline__ int scale_exponent(float amax) {
  const int bits = __float_as_int(amax);
  // 448 = 1.75 * 2^8: one more when the fraction is above 0.75
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return e < -64 ? -64 : e;
}

// One block: the tokens of page `nth` (counted from the first that the call
// writes to) of slot b under `head` (stored K heads first, then V).
struct Block {
  const void* src;   // rows of the head's source
  size_t row0;       // source row of position 0 (wraps where that lies before it)
  int lo, hi;        // new tokens: positions [lo, hi)
  int first;         // position of the page's first token
  int col;           // the page's column in the table
  // where it lies, once its page is known
  uint8_t* codes;
  float* scale_at;
};
__device__ __forceinline__ bool find_rows(const CacheAppend& p, int b, int nth, int head,
                                          Block& k) {
  const CacheCall& c = p.c;
  const Rows r = slot_rows(c, b);
  const int begin = r.base < 0 ? 0 : r.base;  // rows before position 0 are not kept
  const long long col = (long long)(begin >> c.page_shift) + nth;
  const long long first = col << c.page_shift;
  if (r.n_new == 0 || first >= r.cap) return false;
  k.first = (int)first;
  k.lo = max(begin, k.first);
  k.hi = min(r.cap, k.first + (1 << c.page_shift));
  k.col = (int)col;
  const int kv = head >= c.H_k ? head - c.H_k : p.kv_of[head];
  k.src = head >= c.H_k ? p.V : p.K;
  k.row0 = ((size_t)b * c.H_kv + kv) * c.n_q - (size_t)(long long)r.base;
  return k.lo < k.hi;
}
__device__ __forceinline__ bool find_page(const CacheAppend& p, int D, int b, int head, Block& k) {
  const CacheCall& c = p.c;
  const int page = page_at(c, b, k.col);
  if (page < 0) return false;  // a hole: nowhere to put them
  const bool is_v = head >= c.H_k;
  const int ph = is_v ? head - c.H_k : head;  // head in the record
  uint8_t* rec = c.layer + (size_t)page * c.page_stride;
  k.codes = rec + (is_v ? c.off_v : 0) + ((size_t)ph << c.page_shift) * D;
  k.scale_at = reinterpret_cast<float*>(rec + (is_v ? c.off_vs : c.off_ks)) + ph;
  return true;
}

__device__ __forceinline__ float largest(const float (&x)[8], float amax) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // finite
  }
  return amax;
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  return make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16,
                    e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16);
}

// The scale of a block whose new rows have `amax`; the older tokens' codes
// follow if it grows.  `old` is the scale before; n threads share the work.
__device__ __forceinline__ float block_scale(const Block& k, int D, float amax, float old, int i0,
                                             int n) {
  const int e = scale_exponent(amax);
  const float scale = pow2f(e);
  if (k.lo == k.first) return scale;  // the block starts over
  if (old >= scale) return old;
  const float f = old * pow2f(-e);
  for (int i = i0; i < (k.lo - k.first) * (D / 4); i += n) {
    uint32_t* w = reinterpret_cast<uint32_t*>(k.codes) + i;
    uint32_t lo, hi;
    e4m3x4_f16x4(*w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    *w = e4m3x2(a.x * f, a.y * f) | e4m3x2(z.x * f, z.y * f) << 16;
  }
  return scale;
}

// Few rows: a warp takes a block.
template <int D, bool F32>
__global__ void __launch_bounds__(kWarps * 32)
    append_few_kernel(const __grid_constant__ CacheAppend p) {
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows that a warp reads at once
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5), n_heads = p.c.H_k + p.c.H_kv;
  const int head = unit % n_heads;
  Block k;
  if (!find_rows(p, blockIdx.y, unit / n_heads, head, k) ||
      !find_page(p, D, blockIdx.y, head, k))
    return;
  const int rl = lane / kLanes, dl = lane % kLanes * 8;
  const float old = *k.scale_at;
  float amax = 0.f, x[8];
  Raw8<F32> raw;
  for (int j = k.lo + rl; j < k.hi; j += kRows) {
    load8(k.src, (k.row0 + j) * D + dl, raw);
    values8(raw, x);
    amax = largest(x, amax);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  // (the shuffles also see to it that every lane has read `old` before lane 0 writes)
  __syncwarp();
  const float scale = block_scale(k, D, amax, old, lane, 32);
  if (lane == 0) *k.scale_at = scale;
  const float inv = 1.f / scale;  // exact: a power of two
  for (int j = k.lo + rl; j < k.hi; j += kRows) {
    load8(k.src, (k.row0 + j) * D + dl, raw);
    values8(raw, x);
    *reinterpret_cast<uint2*>(k.codes + (size_t)(j - k.first) * D + dl) = encode8(x, inv);
  }
}

// Many rows: a CTA takes a block and keeps kGroups groups of 8 values a thread, as
// they lie in memory.  The rows are on their way while the page is looked up.
template <int D, bool F32>
__global__ void __launch_bounds__(512) append_many_kernel(const __grid_constant__ CacheAppend p) {
  __shared__ float top[16];
  constexpr int kLanes = D / 8;
  const int n_heads = p.c.H_k + p.c.H_kv, unit = blockIdx.x, head = unit % n_heads;
  Block k;
  if (!find_rows(p, blockIdx.y, unit / n_heads, head, k)) return;
  const int rl = threadIdx.x / kLanes, dl = threadIdx.x % kLanes * 8, step = blockDim.x / kLanes;
  Raw8<F32> raw[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int j = k.first + rl + i * step;
    raw[i] = {};
    if (j >= k.lo && j < k.hi) load8(k.src, (k.row0 + j) * D + dl, raw[i]);
  }
  if (!find_page(p, D, blockIdx.y, head, k)) return;
  const float old = *k.scale_at;
  float amax = 0.f, x[8];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    values8(raw[i], x);
    amax = largest(x, amax);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = amax;
  __syncthreads();  // (every thread has read `old`)
  for (int i = 0; i < (int)blockDim.x / 32; ++i) amax = fmaxf(amax, top[i]);
  const float scale = block_scale(k, D, amax, old, threadIdx.x, blockDim.x);
  if (threadIdx.x == 0) *k.scale_at = scale;
  const float inv = 1.f / scale;  // exact: a power of two
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int j = k.first + rl + i * step;
    values8(raw[i], x);
    if (j >= k.lo && j < k.hi)
      *reinterpret_cast<uint2*>(k.codes + (size_t)(j - k.first) * D + dl) = encode8(x, inv);
  }
}

template <int D, bool F32>
cudaError_t launch(const CacheAppend& p, cudaStream_t s) {
  const CacheCall& c = p.c;
  // pages that n_q rows in a row can touch: the first may begin anywhere
  const long long pages = ((long long)c.n_q + (1 << c.page_shift) - 2 >> c.page_shift) + 1;
  const long long units = pages * (c.H_k + c.H_kv);
  trace_begin(s);
  // groups of 8 values in a block: 64 (16 x 32) to 2048 (128 x 128)
  const int groups = (D / 8) << c.page_shift;
  if (c.n_q < kManyRows || groups <= 256)
    append_few_kernel<D, F32>
        <<<dim3((unsigned)((units + kWarps - 1) / kWarps), (unsigned)c.n_seqs), kWarps * 32, 0,
           s>>>(p);
  else
    append_many_kernel<D, F32>
        <<<dim3((unsigned)units, (unsigned)c.n_seqs), groups / kGroups, 0, s>>>(p);
  trace_end(s, "cache_append");
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppend& p, int d_h, cudaStream_t s) {
  switch (d_h) {
    case 32: return p.f32 ? launch<32, true>(p, s) : launch<32, false>(p, s);
    case 64: return p.f32 ? launch<64, true>(p, s) : launch<64, false>(p, s);
    case 128: return p.f32 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace saf
