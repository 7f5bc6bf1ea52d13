// cache_common.cuh — the paged 8-bit cache as its kernels see it: the layout
// of a layer's record in a page, the rows of one call, and the pieces of PTX
// that only these kernels use.
//
// A page holds `page_size` tokens of every layer; one layer's record in it is
//   K codes [H_k, page, d] | V codes [H_kv, page, d] | K scales | V scales
// with e4m3 codes and one fp32 scale for each (page, head).  K is stored for
// the H_k heads that serve at least one dynamic query head.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace saf {

// ------------------------------------------------------------ PTX
// One look at the phase: the thread is not suspended.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 4-D tiled copy global -> shared, whole in the two inner dimensions.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c2), "r"(c3)
      : "memory");
}

// tmem_ld_x16 with the maximum of the 16 values as floats (a NaN does not
// count) in `top`; valid after tmem_wait_ld as well (sm_103).
__device__ __forceinline__ void tmem_ld_max_x16(uint32_t taddr, uint32_t (&r)[16], float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=f"(top)
      : "r"(taddr)
      : "memory");
}

// 16-byte asynchronous copy global -> shared; `bytes` (0..16) are read, the
// rest of the destination is zero-filled.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t a) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a));
}

__device__ __forceinline__ uint32_t lds_word(uint32_t a) {
  uint32_t w[1];
  lds_words(w, a);
  return w[0];
}

// e4m3 and e5m2 of two f16 values, saturating; the NaN code for NaN
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_e5m2x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
// Two e5m2 codes as packed f16 (e5m2 is f16's upper byte).
__device__ __forceinline__ uint32_t e5m2x2_f16x2(uint32_t v) {
  return __byte_perm(v, 0, 0x1404);
}

// Two e4m3 codes (low and high byte of v) as packed f16: exact (f16 holds
// every e4m3 value); the NaN code becomes NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  uint16_t a, b;
  asm("mov.b32 {%0, %1}, %2;" : "=h"(a), "=h"(b) : "r"(w));
  lo = e4m3x2_f16x2(a);
  hi = e4m3x2_f16x2(b);
}

// ... of two values
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// D += A B: 16 x 16 by 16 x 8, f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Of a block's scale (positive and normal).
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ weights in f16
// The second product takes its weights in f16, as p = 2^{y - m} for the exponents y
// of a row and a base m that follows their maximum: m moves to kRoom below it once it
// lies more than kRoom + kLag below.  So the largest weight is 2^11 to 2^15, in f16's
// upper range, and a weight loses bits only where it is less than 2^-25 of the
// largest (it is then off by at most 2^-36 of it); below 2^-36 it is lost.  The sum
// of the softmax takes the weights in fp32.  (A base at the maximum itself loses
// weights from 2^-14 on and all below 2^-25: 131072 keys 17.5 nats below one, a share
// of 0.0033, came out as 0.)
constexpr float kRoom = 11.f, kLag = 4.f;

// 2^e as fp32 for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// A bounded wait whose rare part is a call, for a thread that a whole CTA waits on:
// what follows the wait then lies right behind it.
static __device__ __noinline__ void wait_long(uint32_t bar, uint32_t parity, volatile int* abort,
                                              int* status, int site) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (mbar_test_wait(bar, parity)) return;
    if (*abort) return;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      *abort = 1;
      atomicCAS(status, 0, site);
      return;
    }
  }
}
__device__ __forceinline__ void poll_bar(uint64_t* bar, uint32_t parity, const WaitCtl& w,
                                         int site) {
  const uint32_t a = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < 512; ++i)
    if (mbar_test_wait(a, parity)) return;
  wait_long(a, parity, w.abort, w.status, site);
}

// ------------------------------------------------------------ the rows of a call
// Slot b takes n_new(b) of the n_q rows that the call holds for each slot;
// row t stands at position seq_len - n_new + t.  Lengths beyond the page
// table are cut to it: no page can hold what lies behind.
struct Rows {
  int n_new;  // rows of this slot
  int base;   // position of row 0 (negative: the first rows see nothing)
  int cap;    // keys that exist for the slot
};
__device__ __forceinline__ Rows slot_rows(const CacheCall& c, int b) {
  Rows r;
  const int len = c.seq_len[b];
  int n = c.n_new ? c.n_new[b] : c.n_q;
  n = n < 0 ? 0 : (n > c.n_q ? c.n_q : n);
  r.n_new = n;
  // a negative length counts as zero; len - n cannot overflow (len >= 0, n >= 0)
  const int l = len < 0 ? 0 : len;
  r.base = l - n;
  const int room = c.max_pages << c.page_shift;  // fits: checked on the host
  r.cap = l < room ? l : room;
  return r;
}

// The page of table row b, column col; -1 where the entry names no page of
// the pool (a hole: its tokens weigh nothing).
__device__ __forceinline__ int page_at(const CacheCall& c, int b, int col) {
  const int p = __ldg(c.page_table + (size_t)b * c.max_pages + col);
  return (unsigned)p < (unsigned)c.n_pages ? p : -1;
}

// 4 components of a row's mean as bf16: o over the sum l of its weights.  A row
// without weight gets 0 even where a key that it sees holds NaN.
__device__ __forceinline__ uint2 mean4(const float4& o, float l) {
  if (l == 0.f) return make_uint2(0u, 0u);
  const float inv = 1.f / l;
  return make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// ------------------------------------------------------------ joining parts
// A unit of attention that was cut leaves one part per CTA: for each row the
// base m of its exponents (to base 2), l = sum of the weights relative to m,
// and the weighted sum o, of which a thread takes 4 components.  Parts are added
// in the order of the CTAs.
struct Part {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void add_part(Part& a, const Part& b) {
  // (a part that saw nothing holds zeros: it takes no part, but a NaN does)
  const float top = fmaxf(a.m, b.m);
  const float fa = top == -INFINITY ? 1.f : fast_exp2(a.m - top);
  const float fb = top == -INFINITY ? 1.f : fast_exp2(b.m - top);
  a.m = top;
  a.l = fmaf(a.l, fa, b.l * fb);
  a.o.x = fmaf(a.o.x, fa, b.o.x * fb);
  a.o.y = fmaf(a.o.y, fa, b.o.y * fb);
  a.o.z = fmaf(a.o.z, fa, b.o.z * fb);
  a.o.w = fmaf(a.o.w, fa, b.o.w * fb);
}
// Threads of a joining block, and what it splits them by: `split` of them take
// every split-th part of the same 4 components.  What a unit of many parts costs
// is the latency of its loads, so many parts want many threads; few parts want
// few blocks.  For the same reason blocks are counted by units where there are
// fewer of them than CTAs.  (One token against 29242, 4 K/V heads in 152 parts
// each: 41 us with a thread for all parts of its components, 14.1 us so.)
constexpr int kJoinThreads = 128, kJoinSplit = 8;
inline int join_split(long long ctas, long long units) {
  return ctas > 8 * units ? kJoinSplit : 1;
}
// All threads of the block call this; load(k) reads part k of the thread's
// components.  The result is that of the threads with s = 0.
template <int kAhead, class Load>
__device__ __forceinline__ Part join_parts(int s, int split, int n, bool live, const Load& load) {
  __shared__ Part others[kJoinThreads];
  Part a{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (live)
    for (int k0 = s; k0 < n; k0 += kAhead * split) {
      Part x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k * split < n) x[k] = load(k0 + k * split);
      float top = a.m;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k * split < n) top = fmaxf(top, x[k].m);
      const float f0 = top == -INFINITY ? 1.f : fast_exp2(a.m - top);
      a.m = top;
      a.l *= f0;
      a.o = make_float4(a.o.x * f0, a.o.y * f0, a.o.z * f0, a.o.w * f0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k * split < n) {
          const float f = top == -INFINITY ? 1.f : fast_exp2(x[k].m - top);
          a.l = fmaf(f, x[k].l, a.l);
          a.o.x = fmaf(f, x[k].o.x, a.o.x);
          a.o.y = fmaf(f, x[k].o.y, a.o.y);
          a.o.z = fmaf(f, x[k].o.z, a.o.z);
          a.o.w = fmaf(f, x[k].o.w, a.o.w);
        }
    }
  if (split > 1) {
    others[threadIdx.x] = a;
    __syncthreads();
    if (s == 0)
      for (int k = 1; k < split; ++k) add_part(a, others[threadIdx.x + k * (kJoinThreads / split)]);
  }
  return a;
}

}  // namespace saf
