// rotary.cu — rotary positions of Q and K, and their gradient.
//
// A pair (x1, x2) of a row at position p is turned by the angle p f:
//     (x1 cos pf - x2 sin pf,  x2 cos pf + x1 sin pf) * scale,
// backwards (the gradient) by -p f.  The angle is not formed in floating point:
// f is kept as a fraction of a turn in units of 2^-64, so p f modulo one turn is
// the low 64 bits of an integer product, exact for every position (in fp32 the
// angle of position 10^6 would be off by 0.06 radians).  Its upper 32 bits, as a
// signed fraction of half a turn, go to sincospif: off by 2^-32 of a turn from the
// cut and 2^-24 of itself from the conversion.
//
// The rows are read once and written once, so the kernel is bound by memory.  A block
// takes a few tokens, forms their cosines and sines once in shared memory and uses
// them for every head of Q and K; a thread moves 16-byte vectors, four units of two
// vectors in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace saf {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a block
constexpr int kUnroll = 4;

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

// W consecutive elements.
template <typename T, int W>
struct Vec {
  union {
    typename Raw<sizeof(T) * W>::type raw;
    uint32_t word[sizeof(T) * W >= 4 ? sizeof(T) * W / 4 : 1];
    uint16_t half;
  };
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word[i]);
    else if constexpr (W == 1) return __uint_as_float((uint32_t)half << 16);
    else return __uint_as_float(i & 1 ? word[i >> 1] & 0xffff0000u : word[i >> 1] << 16);
  }
  __device__ __forceinline__ void set2(int i, float a, float b) {  // i even
    if constexpr (sizeof(T) == 4) {
      word[i] = __float_as_uint(a);
      word[i + 1] = __float_as_uint(b);
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      word[i >> 1] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  __device__ __forceinline__ void set1(float a) {
    if constexpr (sizeof(T) == 4) word[0] = __float_as_uint(a);
    else half = __bfloat16_as_ushort(__float2bfloat16_rn(a));
  }
};

// n / d for 0 <= n < 2^31 by one multiplication (d >= 1): m = 2^32 (2^s - d) / d + 1
// with 2^s the least power of two >= d.
__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.m) + n) >> f.s;
}

template <typename T, int W, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  extern __shared__ float tab[];  // [tokens][half] cosines, then as many sines
  __shared__ int64_t row_at[4][kMaxTokens];  // q, k, q_out, k_out: where a token's row starts
  __shared__ int pos_of[kMaxTokens], state_of[kMaxTokens];  // 0: left alone, 1: turned, 2: cleared
  const int half = p.rot / 2;
  float* cosv = tab;
  float* sinv = tab + p.tokens * half;
  const long long n0 = (long long)blockIdx.x * p.tokens;
  const int nt = (int)min((long long)p.tokens, (long long)p.B * p.T - n0);
  if ((int)threadIdx.x < nt) {
    const uint32_t n = (uint32_t)(n0 + threadIdx.x);
    const uint32_t b = fast_div(n, p.by_T), t = n - b * (uint32_t)p.T;
    int pos = (int)t;
    bool live = true;
    if (p.positions) {
      pos = p.positions[n];
    } else if (p.cu) {
      // the last sequence that starts at or before the row, and holds it
      int lo = 0, hi = p.n_seqs;  // cu[lo] <= t for lo > 0 or t >= cu[0]; cu[hi] > t or hi = n_seqs
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= (int)t) lo = mid;
        else hi = mid;
      }
      const int a = p.n_seqs > 0 ? p.cu[lo] : 0;
      live = p.n_seqs > 0 && a <= (int)t && (int)t < p.cu[lo + 1];
      pos = (int)t - a;
    } else if (p.seq_len) {
      const int fresh = p.n_new ? max(0, min(p.n_new[b], p.T)) : p.T;
      live = (int)t < fresh;
      pos = p.seq_len[b] - fresh + (int)t;
    }
    pos_of[threadIdx.x] = pos;
    state_of[threadIdx.x] = live ? 1 : p.clear ? 2 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      row_at[i][threadIdx.x] = (int64_t)b * p.x[i].seq + (int64_t)t * p.x[i].row;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = (int)fast_div((uint32_t)i, p.by_half), j = i - tok * half;
    const uint64_t phase = (uint64_t)(int64_t)pos_of[tok] * p.turns[j];  // modulo one turn
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    cosv[i] = c * p.scale;
    sinv[i] = s * p.scale_sin;
  }
  __syncthreads();
  const int total = nt * (int)p.row_units;
  for (int i0 = threadIdx.x; i0 < total; i0 += kThreads * kUnroll) {
    Vec<T, W> a[kUnroll], b[kUnroll];
    T *to_a[kUnroll], *to_b[kUnroll];
    int at[kUnroll];  // >= 0: offset of the pair's cosines; -1: copied; -2: cleared; -3: nothing
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * kThreads;
      at[k] = -3;
      to_a[k] = to_b[k] = nullptr;
      if (i >= total) continue;
      const int tok = (int)fast_div((uint32_t)i, p.by_row);
      const int r = i - tok * (int)p.row_units;
      const int h = (int)fast_div((uint32_t)r, p.by_units), u = r - h * p.units;
      const int st = state_of[tok];
      if (st == 0) continue;
      const bool isk = h >= p.H;
      const int hh = isk ? h - p.H : h;
      const RotaryRows& in = p.x[isk ? 1 : 0];
      const RotaryRows& out = p.x[isk ? 3 : 2];
      const T* src = static_cast<const T*>(in.p) + row_at[isk ? 1 : 0][tok] + (int64_t)hh * in.head;
      T* dst = static_cast<T*>(out.p) + row_at[isk ? 3 : 2][tok] + (int64_t)hh * out.head;
      int ea, eb;
      if (u < p.pair_units) {
        ea = HALF ? u * W : 2 * u * W;
        eb = HALF ? half + u * W : ea + W;
        at[k] = tok * half + u * W;
      } else {
        ea = p.rot + 2 * (u - p.pair_units) * W;
        eb = ea + W;
        at[k] = -1;
      }
      if (st == 2) at[k] = -2;
      to_a[k] = dst + ea;
      to_b[k] = eb < p.d ? dst + eb : nullptr;
      if (st == 2) {
        a[k].raw = {};
        b[k].raw = {};
      } else {
        a[k].raw = *reinterpret_cast<const decltype(a[k].raw)*>(src + ea);
        if (eb < p.d) b[k].raw = *reinterpret_cast<const decltype(b[k].raw)*>(src + eb);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (at[k] >= 0) {
        const float* c = cosv + at[k];
        const float* s = sinv + at[k];
        if constexpr (HALF) {
          if constexpr (W == 1) {
            const float x = a[k].get(0), y = b[k].get(0);
            a[k].set1(x * c[0] - y * s[0]);
            b[k].set1(y * c[0] + x * s[0]);
          } else {
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const float x0 = a[k].get(e), x1 = a[k].get(e + 1);
              const float y0 = b[k].get(e), y1 = b[k].get(e + 1);
              a[k].set2(e, x0 * c[e] - y0 * s[e], x1 * c[e + 1] - y1 * s[e + 1]);
              b[k].set2(e, y0 * c[e] + x0 * s[e], y1 * c[e + 1] + x1 * s[e + 1]);
            }
          }
        } else {
          if constexpr (W == 1) {
            const float x = a[k].get(0), y = b[k].get(0);
            a[k].set1(x * c[0] - y * s[0]);
            b[k].set1(y * c[0] + x * s[0]);
          } else {
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const float x0 = a[k].get(e), y0 = a[k].get(e + 1);
              const float x1 = b[k].get(e), y1 = b[k].get(e + 1);
              const int q0 = e / 2, q1 = W / 2 + e / 2;
              a[k].set2(e, x0 * c[q0] - y0 * s[q0], y0 * c[q0] + x0 * s[q0]);
              b[k].set2(e, x1 * c[q1] - y1 * s[q1], y1 * c[q1] + x1 * s[q1]);
            }
          }
        }
      }
      if (at[k] > -3) {
        *reinterpret_cast<decltype(a[k].raw)*>(to_a[k]) = a[k].raw;
        if (to_b[k]) *reinterpret_cast<decltype(b[k].raw)*>(to_b[k]) = b[k].raw;
      }
    }
  }
}

FastDiv make_div(uint32_t d) {
  FastDiv f;
  f.s = 0;
  while ((1ull << f.s) < d) ++f.s;
  f.m = (uint32_t)((((1ull << f.s) - d) << 32) / d + 1);
  return f;
}

template <typename T>
cudaError_t launch(RotaryParams& p, int W, bool half, int grid, size_t smem, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  trace_begin(s);
  if (W == V && half) rotary_kernel<T, V, true><<<grid, kThreads, smem, s>>>(p);
  else if (W == V) rotary_kernel<T, V, false><<<grid, kThreads, smem, s>>>(p);
  else if (half) rotary_kernel<T, 1, true><<<grid, kThreads, smem, s>>>(p);
  else rotary_kernel<T, 1, false><<<grid, kThreads, smem, s>>>(p);
  trace_end(s, "rotary");
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(RotaryParams& p, bool f32, bool interleaved, int n_sms, cudaStream_t s) {
  const int size = f32 ? 4 : 2, V = 16 / size, half = p.rot / 2;
  // 16-byte vectors where every row and part of a row lies on their boundaries,
  // single elements otherwise
  bool wide = half % V == 0 && p.d % V == 0;
  for (int i = 0; i < 4; ++i) {
    const RotaryRows& x = p.x[i];
    if (p.H_k == 0 && (i & 1)) continue;
    wide &= reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.seq % V == 0 && x.row % V == 0 &&
            x.head % V == 0;
  }
  const int W = wide ? V : 1;
  p.pair_units = half / W;
  p.units = p.pair_units + (p.copy_rest ? ((p.d - p.rot) / W + 1) / 2 : 0);
  p.row_units = (uint32_t)p.units * (p.H + p.H_k);
  // tokens of a block: as many as keep four blocks for each SM (fewer sines to form
  // and more bytes in flight per block against an idle part of the GPU)
  const long long n = (long long)p.B * p.T;
  p.tokens = kMaxTokens;
  while (p.tokens > 1 && (n + p.tokens - 1) / p.tokens < 4ll * n_sms) p.tokens /= 2;
  p.by_T = make_div((uint32_t)p.T);
  p.by_half = make_div((uint32_t)half);
  p.by_row = make_div(p.row_units);
  p.by_units = make_div((uint32_t)p.units);
  const int grid = (int)((n + p.tokens - 1) / p.tokens);
  const size_t smem = (size_t)p.tokens * half * 2 * sizeof(float);
  return f32 ? launch<float>(p, W, !interleaved, grid, smem, s)
             : launch<__nv_bfloat16>(p, W, !interleaved, grid, smem, s);
}

}  // namespace saf
