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
// The rows are read once and written once, so the kernel is bound by memory.  A thread
// has a token and two vectors of 16 bytes of its rows (the two parts of eight pairs), forms
// their cosines and sines once in registers and goes through the heads of Q and K with
// them, three heads' loads in flight; no shared memory, no barrier.  With few tokens the
// heads are shared out over several threads, which then form the same sines.
// Measured: Q and K (bf16, parts of one projection) of 33.4k tokens, 12 + 12 heads of 64, 37 us,
// 5.5 TB/s or 83 % of the copy rate; fp32, 2 x 8190 tokens, 16 + 4 heads of 128, 57 us, 87 %;
// one token of 64 sequences 6 us (launch, position, sine, row: one latency after another).
// With the sines of 16 tokens in shared memory and a barrier the first took 48 us.
// Parts whose half is no whole vector go one element a load: 33.4k tokens of 12 + 12 heads of 80 with
// 20 turned take 121 us, of 128 with 26 turned 184, where their bytes take 38 and 61.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace saf {
namespace {

constexpr int kThreads = 64;  // (256: the last blocks leave more SMs idle, 38.8 us for 37.7)
constexpr int kUnroll = 3;  // heads in flight

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

// The position of row t of sequence b; false where the row is not worked on.
__device__ __forceinline__ bool position(const RotaryParams& p, uint32_t n, uint32_t b, uint32_t t,
                                         int& pos) {
  pos = (int)t;
  if (p.positions) {
    pos = p.positions[n];
  } else if (p.cu) {
    // the last sequence that starts at or before the row holds it, if any does
    int lo = 0, hi = p.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= (int)t) lo = mid;
      else hi = mid;
    }
    if (p.n_seqs == 0) return false;
    const int a = p.cu[lo];
    pos = (int)t - a;
    return a <= (int)t && (int)t < p.cu[lo + 1];
  } else if (p.seq_len) {
    const int fresh = p.n_new ? max(0, min(p.n_new[b], p.T)) : p.T;
    pos = p.seq_len[b] - fresh + (int)t;
    return (int)t < fresh;
  }
  return true;
}

// Turns (TURN) or copies two vectors of every head h0, h0 + step, ... of one tensor.
template <typename T, int W, bool HALF, bool TURN>
__device__ __forceinline__ void heads(const RotaryRows& in, const RotaryRows& out, uint32_t b,
                                      uint32_t t, int n_heads, int h0, int step, int ea, int eb,
                                      bool has_b, const float (&c)[W], const float (&s)[W]) {
  using V = Vec<T, W>;
  const T* src = static_cast<const T*>(in.p) + (int64_t)b * in.seq + (int64_t)t * in.row;
  T* dst = static_cast<T*>(out.p) + (int64_t)b * out.seq + (int64_t)t * out.row;
  for (int h = h0; h < n_heads; h += kUnroll * step) {
    V x[kUnroll], y[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (h + k * step >= n_heads) continue;
      const T* q = src + (int64_t)(h + k * step) * in.head;
      x[k].raw = *reinterpret_cast<const decltype(x[k].raw)*>(q + ea);
      if (TURN || has_b) y[k].raw = *reinterpret_cast<const decltype(x[k].raw)*>(q + eb);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (h + k * step >= n_heads) continue;
      if constexpr (TURN) {
        V& a = x[k];
        V& d = y[k];
        if constexpr (W == 1) {
          const float p = a.get(0), q = d.get(0);
          a.set1(p * c[0] - q * s[0]);
          d.set1(q * c[0] + p * s[0]);
        } else if constexpr (HALF) {
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const float p0 = a.get(e), p1 = a.get(e + 1), q0 = d.get(e), q1 = d.get(e + 1);
            a.set2(e, p0 * c[e] - q0 * s[e], p1 * c[e + 1] - q1 * s[e + 1]);
            d.set2(e, q0 * c[e] + p0 * s[e], q1 * c[e + 1] + p1 * s[e + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const float p0 = a.get(e), q0 = a.get(e + 1), p1 = d.get(e), q1 = d.get(e + 1);
            const int i = e / 2, j = W / 2 + e / 2;
            a.set2(e, p0 * c[i] - q0 * s[i], q0 * c[i] + p0 * s[i]);
            d.set2(e, p1 * c[j] - q1 * s[j], q1 * c[j] + p1 * s[j]);
          }
        }
      }
      T* q = dst + (int64_t)(h + k * step) * out.head;
      *reinterpret_cast<decltype(x[k].raw)*>(q + ea) = x[k].raw;
      if (TURN || has_b) *reinterpret_cast<decltype(x[k].raw)*>(q + eb) = y[k].raw;
    }
  }
}

template <typename T, int W, bool HALF>
__global__ void __launch_bounds__(kThreads, 16)
    rotary_kernel(const __grid_constant__ RotaryParams p) {
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  wait_for_previous();
  const uint32_t r = fast_div(i, p.by_units), u = i - r * (uint32_t)p.units;
  const uint32_t n = fast_div(r, p.by_split);           // the row of B * T
  const int g = (int)(r - n * (uint32_t)p.split);       // the first of its heads
  if (n >= (uint32_t)p.B * (uint32_t)p.T) return;
  const uint32_t b = fast_div(n, p.by_T), t = n - b * (uint32_t)p.T;
  int pos;
  const bool live = position(p, n, b, t, pos);
  if (!live && !p.clear) return;
  const int half = p.rot / 2;
  const bool pair = u < (uint32_t)p.pair_units;
  const int ea = pair ? (HALF ? (int)u * W : 2 * (int)u * W)
                      : p.rot + 2 * ((int)u - p.pair_units) * W;
  const int eb = pair && HALF ? half + (int)u * W : ea + W;
  const bool has_b = eb < p.d;
  // heads are counted over Q and K: this thread's first of K
  const int k0 = ((g - p.H) % p.split + p.split) % p.split;
  float c[W], s[W];
  if (!live) {
    Vec<T, W> zero;
    zero.raw = {};
    for (int x = 0; x < 2; ++x) {
      const RotaryRows& out = p.x[2 + x];
      T* dst = static_cast<T*>(out.p) + (int64_t)b * out.seq + (int64_t)t * out.row;
      for (int h = x ? k0 : g; h < (x ? p.H_k : p.H); h += p.split) {
        *reinterpret_cast<decltype(zero.raw)*>(dst + (int64_t)h * out.head + ea) = zero.raw;
        if (has_b)
          *reinterpret_cast<decltype(zero.raw)*>(dst + (int64_t)h * out.head + eb) = zero.raw;
      }
    }
  } else if (pair) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      // the phase modulo one turn, in 2^-64
      const uint64_t phase = (uint64_t)(int64_t)pos * p.turns[u * W + e];
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s[e], &c[e]);
      c[e] *= p.scale;
      s[e] *= p.scale_sin;
    }
    heads<T, W, HALF, true>(p.x[0], p.x[2], b, t, p.H, g, p.split, ea, eb, true, c, s);
    heads<T, W, HALF, true>(p.x[1], p.x[3], b, t, p.H_k, k0, p.split, ea, eb, true, c, s);
  } else {
    heads<T, W, HALF, false>(p.x[0], p.x[2], b, t, p.H, g, p.split, ea, eb, has_b, c, s);
    heads<T, W, HALF, false>(p.x[1], p.x[3], b, t, p.H_k, k0, p.split, ea, eb, has_b, c, s);
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
cudaError_t launch(const RotaryParams& p, int W, bool half, unsigned grid, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  auto go = [&](auto kernel) { return launch_first(kernel, grid, kThreads, 0, s, "rotary", p); };
  if (W == V) return half ? go(rotary_kernel<T, V, true>) : go(rotary_kernel<T, V, false>);
  return half ? go(rotary_kernel<T, 1, true>) : go(rotary_kernel<T, 1, false>);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams& p, bool f32, bool interleaved, int n_sms, cudaStream_t s) {
  const int size = f32 ? 4 : 2, V = 16 / size, half = p.rot / 2;
  // 16-byte vectors where every row and part of a row lies on their boundaries,
  // single elements otherwise
  bool wide = half % V == 0 && p.d % V == 0;
  for (int i = 0; i < 4; ++i) {
    const RotaryRows& x = p.x[i];
    if ((i & 1 ? p.H_k : p.H) == 0) continue;
    wide &= reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.seq % V == 0 && x.row % V == 0 &&
            x.head % V == 0;
  }
  const int W = wide ? V : 1;
  p.pair_units = half / W;
  p.units = p.pair_units + (p.copy_rest ? ((p.d - p.rot) / W + 1) / 2 : 0);
  // Threads of a token's unit: one, as long as that fills every SM four times (768 threads
  // each); up to one for each head where there are few tokens.
  const long long n = (long long)p.B * p.T, want = 4ll * 768 * n_sms;
  const long long fits = ((1ll << 31) - kThreads) / (n * p.units);
  long long split = (want + n * p.units - 1) / (n * p.units);
  if (split > p.H + p.H_k) split = p.H + p.H_k;
  p.split = (int)(split > fits ? fits : split);
  if (p.split < 1) return cudaErrorInvalidValue;
  p.by_T = make_div((uint32_t)p.T);
  p.by_units = make_div((uint32_t)p.units);
  p.by_split = make_div((uint32_t)p.split);
  const unsigned grid = (unsigned)((n * p.units * p.split + kThreads - 1) / kThreads);
  return f32 ? launch<float>(p, W, !interleaved, grid, s)
             : launch<__nv_bfloat16>(p, W, !interleaved, grid, s);
}

}  // namespace saf
