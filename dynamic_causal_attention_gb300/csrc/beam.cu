// beam.cu — one step of beam search.
//
// Slot b of a group offers, for every token v, the score
//     score(b) + x(b, v) - log sum_w exp x(b, w);
// a finished slot offers one: its score, with the ending token.  The best `beams`
// offers of a group become its slots; equal scores go to the lower b * vocab + v.
//
// The logits are read once, and that is what bounds the call.  A row is cut into
// blocks' parts; a block goes through its part in tiles, the next one's loads in
// flight while a tile is summed.  The K-th largest of the threads' maxima of the first
// tile is a threshold that at least K elements reach, and of later tiles few more; they
// are listed, and the best K of the list are the part's.  The last block of a row joins
// the row's parts, the last row of a group chooses (a counter each, which its last
// block sets back to zero for the next call).
//
// Which of two offers is better must not hang on the rounding of a sum of 10^5
// exponentials.  So an exponential is formed in base two against the thread's
// exponent E = ceil(max x log2 e): with n = round(x log2 e) and the rest f, both
// from x itself (no difference to the maximum is rounded), 2^(n - E) (1 + f q(f)),
// q of degree 5 fitted by the author to 2e-9; a thread's sum is rounded to 2^-44 of the
// block's scale and added to the others' in integers, so the sum does not depend on the
// order, and parts are joined by exact powers of two in fp64.  Scores are compared in
// fp64.  (Logits beyond 2^20 take a second pass against their maximum.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace saf {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kList = 512;             // candidates of a block before the K best are picked
constexpr float kMasked = -2.3e38f;    // below: as -inf
constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-08f;
constexpr float kPlain = 1048576.f;    // |logits| up to here are reduced without a base
constexpr double kUnit = 17592186044416.0;  // 2^44: a block's sum in integers

// What a block (then a row) leaves behind, followed by its K best as (value, token).
struct __align__(16) Part {
  unsigned long long sum;  // in 2^-44
  int e;                   // sum * 2^e * exp(base), or no element where top = -inf
  float base, top;
  int n;                   // best ones that follow
  int pad[2];
};
struct Best {
  float x;
  int v;
};

// Larger is better: x descending, then the index ascending.
__device__ __forceinline__ unsigned long long key_of(float x, int v) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as +0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((unsigned long long)o << 32) | (uint32_t)~v;
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double pow2(int e) {  // 2^e, -1022 <= e <= 1023
  return __longlong_as_double((long long)(e + 1023) << 52);
}

__device__ __forceinline__ bool dead(const BeamParams& p, int slot) {
  const float s = p.scores[slot];
  return !(s >= kMasked && s < INFINITY);
}

__device__ __forceinline__ Best best_of(unsigned long long key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return Best{__uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o), (int)~(uint32_t)key};
}

// How many of keys[0 .. n) are above `key`.
__device__ __forceinline__ int count_above(const unsigned long long* keys, int n,
                                           unsigned long long key) {
  int above = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) above += keys[j] > key;
  return above;
}

// Joins a row's parts and writes its log sum and its K best; every thread of the block.
__device__ void join_row(const BeamParams& p, int slot, unsigned long long* keys) {
  const int S = p.splits, K = p.beams, tid = threadIdx.x, lane = tid & 31, n = S * K;
  const uint8_t* parts = p.parts + (size_t)slot * S * p.part_bytes;
  auto part = [&](int s) { return reinterpret_cast<const Part*>(parts + (size_t)s * p.part_bytes); };
  for (int i = tid; i < n; i += kThreads) {
    const int s = i / K, j = i - s * K;
    const int2 x = __ldcg(reinterpret_cast<const int2*>(part(s) + 1) + j);
    keys[i] = j < __ldcg(&part(s)->n) ? key_of(__int_as_float(x.x), x.y) : 0;
  }
  if (tid >= kThreads - 32) {
    // the largest element, and the part that holds it: its base and exponent are the sum's
    float top = -INFINITY;
    int at = 0;
    for (int s = lane; s < S; s += 32) {
      const float t = __ldcg(&part(s)->top);
      if (t > top) {
        top = t;
        at = s;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, top, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (t > top || (t == top && a < at)) {
        top = t;
        at = a;
      }
    }
    const float base = __ldcg(&part(at)->base);
    const int e = __ldcg(&part(at)->e);
    double sum = 0.0;
    for (int s = lane; s < S; s += 32) {
      const Part* q = part(s);
      const float b = __ldcg(&q->base);
      const double x = (double)__ldcg(&q->sum) * (1.0 / kUnit);
      const int de = __ldcg(&q->e) - e;
      if (!(__ldcg(&q->top) > -INFINITY)) continue;
      if (b == base) {
        if (de > -1000) sum += x * pow2(de);
      } else {  // one of the two holds logits beyond 2^20
        const double d = ((double)b - (double)base) + (double)de * 0.6931471805599453;
        if (d > -700.0) sum += x * exp(d);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0)
      p.row_lse[slot] = top > -INFINITY
                            ? (double)base + ((double)e * 0.6931471805599453 + log(sum))
                            : 0.0;
  }
  __syncthreads();
  Best* row_best = reinterpret_cast<Best*>(p.row_best) + (size_t)slot * K;
  int mine = 0;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long key = keys[i];
    if (key == 0) continue;
    ++mine;
    const int above = count_above(keys, n, key);
    if (above < K) row_best[above] = best_of(key);
  }
  const int valid = __syncthreads_count(mine > 0) >= K ? K : -1;
  if (valid == K) {
    if (tid == 0) p.row_n[slot] = K;
  } else if (tid == 0) {
    int c = 0;
    for (int i = 0; i < n; ++i) c += keys[i] != 0;
    p.row_n[slot] = min(c, K);
  }
}

// Chooses a group's new slots; every thread of the block.
__device__ void choose(const BeamParams& p, int group, uint8_t* scratch) {
  const int K = p.beams, tid = threadIdx.x, slot0 = group * K;
  unsigned long long* score = reinterpret_cast<unsigned long long*>(scratch);  // [K * K] keys
  int* flat = reinterpret_cast<int*>(score + K * K);                           // [K * K]
  int* chosen = flat + K * K;                                                  // [K] parents
  int* token_of = chosen + K;                                                  // [K]
  for (int i = tid; i < K * K; i += kThreads) {
    const int b = i / K, j = i - b * K, slot = slot0 + b;
    unsigned long long key = 0;
    int f = 0;
    if (!dead(p, slot)) {
      if (p.finished && p.finished[slot]) {
        if (j == 0) {
          key = key_of((double)p.scores[slot]);
          f = b * p.vocab + p.end;
        }
      } else if (j < __ldcg(p.row_n + slot)) {
        const Best* best = reinterpret_cast<const Best*>(p.row_best) + (size_t)slot * K + j;
        const double x = (double)p.scores[slot] +
                         ((double)__ldcg(&best->x) - __ldcg(p.row_lse + slot));
        key = key_of(x);
        f = b * p.vocab + __ldcg(&best->v);
      }
    }
    score[i] = key;
    flat[i] = f;
  }
  for (int i = tid; i < K; i += kThreads) chosen[i] = -1;
  __syncthreads();
  for (int i = tid; i < K * K; i += kThreads) {
    const unsigned long long key = score[i];
    if (key == 0) continue;
    const int f = flat[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < K * K; ++j) {
      const unsigned long long other = score[j];
      above += other > key || (other == key && flat[j] < f);
    }
    if (above < K) {
      const int b = f / p.vocab, v = f - b * p.vocab, s = slot0 + above;
      const unsigned long long u = key >> 63 ? key & 0x7fffffffffffffffull : ~key;
      chosen[above] = slot0 + b;
      token_of[above] = v;
      p.parent[s] = slot0 + b;
      p.token[s] = v;
      p.score_out[s] = (float)__longlong_as_double((long long)u);
      if (p.finished_out) p.finished_out[s] = v == p.end;
    }
  }
  __syncthreads();
  for (int i = tid; i < K; i += kThreads)
    if (chosen[i] < 0) {
      // fewer offers than slots: the slot is free
      p.parent[slot0 + i] = -1;
      p.token[slot0 + i] = -1;
      p.score_out[slot0 + i] = -INFINITY;
      if (p.finished_out) p.finished_out[slot0 + i] = 0;
    }
  if (p.history_out) {
    const int n = max(0, min(*p.n_tokens, p.max_tokens)), cols = min(n + 1, p.max_tokens);
#pragma unroll 4
    for (int i = tid; i < K * cols; i += kThreads) {
      const int b = i / cols, c = i - b * cols, from = chosen[b];
      int v = -1;
      if (from >= 0)
        v = c < n ? __ldg(p.history + (size_t)from * p.max_tokens + c) : token_of[b];
      p.history_out[(size_t)(slot0 + b) * p.max_tokens + c] = v;
    }
  }
}

// Grid: slots * splits blocks.  A thread takes NV vectors of 16 bytes of every tile.  Dynamic
// shared memory holds what joining and choosing need.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 3) beam_kernel(const __grid_constant__ BeamParams p) {
  constexpr int PER = 16 / (int)sizeof(T);  // elements of a vector
  extern __shared__ __align__(16) uint8_t scratch[];
  __shared__ __align__(16) float tops[kThreads];  // the best K maxima of each warp
  __shared__ unsigned long long sums[kWarps];
  __shared__ unsigned long long list[kList];
  __shared__ float sh_top[kWarps];
  __shared__ int n_list, last_of;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / p.splits, split = blockIdx.x - slot * p.splits;
  const int K = p.beams;
  const bool skip = dead(p, slot) || (p.finished && p.finished[slot]);
  if (!skip) {
    const T* row = static_cast<const T*>(p.logits) + (size_t)slot * (size_t)p.row_stride;
    // elements ahead of the first 16-byte boundary, whole vectors, elements behind them
    const int head = min(
        (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(T)),
        p.vocab);
    const int nvec = (p.vocab - head) / PER, tail = p.vocab - head - nvec * PER;
    const uint4* vecs = reinterpret_cast<const uint4*>(row + head);
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    const int first = split * p.tiles * (kThreads * NV);
    const int end = min(nvec, first + p.tiles * (kThreads * NV));
    uint4 x[NV];
    auto load = [&](uint4 (&to)[NV], int tile) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + (tile * NV + k) * kThreads + tid;
        to[k] = v < end ? __ldcs(vecs + v) : make_uint4(none, none, none, none);
      }
    };
    load(x, 0);
    auto get = [&](int k, int e) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&x[k])[sizeof(T) == 4 ? e : e >> 1];
      if constexpr (sizeof(T) == 4) return __uint_as_float(w);
      else return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    };
    // the row's unaligned ends, an element a thread of its first part
    float extra = -INFINITY;
    int v_extra = 0;
    if (split == 0 && tid < head + tail) {
      v_extra = tid < head ? tid : p.vocab - tail + (tid - head);
      extra = (float)row[v_extra];
      if (!(extra < INFINITY)) extra = -INFINITY;
    }
    if (tid == 0) n_list = 0;
    // The maximum of the tile: NaN is passed over, +inf (which counts as masked) cleared.
    auto tile_top = [&]() {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < PER; e += 2) m = fmax3(m, get(k, e), get(k, e + 1));
      return m;
    };
    auto clean_top = [&]() {
      float m = tile_top();
      if (!(m < INFINITY)) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          uint32_t* w = reinterpret_cast<uint32_t*>(&x[k]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
              if (!(__uint_as_float(w[i]) < INFINITY)) w[i] = 0xff800000u;
            } else {
              if (!(__uint_as_float(w[i] << 16) < INFINITY)) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
              if (!(__uint_as_float(w[i] & 0xffff0000u) < INFINITY))
                w[i] = (w[i] & 0xffffu) | 0xff800000u;
            }
          }
        }
        m = tile_top();
      }
      return m >= kMasked ? m : -INFINITY;
    };
    float m = fmaxf(clean_top(), extra >= kMasked ? extra : -INFINITY);
    // the warp's maxima, sorted downwards (bitonic)
    float srt = m;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
      for (int step = size / 2; step > 0; step /= 2) {
        const float o = __shfl_xor_sync(0xffffffffu, srt, step);
        const bool up = (lane & size) != 0, low = (lane & step) == 0;
        srt = (up == low) ? fminf(srt, o) : fmaxf(srt, o);
      }
    if (lane < K) tops[warp * K + lane] = srt;
    __syncthreads();
    // the K-th largest of the threads' maxima: at least K elements are not below it
    float floor_k = -INFINITY;
    if (warp * 32 < kWarps * K) {
      const float mine = tid < kWarps * K ? tops[tid] : -INFINITY;
      int above = 0, not_below = 0;
#pragma unroll 4
      for (int j = 0; j < kWarps * K / 4; ++j) {
        const float4 t = reinterpret_cast<const float4*>(tops)[j];
        above += (t.x > mine) + (t.y > mine) + (t.z > mine) + (t.w > mine);
        not_below += (t.x >= mine) + (t.y >= mine) + (t.z >= mine) + (t.w >= mine);
      }
      if (mine > -INFINITY && above < K && not_below >= K) floor_k = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        floor_k = fmaxf(floor_k, __shfl_xor_sync(0xffffffffu, floor_k, o));
    }
    if (lane == 0) sh_top[warp] = floor_k;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) floor_k = fmaxf(floor_k, sh_top[w]);
    floor_k = fmaxf(floor_k, kMasked);  // fewer than K maxima: every element that counts

    // The sum of exponentials, 2^e times `sum`, and the elements that reach the threshold.
    // Logits below -2^20 are taken as -2^20: that counts only where the part has no
    // larger ones, and then the second pass below does.
    float top = -INFINITY, sum = 0.f;
    int e_run = (int)(-kPlain * kLog2e);
    const uint64_t l2 = f2_pack(kLog2e, kLog2e), ll2 = f2_pack(kLog2eLo, kLog2eLo);
    const uint64_t magic = f2_pack(12582912.f, 12582912.f);  // 1.5 * 2^23: rounds to integers
    const uint64_t nmagic = f2_pack(-12582912.f, -12582912.f);
    const uint64_t c6 = f2_pack(0.00015353362f, 0.00015353362f);
    const uint64_t c5 = f2_pack(0.0013398874f, 0.0013398874f);
    const uint64_t c4 = f2_pack(0.009618437f, 0.009618437f);
    const uint64_t c3 = f2_pack(0.055503324f, 0.055503324f);
    const uint64_t c2 = f2_pack(0.24022648f, 0.24022648f);
    const uint64_t c1 = f2_pack(0.6931472f, 0.6931472f);
    const uint64_t one = f2_pack(1.f, 1.f);
    auto offer = [&](float v, int at) {
      if (v >= floor_k) {
        const int i = atomicAdd(&n_list, 1);
        if (i < kList) list[i] = key_of(v, at);
      }
    };
    for (int tile = 0; tile < p.tiles; ++tile) {
      uint4 next[NV];
      if (tile + 1 < p.tiles) load(next, tile + 1);
      if (tile > 0) m = clean_top();
      if (m > top) {
        top = m;
        const int e = (int)ceilf(fminf(fmaxf(m, -kPlain), kPlain) * kLog2e);
        if (e > e_run) {
          sum = e - e_run > 120 ? 0.f : sum * __uint_as_float((uint32_t)(127 - (e - e_run)) << 23);
          e_run = e;
        }
      }
      const float low = fmaxf(top - 80.f, -kPlain);  // exp of less adds nothing that counts
      const int shift = 0x4b400000 + e_run;          // the magic number's bits, and E
      uint64_t acc[2] = {0ull, 0ull};
      auto add = [&](float x0, float x1, int w) {
        const uint64_t y = f2_pack(fmaxf(x0, low), fmaxf(x1, low));
        const uint64_t t = f2_fma(y, l2, magic);
        const uint64_t n = f2_add(t, nmagic) ^ 0x8000000080000000ull;  // -n
        uint64_t f = f2_fma(y, l2, n);
        f = f2_fma(y, ll2, f);
        uint64_t q = f2_fma(c6, f, c5);
        q = f2_fma(q, f, c4);
        q = f2_fma(q, f, c3);
        q = f2_fma(q, f, c2);
        q = f2_fma(q, f, c1);
        q = f2_fma(q, f, one);
        float t0, t1, q0, q1;
        f2_unpack(t, t0, t1);
        f2_unpack(q, q0, q1);
        // 2^(n - E) goes into the exponent: n - E lies in [-118, 1]
        q0 = __uint_as_float(__float_as_uint(q0) + ((__float_as_uint(t0) - shift) << 23));
        q1 = __uint_as_float(__float_as_uint(q1) + ((__float_as_uint(t1) - shift) << 23));
        acc[w] = f2_add(acc[w], f2_pack(q0, q1));
      };
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < PER; e += 2) add(get(k, e), get(k, e + 1), (e >> 1) & 1);
      if (tile == 0 && split == 0 && warp == 0) add(extra, -INFINITY, 0);
      float s0, s1;
      f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
      sum += s0 + s1;
      if (m >= floor_k) {
        const int at = head + (first + tile * NV * kThreads + tid) * PER;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < PER; ++e) offer(get(k, e), at + k * kThreads * PER + e);
        if (tile == 0) offer(extra, v_extra);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) x[k] = next[k];
    }
    // the block's maximum, then the threads' sums against its exponent
    float block_top = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      block_top = fmaxf(block_top, __shfl_xor_sync(0xffffffffu, block_top, o));
    __syncthreads();
    if (lane == 0) sh_top[warp] = block_top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) block_top = fmaxf(block_top, sh_top[w]);
    const bool far = !(fabsf(block_top) <= kPlain);  // (also: no element)
    const float base = far ? block_top : 0.f;
    const int e_top = far ? 0 : (int)ceilf(block_top * kLog2e);
    unsigned long long fixed = 0;
    // an element of this thread's part, read again
    auto again = [&](auto&& f) {
      for (int v = first + tid; v < end; v += kThreads) {
        const T* q = reinterpret_cast<const T*>(vecs + v);
        for (int e = 0; e < PER; ++e) {
          const float y = (float)q[e];
          if (y >= kMasked && y < INFINITY) f(y, head + v * PER + e);
        }
      }
      if (extra >= kMasked) f(extra, v_extra);
    };
    if (!far) {
      if (top > -INFINITY && e_run - e_top > -100)
        fixed = __double2ull_rn((double)sum * (kUnit * pow2(e_run - e_top)));
    } else if (block_top > -INFINITY) {
      float s = 0.f;
      again([&](float y, int) { s += expf(y - block_top); });
      fixed = __double2ull_rn((double)s * kUnit);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
    if (lane == 0) sums[warp] = fixed;
    __syncthreads();
    Part* part = reinterpret_cast<Part*>(p.parts +
                                         ((size_t)slot * p.splits + split) * p.part_bytes);
    Best* best = reinterpret_cast<Best*>(part + 1);
    const int n = n_list;
    if (n > kList) {
      // too many to list (equal ones, or rising ones): the K best one after another, each
      // the best below the one before
      unsigned long long before = ~0ull;
      for (int r = 0; r < K; ++r) {
        unsigned long long mine = 0;
        if (top >= floor_k)
          again([&](float y, int at) {
            const unsigned long long key = key_of(y, at);
            if (key < before && key > mine) mine = key;
          });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long other = __shfl_xor_sync(0xffffffffu, mine, o);
          mine = other > mine ? other : mine;
        }
        __syncthreads();
        if (lane == 0) list[warp] = mine;
        __syncthreads();
        before = list[0];
        for (int w = 1; w < kWarps; ++w) before = list[w] > before ? list[w] : before;
        if (tid == 0) best[r] = best_of(before);
      }
    } else {
      for (int i = tid; i < n; i += kThreads) {
        const int above = count_above(list, n, list[i]);
        if (above < K) best[above] = best_of(list[i]);
      }
    }
    if (tid == 0) {
      unsigned long long all = 0;
      for (int w = 0; w < kWarps; ++w) all += sums[w];
      part->sum = all;
      part->e = e_top;
      part->base = base;
      part->top = block_top;
      part->n = min(n, K);
    }
  }
  // the last block of the row joins its parts, the last row's of the group chooses
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const bool last = atomicAdd(p.row_count + slot, 1) == p.splits - 1;
    if (last) p.row_count[slot] = 0;
    last_of = last;
  }
  __syncthreads();
  if (!last_of) return;
  __threadfence();
  if (!skip) join_row(p, slot, reinterpret_cast<unsigned long long*>(scratch));
  __threadfence();
  __syncthreads();
  const int group = slot / K;
  if (tid == 0) {
    const bool last = atomicAdd(p.group_count + group, 1) == K - 1;
    if (last) p.group_count[group] = 0;
    last_of = last;
  }
  __syncthreads();
  if (!last_of) return;
  __threadfence();
  choose(p, group, scratch);
}

size_t take(size_t& off, size_t bytes) {
  const size_t o = off;
  off = (off + bytes + 255) & ~(size_t)255;
  return o;
}

}  // namespace

BeamWs beam_ws(int n_groups, int beams, int vocab, int n_sms) {
  BeamWs w;
  const size_t slots = (size_t)n_groups * beams;
  // A thread takes 16 elements of a tile, 8 where that leaves SMs without a block; a
  // block up to 8 tiles, as long as every SM gets its three blocks four times over.
  auto blocks = [&](int elements, int tiles) {
    return (long long)slots * ((vocab + elements * tiles * kThreads - 1) /
                               (elements * tiles * kThreads));
  };
  w.held = blocks(16, 1) < n_sms ? 8 : 16;
  w.tiles = 1;
  while (w.tiles < 8 && blocks(w.held, 2 * w.tiles) >= 12ll * n_sms) w.tiles *= 2;
  // (whole vectors are counted from the row's first 16-byte boundary: never more than
  // vocab elements' worth)
  w.splits = (int)(blocks(w.held, w.tiles) / (long long)slots);
  if (w.splits < 1) w.splits = 1;
  w.part_bytes = sizeof(Part) + (sizeof(Best) * beams + 15) / 16 * 16;
  size_t off = 0;
  w.row_count = take(off, slots * 4);
  w.group_count = take(off, (size_t)n_groups * 4);
  w.row_n = take(off, slots * 4);
  w.row_lse = take(off, slots * 8);
  w.row_best = take(off, slots * beams * sizeof(Best));
  w.parts = take(off, slots * w.splits * w.part_bytes);
  w.total = off;
  return w;
}

cudaError_t launch_beam(const BeamParams& p, bool f32, int held, cudaStream_t s) {
  const size_t join = (size_t)p.splits * p.beams * 8;
  const size_t pick = (size_t)p.beams * p.beams * 12 + 8 * (size_t)p.beams;
  const size_t smem = join > pick ? join : pick;
  const unsigned grid = (unsigned)(p.n_groups * p.beams) * (unsigned)p.splits;
  auto go = [&](auto kern) -> cudaError_t {
    if (smem > 40 * 1024) {
      const cudaError_t e =
          set_max_dynamic_smem(reinterpret_cast<const void*>(kern), 200 * 1024);
      if (e != cudaSuccess) return e;
    }
    trace_begin(s);
    kern<<<grid, kThreads, smem, s>>>(p);
    trace_end(s, "beam");
    return cudaGetLastError();
  };
  if (f32) return held == 16 ? go(beam_kernel<float, 4>) : go(beam_kernel<float, 2>);
  return held == 16 ? go(beam_kernel<__nv_bfloat16, 2>) : go(beam_kernel<__nv_bfloat16, 1>);
}

}  // namespace saf
