// beam.cu — one step of beam search.
//
// Slot b of a group offers, for every token v, the score
//     score(b) + x(b, v) - log sum_w exp x(b, w);
// a finished slot offers one: its score, with the ending token.  The best `beams`
// offers of a group become its slots; a slot's own offers go by their logits, equal scores of
// different slots to the lower one, equal logits to the lower token.
//
// The logits are read once, and that is what bounds the call.  A row is cut into
// blocks' parts; a block goes through its part in tiles, the next one's loads in
// flight while a tile is summed.  The K-th largest of the threads' maxima of the first
// tile is a threshold that at least K elements reach, and of later tiles few more; they
// are listed, and the best K of the list are the part's.  The last block of a row joins
// the row's parts, the last row of a group chooses (a counter each, which its last
// block sets back to zero for the next call).
// Measured: 64 groups of 8 beams over 128003 fp32 logits (a fifth of the slots finished), 55 us
// where the other slots' 210 MB take 32 at the copy rate: about 40 until they have come (5.3 TB/s),
// the last blocks' join and choice 8, their histories of 1000 tokens 4.  The same in bf16 52 us, of
// 105 MB (16 us): as many logits at half the bytes, so it is bound by its instructions (65 % of the
// issue slots, 53 in fp32).  12 x 4 beams over 50001 15 us, 1 x 4 over 32000 12 us: a chain of
// latencies (tile 2 us, join 4, choice 2, two fences and counters).
//
// Which of two offers is better should not hang on the rounding of a sum of 10^5
// exponentials.  An exponential is 2^(x log2 e - E) with the thread's exponent
// E = ceil(max x log2 e): the argument from x itself, by a multiplication that is
// rounded after E is subtracted, and the part of log2 e that fp32 does not hold; so it is
// exact to 2^-24 of what is left, and the function to 2^-22.  A thread's sum is rounded to
// 2^-40 of the block's scale and added to the others' in integers, so it does not
// depend on the order, and parts are joined by exact powers of two in fp64.  Scores are
// compared in fp64.  (Logits beyond 2^20 take a second pass against their maximum.)
// A polynomial in place of the function (2e-9) cost 18 more instructions for each pair
// of logits and twice the time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace saf {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStages = 3;              // tiles of a block's ring
constexpr int kHits = 184;             // vectors of a part that reach its threshold
constexpr float kMasked = -2.3e38f;    // below: as -inf
constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-08f;
constexpr float kPlain = 1048576.f;    // |logits| up to here are reduced without a base
constexpr int kUnit = 40;              // sums in integers count 2^-40: those of 2^22 ones fit

// What a block (then a row) leaves behind, followed by its K best as (value, token).
struct __align__(16) Part {
  unsigned long long sum;  // in 2^-40
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

// x 2^e in units of 2^-40, rounded down (x >= 0 and finite; fp64 has 1/64 of fp32's rate
// here, so this is done in integers).
__device__ __forceinline__ unsigned long long in_units(float x, int e) {
  const uint32_t u = __float_as_uint(x);
  const int sh = (int)(u >> 23) - 127 - 23 + kUnit + e;
  const unsigned long long m = (u & 0x7fffffu) | 0x800000u;
  return u < 0x800000u || sh < -23 ? 0 : sh >= 0 ? m << sh : m >> -sh;
}

// Whether a score is one (not -inf, masked or NaN).
__device__ __forceinline__ bool alive(float score) { return score >= kMasked && score < INFINITY; }

__device__ __forceinline__ Best best_of(unsigned long long key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return Best{__uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o), (int)~(uint32_t)key};
}

// Of two parts of a row one holds logits beyond 2^20: the sum of the one with the smaller
// element in units of the other's.
__device__ __noinline__ unsigned long long far_sum(float from, float to, int e,
                                                   unsigned long long x) {
  const double d = (double)from - (double)to + (double)e * 0.6931471805599453;
  return d > -40.0 ? (unsigned long long)((double)x * exp(d)) : 0;
}

// (top, base, e, sum) takes in another part of the row: of two sums the one with the smaller
// exponent is shifted; the part with the larger element keeps its base.
__device__ __forceinline__ void join_sum(float& top, float& base, int& e, unsigned long long& sum,
                                         float t, float b, int ex, unsigned long long x) {
  if (!(t > -INFINITY)) return;
  if (!(top > -INFINITY)) {
    top = t;
    base = b;
    e = ex;
    sum = x;
    return;
  }
  if (b != base) {
    if (t > top) {
      sum = x + far_sum(base, b, e - ex, sum);
      base = b;
      e = ex;
    } else {
      sum += far_sum(b, base, ex - e, x);
    }
  } else {
    const int up = max(e, ex);
    sum = (up - e < 64 ? sum >> (up - e) : 0) + (up - ex < 64 ? x >> (up - ex) : 0);
    e = up;
  }
  top = fmaxf(top, t);
}

// How many of keys[0 .. n) are above `key`.
__device__ __forceinline__ int count_above(const unsigned long long* keys, int n,
                                           unsigned long long key) {
  int above = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) above += keys[j] > key;
  return above;
}

// What the last blocks work on, in dynamic shared memory.
struct Joined {
  unsigned long long *keys, *best, *score;  // [R * S * K], [K * K], [K * K]
  double* lse;                              // [K]
  int *flat, *chosen, *token;               // [K * K], [K], [K]
};

// Whether a slot offers tokens of its own.
__device__ __forceinline__ bool offers(const BeamParams& p, int slot) {
  // (scores may be score_out, and finished its output: no read-only loads)
  const uint8_t done = p.finished ? p.finished[slot] : 0;
  return alive(p.scores[slot]) && !done;
}

// Joins the parts of R rows from slot0 on: log sums and, best first, K keys of each row
// (0: none); every thread of the block.
__device__ void join_rows(const BeamParams& p, int slot0, int R, const Joined& j) {
  const int S = p.splits, K = p.beams, tid = threadIdx.x, lane = tid & 31, n = S * K;
  auto part = [&](int r, int s) {
    return reinterpret_cast<const int4*>(p.parts + ((size_t)(slot0 + r) * S + s) * p.part_bytes);
  };
  for (int i = tid; i < R * K; i += kThreads) j.best[i] = 0;
  // a warp to a row: its largest element, and against the exponent of that part the
  // sum (j.score, j.flat and j.chosen hold sums, exponents and bases until the row's
  // logarithm is taken)
  for (int r = tid >> 5; r < R; r += kWarps) {
    float top = -INFINITY, base = 0.f;
    int e = 0;
    unsigned long long sum = 0;
    // (parts of a slot that offers nothing hold anything: they are read, not used)
    const bool some = offers(p, slot0 + r);
#pragma unroll 1
    for (int s = lane; s < S; s += 32) {
      const int4 a = __ldcg(part(r, s)), b = __ldcg(part(r, s) + 1);
      const unsigned long long x =
          (unsigned long long)(uint32_t)a.x | (unsigned long long)(uint32_t)a.y << 32;
      const float t = some ? __int_as_float(b.x) : -INFINITY, bs = __int_as_float(a.w);
      join_sum(top, base, e, sum, t, bs, a.z, x);
    }
    if (some) {
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, top, o);
        const float bs = __shfl_xor_sync(0xffffffffu, base, o);
        const int ex = __shfl_xor_sync(0xffffffffu, e, o);
        const unsigned long long x = __shfl_xor_sync(0xffffffffu, sum, o);
        join_sum(top, base, e, sum, t, bs, ex, x);
      }
    }
    if (lane == 0) {
      j.score[r] = top > -INFINITY ? sum : 0;
      j.flat[r] = e;
      j.chosen[r] = __float_as_int(base);
    }
  }
#pragma unroll 2
  for (int i = tid; i < R * n; i += kThreads) {
    const int r = i / n, k = i - r * n, s = k / K, at = k - s * K;
    const int2 x = __ldcg(reinterpret_cast<const int2*>(part(r, s) + 2) + at);
    const int count = __ldcg(&reinterpret_cast<const Part*>(part(r, s))->n);
    j.keys[i] = offers(p, slot0 + r) && at < count ? key_of(__int_as_float(x.x), x.y) : 0;
  }
  __syncthreads();
  if (tid >= kThreads - 32) {
    // all rows' logarithms by one warp (the one with the fewest entries below): fp64
    // instructions take as long for one lane as for 32
    for (int r = lane; r < R; r += 32) {
      const unsigned long long sum = j.score[r];
      const double e = (double)(j.flat[r] - kUnit) * 0.6931471805599453;
      j.lse[r] = sum == 0 ? 0.0 : (double)__int_as_float(j.chosen[r]) + (e + log((double)sum));
    }
  }
  for (int i = tid; i < R * n; i += kThreads) {
    const unsigned long long key = j.keys[i];
    if (key == 0) continue;
    const int r = i / n, above = count_above(j.keys + r * n, n, key);
    if (above < K) j.best[r * K + above] = key;
  }
  __syncthreads();
}

// Chooses a group's new slots from its rows' best; every thread of the block.
__device__ void choose(const BeamParams& p, int group, const Joined& j) {
  const int K = p.beams, tid = threadIdx.x, slot0 = group * K;
  const int filled = p.history_out ? max(0, min(*p.n_tokens, p.max_tokens)) : 0;
  for (int i = tid; i < K * K; i += kThreads) {
    const int b = i / K, slot = slot0 + b;
    unsigned long long key = 0;
    int f = 0;
    const float start = p.scores[slot];  // (scores may be score_out: no read-only load)
    const uint8_t done = p.finished ? p.finished[slot] : 0;
    if (alive(start)) {
      if (done) {
        if (i == b * K) {
          key = key_of((double)start);
          f = b * p.vocab + p.end;
        }
      } else if (j.best[i] != 0) {
        // (an offer whose score is none in fp32 would be a slot that never goes on)
        const Best best = best_of(j.best[i]);
        const double score = (double)start + ((double)best.x - j.lse[b]);
        key = alive((float)score) ? key_of(score) : 0;
        f = b * p.vocab + best.v;
      }
    }
    j.score[i] = key;
    j.flat[i] = f;
  }
  for (int i = tid; i < K; i += kThreads) j.chosen[i] = -1;
  __syncthreads();
  // Equal scores go to the lower slot, and of a slot, whose offers lie here best first, to the
  // larger logit, then the lower token: to the lower place.  (64 bits can round different logits
  // of a slot to one score, far from 0 or beside a large log sum.)
  for (int i = tid; i < K * K; i += kThreads) {
    const unsigned long long key = j.score[i];
    if (key == 0) continue;
    int above = 0;  // (without branches: 64 rounds took 5 us with them)
#pragma unroll 8
    for (int k = 0; k < K * K; ++k) {
      const unsigned long long other = j.score[k];
      above += (int)(other > key) | ((int)(other == key) & (int)(k < i));
    }
    if (above < K) {
      const int f = j.flat[i], b = f / p.vocab, v = f - b * p.vocab, s = slot0 + above;
      const unsigned long long u = key >> 63 ? key & 0x7fffffffffffffffull : ~key;
      j.chosen[above] = slot0 + b;
      j.token[above] = v;
      p.parent[s] = slot0 + b;
      p.token[s] = v;
      p.score_out[s] = (float)__longlong_as_double((long long)u);
      if (p.finished_out) p.finished_out[s] = v == p.end;
    }
  }
  __syncthreads();
  for (int i = tid; i < K; i += kThreads)
    if (j.chosen[i] < 0) {
      // fewer offers than slots: the slot is free
      p.parent[slot0 + i] = -1;
      p.token[slot0 + i] = -1;
      p.score_out[slot0 + i] = -INFINITY;
      if (p.finished_out) p.finished_out[slot0 + i] = 0;
    }
  if (p.history_out) {
    // a warp to a row, 16 columns of each lane in flight
    const int cols = min(filled + 1, p.max_tokens), lane = tid & 31;
    for (int b = tid >> 5; b < K; b += kWarps) {
      const int from = j.chosen[b], last = from >= 0 ? j.token[b] : -1;
      const int32_t* src = p.history + (size_t)max(from, 0) * p.max_tokens;
      int32_t* dst = p.history_out + (size_t)(slot0 + b) * p.max_tokens;
      for (int c0 = lane; c0 < cols; c0 += 512) {
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = c0 + 32 * i;
          v[i] = c >= filled ? last : from >= 0 ? src[c] : -1;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c0 + 32 * i < cols) dst[c0 + 32 * i] = v[i];
      }
    }
  }
}

// Whether this block is the last of `of` to come here (what the others wrote before is then
// visible to it); the counter is zero again afterwards.
__device__ __forceinline__ bool last_here(int* counter, int of, int* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    // the barrier and this fence order the whole block's writes before the count
    __threadfence();
    const bool last = atomicAdd(counter, 1) == of - 1;
    if (last) {
      *counter = 0;
      __threadfence();
    }
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

// The K-th largest of the threads' values m (kMasked if fewer count): at least K elements of
// which the m are maxima are not below it.
__device__ __noinline__ float kth_largest(float m, int K, float* tops, float* sh_top) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // each warp's, sorted downwards (bitonic)
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int step = size / 2; step > 0; step /= 2) {
      const float o = __shfl_xor_sync(0xffffffffu, m, step);
      const bool up = (lane & size) != 0, low = (lane & step) == 0;
      m = (up == low) ? fminf(m, o) : fmaxf(m, o);
    }
  if (lane < K) tops[warp * K + lane] = m;
  __syncthreads();
  float kth = -INFINITY;
  if (warp * 32 < kWarps * K) {
    const float mine = tid < kWarps * K ? tops[tid] : -INFINITY;
    int above = 0, not_below = 0;
#pragma unroll 4
    for (int j = 0; j < kWarps * K / 4; ++j) {
      const float4 t = reinterpret_cast<const float4*>(tops)[j];
      above += (t.x > mine) + (t.y > mine) + (t.z > mine) + (t.w > mine);
      not_below += (t.x >= mine) + (t.y >= mine) + (t.z >= mine) + (t.w >= mine);
    }
    if (mine > -INFINITY && above < K && not_below >= K) kth = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kth = fmaxf(kth, __shfl_xor_sync(0xffffffffu, kth, o));
  }
  if (lane == 0) sh_top[warp] = kth;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) kth = fmaxf(kth, sh_top[w]);
  return fmaxf(kth, kMasked);
}

// Grid: slots * splits blocks.  A thread takes NV vectors of 16 bytes of every tile.  Dynamic
// shared memory holds the ring of tiles, then what joining and choosing need.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 4) beam_kernel(const __grid_constant__ BeamParams p) {
  constexpr int PER = 16 / (int)sizeof(T);  // elements of a vector
  extern __shared__ __align__(16) uint8_t scratch[];
  __shared__ __align__(16) float tops[kThreads];  // the best K maxima of each warp
  // The warps' maxima have a place of their own: the second pass's threshold writes `tops`
  // while slower warps may still read them, no barrier lying between.
  __shared__ float warp_top[kWarps];
  __shared__ unsigned long long sums[kWarps];
  __shared__ uint4 hit[kHits];
  __shared__ int hit_at[kHits];
  __shared__ float sh_top[kWarps];
  __shared__ int n_hits, n_list, last_of;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / p.splits, split = blockIdx.x - slot * p.splits;
  const int K = p.beams;
  wait_for_previous();
  if (offers(p, slot)) {
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
    // Tiles come through a ring in shared memory in which each thread has places of its own:
    // it copies what it reads itself, so no barrier is needed, and no registers
    // hold what is in flight.
    uint4* ring = reinterpret_cast<uint4*>(scratch) + tid;
    constexpr int kTile = kThreads * NV;  // vectors
    auto whole = [&](int tile) { return first + (tile + 1) * kTile <= end; };
    auto issue = [&](int tile) {
      if (tile < p.tiles) {
        uint4* to = ring + tile % kStages * kTile;
        const uint4* from = vecs + (first + tile * kTile + tid);
        if (whole(tile)) {
#pragma unroll
          for (int k = 0; k < NV; ++k) copy_async_16(to + k * kThreads, from + k * kThreads);
        } else {
          for (int k = 0; k < NV; ++k)
            if (first + tile * kTile + k * kThreads + tid < end)
              copy_async_16(to + k * kThreads, from + k * kThreads);
        }
      }
      commit_copies();
    };
    for (int t = 0; t < kStages - 1; ++t) issue(t);
    uint4 x[NV];
    auto fetch = [&](int tile) {
      wait_copies<kStages - 2>();  // (one group a tile: this tile's is done)
      const uint4* from = ring + tile % kStages * kTile;
#pragma unroll
      for (int k = 0; k < NV; ++k) x[k] = from[k * kThreads];
      if (!whole(tile)) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (first + tile * kTile + k * kThreads + tid >= end)
            x[k] = make_uint4(none, none, none, none);
      }
    };
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
      if (!(extra >= kMasked && extra < INFINITY)) extra = -INFINITY;
    }
    if (tid == 0) n_hits = n_list = 0;
    fetch(0);
    // The maximum of the tile (NaN is passed over; it shows in the sum).
    float vec_top[NV];
    auto tile_top = [&]() {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        vec_top[k] = fmaxf(get(k, 0), get(k, 1));
#pragma unroll
        for (int e = 2; e < PER; e += 2) vec_top[k] = fmax3(vec_top[k], get(k, e), get(k, e + 1));
        m = fmaxf(m, vec_top[k]);
      }
      return m >= kMasked ? m : -INFINITY;
    };
    float m = fmaxf(tile_top(), extra);
    const float floor_k = kth_largest(m, K, tops, sh_top);

    // The sum of exponentials, 2^e times `sum`, and the elements that reach the threshold.
    // (Against the first exponent, 2^-(2^20 log2 e), logits below -2^20 add nothing: where a part
    // has no larger ones, the second pass below sums them.)
    float top = -INFINITY, sum = 0.f;
    int e_run = (int)(-kPlain * kLog2e);
    const uint64_t l2 = f2_pack(kLog2e, kLog2e), ll2 = f2_pack(kLog2eLo, kLog2eLo);
    for (int tile = 0; tile < p.tiles; ++tile) {
      if (tile > 0) {
        fetch(tile);
        m = tile_top();
      }
      issue(tile + kStages - 1);
      if (m > top) {
        top = m;
        const int e = (int)ceilf(fminf(fmaxf(m, -kPlain), kPlain) * kLog2e);
        if (e > e_run) {
          sum = e - e_run > 120 ? 0.f : sum * __uint_as_float((uint32_t)(127 - (e - e_run)) << 23);
          e_run = e;
        }
      }
      const uint64_t ne = f2_pack(-(float)e_run, -(float)e_run);
      uint64_t acc[2] = {0ull, 0ull};
      auto add = [&](float x0, float x1, int w) {
        const uint64_t y = f2_pack(x0, x1);
        float t0, t1;
        f2_unpack(f2_fma(y, ll2, f2_fma(y, l2, ne)), t0, t1);
        acc[w] = f2_add(acc[w], f2_pack(fast_exp2(t0), fast_exp2(t1)));
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
          if (vec_top[k] >= floor_k) {
            const int i = atomicAdd(&n_hits, 1);
            if (i < kHits) {
              hit[i] = x[k];
              hit_at[i] = at + k * kThreads * PER;
            }
          }
      }
    }
    wait_copies<0>();
    // the block's maximum, then the threads' sums against its exponent
    float block_top = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      block_top = fmaxf(block_top, __shfl_xor_sync(0xffffffffu, block_top, o));
    if (lane == 0) warp_top[warp] = block_top;
    // NaN or +inf among the logits (they count as masked), or some beyond 2^20: all of the
    // part is gone through again, element by element
    const bool slow = __syncthreads_or(!(sum < INFINITY) || !(top < INFINITY)) != 0;
    auto again = [&](auto&& f) {
      for (int v = first + tid; v < end; v += kThreads) {
        const T* q = reinterpret_cast<const T*>(vecs + v);
#pragma unroll 1
        for (int e = 0; e < PER; ++e) {
          const float y = (float)q[e];
          if (y >= kMasked && y < INFINITY) f(y, head + v * PER + e);
        }
      }
      if (extra > -INFINITY) f(extra, v_extra);
    };
    if (slow) {
      top = -INFINITY;
      again([&](float y, int) { top = fmaxf(top, y); });
      block_top = top;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        block_top = fmaxf(block_top, __shfl_xor_sync(0xffffffffu, block_top, o));
      if (lane == 0) warp_top[warp] = block_top;
      __syncthreads();
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) block_top = fmaxf(block_top, warp_top[w]);
    const bool far = !(fabsf(block_top) <= kPlain);  // (also: no element)
    const float base = far ? block_top : 0.f;
    const int e_top = far ? 0 : (int)ceilf(block_top * kLog2e);
    unsigned long long fixed = 0;
    if (!far && !slow) {
      if (top > -INFINITY) fixed = in_units(sum, max(e_run - e_top, -200));
    } else if (block_top > -INFINITY) {
      // sixteen terms in fp32, as in a tile, then in integers: one after another the roundings
      // of a thread's 136 would add up to 2^-19
      float s = 0.f;
      int n = 0;
      again([&](float y, int) {
        y -= base;
        s += fast_exp2(fmaf(y, kLog2eLo, fmaf(y, kLog2e, -(float)e_top)));
        if (++n == 16) {
          fixed += in_units(s, 0);
          s = 0.f;
          n = 0;
        }
      });
      fixed += in_units(s, 0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
    if (lane == 0) sums[warp] = fixed;
    Part* part = reinterpret_cast<Part*>(p.parts +
                                         ((size_t)slot * p.splits + split) * p.part_bytes);
    Best* best = reinterpret_cast<Best*>(part + 1);
    // the elements that reach the threshold, in the ring's place (no tile is needed any more)
    unsigned long long* list = reinterpret_cast<unsigned long long*>(scratch);
    constexpr int list_size = kStages * kTile * 16 / 8;
    static_assert(list_size >= kHits * PER + 16, "what the hits hold, and the ends, fits");
    int n = n_hits;
    bool listed = !slow && n <= kHits;
    if (!listed) {
      // too many reach the threshold of the first tile (or NaN spoiled it): that of
      // the whole part, and another pass for what reaches it
      const float floor_all = kth_largest(top, K, tops, sh_top);
      __syncthreads();
      again([&](float y, int at) {
        if (y >= floor_all) {
          const int i = atomicAdd(&n_list, 1);
          if (i < list_size) list[i] = key_of(y, at);
        }
      });
    } else {
      for (int i = tid; i < n * PER; i += kThreads) {
        const int v = i / PER, e = i % PER;
        const float y = (float)reinterpret_cast<const T*>(&hit[v])[e];
        if (y >= floor_k) list[atomicAdd(&n_list, 1)] = key_of(y, hit_at[v] + e);
      }
      if (extra >= floor_k) list[atomicAdd(&n_list, 1)] = key_of(extra, v_extra);
    }
    __syncthreads();
    n = n_list;
    listed = n <= list_size;
    if (!listed) {
      // so many equal ones: the K best one after another, each the best below the one before
      unsigned long long before = ~0ull;
      for (n = 0; n < K; ++n) {
        unsigned long long mine = 0;
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
        if (before == 0) break;  // fewer than K
        if (tid == 0) best[n] = best_of(before);
      }
    } else {
      for (int i = tid; i < n; i += kThreads) {
        const int above = count_above(list, n, list[i]);
        if (above < K) best[above] = best_of(list[i]);
      }
    }
    __syncthreads();
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
  // The last block joins and chooses: of the group where its rows' parts are few, else
  // of each row, and then of the group's rows.
  const int group = slot / K, slot0 = group * K, R = p.one_join ? K : 1;
  Joined j;
  j.keys = reinterpret_cast<unsigned long long*>(scratch);
  j.best = j.keys + R * p.splits * K;
  j.score = j.best + K * K;
  j.lse = reinterpret_cast<double*>(j.score + K * K);
  j.flat = reinterpret_cast<int*>(j.lse + K);
  j.chosen = j.flat + K * K;
  j.token = j.chosen + K;
  if (p.one_join) {
    if (!last_here(p.group_count + group, K * p.splits, &last_of)) return;
    join_rows(p, slot0, K, j);
  } else {
    if (!last_here(p.row_count + slot, p.splits, &last_of)) return;
    join_rows(p, slot, 1, j);
    for (int i = tid; i < K; i += kThreads) p.row_best[(size_t)slot * K + i] = j.best[i];
    if (tid == 0) p.row_lse[slot] = j.lse[0];
    if (!last_here(p.group_count + group, K, &last_of)) return;
    for (int i = tid; i < K * K; i += kThreads)
      j.best[i] = __ldcg(p.row_best + (size_t)slot0 * K + i);
    for (int i = tid; i < K; i += kThreads) j.lse[i] = __ldcg(p.row_lse + slot0 + i);
    __syncthreads();
  }
  choose(p, group, j);
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
  // (of each tile about as many vectors as beams reach the first one's threshold: half of
  // the places for them are left for chance)
  while (w.tiles < 8 && 2 * w.tiles * beams <= kHits / 2 &&
         blocks(w.held, 2 * w.tiles) >= 12ll * n_sms)
    w.tiles *= 2;
  // (whole vectors are counted from the row's first 16-byte boundary: never more than
  // vocab elements' worth)
  w.splits = (int)(blocks(w.held, w.tiles) / (long long)slots);
  // all parts of a group are joined at once where each thread has but a few of their
  // best (an entry counts those of its row)
  w.one_join = (long long)beams * beams * w.splits <= 4 * kThreads;
  if (w.splits < 1) w.splits = 1;
  w.part_bytes = sizeof(Part) + (sizeof(Best) * beams + 15) / 16 * 16;
  size_t off = 0;
  w.row_count = take(off, slots * 4);
  w.group_count = take(off, (size_t)n_groups * 4);
  w.row_lse = take(off, slots * 8);
  w.row_best = take(off, slots * beams * 8);
  w.parts = take(off, slots * w.splits * w.part_bytes);
  w.total = off;
  return w;
}

cudaError_t launch_beam(const BeamParams& p, bool f32, int held, cudaStream_t s) {
  const size_t K = p.beams;
  const size_t join = (p.one_join ? K : 1) * p.splits * K * 8 + K * K * 20 + K * 16;
  const size_t ring = (size_t)kStages * held * (f32 ? 4 : 2) * kThreads;  // join follows it
  const size_t smem = join > ring ? join : ring;
  const unsigned grid = (unsigned)(p.n_groups * p.beams) * (unsigned)p.splits;
  auto go = [&](auto kern) -> cudaError_t {
    if (smem > 40 * 1024) {
      const cudaError_t e =
          set_max_dynamic_smem(reinterpret_cast<const void*>(kern), 200 * 1024);
      if (e != cudaSuccess) return e;
    }
    return launch_first(kern, grid, kThreads, smem, s, "beam", p);
  };
  if (f32) return held == 16 ? go(beam_kernel<float, 4>) : go(beam_kernel<float, 2>);
  return held == 16 ? go(beam_kernel<__nv_bfloat16, 2>) : go(beam_kernel<__nv_bfloat16, 1>);
}

}  // namespace saf
