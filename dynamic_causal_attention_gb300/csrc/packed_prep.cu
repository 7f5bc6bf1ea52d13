// packed_prep.cu — what precedes and follows the packed attention's kernels.
//
// packed_prep_kernel, one launch ahead of the forward and of the backward:
//   block 0      the plan: a record (first row of the sequence, its rows, tile X, the
//                sequence's first tile) for every tile of 128 rows, sorted by falling X
//                (steps of the forward) and by falling number of query tiles (steps of
//                the backward).  A sequence of n tiles has one tile with every key
//                1..n in either order, so with the sequences sorted by falling n those that have
//                key k are the first cnt[k], and a record's place is start[k] + place
//                of its sequence: one counting sort of the sequences gives both.
//                Neighbours in the first order share X and a frozen head's weights.
//   then         the frozen heads' generator tables, 128 entries a block
//   the last     rows of no sequence, cleared where asked
// 7 us for 16 sequences with its launch: of that a chain of scans by one block 3, beside tables of
// 4096 entries (2).  The tables are made for max_len, whatever the batch's longest sequence: each
// block looks for the range over all of it, and a head whose range needs the exact exponentials
// forms log Z of every row.  Forward of six prompts of up to 100 tokens, 12 heads (3 frozen): 12 us with
// max_len 4096, 34 with 32768, 270 with 131072; with such heads 126 us, 3.1 and 33 ms.
// packed_pre / packed_post: the backward's row passes (D = rowsum(dO o O), -lse log2 e,
// zeros of dQ's accumulator; dQ from it), by tiles and heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "packed.h"
#include "ptx.cuh"

namespace saf {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMasked = -2.3e38f;              // below: as -inf
constexpr float kMaxFactoredRange = 80.0f;       // as for batches of one length
constexpr int kPrepThreads = 512, kPrepWarps = kPrepThreads / 32;
constexpr int kClearBlocks = 64;

struct PlanShared {
  int hist[kMaxPackedTiles + 2];    // sequences of n tiles, then the next place of such a one
  int cnt[kMaxPackedTiles + 2];     // sequences of at least k tiles
  int start[kMaxPackedTiles + 2];   // records of keys above k
  int gstart[kMaxPackedTiles + 2];  // groups of keys above k
  int warp_max[kPrepWarps], warp_sum[kPrepWarps];
  int end, tiles, group;
  unsigned long long longest;       // (rows, first tile) of the longest sequence
};

// Suffix sums of value(0 .. n - 1), two at a time: put(i, sums of j >= i, value(i)), by one
// warp.  The sums of all come back.
template <class F, class G>
__device__ int2 warp_suffix(int n, F value, G put) {
  const int lane = threadIdx.x & 31;
  int2 carry = make_int2(0, 0);
  for (int base = (n - 1) / 32 * 32; base >= 0; base -= 32) {
    const int i = base + lane;
    const int2 v = i < n ? value(i) : make_int2(0, 0);
    int2 s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int tx = __shfl_down_sync(0xffffffffu, s.x, o);
      const int ty = __shfl_down_sync(0xffffffffu, s.y, o);
      if (lane + o < 32) {
        s.x += tx;
        s.y += ty;
      }
    }
    if (i < n) put(i, make_int2(carry.x + s.x, carry.y + s.y), v);
    carry.x += __shfl_sync(0xffffffffu, s.x, 0);
    carry.y += __shfl_sync(0xffffffffu, s.y, 0);
  }
  return carry;
}

__device__ void make_plan(const PackedPrep& p, PlanShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n_seqs, m = p.max_tiles;
  if (tid == 0) {
    *p.status = 0;
    p.hdr[2] = p.hdr[3] = 0;
    sh.end = max(0, min(p.cu[0], p.total));
    sh.tiles = 0;
    sh.longest = 0;
  }
  for (int i = tid; i < m + 2; i += kPrepThreads) sh.hist[i] = 0;
  __syncthreads();
  // Ends of the sequences (never falling, whatever cu holds, so that no row is in two
  // of them), their tiles, and the sum of the tiles before.
  for (int b0 = 0; b0 < n; b0 += kPrepThreads) {
    const int b = b0 + tid;
    const int carry_end = sh.end, carry_tiles = sh.tiles;
    int e = b < n ? max(0, min(p.cu[b + 1], p.total)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int t = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) e = max(e, t);
    }
    if (lane == 31) sh.warp_max[warp] = e;
    __syncthreads();
    int before = carry_end;
    for (int w = 0; w < warp; ++w) before = max(before, sh.warp_max[w]);
    e = max(e, before);
    const int prev = __shfl_up_sync(0xffffffffu, e, 1);
    const int a = lane > 0 ? prev : before;
    const int len = b < n ? min(e - a, p.max_len) : 0;
    const int nt = (len + 127) / 128;
    int s = nt;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) sh.warp_sum[warp] = s;
    __syncthreads();
    int tile0 = carry_tiles + s - nt;
    for (int w = 0; w < warp; ++w) tile0 += sh.warp_sum[w];
    if (b < n) {
      p.seqs[b] = make_int4(a, len, tile0, 0);
      atomicAdd(&sh.hist[nt], 1);
      if (p.backward) atomicMax(&sh.longest, (unsigned long long)len << 32 | (unsigned)tile0);
    }
    __syncthreads();
    if (tid == kPrepThreads - 1) {
      sh.end = e;
      sh.tiles = tile0 + nt;
    }
    __syncthreads();
  }
  if (warp == 0) {
    warp_suffix(m + 2, [&](int i) { return make_int2(sh.hist[i], 0); },
                [&](int i, int2 s, int2) { sh.cnt[i] = s.x; });
    __syncwarp();
    const int tiles = sh.tiles;
    // Tiles share generated weights where there are more items than SMs; with fewer, an
    // item that carries several tiles only takes longer (dV of a K/V head of 32 and 40
    // documents of up to 300 tokens: 16.4 us shared, 11 not; of 3 of 64 and 16 documents of
    // up to 4096: 49.7 and 62.9).
    const int g = tiles * p.per_tile > p.num_sms ? p.group : 1;
    // places of the records and of the groups of a key: as many as larger keys have
    const int2 all = warp_suffix(
        m + 2,
        [&](int i) { return i ? make_int2(sh.cnt[i], (sh.cnt[i] + g - 1) / g) : make_int2(0, 0); },
        [&](int i, int2 s, int2 v) {
          sh.start[i] = s.x - v.x;
          sh.gstart[i] = s.y - v.y;
        });
    if (lane == 0) {
      sh.group = g;
      p.hdr[0] = tiles;
      p.hdr[1] = all.y;
      p.hdr[4] = (int)(unsigned)sh.longest;
    }
  }
  __syncthreads();
  for (int i = tid; i <= m; i += kPrepThreads) sh.hist[i] = sh.cnt[i + 1];
  __syncthreads();
  const int g = sh.group;
  for (int b = warp; b < n; b += kPrepWarps) {
    const int4 q = p.seqs[b];
    const int nt = (q.y + 127) / 128;
    int place = 0;
    if (lane == 0 && nt > 0) place = atomicAdd(&sh.hist[nt], 1);
    place = __shfl_sync(0xffffffffu, place, 0);
    for (int X = lane; X < nt; X += 32) {
      const int4 rec = make_int4(q.x, q.y, X, q.z);
      const int kf = X + 1, kb = nt - X;
      p.by_key[sh.start[kf] + place] = rec;
      p.by_query[sh.start[kb] + place] = rec;
      // (groups come by falling steps: of the transposed form by the query tiles of their
      // first sequence, which has the most)
      if (place % g == 0)
        p.groups[sh.gstart[p.backward ? kb : kf] + place / g] =
            make_int2(sh.start[kf] + place, min(g, sh.cnt[kf] - place));
    }
  }
}

// Entry t of alpha or rho: -inf behind the longest sequence and for masks.
__device__ __forceinline__ float entry(const float* v, int t, int n) {
  const float x = t < n ? v[t] : -INFINITY;
  return x < kMasked ? -INFINITY : x;
}

// Entries row0 .. row0 + 127 of a frozen head's tables (the formulas of static_prep_kernel).
__device__ void make_tables(const PackedPrep& p, int hs, int row0, float* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = p.T, h = p.static_heads[hs], n = p.max_len;
  const float* alpha = p.alpha + (size_t)h * p.T_pat;
  const float* rho = p.rho + (size_t)h * p.T_pat;
  // finite ranges of the whole head (every block agrees)
  float amax = -INFINITY, amin = INFINITY, rmax = -INFINITY, rmin = INFINITY;
#pragma unroll 4
  for (int t = tid; t < n; t += kPrepThreads) {
    const float a = entry(alpha, t, n), r = entry(rho, t, n);
    if (isfinite(a)) { amax = fmaxf(amax, a); amin = fminf(amin, a); }
    if (isfinite(r)) { rmax = fmaxf(rmax, r); rmin = fminf(rmin, r); }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    amin = fminf(amin, __shfl_xor_sync(0xffffffffu, amin, o));
    rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, o));
    rmin = fminf(rmin, __shfl_xor_sync(0xffffffffu, rmin, o));
  }
  if (lane == 0) {
    red[warp] = amax;
    red[kPrepWarps + warp] = amin;
    red[2 * kPrepWarps + warp] = rmax;
    red[3 * kPrepWarps + warp] = rmin;
  }
  __syncthreads();
  for (int w = 0; w < kPrepWarps; ++w) {
    amax = fmaxf(amax, red[w]);
    amin = fminf(amin, red[kPrepWarps + w]);
    rmax = fmaxf(rmax, red[2 * kPrepWarps + w]);
    rmin = fminf(rmin, red[3 * kPrepWarps + w]);
  }
  const bool none = !(amax > -INFINITY) || !(rmax > -INFINITY);
  const bool exact = !none && (amax - amin) + (rmax - rmin) > kMaxFactoredRange;
  float* a_tab = p.a_tab + (size_t)hs * T;
  float* r_tab = p.r_tab + (size_t)hs * (T + 128);
  if (row0 == 0 && tid == 0) {
    p.mode[hs] = exact ? 1 : 0;
    p.shift[hs] = exact || none ? 0.f : amax + rmax;
  }
  if (row0 == 0 && tid < 128) r_tab[tid < 127 ? tid : T + 127] = exact ? -INFINITY : 0.f;
  if (tid < 128) {
    const int t = row0 + tid;
    const float a = entry(alpha, t, n), r = entry(rho, t, n);
    a_tab[t] = exact ? a * kLog2e : none ? 0.f : expf(a - amax);
    r_tab[127 + t] = exact ? r * kLog2e : none ? 0.f : expf(r - rmax);
  }
  if (!exact) return;
  // log Z of each row: an online log-sum-exp per lane, merged in a fixed order
  for (int k0 = 0; k0 < 128 / kPrepWarps; ++k0) {
    const int i = row0 + warp * (128 / kPrepWarps) + k0;
    float mx = -INFINITY, sm = 0.f;
    for (int k = lane; k <= i && k < n; k += 32) {
      const float t = entry(alpha, k, n) + entry(rho, i - k, n);
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
      const float lz = mx > -INFINITY ? mx + logf(sm) : -INFINITY;
      p.logZ[(size_t)hs * T + i] = lz;
      p.row_tab[(size_t)hs * T + i] = mx > -INFINITY ? -lz * kLog2e : -INFINITY;
    }
  }
}

// Rows row0 .. row0 + n - 1, by threads t0, t0 + step, ...
__device__ void clear_range(const PackedPrep& p, long long row0, long long n, long long t0,
                            long long step) {
  for (int i = 0; i < p.n_rows; ++i) {
    const ClearRows& x = p.rows[i];
    const int units = p.d / 8;
    for (long long j = t0; j < n * x.heads * units; j += step) {
      const int u = (int)(j % units);
      const long long hr = j / units;
      const int h = (int)(hr % x.heads);
      *reinterpret_cast<uint4*>(x.p + (row0 + hr / x.heads) * x.row + (int64_t)h * x.head + 8 * u) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (p.lse)
    for (long long j = t0; j < n * p.H; j += step)
      p.lse[j / n * p.total + row0 + j % n] = -INFINITY;
}

// What is not worked on: rows before the first and behind the last sequence, and rows of a
// sequence from max_len on.
__device__ void clear_rows(const PackedPrep& p, int block) {
  const int first = max(0, min(p.cu[0], p.total));
  const int last = max(first, min(p.cu[p.n_seqs], p.total));
  const long long t0 = (long long)block * kPrepThreads + threadIdx.x;
  const long long step = (long long)kClearBlocks * kPrepThreads;
  clear_range(p, 0, first, t0, step);
  clear_range(p, last, p.total - last, t0, step);
  for (int b = block; b < p.n_seqs; b += kClearBlocks) {
    const int a = max(0, min(p.cu[b], p.total)), e = max(0, min(p.cu[b + 1], p.total));
    if (e - a > p.max_len)
      clear_range(p, a + p.max_len, e - a - p.max_len, threadIdx.x, kPrepThreads);
  }
}

// Grid: 1 + tables * n_static + (clear ? kClearBlocks : 0).
__global__ void __launch_bounds__(kPrepThreads)
    packed_prep_kernel(const __grid_constant__ PackedPrep p) {
  __shared__ PlanShared plan;
  const int chunks = p.max_tiles;
  const int b = (int)blockIdx.x - 1;
  wait_for_previous();
  if (b < 0) make_plan(p, plan);
  else if (b < chunks * p.n_static)
    make_tables(p, b / chunks, (b % chunks) * 128, reinterpret_cast<float*>(plan.hist));
  else clear_rows(p, b - chunks * p.n_static);
}

// Place of a key among the block's keys (all different, those behind n the largest).
__device__ __forceinline__ int place_of(uint32_t key, const uint32_t* keys, int n) {
  int below = 0;
#pragma unroll 19  // (half of 152 CTAs' keys in flight: 16 rounds 4 us shorter than by fours)
  for (int i = 0; i < n; i += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
    below += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
  }
  return below;
}

// The dynamic pass's items shared out over its CTAs, by one block beside the row pass: round by
// round the costliest item of a round goes to the CTA with the least to do so far.  A
// step costs 2, an item's beginning and end 1.  (By the snake order 16 % of the SMs' time was
// idle with 16 documents of up to 4096 tokens and 9 heads of 64, 17 % with 3 of up to 8192 and
// 8 K/V heads: 397 and 793 us against 368 and 695.  Items handed out as CTAs come free,
// through a ring in shared memory to the five roles, cost each step 9 %.)  A round takes 1.5 us
// beside the row pass; where there are many, the snake order shares out as well (400 documents
// of up to 300 tokens and 16 heads of 64: the row pass would take 135 us in place of 89).
constexpr int kRankedRounds = 48;
__device__ void share_out(const PackedRows& p) {
  constexpr int AHEAD = 4;  // rounds whose records are on their way
  __shared__ __align__(16) int4 ring[AHEAD][256];
  __shared__ __align__(16) uint32_t by_load[256], by_cost[256];
  __shared__ int load_of[256], cta_at[256];
  const int tid = threadIdx.x, n_ctas = p.n_ctas, nt = p.hdr[0], n = nt * p.items.n_kv;
  const int rounds = (n + n_ctas - 1) / n_ctas;
  if (rounds > order_rounds(p.d_h)) return;
  if (rounds > kRankedRounds) {
#pragma unroll 4
    for (int r = 0; r <= rounds; ++r) {
      const int it = snake_item(r, tid, n_ctas);
      if (tid < n_ctas)
        p.order[r * n_ctas + tid] =
            it < n ? packed_bwd_item(p.items, nt, it) : make_int4(0, 0, 0, 0);
    }
    return;
  }
  // A thread's record of round r, by a copy of its own into its place of the ring (beside the row
  // pass a load takes 1.5 us: one round ahead, 16 rounds took 33 us, longer than all rows)
  auto issue = [&](int r) {
    const int it = r * n_ctas + tid;
    if (tid < n_ctas && it < n)
      copy_async_16(&ring[r % AHEAD][tid], p.items.tiles + packed_bwd_place(p.items, nt, it).x);
    commit_copies();
  };
  // costs in units that keep a CTA's sum below 2^24
  int shift = 0;
  while (((long long)rounds * (1 + 2 * p.items.most_steps)) >> shift >= 1 << 24) ++shift;
  load_of[tid] = 0;
  by_load[tid] = by_cost[tid] = 0xffffffffu;  // (what is behind the last CTA stays so)
  for (int r = 0; r < AHEAD - 1; ++r) issue(r);
  for (int r = 0; r < rounds; ++r) {
    wait_copies<AHEAD - 2>();
    int4 rec = make_int4(0, 0, 0, 0);
    const int it = r * n_ctas + tid;
    if (tid < n_ctas && it < n) {
      rec = ring[r % AHEAD][tid];
      rec.z |= packed_bwd_place(p.items, nt, it).y << 16;
    }
    issue(r + AHEAD - 1);
    const int cost = rec.y > 0 ? (1 + 2 * (int)p.items.dyn_count[rec.z >> 16] *
                                          ((rec.y + 127) / 128 - (rec.z & 0xffff))) >> shift
                               : 0;
    const uint32_t lk = (uint32_t)load_of[tid] << 8 | tid, ck = (0xffffffu - cost) << 8 | tid;
    if (tid < n_ctas) {
      by_load[tid] = lk;
      by_cost[tid] = ck;
    }
    __syncthreads();
    // (records come by falling steps: they need no ranking where every K/V head
    // serves as many query heads)
    int place = tid;
    if (tid < n_ctas) {
      cta_at[place_of(lk, by_load, n_ctas)] = tid;
      if (!p.items.even) place = place_of(ck, by_cost, n_ctas);
    }
    __syncthreads();
    if (tid < n_ctas) {
      const int cta = cta_at[place];
      p.order[r * n_ctas + cta] = rec;
      load_of[cta] += cost;
    }
    __syncthreads();
  }
  wait_copies<0>();
  if (tid < n_ctas) p.order[rounds * n_ctas + tid] = make_int4(0, 0, 0, 0);
}

// Sum of eight products.
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&b);
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __bfloat1622float2(a2[k]), y = __bfloat1622float2(b2[k]);
    s = fmaf(x.x, y.x, s);
    s = fmaf(x.y, y.y, s);
  }
  return s;
}

// D of the first rows of a sequence is formed from P and dP themselves.  With few keys dP - D
// nearly cancels (of a first row it is zero), and D from the rounded out is off by 2^-9 of
// what cancels: gradients of sequences of two tokens were 2.2 times as far from those in 64 bits as
// ones rounded once, 1.35 with this (of 12 tokens 1.75 and 1.45).
constexpr int kExactRows = 8;

// Rows 0 .. kExactRows - 1 of a sequence of `len` from row `first` on, by the block: D/8 lanes a
// pair of a row and a key, whose loads do not wait for one another's.
template <int LPR>
__device__ __forceinline__ void exact_rows(const PackedRows& p, int first, int len, int h,
                                           float* out) {
  constexpr int kAhead = LPR == 16 ? 1 : 2;  // (two of d_h = 128 spill)
  __shared__ float part[kExactRows * kExactRows];
  const int sub = threadIdx.x % LPR;
  const int64_t kv = h / p.group_kv;
#pragma unroll kAhead
  for (int i = threadIdx.x / LPR; i < kExactRows * kExactRows; i += 256 / LPR) {
    const int r = i / kExactRows, j = i % kExactRows;
    const bool sees = r < len && j <= r;
    const int64_t row = first + (sees ? r : 0), key = first + (sees ? j : 0);
    auto at = [&](const __nv_bfloat16* x, int64_t n, int64_t by_row, int64_t head,
                  int64_t by_head) {
      return *reinterpret_cast<const uint4*>(x + n * by_row + head * by_head + sub * 8);
    };
    float s = dot8(at(p.q, row, p.q_row, h, p.q_head), at(p.k, key, p.k_row, kv, p.k_head));
    float dp = dot8(at(p.dout, row, p.do_row, h, p.do_head), at(p.v, key, p.v_row, kv, p.v_head));
    const float l2 = p.lse[(int64_t)h * p.total + row] * kLog2e;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      dp += __shfl_xor_sync(0xffffffffu, dp, o);
    }
    if (sub == 0) part[i] = sees ? exp2f(s * p.scale * kLog2e - l2) * dp : 0.f;
  }
  __syncthreads();  // (and the block's D of these rows is written)
  if (threadIdx.x < kExactRows && (int)threadIdx.x < len) {
    float d = 0.f;
    for (int j = 0; j < kExactRows; ++j) d += part[threadIdx.x * kExactRows + j];
    out[threadIdx.x] = -d;
  }
}

// A tile's rows under one head: D/8 lanes a row, 8 elements each.
template <int D>
__global__ void __launch_bounds__(256, 6) packed_pre_kernel(const __grid_constant__ PackedRows p) {
  constexpr int LPR = D / 8;
  wait_for_previous();
  if ((int)blockIdx.y == 0 && p.order) {
    if (blockIdx.x == 0) share_out(p);
    return;
  }
  if ((int)blockIdx.x >= p.hdr[0]) return;
  // (first tiles of sequences, which have more to do, come first)
  const int4 t = p.tiles[p.hdr[0] - 1 - (int)blockIdx.x];
  const int h = (int)blockIdx.y - (p.order ? 1 : 0), hs = p.static_slot[h], kv = h / p.group_kv;
  const int tile = t.w + t.z, valid = min(128, t.y - t.z * 128), longest = p.hdr[4];
  const bool zero_k = h == kv * p.group_kv && !p.kv_has_dyn[kv];
  const int sub = threadIdx.x % LPR;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
  for (int r = threadIdx.x / LPR; r < 128; r += 256 / LPR) {
    const int64_t row = t.x + t.z * 128 + r;
    const bool mine = r < valid;
    if (zero_k && mine)
      *reinterpret_cast<uint4*>(p.dK + row * p.dk_row + (int64_t)kv * p.dk_head + sub * 8) = zero;
    if (hs >= 0) {
      if (mine)
        *reinterpret_cast<uint4*>(p.dQ + row * p.dq_row + (int64_t)h * p.dq_head + sub * 8) = zero;
      if (sub == 0 && t.w == longest) {
        // the weight of a query's row: 1 / Z', or -log2 Z (exact); none behind the end.  A
        // frozen head's depends on the position alone, so the longest sequence's serve all.
        const float l = mine ? p.lse[(int64_t)h * p.total + row] : -INFINITY;
        const bool some = l > -INFINITY;
        const float v = p.mode[hs] ? (some ? -l * kLog2e : -INFINITY)
                                   : (some ? expf(p.shift[hs] - l) : 0.f);
        p.row_vals[(size_t)hs * p.T + t.z * 128 + r] = v;
      }
      continue;
    }
    float acc = 0.f;
    if (mine) {
      const uint4 a = *reinterpret_cast<const uint4*>(p.out + row * p.out_row +
                                                      (int64_t)h * p.out_head + sub * 8);
      const uint4 b = *reinterpret_cast<const uint4*>(p.dout + row * p.do_row +
                                                      (int64_t)h * p.do_head + sub * 8);
      acc = dot8(a, b);
      float4* z = reinterpret_cast<float4*>(p.dq_acc + ((int64_t)h * p.total + row) * D + sub * 8);
      z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (sub == 0) {
      const size_t at = ((size_t)h * p.nt_max + tile) * 128 + r;
      p.Dvec[at] = mine ? -acc : 0.f;
      p.lse2[at] = mine ? -p.lse[(int64_t)h * p.total + row] * kLog2e : -INFINITY;
    }
  }
  if (t.z == 0 && hs < 0)
    exact_rows<LPR>(p, t.x, t.y, h, p.Dvec + ((size_t)h * p.nt_max + tile) * 128);
}

template <int D>
__global__ void __launch_bounds__(256) packed_post_kernel(const __grid_constant__ PackedRows p) {
  constexpr int LPR = D / 8;
  const int h = blockIdx.y;
  wait_for_previous();
  if ((int)blockIdx.x >= p.hdr[0] || p.static_slot[h] >= 0) return;
  const int4 t = p.tiles[blockIdx.x];
  const int valid = min(128, t.y - t.z * 128), sub = threadIdx.x % LPR;
  for (int r = threadIdx.x / LPR; r < valid; r += 256 / LPR) {
    const int64_t row = t.x + t.z * 128 + r;
    const float* src = p.dq_acc + ((int64_t)h * p.total + row) * D + sub * 8;
    const float4 a = *reinterpret_cast<const float4*>(src);
    const float4 b = *reinterpret_cast<const float4*>(src + 4);
    uint4 q;
    q.x = pack_bf16x2(a.x * p.scale, a.y * p.scale);
    q.y = pack_bf16x2(a.z * p.scale, a.w * p.scale);
    q.z = pack_bf16x2(b.x * p.scale, b.y * p.scale);
    q.w = pack_bf16x2(b.z * p.scale, b.w * p.scale);
    *reinterpret_cast<uint4*>(p.dQ + row * p.dq_row + (int64_t)h * p.dq_head + sub * 8) = q;
  }
}

}  // namespace

cudaError_t launch_packed_prep(const PackedPrep& p, cudaStream_t s) {
  const int grid = 1 + p.max_tiles * p.n_static + (p.clear ? kClearBlocks : 0);
  return launch_first(packed_prep_kernel, grid, kPrepThreads, 0, s, "packed_prep", p);
}

cudaError_t launch_packed_pre(const PackedRows& p, cudaStream_t s) {
  const dim3 grid(p.nt_max, p.H + (p.order ? 1 : 0));
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, 256, 0, s, "packed_pre", p); };
  switch (p.d_h) {
    case 32: return go(packed_pre_kernel<32>);
    case 64: return go(packed_pre_kernel<64>);
    case 128: return go(packed_pre_kernel<128>);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_packed_post(const PackedRows& p, cudaStream_t s) {
  const dim3 grid(p.nt_max, p.H);
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, 256, 0, s, "packed_post", p); };
  switch (p.d_h) {
    case 32: return go(packed_post_kernel<32>);
    case 64: return go(packed_post_kernel<64>);
    case 128: return go(packed_post_kernel<128>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saf
