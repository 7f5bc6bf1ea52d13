// cache_pages.cu — page tables and reference counts of the paged cache:
// growing rows, forking / reordering / freeing them, and moving the used
// pages together.  Everything is integer work with a fixed outcome: free
// pages are taken lowest first, in the order of the slots; the only atomics
// are integer additions, whose order does not matter.
//
// `grow` and `compact` plan in one CTA, or for large pools in a cluster of
// eight that exchange their sums through each other's shared memory: each walks
// its part of the reference counts with block-wide scans.  The plan is carried
// out with the whole GPU: table entries, counts and the copies of pages, which
// are what takes time.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "cache_common.cuh"

namespace cg = cooperative_groups;

namespace saf {
namespace {

constexpr int kPlan = 1024;          // threads of a planning CTA
constexpr int kCopy = 256;           // threads of a carrying-out CTA
constexpr int kChunk = kCopy * 128;  // bytes that it copies at once

// Exclusive sum over the CTA of x; the total in `total`.
__device__ long long block_scan(long long x, long long* warp_sums /* [33] */, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  long long v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < n ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += y;
    }
    if (lane < n) warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[n - 1];
  return v - x + (warp ? warp_sums[warp - 1] : 0);
}

// Scratch of one call: a header, a record for each slot, two page lists and a
// page map.
struct Scratch {
  int* head;     // [16] grow: goes through, copies, pages taken; compact: -, copies, used
  int4* slots;   // [n_seqs] first column, columns, first of its pages in the list, copy or -1
  int* from;     // [max(n_seqs, n_pages)] pages to copy
  int* to;       // [max(n_seqs, n_pages)]
  int* list;     // [n_pages] grow: free pages; compact: new place of a page
};
__host__ __device__ __forceinline__ size_t round4(size_t x) { return (x + 3) & ~(size_t)3; }
__device__ __forceinline__ Scratch scratch_of(const CachePages& p) {
  Scratch s;
  const size_t n = round4(p.n_pages > p.n_seqs ? p.n_pages : p.n_seqs);
  s.head = p.scratch;
  s.slots = reinterpret_cast<int4*>(p.scratch + 16);
  s.from = p.scratch + 16 + 4 * (size_t)p.n_seqs;
  s.to = s.from + n;
  s.list = s.to + n;
  return s;
}

constexpr int kRowPages = 4 * kPlan;  // four pages for each thread
constexpr int kPlanRows = 2;          // rows of a step of the walk, all loaded at once
constexpr int kStepPages = kPlanRows * kRowPages;

// The counts of pages base + 4 i .. base + 4 i + 3 (i: the thread); pages
// behind the last one count as neither free nor used.
struct Four {
  int v[4];
  unsigned used, exist;  // bit k: page k
};
__device__ __forceinline__ Four four_pages(const int32_t* ref, int n_pages, int base) {
  Four f;
  const int first = base + 4 * (int)threadIdx.x;
  f.used = f.exist = 0;
  if (first + 4 <= n_pages) {
    const int4 x = *reinterpret_cast<const int4*>(ref + first);
    f.v[0] = x.x, f.v[1] = x.y, f.v[2] = x.z, f.v[3] = x.w;
    f.exist = 15;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f.v[k] = first + k < n_pages ? ref[first + k] : 0;
      f.exist |= (first + k < n_pages ? 1u : 0u) << k;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) f.used |= (f.v[k] > 0 ? 1u : 0u) << k;
  return f;
}

// The pages of one CTA of the plan's cluster.
struct Part {
  int begin, end;
};
__device__ __forceinline__ Part part_of(int n_pages) {
  const long long n = gridDim.x, per = ((n_pages + n - 1) / n + 3) & ~3ll;
  Part r;
  r.begin = (int)min((long long)n_pages, per * blockIdx.x);
  r.end = (int)min((long long)n_pages, per * blockIdx.x + per);
  return r;
}

// All threads of the plan, and what they wrote.
__device__ __forceinline__ void plan_sync() {
  if (gridDim.x > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
}

// x summed over the CTA's threads, then over the cluster: the sum of the CTAs
// before this one and of all.  Every thread of the cluster calls it; `box` is a
// shared word used for nothing else.
struct Sums {
  long long before, all;
};
__device__ Sums cluster_sums(long long x, long long* warp_sums, long long* box) {
  long long mine;
  block_scan(x, warp_sums, mine);
  Sums s = {0, mine};
  if (gridDim.x == 1) return s;
  s.all = 0;
  if (threadIdx.x == 0) *box = mine;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (unsigned i = 0; i < gridDim.x; ++i) {
    const long long y = *cluster.map_shared_rank(box, i);
    if (i < blockIdx.x) s.before += y;
    s.all += y;
  }
  return s;
}

// Ranks of the marked pages of a step among all marked pages of the step: of
// the thread's first one in each row; returns the step's total.  One barrier
// before the sums are read; the caller lets two steps use different `sums`.
__device__ __forceinline__ int step_ranks(const unsigned (&marked)[kPlanRows],
                                          int (*sums)[32] /* [kPlanRows] */,
                                          int (&rank)[kPlanRows]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned before = (1u << lane) - 1;
#pragma unroll
  for (int j = 0; j < kPlanRows; ++j) {
    int mine = 0;
    rank[j] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned b = __ballot_sync(~0u, marked[j] >> k & 1);
      rank[j] += __popc(b & before);
      mine += __popc(b);
    }
    if (lane == 0) sums[j][warp] = mine;
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int j = 0; j < kPlanRows; ++j) {
    int x = sums[j][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    const int up_to = __shfl_sync(~0u, x, warp ? warp - 1 : 0);
    rank[j] += total + (warp ? up_to : 0);
    total += __shfl_sync(~0u, x, 31);
  }
  return total;
}

// Copies pages from[k] -> to[k], k < n, in chunks over the whole grid.
__device__ void copy_pages(const CachePages& p, const int* from, const int* to, int n) {
  const long long chunks = ((long long)p.page_bytes + kChunk - 1) / kChunk;
  for (long long i = blockIdx.x; i < chunks * n; i += gridDim.x) {
    const int k = (int)(i / chunks);
    const size_t off = (size_t)(i % chunks) * kChunk;
    const uint8_t* src = p.pool + (size_t)from[k] * p.page_stride;
    uint8_t* dst = p.pool + (size_t)to[k] * p.page_stride;
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t o = off + ((size_t)u * kCopy + threadIdx.x) * 16;
      if (o < p.page_bytes) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + o));
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t o = off + ((size_t)u * kCopy + threadIdx.x) * 16;
      if (o < p.page_bytes) __stcs(reinterpret_cast<uint4*>(dst + o), v[u]);
    }
  }
}

// ------------------------------------------------------------ grow
struct Need {
  int n;        // tokens granted if the call goes through
  int begin;    // first new column
  int columns;  // new columns
  int tail;     // page to copy, or -1
};
__device__ __forceinline__ Need slot_need(const CachePages& p, int s) {
  Need d;
  const int len = max(0, p.seq_len[s]), n = max(0, p.n_new[s]), size = 1 << p.page_shift;
  const long long room = (long long)p.max_pages << p.page_shift;
  d.n = len + (long long)n <= room ? n : 0;
  d.begin = (int)(((long long)len + size - 1) >> p.page_shift);
  d.columns = d.n > 0 ? (int)(((long long)len + d.n + size - 1) >> p.page_shift) - d.begin : 0;
  d.tail = -1;
  if (d.n > 0 && (len & (size - 1))) {
    const int t = p.table[(size_t)s * p.max_pages + (len >> p.page_shift)];
    if ((unsigned)t < (unsigned)p.n_pages && p.ref[t] > 1) d.tail = t;
  }
  return d;
}
// A row may hold pages behind its length: tokens were taken back.  New columns, from
// the first on, that hold a page which no other row holds need none; returns their
// number.  To be asked before the counts change.
__device__ __forceinline__ int held_columns(const CachePages& p, int s, const Need& d) {
  const int32_t* row = p.table + (size_t)s * p.max_pages + d.begin;
  constexpr int kAhead = 4;  // loads in flight
  for (int c = 0; c < d.columns; c += kAhead) {
    int t[kAhead], r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t[k] = c + k < d.columns ? row[c + k] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = (unsigned)t[k] < (unsigned)p.n_pages ? p.ref[t[k]] : 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (r[k] != 1) return min(c + k, d.columns);
  }
  return d.columns;
}

// The plan: each slot's share of the free pages (a copy of its last page
// first, then its new columns), and whether there are enough.
__global__ void __launch_bounds__(kPlan) grow_plan_kernel(const __grid_constant__ CachePages p) {
  __shared__ long long sums[33];
  __shared__ int ranks[2][kPlanRows][32];
  __shared__ long long box;
  asm volatile("griddepcontrol.launch_dependents;");
  const Scratch w = scratch_of(p);
  // needs in the low 44 bits, copies above; every CTA adds up all slots
  const int per = (p.n_seqs + kPlan - 1) / kPlan;
  const int s0 = min(p.n_seqs, (int)threadIdx.x * per), s1 = min(p.n_seqs, s0 + per);
  // each CTA writes the slots of its share of the threads
  const bool owner = (int)(threadIdx.x * gridDim.x / kPlan) == (int)blockIdx.x;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Need d = slot_need(p, s);
    const int held = held_columns(p, s, d);
    if (owner) w.slots[s].x = held;
    mine += d.columns - held + (d.tail >= 0) + ((long long)(d.tail >= 0) << 44);
  }
  long long all;
  long long at = block_scan(mine, sums, all);
  const long long total = all & ((1ll << 44) - 1);
  const Part part = part_of(p.n_pages);
  // the first row stays in registers: all there is of a small pool
  const Four first_row = four_pages(p.ref, part.end, part.begin);
  long long n_mine = __popc(~first_row.used & first_row.exist);
#pragma unroll 4
  for (int base = part.begin + kRowPages; base < part.end; base += kRowPages) {
    const Four f = four_pages(p.ref, part.end, base);
    n_mine += __popc(~f.used & f.exist);
  }
  // (also: no CTA writes before all have read the lengths)
  const Sums free_pages = cluster_sums(n_mine, sums, &box);
  const bool ok = total <= free_pages.all;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.head[0] = ok ? 1 : 0;
    w.head[1] = ok ? (int)(all >> 44) : 0;
    w.head[2] = ok ? (int)total : 0;
    const long long lack = ok ? 0 : total - free_pages.all;
    *p.count = lack > 0x7fffffff ? 0x7fffffff : (int)lack;
  }
  // the first `total` free pages go into the list and get a count of one; the
  // other counts are copied where the call has its own output
  const bool in_place = p.ref == p.ref_out;
  long long rank0 = free_pages.before;
  for (int base = part.begin, step = 0; base < part.end; base += kStepPages, ++step) {
    if (in_place && (!ok || rank0 >= total)) break;
    Four f[kPlanRows];
    unsigned marked[kPlanRows];
    int rank[kPlanRows];
#pragma unroll
    for (int j = 0; j < kPlanRows; ++j) {
      f[j] = j == 0 && step == 0 ? first_row
                                 : four_pages(p.ref, part.end, base + j * kRowPages);
      marked[j] = ~f[j].used & f[j].exist;
    }
    const int n = step_ranks(marked, ranks[step & 1], rank);
#pragma unroll
    for (int j = 0; j < kPlanRows; ++j) {
      const int first = base + j * kRowPages + 4 * (int)threadIdx.x;
      long long at_rank = rank0 + rank[j];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool free = marked[j] >> k & 1, take = ok && free && at_rank < total;
        if (take) {
          w.list[at_rank] = first + k;
          f[j].v[k] = 1;
          if (in_place) p.ref_out[first + k] = 1;
        }
        at_rank += free;
      }
      if (!in_place) {
        if (f[j].exist == 15)
          *reinterpret_cast<int4*>(p.ref_out + first) =
              make_int4(f[j].v[0], f[j].v[1], f[j].v[2], f[j].v[3]);
        else
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (f[j].exist >> k & 1) p.ref_out[first + k] = f[j].v[k];
      }
    }
    rank0 += n;
  }
  plan_sync();  // the list is whole; nobody reads a box any more
  if (!owner) return;
  for (int s = s0; s < s1; ++s) {
    const Need d = slot_need(p, s);
    const int held = w.slots[s].x, columns = d.columns - held;
    const long long base = at & ((1ll << 44) - 1);
    const bool copy = d.tail >= 0;
    int4 rec = make_int4(d.begin + held, ok ? columns : 0, (int)base + copy, -1);
    if (ok && copy) {
      w.from[at >> 44] = d.tail;
      w.to[at >> 44] = w.list[base];
      rec.w = w.list[base];
    }
    w.slots[s] = rec;
    at += columns + copy + ((long long)copy << 44);
    p.granted[s] = ok ? d.n : 0;
    p.seq_len_out[s] = max(0, p.seq_len[s]) + (ok ? d.n : 0);
  }
}

// Whether x is among the n ascending pages of the list.
__device__ __forceinline__ bool in_list(const int* list, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (list[mid] < x)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo < n && list[lo] == x;
}

__global__ void __launch_bounds__(kCopy) grow_apply_kernel(const __grid_constant__ CachePages p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Scratch w = scratch_of(p);
  const bool in_place = p.table == p.table_out;
  if (!w.head[0] && in_place) return;
  for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
    const int4 r = w.slots[s];  // first new column, columns, place in the list, copy or -1
    const size_t row = (size_t)s * p.max_pages;
    // the column whose page becomes the slot's own: that of its length before
    const int own = r.w >= 0 ? p.seq_len_out[s] - p.granted[s] >> p.page_shift : -1;
    if (own >= 0 && threadIdx.x == 0) {
      atomicSub(p.ref_out + p.table[row + own], 1);
      p.table_out[row + own] = r.w;
    }
    const int c0 = in_place ? r.x : 0, c1 = in_place ? r.x + r.y : p.max_pages;
    for (int c = c0 + threadIdx.x; c < c1; c += kCopy)
      if (c >= r.x && c < r.x + r.y) {
        // a page that the row holds here, with others or behind a column that needed one,
        // is given up.  (One that was free when the call began is nobody's, whatever the
        // entry says, or was taken in this call.)
        const int was = p.table[row + c];
        p.table_out[row + c] = w.list[r.z + c - r.x];
        if ((unsigned)was < (unsigned)p.n_pages && !in_list(w.list, w.head[2], was) &&
            *(volatile int32_t*)(p.ref_out + was) > 0)
          atomicSub(p.ref_out + was, 1);
      } else if (c != own)
        p.table_out[row + c] = p.table[row + c];
  }
  copy_pages(p, w.from, w.to, w.head[1]);
}

// ------------------------------------------------------------ fork
// Each CTA takes `width` columns of every row: it reads them all before it
// writes, so the table may be updated in place.  The last CTA takes the
// lengths.
__global__ void __launch_bounds__(512)
    fork_kernel(const __grid_constant__ CachePages p, int width, int n_blocks) {
  extern __shared__ int32_t old[];
  if ((int)blockIdx.x == n_blocks) {
    for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) old[s] = p.seq_len[s];
    __syncthreads();
    for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
      const int q = p.parent[s];
      p.seq_len_out[s] = (unsigned)q < (unsigned)p.n_seqs ? old[q] : 0;
    }
    return;
  }
  const int c0 = blockIdx.x * width, n = min(width, p.max_pages - c0);
  // an element's row and column, a power of two apart
  const int shift = width == 8 ? 3 : (width == 4 ? 2 : width - 1);
  const int all = p.n_seqs << shift;
#pragma unroll 8
  for (int i = threadIdx.x; i < all; i += 512) {
    const int s = i >> shift, c = i & (width - 1);
    if (c < n) old[i] = p.table[(size_t)s * p.max_pages + c0 + c];
  }
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < all; i += 512) {
    const int s = i >> shift, c = i & (width - 1);
    if (c >= n) continue;
    const int q = p.parent[s];
    const int was = old[i];
    const int is = (unsigned)q < (unsigned)p.n_seqs ? old[(q << shift) + c] : -1;
    if (was != is || p.table != p.table_out) p.table_out[(size_t)s * p.max_pages + c0 + c] = is;
    if (was != is) {
      if ((unsigned)was < (unsigned)p.n_pages) atomicSub(p.ref_out + was, 1);
      if ((unsigned)is < (unsigned)p.n_pages) atomicAdd(p.ref_out + is, 1);
    }
  }
}

// ------------------------------------------------------------ compact
__global__ void __launch_bounds__(kPlan)
    compact_plan_kernel(const __grid_constant__ CachePages p) {
  __shared__ long long sums[33];
  __shared__ int ranks[4][kPlanRows][32];
  __shared__ long long boxes[2];
  asm volatile("griddepcontrol.launch_dependents;");
  const Scratch w = scratch_of(p);
  const Part part = part_of(p.n_pages);
  // the first row stays in registers: all there is of a small pool
  const Four first_row = four_pages(p.ref, part.end, part.begin);
  long long n_mine = __popc(first_row.used);
#pragma unroll 4
  for (int base = part.begin + kRowPages; base < part.end; base += kRowPages)
    n_mine += __popc(four_pages(p.ref, part.end, base).used);
  const int n_used = (int)cluster_sums(n_mine, sums, &boxes[0]).all;
  // free pages before n_used take the used pages behind it, in order: `front`
  // marks the former and `back` the latter
  auto bits = [&](const Four& f, int base, unsigned& front, unsigned& back) {
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m |= (base + 4 * (int)threadIdx.x + k < n_used ? 1u : 0u) << k;
    front = ~f.used & f.exist & m;
    back = f.used & ~m;
  };
  long long both = 0;  // front in the low half, back above
#pragma unroll 4
  for (int base = part.begin; base < part.end; base += kRowPages) {
    unsigned front, back;
    bits(base == part.begin ? first_row : four_pages(p.ref, part.end, base), base, front, back);
    both += __popc(front) + ((long long)__popc(back) << 32);
  }
  const Sums place = cluster_sums(both, sums, &boxes[1]);
  int at_to = (int)(place.before & 0xffffffff), at_from = (int)(place.before >> 32);
  for (int base = part.begin, step = 0; base < part.end; base += kStepPages, ++step) {
    unsigned front[kPlanRows], back[kPlanRows];
    int rank[kPlanRows];
#pragma unroll
    for (int j = 0; j < kPlanRows; ++j)
      bits(j == 0 && step == 0 ? first_row
                               : four_pages(p.ref, part.end, base + j * kRowPages),
           base + j * kRowPages, front[j], back[j]);
    const int first = base + 4 * (int)threadIdx.x;
    if (base < n_used) {
      const int n = step_ranks(front, ranks[step & 1], rank);
#pragma unroll
      for (int j = 0; j < kPlanRows; ++j) {
        int k0 = at_to + rank[j];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (front[j] >> k & 1) w.to[k0++] = first + j * kRowPages + k;
      }
      at_to += n;
    }
    if (base + kStepPages > n_used) {
      const int n = step_ranks(back, ranks[2 + (step & 1)], rank);
#pragma unroll
      for (int j = 0; j < kPlanRows; ++j) {
        int k0 = at_from + rank[j];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int page = first + j * kRowPages + k;
          if (back[j] >> k & 1)
            w.from[k0++] = page;
          else if (page >= n_used && page < part.end)
            w.list[page] = page;  // a free page's entry, should a row hold one
        }
      }
      at_from += n;
    }
  }
  plan_sync();  // the lists are whole; nobody reads a box any more
  const int n = (int)(place.all >> 32);
  for (int k = blockIdx.x * kPlan + threadIdx.x; k < n; k += gridDim.x * kPlan)
    w.list[w.from[k]] = w.to[k];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.head[1] = n;
    w.head[2] = n_used;
    *p.count = n_used;
  }
}

__global__ void __launch_bounds__(kCopy)
    compact_apply_kernel(const __grid_constant__ CachePages p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Scratch w = scratch_of(p);
  const int n = w.head[1], n_used = w.head[2];
  const size_t tid = (size_t)blockIdx.x * kCopy + threadIdx.x, all = (size_t)gridDim.x * kCopy;
  for (size_t k = tid; k < (size_t)n; k += all) {
    const int from = w.from[k], to = w.to[k];
    p.ref_out[to] = p.ref[from];
    if (p.ref == p.ref_out) p.ref_out[from] = 0;
  }
  if (p.ref != p.ref_out)  // the places of moved pages are written above
    for (size_t i = tid; i < (size_t)p.n_pages; i += all) {
      const int r = p.ref[i];
      if ((int)i >= n_used)
        p.ref_out[i] = r > 0 ? 0 : r;
      else if (r > 0)
        p.ref_out[i] = r;
    }
  const bool in_place = p.table == p.table_out;
#pragma unroll 4
  for (size_t i = tid; i < (size_t)p.n_seqs * p.max_pages; i += all) {
    const int page = p.table[i];
    const int is = page >= n_used && page < p.n_pages ? w.list[page] : page;
    if (is != page || !in_place) p.table_out[i] = is;
  }
  copy_pages(p, w.from, w.to, n);
}

// Launched while its predecessor runs (both plans allow it at their start); waits
// for the predecessor's end.
template <class K>
cudaError_t launch_after(K kernel, const char* name, const CachePages& p, int grid,
                         cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kCopy);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  trace_end(s, name);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// One CTA plans for a pool of up to 8192 pages, a cluster of eight for more
// (2048 pages: one CTA 6 us; 65536 pages: one CTA 25 us).
template <class K>
cudaError_t launch_plan(K kernel, const char* name, const CachePages& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const unsigned n = p.n_pages > 8192 ? 8 : 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(kPlan);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin(s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  trace_end(s, name);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t copy_words(int32_t* to, const int32_t* from, size_t n, cudaStream_t s) {
  if (to == from || n == 0) return cudaSuccess;
  return cudaMemcpyAsync(to, from, n * 4, cudaMemcpyDeviceToDevice, s);
}

}  // namespace

size_t cache_pages_scratch_words(int n_seqs, int n_pages) {
  const size_t n = round4(n_pages > n_seqs ? n_pages : n_seqs);
  return 16 + 4 * (size_t)n_seqs + 2 * n + round4(n_pages);
}

cudaError_t launch_cache_fork(const CachePages& p, cudaStream_t s) {
  cudaError_t e = copy_words(p.ref_out, p.ref, p.n_pages, s);
  if (e != cudaSuccess) return e;
  // 8 columns are a 32-byte sector; fewer where 8 of every row do not fit
  int width = 8;
  while (width > 1 && (size_t)p.n_seqs * width * 4 > 200 * 1024) width >>= 1;
  const size_t smem = (size_t)p.n_seqs * width * 4;
  const int n_blocks = (p.max_pages + width - 1) / width;
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(fork_kernel), 200 * 1024);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  fork_kernel<<<n_blocks + 1, 512, smem, s>>>(p, width, n_blocks);
  trace_end(s, "cache_fork");
  return cudaGetLastError();
}

cudaError_t launch_cache_grow(const CachePages& p, int n_sms, cudaStream_t s) {
  const cudaError_t e = launch_plan(grow_plan_kernel, "cache_grow_plan", p, s);
  if (e != cudaSuccess) return e;
  return launch_after(grow_apply_kernel, "cache_grow", p, 4 * n_sms, s);
}

cudaError_t launch_cache_compact(const CachePages& p, int n_sms, cudaStream_t s) {
  const cudaError_t e = launch_plan(compact_plan_kernel, "cache_compact_plan", p, s);
  if (e != cudaSuccess) return e;
  return launch_after(compact_apply_kernel, "cache_compact", p, 4 * n_sms, s);
}

}  // namespace saf
