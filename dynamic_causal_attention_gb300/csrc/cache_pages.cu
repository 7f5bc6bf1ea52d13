// cache_pages.cu — page tables and reference counts of the paged cache:
// growing rows, forking / reordering / freeing them, and moving the used
// pages together.  Everything is integer work with a fixed outcome: free
// pages are taken lowest first, in the order of the slots; the only atomics
// are integer additions, whose order does not matter.
//
// `grow` and `compact` each plan in one CTA (a run of the counts for each
// thread, one block scan) and carry the plan out with the whole GPU: table
// entries, counts and the copies of pages, which are what takes time.
#include <cuda_runtime.h>

#include "cache_common.cuh"

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
  int* head;     // [16] total, copies, used
  int4* slots;   // [n_seqs] first column, columns, first of its pages in the list, -
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

// The pages of one thread: a run of whole groups of four.
struct Run {
  int begin, end;
};
__device__ __forceinline__ Run page_run(int n_pages) {
  const long long per = ((((long long)n_pages + kPlan - 1) / kPlan) + 3) & ~3ll;
  Run r;
  r.begin = (int)min((long long)n_pages, per * threadIdx.x);
  r.end = (int)min((long long)n_pages, per * threadIdx.x + per);
  return r;
}
// f(page, in use) over the run, counts read four at a time
template <class F>
__device__ __forceinline__ void each_page(const int32_t* ref, Run r, F f) {
  int i = r.begin;
#pragma unroll 4
  for (; i + 4 <= r.end; i += 4) {
    const int4 v = *reinterpret_cast<const int4*>(ref + i);
    f(i, v.x > 0);
    f(i + 1, v.y > 0);
    f(i + 2, v.z > 0);
    f(i + 3, v.w > 0);
  }
  for (; i < r.end; ++i) f(i, ref[i] > 0);
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
    if ((unsigned)t < (unsigned)p.n_pages && p.ref_out[t] > 1) d.tail = t;
  }
  return d;
}

// The plan: each slot's share of the free pages (a copy of its last page
// first, then its new columns), and whether there are enough.
__global__ void __launch_bounds__(kPlan) grow_plan_kernel(const __grid_constant__ CachePages p) {
  __shared__ long long sums[33];
  const Scratch w = scratch_of(p);
  // needs in the low 44 bits, copies above
  const int per = (p.n_seqs + kPlan - 1) / kPlan;
  const int s0 = min(p.n_seqs, (int)threadIdx.x * per), s1 = min(p.n_seqs, s0 + per);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Need d = slot_need(p, s);
    mine += d.columns + (d.tail >= 0) + ((long long)(d.tail >= 0) << 44);
  }
  long long all, n_free;
  long long at = block_scan(mine, sums, all);
  const long long total = all & ((1ll << 44) - 1);
  const Run run = page_run(p.n_pages);
  long long free_mine = 0;
  each_page(p.ref_out, run, [&](int, bool used) { free_mine += !used; });
  long long rank = block_scan(free_mine, sums, n_free);
  const bool ok = total <= n_free;
  if (threadIdx.x == 0) {
    w.head[0] = ok ? 1 : 0;
    w.head[1] = ok ? (int)(all >> 44) : 0;
    const long long lack = ok ? 0 : total - n_free;
    *p.count = lack > 0x7fffffff ? 0x7fffffff : (int)lack;
  }
  if (ok && free_mine > 0 && rank < total)
    each_page(p.ref_out, run, [&](int page, bool used) {
      if (!used && rank < total) w.list[rank] = page;
      rank += !used;
    });
  __syncthreads();  // every thread reads the list
  for (int s = s0; s < s1; ++s) {
    const Need d = slot_need(p, s);
    const long long base = at & ((1ll << 44) - 1);
    const bool copy = d.tail >= 0;
    int4 rec = make_int4(d.begin, ok ? d.columns : 0, (int)base + copy, -1);
    if (ok && copy) {
      w.from[at >> 44] = d.tail;
      w.to[at >> 44] = w.list[base];
      rec.w = w.list[base];
    }
    w.slots[s] = rec;
    at += d.columns + copy + ((long long)copy << 44);
    p.granted[s] = ok ? d.n : 0;
    p.seq_len_out[s] = max(0, p.seq_len[s]) + (ok ? d.n : 0);
  }
}

__global__ void __launch_bounds__(kCopy) grow_apply_kernel(const __grid_constant__ CachePages p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Scratch w = scratch_of(p);
  if (!w.head[0]) return;
  for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
    const int4 r = w.slots[s];
    int32_t* row = p.table_out + (size_t)s * p.max_pages;
    for (int i = threadIdx.x; i < r.y; i += kCopy) {
      const int page = w.list[r.z + i];
      row[r.x + i] = page;
      p.ref_out[page] = 1;
    }
    if (r.w >= 0 && threadIdx.x == 0) {  // the last page becomes the slot's own
      atomicSub(p.ref_out + row[r.x - 1], 1);
      row[r.x - 1] = r.w;
      p.ref_out[r.w] = 1;
    }
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
  for (int i = threadIdx.x; i < p.n_seqs * n; i += blockDim.x) {
    const int s = i / n, c = i - s * n;
    old[s * width + c] = p.table[(size_t)s * p.max_pages + c0 + c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.n_seqs * n; i += blockDim.x) {
    const int s = i / n, c = i - s * n;
    const int q = p.parent[s];
    const int was = old[s * width + c];
    const int is = (unsigned)q < (unsigned)p.n_seqs ? old[q * width + c] : -1;
    p.table_out[(size_t)s * p.max_pages + c0 + c] = is;
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
  const Scratch w = scratch_of(p);
  const Run run = page_run(p.n_pages);
  long long used_mine = 0, n_used, both;
  each_page(p.ref, run, [&](int, bool used) { used_mine += used; });
  block_scan(used_mine, sums, n_used);
  // used pages behind n_used in the low half, free pages before it above
  long long mine = 0;
  each_page(p.ref, run, [&](int page, bool used) {
    if (used ? page >= n_used : page < n_used) mine += used ? 1 : 1ll << 32;
  });
  long long at = block_scan(mine, sums, both);
  each_page(p.ref, run, [&](int page, bool used) {
    if (used && page >= n_used) {
      w.from[at & 0xffffffff] = page;
      at += 1;
    } else if (!used && page < n_used) {
      w.to[at >> 32] = page;
      at += 1ll << 32;
    }
    w.list[page] = page;
  });
  __syncthreads();
  const int n = (int)(both & 0xffffffff);
  for (int k = threadIdx.x; k < n; k += kPlan) w.list[w.from[k]] = w.to[k];
  if (threadIdx.x == 0) {
    w.head[1] = n;
    *p.count = (int)n_used;
  }
}

__global__ void __launch_bounds__(kCopy)
    compact_apply_kernel(const __grid_constant__ CachePages p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Scratch w = scratch_of(p);
  const int n = w.head[1];
  const size_t tid = (size_t)blockIdx.x * kCopy + threadIdx.x, all = (size_t)gridDim.x * kCopy;
  for (size_t k = tid; k < (size_t)n; k += all) {
    const int from = w.from[k], to = w.to[k];
    p.ref_out[to] = p.ref[from];
    p.ref_out[from] = 0;
  }
  for (size_t i = tid; i < (size_t)p.n_seqs * p.max_pages; i += all) {
    const int page = p.table[i];
    const int is = (unsigned)page < (unsigned)p.n_pages ? w.list[page] : page;
    p.table_out[i] = is;
  }
  copy_pages(p, w.from, w.to, n);
}

// Launched while its predecessor runs; waits for the predecessor's end.
template <class K>
cudaError_t launch_after(K kernel, const char* name, const CachePages& p, int grid, cudaStream_t s) {
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
  cudaError_t e = copy_words(p.ref_out, p.ref, p.n_pages, s);
  if (e == cudaSuccess)
    e = copy_words(p.table_out, p.table, (size_t)p.n_seqs * p.max_pages, s);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  grow_plan_kernel<<<1, kPlan, 0, s>>>(p);
  trace_end(s, "cache_grow_plan");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(grow_apply_kernel, "cache_grow", p, 4 * n_sms, s);
}

cudaError_t launch_cache_compact(const CachePages& p, int n_sms, cudaStream_t s) {
  cudaError_t e = copy_words(p.ref_out, p.ref, p.n_pages, s);
  if (e != cudaSuccess) return e;
  trace_begin(s);
  compact_plan_kernel<<<1, kPlan, 0, s>>>(p);
  trace_end(s, "cache_compact_plan");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(compact_apply_kernel, "cache_compact", p, 4 * n_sms, s);
}

}  // namespace saf
