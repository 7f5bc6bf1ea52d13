// internal.h — declarations shared by the host API (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/saf.h"

namespace saf {

// Launch bookkeeping (per host thread): trace_begin() before and trace_end()
// after every kernel launch.  trace_end counts the launch for
// saf_last_launch_count(); when the kernel trace is enabled the pair also
// records two CUDA events on the launch stream around the kernel.
void trace_begin(cudaStream_t s);
void trace_end(cudaStream_t s, const char* kernel);
// Start counting launches for a new entry-point call.
void launch_count_reset();

// Raise `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device.  cudaFuncSetAttribute applies to the current device only, so this
// is done once per (kernel, device); safe to call from several host threads.
cudaError_t set_max_dynamic_smem(const void* kernel, int bytes);

// ------------------------------------------------------------ calibration
struct CalibLaunch {
  const float* A;     // [n, head_count, T, T]
  int n;
  int head_begin;
  int head_count;
  int T;
  int count0;         // samples already merged into these heads
  float* mean;        // [num_heads, T, T]
  float* m2;          // [num_heads, T, T]
  float* ent;         // [num_heads, T, T] sum_n x log x, or null (not tracked)
};
cudaError_t launch_calib_accumulate(const CalibLaunch& p, cudaStream_t s);

struct CalibFinalize {
  int num_heads;
  int T;
  int N;
  int k;
  const float* mean;
  const float* m2;
  double* row_partials;  // [num_heads, T]
  float* A_hat;          // nullable
  float* s_var;
  int32_t* selected;     // nullable when k == 0
  const float* ent;      // KL score only: sum_n x log x state
};
cudaError_t launch_calib_finalize(const CalibFinalize& p, cudaStream_t s);
// Forward-KL score per head (into p.s_var) and its exact top-k.
cudaError_t launch_calib_finalize_kl(const CalibFinalize& p, cudaStream_t s);
// Sharp-mean pattern: causal softmax of each row of the running mean.
cudaError_t launch_calib_sharp(const float* mean, int num_heads, int T, float* out,
                               cudaStream_t s);

// ------------------------------------------------------------ compact fit
struct FitParams {
  const float* A_hat;        // [num_heads, T, T]
  int T;
  const int32_t* candidates; // [n_candidates] head indices, priority order
  int n_candidates;
  int k;
  float kl_max;
  int steps;
  float lr, beta1, beta2, eps;
  float* alpha;              // [n_candidates, T]
  float* rho;                // [n_candidates, T]
  float* kl;                 // [n_candidates]
  int32_t* selected;         // [k] (nullable when k == 0)
  int32_t* n_selected;       // [1]
};
size_t fit_smem_bytes(int T);
cudaError_t launch_fit(const FitParams& p, cudaStream_t s);

// ------------------------------------------------------------ attention
constexpr int kMaxHeads = 256;

// Static-head pre-pass (alpha/rho -> generator tables and log Z).
struct StaticPrep {
  int T;
  int n_static;
  const uint8_t* heads_dev;  // unused (heads passed by value below)
  uint8_t heads[kMaxHeads];  // static head ids
  const float* alpha;        // [H, T]
  const float* rho;          // [H, T]
  float* a_tab;              // [n_static, T]
  float* r_tab;              // [n_static, T + 128] (127 leading pads)
  float* row_tab;            // [n_static, T] : -log2 Z (exact heads only)
  float* logZ;               // [n_static, T] natural log (exact heads only)
  int* mode;                 // [n_static] 0 factored, 1 exact
  float* shift;              // [n_static] factored: max alpha + max rho (0 if all masked)
};
cudaError_t launch_static_prep(const StaticPrep& p, cudaStream_t s);

// Elementwise helpers.
cudaError_t launch_zero_u32(void* dst, size_t n_words, cudaStream_t s);
// [n_slabs, T_src, d] rows (bf16 or fp32) into [n_slabs, T_dst, d] (bf16 or
// fp32): rows t >= T_src of the destination are zero (padding), rows of the
// source past T_dst are dropped (cropping).  d % 4 == 0.
cudaError_t launch_restage_rows(const void* src, bool src_f32, void* dst, bool dst_f32,
                                size_t n_slabs, int T_src, int T_dst, int d, cudaStream_t s);
// [n_rows, T_src] fp32 into [n_rows, T_dst], entries t >= T_src set to `fill`.
cudaError_t launch_restage_vec(const float* src, float* dst, size_t n_rows, int T_src, int T_dst,
                               float fill, cudaStream_t s);

// ------------------------------------------------------------ paged 8-bit cache
// One call on one layer of the cache (see cache_common.cuh for the layout).
struct CacheCall {
  uint8_t* layer;            // the layer's record in page 0
  size_t page_stride;        // bytes from one page to the next
  size_t off_v, off_ks, off_vs;  // V codes, K scales, V scales in the record
  const int32_t* page_table; // [n_seqs, max_pages]
  const int32_t* seq_len;    // [n_seqs], the new tokens among them
  const int32_t* n_new;      // [n_seqs] or null: n_q rows for every slot
  int n_seqs, max_pages, n_pages, page_shift;
  int H, H_kv, group, n_q;   // group = H / H_kv
  int H_k;                   // K heads that are stored
  int16_t k_of[kMaxHeads];   // [H_kv] index among the stored K heads, or -1
  uint8_t is_static[kMaxHeads];
};

struct CacheAppend {
  CacheCall c;
  const void *K, *V;  // [n_seqs, H_kv, n_q, d]
  bool f32;
  int16_t kv_of[kMaxHeads];  // [H_k] the K/V head of a stored K head
};
cudaError_t launch_cache_append(const CacheAppend& p, int d_h, cudaStream_t s);

struct CacheAttn {
  CacheCall c;
  const uint16_t* Q;  // bf16 [n_seqs, H, n_q, d]
  const float *alpha, *rho;  // [H, T_pat]
  int T_pat;
  uint16_t* out;  // bf16 [n_seqs, H, n_q, d]
  float* lse;     // [n_seqs, H, n_q] or null
  // scratch: see cache_attn_ws
  int* status;
  int4* join;     // [n_ctas] the units that were cut, by CTA or by unit
  float* ml;      // [2 n_ctas, rows, 2]
  float* acc;     // [2 n_ctas, rows, d]
};
struct CacheAttnWs {
  size_t status, join, ml, acc, total;
};
CacheAttnWs cache_attn_ws(int d_h, int n_sms);
cudaError_t launch_cache_attn(const CacheAttn& p, int d_h, int n_sms, cudaStream_t s);

// Many rows (cache_chunk.cu): a class is the dynamic or the frozen query heads
// of a K/V head; classes of equal width and kind form a group.
struct CacheChunk {
  CacheAttn a;
  int n_groups;
  int group_width[kMaxHeads];       // heads of each class of the group
  uint8_t group_static[kMaxHeads];
  int group_first[kMaxHeads + 1];   // its first class
  int16_t cls_first[kMaxHeads];     // a class's heads: order[cls_first ...]
  uint8_t cls_kv[kMaxHeads], order[kMaxHeads];
  // units that a slot can have, and of them the first of each group; whether
  // `join` is ordered by units (no more of them than CTAs)
  int slot_units, group_unit[kMaxHeads];
  bool by_unit;
};
CacheAttnWs cache_chunk_ws(int d_h, int n_sms);
cudaError_t launch_cache_chunk(const CacheAttn& p, int d_h, int n_sms, cudaStream_t s);

// Page tables and reference counts (cache_pages.cu); a page is page_bytes
// long, every page_stride bytes.
struct CachePages {
  int n_seqs, max_pages, n_pages, page_shift;
  uint8_t* pool;
  size_t page_stride, page_bytes;
  const int32_t *table, *seq_len, *ref;
  int32_t *table_out, *seq_len_out, *ref_out;
  const int32_t* parent;   // fork: [n_seqs]
  const int32_t* n_new;    // grow: [n_seqs]
  int32_t* granted;        // grow: [n_seqs]
  int32_t* count;          // grow: pages short; compact: pages in use
  int32_t* scratch;
};
size_t cache_pages_scratch_words(int n_seqs, int n_pages);
cudaError_t launch_cache_fork(const CachePages& p, cudaStream_t s);
cudaError_t launch_cache_grow(const CachePages& p, int n_sms, cudaStream_t s);
cudaError_t launch_cache_compact(const CachePages& p, int n_sms, cudaStream_t s);

}  // namespace saf
