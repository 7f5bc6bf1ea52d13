// packed.h — the small kernels around the packed attention: the plan and the tables that
// precede it, and the backward's row passes.
#pragma once

#include "attn_kernels.h"

namespace saf {

constexpr int kMaxPackedLen = 131072;             // longest sequence
constexpr int kMaxPackedTiles = kMaxPackedLen / 128;

// bf16 rows [total, heads, d] of which those of no sequence are cleared.
struct ClearRows {
  __nv_bfloat16* p;
  int64_t row, head;
  int heads;
};

struct PackedPrep {
  int total, n_seqs, max_len, max_tiles;  // max_tiles = ceil(max_len / 128)
  bool backward;             // groups are of the transposed form
  int group;                 // most tiles of a static item
  int per_tile;              // work items of a tile that shares nothing
  int num_sms;
  const int32_t* cu;         // [n_seqs + 1]
  int* status;
  int* hdr;                  // {tiles, groups, two counters of items handed out, first tile of the
                             // longest sequence (backward)}
  int4 *by_key, *by_query;   // records by falling X + 1 and by falling query tiles
  int2* groups;              // (first record of by_key, records) that share X
  int4* seqs;                // [n_seqs] scratch
  // tables of the frozen heads, T = 128 * max_tiles entries a head (see static_prep_kernel)
  int T, T_pat, n_static;
  const float *alpha, *rho;
  float *a_tab, *r_tab, *row_tab, *logZ, *shift;
  int* mode;
  // rows of no sequence: cleared where `clear`
  bool clear;
  ClearRows rows[3];
  int n_rows, d;
  float* lse;                // or null
  int H;
  uint8_t static_heads[kMaxHeads];
};
cudaError_t launch_packed_prep(const PackedPrep& p, cudaStream_t s);

struct PackedRows {
  int nt_max, total, H, group_kv, d_h;
  const int* hdr;
  const int4* tiles;
  const __nv_bfloat16 *out, *dout, *q, *k, *v;
  int64_t out_row, out_head, do_row, do_head, q_row, q_head, k_row, k_head, v_row, v_head;
  const float* lse;          // [H, total]
  float *Dvec, *lse2;        // [H, nt_max * 128]
  float* row_vals;           // [n_static, T], by the position in a sequence
  int T;
  const int* mode;
  const float* shift;
  float* dq_acc;             // [H, total, d]
  __nv_bfloat16 *dQ, *dK;
  int64_t dq_row, dq_head, dk_row, dk_head;
  float scale;
  // the dynamic pass's items, shared out over its CTAs
  int4* order;               // or null: no such pass
  int n_ctas;                // up to 256
  PackedBwdItems items;
  int16_t static_slot[kMaxHeads];  // -1: dynamic
  uint8_t kv_has_dyn[kMaxHeads];
};
cudaError_t launch_packed_pre(const PackedRows& p, cudaStream_t s);
cudaError_t launch_packed_post(const PackedRows& p, cudaStream_t s);

}  // namespace saf
