// serving_api.cu — host side of the rotary positions and of the beam step:
// argument checks and launch parameters.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <utility>

#include "../../include/saf.h"
#include "host_common.h"
#include "internal.h"

namespace saf {
namespace {

saf_status status_of(cudaError_t e) { return e == cudaSuccess ? SAF_OK : SAF_ERR_CUDA; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether rows run into one another: by rising strides, each must pass what lies below it.
bool overlap(const saf_rows& r, int B, int T, int heads, int d) {
  int64_t stride[3] = {r.head, r.row, r.seq};
  int n[3] = {heads, T, B};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[j] > stride[j + 1]) {
        std::swap(stride[j], stride[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  __int128 span = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] < 2) continue;
    if (stride[i] < span) return true;
    span += (__int128)stride[i] * (n[i] - 1);
  }
  return false;
}

constexpr int kMaxBeams = 32;
constexpr int kMaxVocab = 1 << 22;

saf_status check_beam(const saf_beam_dims* d) {
  if (!d) return SAF_ERR_INVALID_ARG;
  if (d->n_groups < 0 || d->beams < 1 || d->vocab < 1 || d->row_stride < d->vocab ||
      d->max_tokens < 0 || d->end < -1 || d->end >= d->vocab)
    return SAF_ERR_INVALID_ARG;
  if (d->dtype != SAF_BF16 && d->dtype != SAF_F32) return SAF_ERR_INVALID_ARG;
  if (d->beams > kMaxBeams || d->vocab > kMaxVocab) return SAF_ERR_UNSUPPORTED;
  // blocks are counted in 31 bits: a row has fewer than vocab / 2048 + 2 of them
  if ((long long)d->n_groups * d->beams * (d->vocab / 2048 + 2) >= (1ll << 31))
    return SAF_ERR_UNSUPPORTED;
  return SAF_OK;
}

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" {

saf_status saf_rotary_turns(const double* radians, int n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!radians || !turns))) return SAF_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!isfinite(radians[i])) return SAF_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double t = radians[i] / 6.283185307179586476925286766559;
    const double part = t - floor(t);  // in [0, 1]: 1 where t is a little below 0
    // whole multiples of 2^-64 (a double has 53 bits), a full turn being none
    turns[i] = part >= 1.0 ? 0 : (uint64_t)ldexp(part, 64);
  }
  return SAF_OK;
}

saf_status saf_rotary(const saf_rotary_dims* dims, const saf_rows* q, const saf_rows* k,
                      const saf_rows* q_out, const saf_rows* k_out, const uint64_t* turns,
                      float scale, const int32_t* positions, const int32_t* cu_seqlens,
                      int n_seqs, const int32_t* seq_len, const int32_t* n_new, unsigned flags,
                      void* stream) {
  launch_count_reset();
  if (!dims) return SAF_ERR_INVALID_ARG;
  const saf_rotary_dims& d = *dims;
  if (d.B < 0 || d.T < 0 || d.H < 0 || d.H_k < 0 || d.d_h < 1 || d.rot < 2 || d.rot % 2 != 0 ||
      d.rot > d.d_h || (d.dtype != SAF_BF16 && d.dtype != SAF_F32))
    return SAF_ERR_INVALID_ARG;
  if ((flags & ~(unsigned)(SAF_ROTARY_INTERLEAVED | SAF_ROTARY_INVERSE | SAF_CLEAR_REST)) != 0)
    return SAF_ERR_INVALID_ARG;
  if ((positions != nullptr) + (cu_seqlens != nullptr) + (seq_len != nullptr) > 1 ||
      (n_new && !seq_len) || n_seqs < 0 || (cu_seqlens && d.B > 1))
    return SAF_ERR_INVALID_ARG;
  // pairs and copied parts of all rows are counted in 31 bits
  if (d.d_h > 256 || d.H > kMaxHeads || d.H_k > kMaxHeads ||
      (long long)d.B * d.T > ((1ll << 31) - 1024) / d.d_h)
    return SAF_ERR_UNSUPPORTED;
  if (d.B == 0 || d.T == 0 || d.H + d.H_k == 0) return SAF_OK;
  if (!turns || !aligned(turns, 8) || !isfinite(scale)) return SAF_ERR_INVALID_ARG;
  const int32_t* ints[] = {positions, cu_seqlens, seq_len, n_new};
  for (const int32_t* p : ints)
    if (!aligned(p, 4)) return SAF_ERR_INVALID_ARG;
  RotaryParams p;
  memset(&p, 0, sizeof(p));
  const saf_rows* rows[4] = {q, k, q_out, k_out};
  const size_t size = d.dtype == SAF_F32 ? 4 : 2;
  bool in_place = true;
  for (int i = 0; i < 4; ++i) {
    const int heads = i & 1 ? d.H_k : d.H;
    if (heads == 0) continue;
    const saf_rows* r = rows[i];
    if (!r || !r->p || !aligned(r->p, size) || r->seq < 0 || r->row < 0 || r->head < 0)
      return SAF_ERR_INVALID_ARG;
    if (i >= 2 && overlap(*r, d.B, d.T, heads, d.d_h)) return SAF_ERR_INVALID_ARG;
    p.x[i] = RotaryRows{r->p, r->seq, r->row, r->head};
    if (i >= 2) {
      const saf_rows* in = rows[i - 2];
      const bool same = in->p == r->p;
      if (same && (in->seq != r->seq || in->row != r->row || in->head != r->head))
        return SAF_ERR_INVALID_ARG;
      in_place &= same;
    }
  }
  // one tensor's output in the place of the other (x: q, k, q_out, k_out)
  if (d.H > 0 && d.H_k > 0 &&
      (p.x[2].p == p.x[1].p || p.x[3].p == p.x[0].p || p.x[2].p == p.x[3].p))
    return SAF_ERR_INVALID_ARG;
  p.B = d.B;
  p.T = d.T;
  p.H = d.H;
  p.H_k = d.H_k;
  p.d = d.d_h;
  p.rot = d.rot;
  p.turns = turns;
  p.scale = scale;
  p.scale_sin = flags & SAF_ROTARY_INVERSE ? -scale : scale;
  p.positions = positions;
  p.cu = cu_seqlens;
  p.n_seqs = n_seqs;
  p.seq_len = seq_len;
  p.n_new = n_new;
  p.clear = (flags & SAF_CLEAR_REST) != 0;
  p.copy_rest = !in_place || p.clear;
  return status_of(launch_rotary(p, d.dtype == SAF_F32, (flags & SAF_ROTARY_INTERLEAVED) != 0,
                                 sm_count(), static_cast<cudaStream_t>(stream)));
}

size_t saf_beam_workspace_size(const saf_beam_dims* dims) {
  if (check_beam(dims) != SAF_OK) return 0;
  const size_t n = beam_ws(dims->n_groups, dims->beams, dims->vocab, sm_count()).total;
  return n < 256 ? 256 : n;
}

saf_status saf_beam_step(const saf_beam_dims* dims, const void* logits, const float* scores,
                         const uint8_t* finished, const int32_t* history, const int32_t* n_tokens,
                         int32_t* parent, int32_t* token, float* score_out, uint8_t* finished_out,
                         int32_t* history_out, void* workspace, size_t ws_bytes, void* stream) {
  launch_count_reset();
  const saf_status st = check_beam(dims);
  if (st != SAF_OK) return st;
  const saf_beam_dims& d = *dims;
  if (d.n_groups == 0) return SAF_OK;
  const bool f32 = d.dtype == SAF_F32;
  if (!logits || !aligned(logits, f32 ? 4 : 2) || !scores || !parent || !token || !score_out)
    return SAF_ERR_INVALID_ARG;
  if ((finished || finished_out) && d.end < 0) return SAF_ERR_INVALID_ARG;
  if ((history == nullptr) != (history_out == nullptr)) return SAF_ERR_INVALID_ARG;
  if (history && (!n_tokens || history == history_out || d.max_tokens < 1))
    return SAF_ERR_INVALID_ARG;
  const void* words[] = {scores, history, n_tokens, parent, token, score_out, history_out};
  for (const void* p : words)
    if (!aligned(p, 4)) return SAF_ERR_INVALID_ARG;
  const BeamWs w = beam_ws(d.n_groups, d.beams, d.vocab, sm_count());
  if (!workspace || !aligned(workspace, 256) || ws_bytes < w.total) return SAF_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  BeamParams p;
  memset(&p, 0, sizeof(p));
  p.n_groups = d.n_groups;
  p.beams = d.beams;
  p.vocab = d.vocab;
  p.end = d.end;
  p.max_tokens = d.max_tokens;
  p.row_stride = d.row_stride;
  p.logits = logits;
  p.scores = scores;
  p.finished = finished;
  p.history = history;
  p.n_tokens = n_tokens;
  p.parent = parent;
  p.token = token;
  p.score_out = score_out;
  p.finished_out = finished_out;
  p.history_out = history_out;
  p.one_join = w.one_join;
  p.tiles = w.tiles;
  p.splits = w.splits;
  p.part_bytes = w.part_bytes;
  p.row_count = reinterpret_cast<int*>(ws + w.row_count);
  p.group_count = reinterpret_cast<int*>(ws + w.group_count);
  p.row_lse = reinterpret_cast<double*>(ws + w.row_lse);
  p.row_best = reinterpret_cast<unsigned long long*>(ws + w.row_best);
  p.parts = ws + w.parts;
  return status_of(launch_beam(p, f32, w.held, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
