// cache_api.cu — host side of the paged 8-bit cache's calls: argument checks,
// the layout of a layer's record, launch parameters.
#include <cuda_runtime.h>
#include <string.h>

#include "../../include/saf.h"
#include "host_common.h"
#include "internal.h"

namespace saf {
namespace {

constexpr int kMaxSlots = 32768;

saf_status check_cache(const saf_cache_dims* d) {
  if (!d) return SAF_ERR_INVALID_ARG;
  if (d->n_seqs < 0 || d->max_pages < 1 || d->n_pages < 1 || d->page_size < 1 || d->H < 1 ||
      d->H_kv < 1 || d->H % d->H_kv != 0 || d->d_h < 1)
    return SAF_ERR_INVALID_ARG;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return SAF_ERR_UNSUPPORTED;
  if (d->d_h != 32 && d->d_h != 64 && d->d_h != 128) return SAF_ERR_UNSUPPORTED;
  if (d->H > kMaxHeads || d->n_seqs > kMaxSlots) return SAF_ERR_UNSUPPORTED;
  // the kernels step past the last key by less than a tile
  if ((long long)d->max_pages * d->page_size > (1ll << 31) - 1024) return SAF_ERR_UNSUPPORTED;
  if (d->page_stride % 16 != 0) return SAF_ERR_INVALID_ARG;
  if (d->page_stride >= (1ull << 32)) return SAF_ERR_UNSUPPORTED;
  return SAF_OK;
}

int page_shift(const saf_cache_dims& d) {
  int s = 4;
  while ((1 << s) < d.page_size) ++s;
  return s;
}

saf_cache_layout layout_of(const saf_cache_dims& d, const uint8_t* head_is_static,
                           int16_t* k_of /* [H_kv] or null */) {
  saf_cache_layout L;
  const int g = d.H / d.H_kv;
  L.H_k = 0;
  for (int k = 0; k < d.H_kv; ++k) {
    bool dyn = false;
    for (int h = k * g; h < (k + 1) * g; ++h) dyn |= head_is_static[h] == 0;
    if (k_of) k_of[k] = dyn ? (int16_t)L.H_k : (int16_t)-1;
    L.H_k += dyn;
  }
  const size_t block = (size_t)d.page_size * d.d_h;
  L.v = L.H_k * block;
  L.k_scale = L.v + d.H_kv * block;
  L.v_scale = L.k_scale + 4 * (size_t)L.H_k;
  L.bytes = (L.v_scale + 4 * (size_t)d.H_kv + 127) / 128 * 128;
  return L;
}

bool bad16(const void* p) { return !p || !aligned16(p); }

// The parts of a call on one layer; SAF_OK or what the call returns.
saf_status make_call(const saf_cache_dims& d, const uint8_t* head_is_static, const void* layer,
                     int n_q, const int32_t* n_new, const int32_t* seq_len,
                     const int32_t* page_table, CacheCall& c) {
  if (!head_is_static || bad16(layer) || !seq_len || !page_table) return SAF_ERR_INVALID_ARG;
  const void* ints[] = {n_new, seq_len, page_table};
  for (const void* p : ints)
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return SAF_ERR_INVALID_ARG;
  memset(&c, 0, sizeof(c));
  const saf_cache_layout L = layout_of(d, head_is_static, c.k_of);
  if (d.page_stride < L.bytes) return SAF_ERR_INVALID_ARG;
  c.layer = static_cast<uint8_t*>(const_cast<void*>(layer));
  c.page_stride = d.page_stride;
  c.off_v = L.v;
  c.off_ks = L.k_scale;
  c.off_vs = L.v_scale;
  c.page_table = page_table;
  c.seq_len = seq_len;
  c.n_new = n_new;
  c.n_seqs = d.n_seqs;
  c.max_pages = d.max_pages;
  c.n_pages = d.n_pages;
  c.page_shift = page_shift(d);
  c.H = d.H;
  c.H_kv = d.H_kv;
  c.group = d.H / d.H_kv;
  c.n_q = n_q;
  c.H_k = L.H_k;
  for (int h = 0; h < d.H; ++h) c.is_static[h] = head_is_static[h] != 0;
  return SAF_OK;
}

// Which kernel takes an attention call of n_q rows.  cache_attn.cu starts fast
// and reads a head's keys once for every 8 or 16 rows (from L2 after the first);
// cache_chunk.cu takes longer to start and reads them once for 256 rows of the
// dynamic heads and once for 256 of each frozen one.  The times are in nanoseconds
// on the whole GPU for a unit of rows and for each of its keys, fitted to 300 calls
// drawn at random that were timed with both, in tables as wide as their longest
// sequence: there the choice cost 0.1% over the better one (by rows alone, 11%).
// (Both kernels have changed by up to 5% since.)  All that the host knows of the
// lengths is the page table's width, so short sequences in wide tables may get the
// slower kernel: 4 x 107 rows of 2 heads against 107 keys take 6 us in a table of 128
// or 512 keys, 8 in one of 4096 (units may then be cut), 14 from 32768 on; a prompt of
// 512 tokens, 16 heads of 4, 28 us in a table of 512 keys and 26 in wider ones.
bool many_rows(const saf_cache_dims& d, const uint8_t* is_static, int n_q) {
  const int g = d.H / d.H_kv;
  const long long rows = (long long)n_q * g, tile = rows <= 8 ? 8 : 16;
  const double keys = (double)d.max_pages * d.page_size;
  long long units = 0;
  for (int kv = 0; kv < d.H_kv; ++kv) {
    int frozen = 0;
    for (int h = kv * g; h < (kv + 1) * g; ++h) frozen += is_static[h] != 0;
    units += ((long long)n_q * (g - frozen) + 255) / 256 + ((long long)n_q + 255) / 256 * frozen;
  }
  const double few_units = (double)d.n_seqs * d.H_kv * ((rows + tile - 1) / tile);
  const double few = 5e3 + few_units * (10 + 0.03 * keys);
  const double many = 18e3 + (double)d.n_seqs * units * (50 + 0.09 * keys);
  return few > many;
}

saf_status status_of(cudaError_t e) { return e == cudaSuccess ? SAF_OK : SAF_ERR_CUDA; }

saf_status make_pages(const saf_cache_dims& d, const int32_t* const (&words)[3],
                      int32_t* const (&outs)[3], CachePages& p) {
  for (int i = 0; i < 3; ++i)
    if (bad16(words[i]) || bad16(outs[i])) return SAF_ERR_INVALID_ARG;
  memset(&p, 0, sizeof(p));
  p.n_seqs = d.n_seqs;
  p.max_pages = d.max_pages;
  p.n_pages = d.n_pages;
  p.page_shift = page_shift(d);
  p.page_stride = d.page_stride;
  p.table = words[0];
  p.seq_len = words[1];
  p.ref = words[2];
  p.table_out = outs[0];
  p.seq_len_out = outs[1];
  p.ref_out = outs[2];
  return SAF_OK;
}

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" {

saf_status saf_cache_layer_layout(const saf_cache_dims* dims, const uint8_t* head_is_static,
                                  saf_cache_layout* layout) {
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  if (!head_is_static || !layout) return SAF_ERR_INVALID_ARG;
  *layout = layout_of(*dims, head_is_static, nullptr);
  return SAF_OK;
}

saf_status saf_cache_append(const saf_cache_dims* dims, const uint8_t* head_is_static, void* layer,
                            const void* K, const void* V, saf_dtype dtype, int n_q,
                            const int32_t* n_new, const int32_t* seq_len,
                            const int32_t* page_table, void* stream) {
  launch_count_reset();
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  if (n_q < 0 || (dtype != SAF_BF16 && dtype != SAF_F32)) return SAF_ERR_INVALID_ARG;
  if ((long long)n_q * dims->H >= (1ll << 31) || n_q > 1 << 30) return SAF_ERR_UNSUPPORTED;
  if (dims->n_seqs == 0 || n_q == 0) return SAF_OK;
  CacheAppend p;
  memset(&p, 0, sizeof(p));
  const saf_status cs =
      make_call(*dims, head_is_static, layer, n_q, n_new, seq_len, page_table, p.c);
  if (cs != SAF_OK) return cs;
  if (bad16(V) || (p.c.H_k > 0 ? bad16(K) : K && !aligned16(K))) return SAF_ERR_INVALID_ARG;
  p.K = K;
  p.V = V;
  p.f32 = dtype == SAF_F32;
  for (int k = 0; k < dims->H_kv; ++k)
    if (p.c.k_of[k] >= 0) p.kv_of[p.c.k_of[k]] = (int16_t)k;
  return status_of(launch_cache_append(p, dims->d_h, static_cast<cudaStream_t>(stream)));
}

size_t saf_cache_attn_workspace_size(const saf_cache_dims* dims, int n_q) {
  if (check_cache(dims) != SAF_OK || n_q < 0) return 0;
  // which kernel runs depends on the frozen heads; 16 rows of a group always take
  // the first: each head of K and V then is one unit there and at least one in the other
  const size_t few = cache_attn_ws(dims->d_h, sm_count()).total;
  const size_t many = cache_chunk_ws(dims->d_h, sm_count()).total;
  return (long long)n_q * (dims->H / dims->H_kv) <= 16 || few > many ? few : many;
}

saf_status saf_cache_attn(const saf_cache_dims* dims, const uint8_t* head_is_static,
                          const void* layer, const void* Q, const float* alpha, const float* rho,
                          int T_pat, int n_q, const int32_t* n_new, const int32_t* seq_len,
                          const int32_t* page_table, void* out, float* lse, void* workspace,
                          size_t ws_bytes, void* stream) {
  launch_count_reset();
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  if (n_q < 0 || T_pat < 0) return SAF_ERR_INVALID_ARG;
  if ((long long)n_q * dims->H >= (1ll << 31) || n_q > 1 << 30) return SAF_ERR_UNSUPPORTED;
  if (dims->n_seqs == 0 || n_q == 0) return SAF_OK;
  CacheAttn p;
  memset(&p, 0, sizeof(p));
  const saf_status cs =
      make_call(*dims, head_is_static, layer, n_q, n_new, seq_len, page_table, p.c);
  if (cs != SAF_OK) return cs;
  bool any_static = false;
  for (int h = 0; h < dims->H; ++h) any_static |= p.c.is_static[h] != 0;
  if (p.c.H_k > 0 ? bad16(Q) : Q && !aligned16(Q)) return SAF_ERR_INVALID_ARG;
  if (any_static && T_pat > 0 && (bad16(alpha) || bad16(rho))) return SAF_ERR_INVALID_ARG;
  if (bad16(out) || (lse && !aligned16(lse)) || !workspace) return SAF_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SAF_ERR_INVALID_ARG;
  const bool many = many_rows(*dims, p.c.is_static, n_q);
  const CacheAttnWs w = (many ? cache_chunk_ws : cache_attn_ws)(dims->d_h, sm_count());
  if (ws_bytes < w.total) return SAF_ERR_INVALID_ARG;
  p.Q = static_cast<const uint16_t*>(Q);
  p.alpha = alpha;
  p.rho = rho;
  p.T_pat = T_pat;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int*>(ws + w.status);
  p.join = reinterpret_cast<int4*>(ws + w.join);
  p.ml = reinterpret_cast<float*>(ws + w.ml);
  p.acc = reinterpret_cast<float*>(ws + w.acc);
  return status_of((many ? launch_cache_chunk : launch_cache_attn)(
      p, dims->d_h, sm_count(), static_cast<cudaStream_t>(stream)));
}

saf_status saf_cache_fork(const saf_cache_dims* dims, const int32_t* parent,
                          const int32_t* page_table, const int32_t* seq_len, const int32_t* ref,
                          int32_t* page_table_out, int32_t* seq_len_out, int32_t* ref_out,
                          void* stream) {
  launch_count_reset();
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  if (dims->n_seqs == 0) return SAF_OK;
  if (bad16(parent)) return SAF_ERR_INVALID_ARG;
  CachePages p;
  const int32_t* const in[3] = {page_table, seq_len, ref};
  int32_t* const out[3] = {page_table_out, seq_len_out, ref_out};
  const saf_status ps = make_pages(*dims, in, out, p);
  if (ps != SAF_OK) return ps;
  p.parent = parent;
  return status_of(launch_cache_fork(p, static_cast<cudaStream_t>(stream)));
}

size_t saf_cache_pages_workspace_size(const saf_cache_dims* dims) {
  if (check_cache(dims) != SAF_OK) return 0;
  return align256(cache_pages_scratch_words(dims->n_seqs, dims->n_pages) * 4);
}

saf_status saf_cache_grow(const saf_cache_dims* dims, void* pool, size_t page_bytes,
                          const int32_t* n_new, const int32_t* page_table, const int32_t* seq_len,
                          const int32_t* ref, int32_t* page_table_out, int32_t* seq_len_out,
                          int32_t* ref_out, int32_t* granted, int32_t* n_short, void* workspace,
                          size_t ws_bytes, void* stream) {
  launch_count_reset();
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  CachePages p;
  const int32_t* const in[3] = {page_table, seq_len, ref};
  int32_t* const out[3] = {page_table_out, seq_len_out, ref_out};
  if (dims->n_seqs == 0) return SAF_OK;
  const saf_status ps = make_pages(*dims, in, out, p);
  if (ps != SAF_OK) return ps;
  if (bad16(pool) || bad16(n_new) || bad16(granted) || bad16(n_short) || bad16(workspace))
    return SAF_ERR_INVALID_ARG;
  if (page_bytes % 16 != 0 || page_bytes > dims->page_stride) return SAF_ERR_INVALID_ARG;
  if (ws_bytes < saf_cache_pages_workspace_size(dims)) return SAF_ERR_INVALID_ARG;
  p.pool = static_cast<uint8_t*>(pool);
  p.page_bytes = page_bytes;
  p.n_new = n_new;
  p.granted = granted;
  p.count = n_short;
  p.scratch = static_cast<int32_t*>(workspace);
  return status_of(launch_cache_grow(p, sm_count(), static_cast<cudaStream_t>(stream)));
}

saf_status saf_cache_compact(const saf_cache_dims* dims, void* pool, size_t page_bytes,
                             const int32_t* page_table, const int32_t* ref,
                             int32_t* page_table_out, int32_t* ref_out, int32_t* n_used,
                             void* workspace, size_t ws_bytes, void* stream) {
  launch_count_reset();
  const saf_status st = check_cache(dims);
  if (st != SAF_OK) return st;
  CachePages p;
  // the lengths are not touched: any pointer that passes the check stands in
  const int32_t* const in[3] = {page_table, ref, ref};
  int32_t* const out[3] = {page_table_out, ref_out, ref_out};
  const saf_status ps = make_pages(*dims, in, out, p);
  if (ps != SAF_OK) return ps;
  if (bad16(pool) || bad16(n_used) || bad16(workspace)) return SAF_ERR_INVALID_ARG;
  if (page_bytes % 16 != 0 || page_bytes > dims->page_stride) return SAF_ERR_INVALID_ARG;
  if (ws_bytes < saf_cache_pages_workspace_size(dims)) return SAF_ERR_INVALID_ARG;
  p.pool = static_cast<uint8_t*>(pool);
  p.page_bytes = page_bytes;
  p.count = n_used;
  p.scratch = static_cast<int32_t*>(workspace);
  return status_of(launch_cache_compact(p, sm_count(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
