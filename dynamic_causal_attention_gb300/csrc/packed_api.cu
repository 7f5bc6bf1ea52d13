// packed_api.cu — host side of the packed attention: argument checks, workspace, tensor
// maps and the launch sequence of the forward and of the backward.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "../../include/saf.h"
#include "host_common.h"
#include "packed.h"

namespace saf {
namespace {

constexpr int kMaxSeqs = 1 << 20;

saf_status check_packed(const saf_packed_dims* d) {
  if (!d) return SAF_ERR_INVALID_ARG;
  if (d->total < 0 || d->n_seqs < 0 || d->max_len < 0 || d->H < 1 || d->H_kv < 1 ||
      d->H % d->H_kv != 0 || d->d_h < 1)
    return SAF_ERR_INVALID_ARG;
  if (d->d_h != 32 && d->d_h != 64 && d->d_h != 128) return SAF_ERR_UNSUPPORTED;
  if (d->H > kMaxHeads || d->n_seqs > kMaxSeqs || d->max_len > kMaxPackedLen)
    return SAF_ERR_UNSUPPORTED;
  // rows are counted over the heads in 31 bits, tiles of all sequences under all heads too
  if (((long long)d->total + 256) * d->H >= (1ll << 31)) return SAF_ERR_UNSUPPORTED;
  return SAF_OK;
}

int tiles_of(int rows) { return (rows + 127) / 128; }

// Tiles that any sequences within the dims can have.
int max_tiles(const saf_packed_dims& d) {
  const long long by_rows = (long long)d.total / 128 + d.n_seqs;
  const long long by_len = (long long)d.n_seqs * tiles_of(d.max_len);
  const long long by_one = d.total;  // a tile has a row at least
  long long n = by_rows < by_len ? by_rows : by_len;
  if (n > by_one) n = by_one;
  return (int)n;
}

struct PackedWs {
  size_t status, hdr, by_key, by_query, groups, seqs;
  size_t a_tab, r_tab, row_tab, logZ, mode, shift;
  size_t Dvec, lse2, row_vals, dq_acc, dv_acc, order, total;
};

PackedWs packed_ws(const saf_packed_dims& d, bool backward) {
  PackedWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  const size_t nt = max_tiles(d), H = d.H, T = (size_t)tiles_of(d.max_len) * 128;
  w.status = take(256);
  w.hdr = take(32);
  w.by_key = take(nt * 16);
  w.by_query = take(nt * 16);
  w.groups = take(nt * 8);
  w.seqs = take((size_t)d.n_seqs * 16);
  w.a_tab = take(H * T * 4);
  w.r_tab = take(H * (T + 128) * 4);
  w.row_tab = take(H * T * 4);
  w.logZ = take(H * T * 4);
  w.mode = take(H * 4);
  w.shift = take(H * 4);
  const size_t b = backward ? 1 : 0;
  w.Dvec = take(b * H * nt * 512);
  w.lse2 = take(b * H * nt * 512);
  w.row_vals = take(b * H * T * 4);
  w.dq_acc = take(b * H * d.total * d.d_h * 4);
  w.dv_acc = take(b * d.H_kv * d.total * d.d_h * 4);
  w.order = take(b * (order_rounds(d.d_h) + 1) * 256 * 16);
  w.total = off;
  return w;
}

// SAF_OK where rows [total, heads, d_h] can be read (written: `out`) through r.
saf_status check_rows(const saf_rows* r, const saf_packed_dims& d, int heads, bool out) {
  if (!r || !r->p || !aligned16(r->p)) return SAF_ERR_INVALID_ARG;
  const bool many_rows = d.total > 1, many_heads = heads > 1;
  if (r->row >= (1ll << 30) || r->head >= (1ll << 38)) return SAF_ERR_UNSUPPORTED;
  if ((many_rows && (r->row < d.d_h || r->row % 8 != 0)) ||
      (many_heads && (r->head < d.d_h || r->head % 8 != 0)))
    return SAF_ERR_INVALID_ARG;
  // an output's rows must not run into one another: rows of heads or heads of rows
  if (out && many_rows && many_heads && r->row < (int64_t)(heads - 1) * r->head + d.d_h &&
      r->head < (int64_t)(d.total - 1) * r->row + d.d_h)
    return SAF_ERR_INVALID_ARG;
  return SAF_OK;
}

// Strides as the kernels take them (of an extent of one they may be anything).
int64_t row_of(const saf_rows& r, const saf_packed_dims& d) { return d.total > 1 ? r.row : d.d_h; }
int64_t head_of(const saf_rows& r, int heads) { return heads > 1 ? r.head : 0; }

bool encode(CUtensorMap* m, const saf_rows& r, const saf_packed_dims& d, int heads) {
  return encode_heads(m, r.p, d.total, heads, d.d_h, row_of(r, d) * 2,
                      heads > 1 ? r.head * 2 : (int64_t)d.d_h * 2);
}

struct Call {
  const saf_packed_dims& d;
  HeadSplit hs;
  int Hkv, g, nt;
  PackedWs w;
  uint8_t* ws;
  cudaStream_t s;
  template <class T>
  T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }
};

PackedPrep make_prep(const Call& c, const int32_t* cu, const float* alpha, const float* rho,
                     bool backward, bool clear) {
  PackedPrep p;
  memset(&p, 0, sizeof(p));
  p.total = c.d.total;
  p.n_seqs = c.d.n_seqs;
  p.max_len = c.d.max_len;
  p.max_tiles = tiles_of(c.d.max_len);
  // (the accumulators that fit beside the tiles of weights: static_group)
  p.backward = backward;
  p.group = static_group(c.d.d_h, 4, backward);
  p.per_tile = c.d.H;
  if (backward) {
    // dV of the K/V heads that frozen heads read
    p.per_tile = 0;
    for (int kv = 0; kv < c.Hkv; ++kv) {
      int frozen = 0;
      for (int h = kv * c.g; h < (kv + 1) * c.g; ++h) frozen |= c.hs.is_static[h];
      p.per_tile += frozen;
    }
  }
  p.num_sms = sm_count();
  p.cu = cu;
  p.status = c.at<int>(c.w.status);
  p.hdr = c.at<int>(c.w.hdr);
  p.by_key = c.at<int4>(c.w.by_key);
  p.by_query = c.at<int4>(c.w.by_query);
  p.groups = c.at<int2>(c.w.groups);
  p.seqs = c.at<int4>(c.w.seqs);
  p.T = p.max_tiles * 128;
  p.T_pat = c.d.T_pat;
  p.n_static = c.hs.n_static;
  p.alpha = alpha;
  p.rho = rho;
  p.a_tab = c.at<float>(c.w.a_tab);
  p.r_tab = c.at<float>(c.w.r_tab);
  p.row_tab = c.at<float>(c.w.row_tab);
  p.logZ = c.at<float>(c.w.logZ);
  p.mode = c.at<int>(c.w.mode);
  p.shift = c.at<float>(c.w.shift);
  p.clear = clear;
  p.d = c.d.d_h;
  p.H = c.d.H;
  memcpy(p.static_heads, c.hs.st, sizeof(p.static_heads));
  return p;
}

void clear_too(PackedPrep& p, const saf_rows& r, const saf_packed_dims& d, int heads) {
  p.rows[p.n_rows++] =
      ClearRows{static_cast<__nv_bfloat16*>(r.p), row_of(r, d), head_of(r, heads), heads};
}

void fill_fwd(PackedFwdParams& p, const Call& c) {
  memset(&p, 0, sizeof(p));
  p.H = c.d.H;
  p.T = tiles_of(c.d.max_len) * 128;
  p.H_kv = c.Hkv;
  p.group_kv = c.g;
  p.n_static = c.hs.n_static;
  p.n_dynamic = c.hs.n_dynamic;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d.d_h);
  memcpy(p.static_heads, c.hs.st, sizeof(p.static_heads));
  memcpy(p.dynamic_heads, c.hs.dy, sizeof(p.dynamic_heads));
  p.a_tab = c.at<float>(c.w.a_tab);
  p.r_tab = c.at<float>(c.w.r_tab);
  p.row_tab = c.at<float>(c.w.row_tab);
  p.logZ = c.at<float>(c.w.logZ);
  p.mode = c.at<int>(c.w.mode);
  p.shift = c.at<float>(c.w.shift);
  p.status = c.at<int>(c.w.status);
  p.hdr = c.at<int>(c.w.hdr);
  p.counter = c.at<int>(c.w.hdr) + 2;
  p.groups = c.at<int2>(c.w.groups);
  p.total = c.d.total;
}

// Blocks for `n` items per tile: the plan may hold fewer.
int items_for(const Call& c, int n) {
  const long long m = (long long)c.nt * n;
  return m > (1 << 30) ? 1 << 30 : (int)m;
}

saf_status common_checks(const saf_packed_dims* dims, const int32_t* cu, const float* alpha,
                         const float* rho, const uint8_t* head_is_static, const void* workspace,
                         unsigned flags, HeadSplit& hs) {
  if (!head_is_static || !cu || !workspace) return SAF_ERR_INVALID_ARG;
  if ((flags & ~(unsigned)SAF_CLEAR_REST) != 0) return SAF_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu) & 3u) != 0) return SAF_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SAF_ERR_INVALID_ARG;
  hs = split_heads(head_is_static, dims->H);
  if (hs.n_static > 0) {
    if (!alpha || !rho || (reinterpret_cast<uintptr_t>(alpha) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(rho) & 3u) != 0 || dims->T_pat < dims->max_len)
      return SAF_ERR_INVALID_ARG;
  }
  return SAF_OK;
}

}  // namespace
}  // namespace saf

using namespace saf;

#define SAF_TRY(expr)                           \
  do {                                          \
    cudaError_t e_ = (expr);                    \
    if (e_ != cudaSuccess) return SAF_ERR_CUDA; \
  } while (0)

#define SAF_CHECK(expr)               \
  do {                                \
    const saf_status s_ = (expr);     \
    if (s_ != SAF_OK) return s_;      \
  } while (0)

extern "C" {

size_t saf_packed_attn_workspace_size(const saf_packed_dims* dims, int backward) {
  if (check_packed(dims) != SAF_OK) return 0;
  return packed_ws(*dims, backward != 0).total;
}

saf_status saf_packed_attn_fwd(const saf_packed_dims* dims, const saf_rows* Q, const saf_rows* K,
                               const saf_rows* V, const int32_t* cu_seqlens, const float* alpha,
                               const float* rho, const uint8_t* head_is_static,
                               const saf_rows* out, float* lse, unsigned flags, void* workspace,
                               size_t ws_bytes, void* stream) {
  launch_count_reset();
  SAF_CHECK(check_packed(dims));
  const saf_packed_dims& d = *dims;
  if (d.total == 0) return SAF_OK;
  Call c{d, {}, d.H_kv, d.H / d.H_kv, max_tiles(d), packed_ws(d, false),
         static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
  SAF_CHECK(common_checks(dims, cu_seqlens, alpha, rho, head_is_static, workspace, flags, c.hs));
  if (c.hs.n_dynamic > 0) {
    SAF_CHECK(check_rows(Q, d, d.H, false));
    SAF_CHECK(check_rows(K, d, d.H_kv, false));
  }
  SAF_CHECK(check_rows(V, d, d.H_kv, false));
  SAF_CHECK(check_rows(out, d, d.H, true));
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return SAF_ERR_INVALID_ARG;
  if (ws_bytes < c.w.total) return SAF_ERR_INVALID_ARG;

  PackedPrep prep = make_prep(c, cu_seqlens, alpha, rho, false, (flags & SAF_CLEAR_REST) != 0);
  clear_too(prep, *out, d, d.H);
  prep.lse = lse;
  SAF_TRY(launch_packed_prep(prep, c.s));
  if (c.nt == 0) return SAF_OK;

  PackedFwdLaunch L;
  memset(&L, 0, sizeof(L));
  fill_fwd(L.p, c);
  L.p.tiles = c.at<int4>(c.w.by_key);
  L.p.out = static_cast<__nv_bfloat16*>(out->p);
  L.p.out_row = row_of(*out, d);
  L.p.out_head = head_of(*out, d.H);
  L.p.lse = lse;
  L.p.n_items = items_for(c, d.H);
  // without dynamic heads the maps of Q and K are not used, but must be valid
  const bool dyn = c.hs.n_dynamic > 0;
  if (!encode(&L.tm_q, dyn ? *Q : *V, d, dyn ? d.H : d.H_kv) ||
      !encode(&L.tm_k, dyn ? *K : *V, d, d.H_kv) || !encode(&L.tm_v, *V, d, d.H_kv))
    return SAF_ERR_CUDA;
  // (the map of out is used where a tile is staged in shared memory)
  if (d.d_h != 64) L.tm_o = L.tm_v;
  else if (!encode(&L.tm_o, *out, d, d.H)) return SAF_ERR_CUDA;
  L.d_h = d.d_h;
  L.num_sms = sm_count();
  SAF_TRY(launch_packed_fwd(L, false, c.s));
  return SAF_OK;
}

saf_status saf_packed_attn_bwd(const saf_packed_dims* dims, const saf_rows* Q, const saf_rows* K,
                               const saf_rows* V, const saf_rows* out, const float* lse,
                               const saf_rows* dout, const int32_t* cu_seqlens,
                               const float* alpha, const float* rho,
                               const uint8_t* head_is_static, const saf_rows* dQ,
                               const saf_rows* dK, const saf_rows* dV, unsigned flags,
                               void* workspace, size_t ws_bytes, void* stream) {
  launch_count_reset();
  SAF_CHECK(check_packed(dims));
  const saf_packed_dims& d = *dims;
  if (d.total == 0) return SAF_OK;
  Call c{d, {}, d.H_kv, d.H / d.H_kv, max_tiles(d), packed_ws(d, true),
         static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
  SAF_CHECK(common_checks(dims, cu_seqlens, alpha, rho, head_is_static, workspace, flags, c.hs));
  const bool dyn = c.hs.n_dynamic > 0;
  if (dyn) {
    SAF_CHECK(check_rows(Q, d, d.H, false));
    SAF_CHECK(check_rows(K, d, d.H_kv, false));
    SAF_CHECK(check_rows(out, d, d.H, false));
  }
  SAF_CHECK(check_rows(V, d, d.H_kv, false));
  SAF_CHECK(check_rows(dout, d, d.H, false));
  SAF_CHECK(check_rows(dQ, d, d.H, true));
  SAF_CHECK(check_rows(dK, d, d.H_kv, true));
  SAF_CHECK(check_rows(dV, d, d.H_kv, true));
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return SAF_ERR_INVALID_ARG;
  if (ws_bytes < c.w.total) return SAF_ERR_INVALID_ARG;

  PackedPrep prep = make_prep(c, cu_seqlens, alpha, rho, true, (flags & SAF_CLEAR_REST) != 0);
  clear_too(prep, *dQ, d, d.H);
  clear_too(prep, *dK, d, d.H_kv);
  clear_too(prep, *dV, d, d.H_kv);
  SAF_TRY(launch_packed_prep(prep, c.s));
  if (c.nt == 0) return SAF_OK;

  PackedRows r;
  memset(&r, 0, sizeof(r));
  r.nt_max = c.nt;
  r.total = d.total;
  r.H = d.H;
  r.group_kv = c.g;
  r.d_h = d.d_h;
  r.hdr = c.at<int>(c.w.hdr);
  r.tiles = c.at<int4>(c.w.by_key);
  if (dyn) {
    r.out = static_cast<const __nv_bfloat16*>(out->p);
    r.out_row = row_of(*out, d);
    r.out_head = head_of(*out, d.H);
    r.q = static_cast<const __nv_bfloat16*>(Q->p);
    r.q_row = row_of(*Q, d);
    r.q_head = head_of(*Q, d.H);
    r.k = static_cast<const __nv_bfloat16*>(K->p);
    r.k_row = row_of(*K, d);
    r.k_head = head_of(*K, c.Hkv);
    r.v = static_cast<const __nv_bfloat16*>(V->p);
    r.v_row = row_of(*V, d);
    r.v_head = head_of(*V, c.Hkv);
  }
  r.dout = static_cast<const __nv_bfloat16*>(dout->p);
  r.do_row = row_of(*dout, d);
  r.do_head = head_of(*dout, d.H);
  r.lse = lse;
  r.Dvec = c.at<float>(c.w.Dvec);
  r.lse2 = c.at<float>(c.w.lse2);
  r.row_vals = c.at<float>(c.w.row_vals);
  r.T = tiles_of(d.max_len) * 128;
  r.mode = c.at<int>(c.w.mode);
  r.shift = c.at<float>(c.w.shift);
  r.dq_acc = c.at<float>(c.w.dq_acc);
  r.dQ = static_cast<__nv_bfloat16*>(dQ->p);
  r.dq_row = row_of(*dQ, d);
  r.dq_head = head_of(*dQ, d.H);
  r.dK = static_cast<__nv_bfloat16*>(dK->p);
  r.dk_row = row_of(*dK, d);
  r.dk_head = head_of(*dK, c.Hkv);
  r.scale = 1.0f / sqrtf((float)d.d_h);
  memset(r.static_slot, 0xff, sizeof(r.static_slot));  // -1
  for (int i = 0; i < c.hs.n_static; ++i) r.static_slot[c.hs.st[i]] = (int16_t)i;
  for (int h = 0; h < d.H; ++h) r.kv_has_dyn[h / c.g] |= !c.hs.is_static[h];

  // the dynamic pass: query heads by K/V head, and its items
  PackedBwdLaunch bl;
  memset(&bl, 0, sizeof(bl));
  if (dyn) {
    PackedBwdParams& p = bl.p;
    int n = 0;
    for (int kv = 0; kv < c.Hkv; ++kv) {
      p.dyn_begin[kv] = (uint16_t)n;
      for (int h = kv * c.g; h < (kv + 1) * c.g; ++h)
        if (!c.hs.is_static[h]) p.dyn_by_kv[n++] = (uint8_t)h;
      p.dyn_count[kv] = (uint16_t)(n - p.dyn_begin[kv]);
      if (p.dyn_count[kv] > 0) p.items.kv_list[p.n_kv++] = (uint8_t)kv;
    }
    // K/V heads of a group of items.  The CTAs add into dQ's sums, and read Q and dO, of one
    // query head of each K/V head of the group at a time; half of L2 and a little more
    // holds them, about 82 MB.  Up to 160 MB one group is better all the same, as items
    // share out better: 352 us against 368 with two (9 heads of 64, 33k rows).  With 245 MB three
    // groups take 340 us, one 370 (16 heads of 64, 30k rows); with 201 MB two 924, three
    // 1002 (12 heads of 128, 2 x 8192 rows); with 268 three 2370, two 2446, four 2419 (16 heads of
    // 128, 16384 rows).  (Nothing was measured between 154 and 201 MB.)
    int heads = 1;
    for (int i = 0; i < p.n_kv; ++i)
      heads = p.dyn_count[p.items.kv_list[i]] > heads ? p.dyn_count[p.items.kv_list[i]] : heads;
    const double mb = (double)p.n_kv * d.total * d.d_h * 8.0 / 1e6;
    int groups = mb <= 160.0 ? 1 : (int)(mb / 82.0 + 0.5);
    if (groups > p.n_kv) groups = p.n_kv;
    p.items.tiles = c.at<int4>(c.w.by_query);
    p.items.n_kv = p.n_kv;
    p.items.per_group = (p.n_kv + groups - 1) / groups;
    p.items.most_steps = heads * tiles_of(d.max_len);
    p.items.even = n == heads * p.n_kv;
    memcpy(p.items.dyn_count, p.dyn_count, sizeof(p.dyn_count));
    p.n_items = items_for(c, p.n_kv);
    bl.num_sms = sm_count() < 256 ? sm_count() : 256;
    p.order = c.at<int4>(c.w.order);
    r.order = c.at<int4>(c.w.order);
    r.n_ctas = p.n_items < bl.num_sms ? p.n_items : bl.num_sms;
    r.items = p.items;
  }
  SAF_TRY(launch_packed_pre(r, c.s));

  float* dv_acc = c.at<float>(c.w.dv_acc);
  uint8_t kv_has_static[kMaxHeads] = {0};
  for (int h = 0; h < d.H; ++h) kv_has_static[h / c.g] |= c.hs.is_static[h];
  if (c.hs.n_static > 0) {
    // dV = P^T dO of the frozen heads: written where no dynamic head shares V, left
    // in fp32 for the dynamic pass elsewhere
    PackedFwdLaunch L;
    memset(&L, 0, sizeof(L));
    fill_fwd(L.p, c);
    L.p.counter = c.at<int>(c.w.hdr) + 3;
    L.p.tiles = c.at<int4>(c.w.by_key);
    L.p.out = static_cast<__nv_bfloat16*>(dV->p);
    L.p.out_row = row_of(*dV, d);
    L.p.out_head = head_of(*dV, c.Hkv);
    L.p.out_acc = dv_acc;
    L.p.row_vals = r.row_vals;
    memcpy(L.p.kv_has_dyn, r.kv_has_dyn, sizeof(L.p.kv_has_dyn));
    int n = 0;
    for (int kv = 0; kv < c.Hkv; ++kv) {
      L.p.st_begin[kv] = (uint16_t)n;
      for (int h = kv * c.g; h < (kv + 1) * c.g; ++h)
        if (c.hs.is_static[h]) L.p.st_by_kv[n++] = (uint8_t)r.static_slot[h];
      L.p.st_count[kv] = (uint16_t)(n - L.p.st_begin[kv]);
      if (L.p.st_count[kv] > 0) L.p.kv_list[L.p.n_kv_st++] = (uint8_t)kv;
    }
    L.p.n_items = items_for(c, L.p.n_kv_st);
    if (!encode(&L.tm_v, *dout, d, d.H)) return SAF_ERR_CUDA;
    L.tm_q = L.tm_k = L.tm_o = L.tm_v;
    L.d_h = d.d_h;
    L.num_sms = sm_count();
    SAF_TRY(launch_packed_fwd(L, true, c.s));
  }
  if (dyn) {
    PackedBwdLaunch& L = bl;
    PackedBwdParams& p = L.p;
    p.H = d.H;
    p.H_kv = c.Hkv;
    memcpy(p.kv_has_static, kv_has_static, sizeof(p.kv_has_static));
    p.scale = r.scale;
    p.scale_log2 = 1.4426950408889634f * r.scale;
    p.dv_acc = dv_acc;
    p.lse2 = r.lse2;
    p.Dvec = r.Dvec;
    p.dq_acc = r.dq_acc;
    p.dK = r.dK;
    p.dk_row = r.dk_row;
    p.dk_head = r.dk_head;
    p.dV = static_cast<__nv_bfloat16*>(dV->p);
    p.dv_row = row_of(*dV, d);
    p.dv_head = head_of(*dV, c.Hkv);
    p.status = c.at<int>(c.w.status);
    p.hdr = r.hdr;
    p.total = d.total;
    p.nt_max = c.nt;
    if (!encode(&L.tm_q, *Q, d, d.H) || !encode(&L.tm_k, *K, d, c.Hkv) ||
        !encode(&L.tm_v, *V, d, c.Hkv) || !encode(&L.tm_do, *dout, d, d.H) ||
        !encode_rows_f32(&L.tm_dq, r.dq_acc, (uint64_t)d.H * d.total, d.d_h))
      return SAF_ERR_CUDA;
    L.d_h = d.d_h;
    SAF_TRY(launch_packed_bwd(L, c.s));
    SAF_TRY(launch_packed_post(r, c.s));
  }
  return SAF_OK;
}

}  // extern "C"
