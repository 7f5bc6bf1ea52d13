"""Torch-facing entry points of libsaf (device memory and streams only).

These wrappers allocate outputs and the workspace with torch, pass raw
device addresses and the current CUDA stream to the C ABI, and raise on any
non-OK status.  All arithmetic runs in libsaf's kernels.
"""

from __future__ import annotations

import math

import numpy as np
import torch

from . import _binding as B

__all__ = ["HybridAttention", "Calibration", "PackedAttention", "PagedCache", "Rotary",
           "rotary_frequencies", "BeamSearch", "fit_compact", "num_select", "SafError"]

SafError = B.SafError


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device=None):
    return torch.cuda.current_stream(device).cuda_stream


def _raw_stream(index):
    """The current stream of a device as an integer (what ``_stream`` gives, without a Stream
    object: a call on the cache is a few microseconds)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _check(st, where):
    if st != B.SAF_OK:
        raise B.SafError(st, where)


class HybridAttention:
    """One hybrid causal attention layer of shape (B, H, T, d_h).

    ``head_is_static`` marks the frozen heads (host booleans, length H).
    ``dtype`` is torch.bfloat16 or torch.float32 (fp32 I/O is computed in
    bf16 inside the library).  ``H_kv`` < H groups the K/V heads: query head
    h reads K/V head h // (H // H_kv), and K, V, dK, dV are [B, H_kv, T, d_h].
    """

    def __init__(self, B_: int, H: int, T: int, d_h: int, head_is_static,
                 dtype=torch.bfloat16, device="cuda", want_param_grads=False, H_kv=None):
        self.shape = (B_, H, T, d_h)
        self.H_kv = H if H_kv is None else H_kv
        self.dtype = dtype
        self.device = torch.device(device)
        code = B.SAF_BF16 if dtype == torch.bfloat16 else B.SAF_F32
        self.dims = B._dims(B_, H, T, d_h, code, self.H_kv)
        self.head_is_static = bytes(np.asarray(head_is_static, dtype=np.uint8).tolist())
        assert len(self.head_is_static) == H
        self.ws_bytes = B.saf_hybrid_attn_workspace_size(self.dims, int(want_param_grads))
        if self.ws_bytes == 0:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "saf_hybrid_attn_workspace_size")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    def forward(self, q, k, v, alpha, rho, out=None, lse=None):
        B_, H, T, d = self.shape
        if out is None:
            out = torch.empty((B_, H, T, d), dtype=self.dtype, device=self.device)
        if lse is None:
            lse = torch.empty((B_, H, T), dtype=torch.float32, device=self.device)
        st = B.saf_hybrid_attn_fwd(self.dims, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(rho),
                                   self.head_is_static, _ptr(out), _ptr(lse),
                                   _ptr(self.workspace), self.ws_bytes, _stream(self.device))
        _check(st, "saf_hybrid_attn_fwd")
        return out, lse

    def backward(self, q, k, v, out, lse, dout, alpha, rho, want_param_grads=False,
                 grads=None):
        B_, H, T, d = self.shape
        if grads is None:
            mk = lambda h: torch.empty((B_, h, T, d), dtype=self.dtype, device=self.device)
            dq, dk, dv = mk(H), mk(self.H_kv), mk(self.H_kv)
            da = dr = None
            if want_param_grads:
                da = torch.empty((H, T), dtype=torch.float32, device=self.device)
                dr = torch.empty((H, T), dtype=torch.float32, device=self.device)
        else:
            dq, dk, dv, da, dr = grads
        st = B.saf_hybrid_attn_bwd(self.dims, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                   _ptr(dout), _ptr(alpha), _ptr(rho), self.head_is_static,
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(da), _ptr(dr),
                                   _ptr(self.workspace), self.ws_bytes, _stream(self.device))
        _check(st, "saf_hybrid_attn_bwd")
        return dq, dk, dv, da, dr

    def device_status(self):
        return B.saf_get_device_status(_ptr(self.workspace), 0, _stream(self.device))


class Calibration:
    """Streaming calibration state for ``num_heads`` heads of length T."""

    def __init__(self, num_heads: int, T: int, device="cuda", track_kl=False):
        self.device = torch.device(device)
        with torch.cuda.device(self.device):
            st, self.handle = B.saf_calib_create_ex(
                num_heads, T, B.SAF_CALIB_TRACK_KL if track_kl else 0)
        _check(st, "saf_calib_create_ex")
        self.num_heads, self.T = num_heads, T

    def accumulate(self, A, head_begin=0):
        n, hc = A.shape[0], A.shape[1]
        st = B.saf_calib_accumulate(self.handle, _ptr(A), n, head_begin, hc, _stream(self.device))
        _check(st, "saf_calib_accumulate")

    def finalize(self, k, want_mean=True):
        A_hat = None
        if want_mean:
            A_hat = torch.empty((self.num_heads, self.T, self.T), dtype=torch.float32,
                                device=self.device)
        s_var = torch.empty(self.num_heads, dtype=torch.float32, device=self.device)
        sel = torch.empty(max(k, 1), dtype=torch.int32, device=self.device)
        st = B.saf_calib_finalize(self.handle, k, _ptr(A_hat), _ptr(s_var), _ptr(sel),
                                  _stream(self.device))
        _check(st, "saf_calib_finalize")
        return A_hat, s_var, sel[:k]

    def finalize_kl(self, k):
        """Forward-KL selector: (s_kl [num_heads], the k lowest-scoring heads)."""
        s_kl = torch.empty(self.num_heads, dtype=torch.float32, device=self.device)
        sel = torch.empty(max(k, 1), dtype=torch.int32, device=self.device)
        st = B.saf_calib_finalize_kl(self.handle, k, _ptr(s_kl), _ptr(sel), _stream(self.device))
        _check(st, "saf_calib_finalize_kl")
        return s_kl, sel[:k]

    def finalize_sharp(self):
        """Sharp-mean pattern [num_heads, T, T] of a handle fed logits: the
        causal softmax of each row of the logits' mean."""
        out = torch.empty((self.num_heads, self.T, self.T), dtype=torch.float32,
                          device=self.device)
        st = B.saf_calib_finalize_sharp(self.handle, _ptr(out), _stream(self.device))
        _check(st, "saf_calib_finalize_sharp")
        return out

    def reset(self):
        _check(B.saf_calib_reset(self.handle), "saf_calib_reset")

    def close(self):
        if self.handle is not None:
            B.saf_calib_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """Keys and values of past tokens in pages of a pool, held in 8 bits, for serving the
    hybrid layers token by token.

    ``layers`` has one list of host booleans of length H for each layer: its frozen heads.
    ``H_kv`` < H groups the K/V heads as in HybridAttention.  The cache has ``n_seqs`` slots
    (rows of ``page_table`` [n_seqs, max_pages], int32), ``n_pages`` pages of ``page_size``
    tokens each, a token count for each slot (``seq_len``) and a count of the rows that hold
    each page (``ref``); all live on the GPU and may be given by the caller.  A page holds its
    tokens of every layer: ``pool`` is [n_pages, bytes of a page].

    One step of serving::

        granted, n_short = cache.grow(n_new)         # pages for the tokens to come
        for layer ...:
            cache.append(layer, k, v, n_new=granted)
            out, lse = cache.attend(layer, q, alpha, rho, n_new=granted)

    ``fork`` copies, reorders and frees slots, ``compact`` moves the used pages together.
    Nothing synchronises, and every call can be captured in a CUDA graph.  ``max_new`` is the
    largest number of rows for each slot that ``attend`` will be given; calls on one cache share
    its workspace, so they belong on one stream at a time.
    """

    def __init__(self, layers, H: int, d_h: int, *, n_seqs: int, max_pages: int, n_pages: int,
                 page_size: int = 64, H_kv=None, max_new: int = 1, device="cuda", pool=None,
                 page_table=None, seq_len=None, ref=None):
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self.H, self.d_h, self.H_kv = H, d_h, H if H_kv is None else H_kv
        self.n_seqs, self.max_pages, self.n_pages = n_seqs, max_pages, n_pages
        self.page_size, self.max_new = page_size, max_new
        self.layouts, self.offsets, self._static, self._frozen = [], [], [], []
        if n_seqs < 1:
            raise B.SafError(B.SAF_ERR_INVALID_ARG, f"PagedCache: {n_seqs} slots")
        geometry = (n_seqs, max_pages, n_pages, page_size, H, self.H_kv, d_h)
        at = 0
        for mask in layers:
            m = bytes(int(bool(x)) for x in mask)
            if len(m) != H:
                raise B.SafError(B.SAF_ERR_INVALID_ARG, f"PagedCache: a mask of {len(m)} heads")
            st, layout = B.saf_cache_layer_layout(B._cache_dims(*geometry, 0), m)
            _check(st, "saf_cache_layer_layout")
            self._static.append(m)
            self._frozen.append(any(m))
            self.layouts.append(layout)
            self.offsets.append(at)
            at += layout.bytes
        self.page_bytes = at
        new = lambda shape, fill: torch.full(shape, fill, dtype=torch.int32, device=self.device)
        if pool is None:
            pool = torch.zeros((n_pages, at), dtype=torch.uint8, device=self.device)
        self._tables = (new((n_seqs, max_pages), -1) if page_table is None else page_table,
                        new((n_seqs,), 0) if seq_len is None else seq_len,
                        new((n_pages,), 0) if ref is None else ref)
        if not (pool.dim() == 2 and pool.shape == (n_pages, at) and pool.stride(1) == 1
                and pool.dtype == torch.uint8 and pool.device == self.device):
            raise B.SafError(B.SAF_ERR_INVALID_ARG, f"PagedCache: pool is not [{n_pages}, {at}] bytes")
        self._pool = pool
        self._shapes = (torch.Size((n_seqs, max_pages)), torch.Size((n_seqs,)),
                        torch.Size((n_pages,)))
        self._table_like(self._tables, "PagedCache")
        self._pool_shape, self._strides = pool.shape, pool.stride()
        # a pool of one page may report any stride
        self.dims = B._cache_dims(*geometry, pool.stride(0) if n_pages > 1 else at)
        with torch.cuda.device(self.device):
            attn = B.saf_cache_attn_workspace_size(self.dims, max_new)
            pages = B.saf_cache_pages_workspace_size(self.dims)
        if attn == 0 or pages == 0:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "saf_cache_attn_workspace_size")
        self.ws_bytes, self._pages_bytes = attn, pages
        self.workspace = torch.empty(attn, dtype=torch.uint8, device=self.device)
        self.workspace[:256].zero_()  # the status before the first call
        self._pages_ws = torch.empty(pages, dtype=torch.uint8, device=self.device)

    page_table = property(lambda self: self._tables[0], doc="[n_seqs, max_pages] int32")
    seq_len = property(lambda self: self._tables[1], doc="[n_seqs] int32: tokens of each slot")
    ref = property(lambda self: self._tables[2], doc="[n_pages] int32: rows that hold a page")
    pool = property(lambda self: self._pool, doc="[n_pages, bytes of a page]")

    # ---- checks
    def _need(self, t, shape, dtype, what):
        if (t.dtype is not dtype or not t.is_cuda or t.get_device() != self._index
                or t.shape != shape or not t.is_contiguous()):
            raise B.SafError(B.SAF_ERR_INVALID_ARG,
                             f"{what}: want a contiguous {dtype} tensor {tuple(shape)} on {self.device}")
        return t.data_ptr()

    def _table_like(self, three, what):
        return tuple(self._need(t, s, torch.int32, what) for t, s in zip(three, self._shapes))

    # The tables and the pool belong to the caller, who may give them other storage: every call
    # takes their addresses anew, and checks them like its other arguments.
    def _table_at(self, i):
        return self._need(self._tables[i], self._shapes[i], torch.int32, "PagedCache: its tables")

    def _tables_at(self):
        return self._table_at(0), self._table_at(1), self._table_at(2)

    def _pool_at(self):
        p = self._pool
        if (p.dtype is not torch.uint8 or not p.is_cuda or p.get_device() != self._index
                or p.shape != self._pool_shape or p.stride() != self._strides):
            raise B.SafError(B.SAF_ERR_INVALID_ARG,
                             "PagedCache: the pool has another shape, type, device or stride now")
        return p.data_ptr()

    def _per_slot(self, t, what):
        return None if t is None else self._need(t, self._shapes[1], torch.int32, what)

    def _call(self, entry, *args):
        """The C entry on this cache's device and its current stream."""
        if torch.cuda.current_device() == self._index:
            st = entry(*args, _raw_stream(self._index))
        else:
            with torch.cuda.device(self.device):
                st = entry(*args, _raw_stream(self._index))
        if st != B.SAF_OK:
            raise B.SafError(st, entry.__name__)

    # ---- tokens
    def append(self, layer: int, k, v, n_new=None):
        """Quantise new rows k, v [n_seqs, H_kv, n, d_h] (bf16 or fp32) into the pages of
        ``layer``: the last n_new[s] (None: n) tokens of each slot, as counted by seq_len.
        k may be None where the layer stores no K."""
        n = v.shape[2] if v.dim() == 4 else -1
        shape = (self.n_seqs, self.H_kv, n, self.d_h)
        if v.dtype not in (torch.bfloat16, torch.float32):
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "append: v is neither bf16 nor fp32")
        pv = self._need(v, shape, v.dtype, "append: v")
        pk = None if k is None else self._need(k, shape, v.dtype, "append: k")
        self._call(B.saf_cache_append, self.dims, self._static[layer],
                   self._pool_at() + self.offsets[layer], pk, pv,
                   B.SAF_F32 if v.dtype == torch.float32 else B.SAF_BF16, n,
                   self._per_slot(n_new, "append: n_new"), self._table_at(1), self._table_at(0))

    def attend(self, layer: int, q, alpha=None, rho=None, n_new=None, out=None, lse=None):
        """The hybrid attention of q [n_seqs, H, n, d_h] (bf16), the last n_new[s] (None: n)
        tokens of each slot, over the cache.  alpha, rho [H, T] are needed where the layer has
        frozen heads.  Returns (out, lse); rows behind n_new are left as they were in buffers that
        are given, and 0 and -inf in those that the call makes (two small launches more)."""
        n = q.shape[2] if q.dim() == 4 else -1
        shape = (self.n_seqs, self.H, n, self.d_h)
        pq = self._need(q, shape, torch.bfloat16, "attend: q")
        if n > self.max_new:
            raise B.SafError(B.SAF_ERR_INVALID_ARG, f"attend: {n} rows, max_new is {self.max_new}")
        # what is made here and may keep rows that no slot takes starts as the results of rows
        # without a key
        if out is None:
            out = torch.empty_like(q) if n_new is None else torch.zeros_like(q)
        if lse is None:
            lse = torch.empty(shape[:3], dtype=torch.float32, device=self.device)
            if n_new is not None:
                lse.fill_(-math.inf)
        pa = pr = None
        T = 0
        if alpha is not None:
            T = alpha.shape[-1]
            pa = self._need(alpha, (self.H, T), torch.float32, "attend: alpha")
            pr = None if rho is None else self._need(rho, (self.H, T), torch.float32, "attend: rho")
        if self._frozen[layer] and (alpha is None or rho is None):
            raise B.SafError(B.SAF_ERR_INVALID_ARG, "attend: frozen heads need alpha and rho")
        self._call(B.saf_cache_attn, self.dims, self._static[layer],
                   self._pool_at() + self.offsets[layer], pq, pa, pr, T, n,
                   self._per_slot(n_new, "attend: n_new"), self._table_at(1), self._table_at(0),
                   self._need(out, shape, torch.bfloat16, "attend: out"),
                   self._need(lse, shape[:3], torch.float32, "attend: lse"),
                   self.workspace.data_ptr(), self.ws_bytes)
        return out, lse

    def views(self, layer: int):
        """(K codes, V codes, K scales, V scales) of a layer as views of the pool: codes
        [n_pages, heads, page_size, d_h] e4m3, scales [n_pages, heads] fp32."""
        L, n, d = self.layouts[layer], self.n_pages, self.d_h
        rec = self.pool[:, self.offsets[layer]:self.offsets[layer] + L.bytes]
        part = lambda a, b, h: rec[:, a:b].view(n, h, self.page_size, d).view(torch.float8_e4m3fn)
        return (part(0, L.v, L.H_k), part(L.v, L.k_scale, self.H_kv),
                rec[:, L.k_scale:L.v_scale].view(torch.float32),
                rec[:, L.v_scale:L.v_scale + 4 * self.H_kv].view(torch.float32))

    # ---- pages
    def grow(self, n_new, into=None):
        """Room for n_new[s] more tokens in every slot (copying a last page that is shared);
        seq_len advances.  To take tokens back lower seq_len: the row keeps its pages, and grow
        uses them again where no other row holds them.  Returns (granted [n_seqs], n_short [1]): what each slot got, all zero
        when n_short pages are missing.  ``into``: (page_table, seq_len, ref) to write instead of
        the cache's own."""
        at = self._tables_at()
        to = at if into is None else self._table_like(into, "grow: into")
        granted = torch.empty(self.n_seqs, dtype=torch.int32, device=self.device)
        n_short = torch.empty(1, dtype=torch.int32, device=self.device)
        self._call(B.saf_cache_grow, self.dims, self._pool_at(), self.page_bytes,
                   self._per_slot(n_new, "grow: n_new"), *at, *to, granted.data_ptr(),
                   n_short.data_ptr(), self._pages_ws.data_ptr(), self._pages_bytes)
        return granted, n_short

    def fork(self, parent, into=None):
        """Slot s takes over the pages and length of slot parent[s] (int32 [n_seqs]); a parent
        outside [0, n_seqs) frees it.  ``into`` as in grow."""
        at = self._tables_at()
        to = at if into is None else self._table_like(into, "fork: into")
        self._call(B.saf_cache_fork, self.dims, self._per_slot(parent, "fork: parent"), *at, *to)

    def compact(self, into=None):
        """Move the used pages into the lowest page numbers.  Returns their number (int32 [1]).
        ``into``: (page_table, ref) to write instead of the cache's own."""
        table, ref = self._table_at(0), self._table_at(2)
        to = (table, ref)
        if into is not None:
            to = (self._need(into[0], self._shapes[0], torch.int32, "compact: into"),
                  self._need(into[1], self._shapes[2], torch.int32, "compact: into"))
        n_used = torch.empty(1, dtype=torch.int32, device=self.device)
        self._call(B.saf_cache_compact, self.dims, self._pool_at(), self.page_bytes, table, ref,
                   *to, n_used.data_ptr(), self._pages_ws.data_ptr(), self._pages_bytes)
        return n_used

    def device_status(self):
        return B.saf_get_device_status(_ptr(self.workspace), 0, _stream(self.device))


class _OnDevice:
    """What the classes below share: their device, checks of arguments, the call itself."""

    def _place(self, device):
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index

    def _bad(self, what):
        return B.SafError(B.SAF_ERR_INVALID_ARG, what)

    def _counts(self, what, *counts):
        """Refuses what the C structs' ints do not hold (ctypes would cut it)."""
        for n in counts:
            if not 0 <= n < 1 << 31:
                raise self._bad(f"{what}: {n} is out of range")

    # (get_device of a CPU tensor is -1: no device of ours)
    def _need(self, t, shape, dtype, what):
        """The address of a contiguous tensor of this shape, type and device."""
        if (t.dtype is not dtype or t.get_device() != self._index or t.shape != shape
                or not t.is_contiguous()):
            raise self._bad(f"{what}: want a contiguous {dtype} tensor {tuple(shape)} on "
                            f"{self.device}")
        return t.data_ptr()

    def _rows(self, t, shape, dtype, what):
        """saf_rows of [total, heads, d] or [B, heads, T, d] rows in any order."""
        st = t.stride()
        if (t.dtype is not dtype or t.get_device() != self._index or t.shape != shape
                or (st[-1] != 1 and shape[-1] != 1)):
            raise self._bad(f"{what}: want a {dtype} tensor {tuple(shape)} on {self.device} "
                            "whose rows are contiguous")
        if len(st) == 3:
            return B.saf_rows(t.data_ptr(), 0, st[0], st[1])
        return B.saf_rows(t.data_ptr(), st[0], st[2], st[1])

    def _fresh(self, shape):
        """New bf16 rows [total, heads, d] and their saf_rows (which need no checks: those of three
        tensors take 2 us of a call)."""
        t = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        return t, B.saf_rows(t.data_ptr(), 0, shape[1] * shape[2], shape[2])

    def _call(self, entry, *args):
        """The C entry on this object's device and its current stream."""
        if torch.cuda.current_device() == self._index:
            st = entry(*args, _raw_stream(self._index))
        else:
            with torch.cuda.device(self.device):
                st = entry(*args, _raw_stream(self._index))
        if st != B.SAF_OK:
            raise B.SafError(st, entry.__name__)


def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, stretch: float = 1.0,
                       kind: str = "ramp", trained: int = 4096, slow: float = 1.0,
                       fast: float = 32.0):
    """Radians a token of each of the rot_dim / 2 turned pairs, in 64 bits: base^(-2 j / rot_dim),
    for contexts ``stretch`` times longer than the ``trained`` one changed by ``kind``:

    * ``linear``  every frequency divided by ``stretch``
    * ``base``    a larger base, so that the slowest pair is divided by ``stretch`` and the
                  fastest stays
    * ``ramp``    pairs with at least ``fast`` turns over the trained context stay, those with at
                  most ``slow`` are divided by ``stretch``, those between are mixed
    """
    if rot_dim < 2 or rot_dim % 2 or base <= 0 or stretch <= 0 or trained < 1 or fast <= slow:
        raise B.SafError(B.SAF_ERR_INVALID_ARG, "rotary_frequencies")
    if kind not in ("linear", "base", "ramp"):
        raise B.SafError(B.SAF_ERR_INVALID_ARG, f"rotary_frequencies: kind {kind!r}")
    if kind == "base" and stretch != 1.0:
        if rot_dim < 4:
            raise B.SafError(B.SAF_ERR_INVALID_ARG, "rotary_frequencies: one pair has no base")
        base = base * stretch ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * np.arange(rot_dim // 2, dtype=np.float64) / rot_dim)
    if kind == "base" or stretch == 1.0:
        return f
    if kind == "linear":
        return f / stretch
    keep = np.clip((trained * f / (2.0 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
    return np.where(keep == 1.0, f, f * keep + f / stretch * (1.0 - keep))


class Rotary(_OnDevice):
    """Rotary positions for Q and K: pairs of components turned by position times frequency.

    ``freqs`` are the frequencies (radians a token, one for each turned pair: see
    rotary_frequencies); without it they are those of ``rot_dim`` (default: d_h) and ``base``.
    The first 2 * len(freqs) components of a row are turned, the rest copied.  ``layout`` is
    "half" (pairs j, j + rot_dim / 2) or "interleaved" (2 j, 2 j + 1); the turned pairs are
    multiplied by ``scale``.  Angles are exact modulo a turn at any position.
    """

    def __init__(self, d_h: int, *, rot_dim=None, base: float = 10000.0, freqs=None,
                 layout: str = "half", scale: float = 1.0, device="cuda"):
        self._place(device)
        if freqs is None:
            freqs = rotary_frequencies(d_h if rot_dim is None else rot_dim, base)
        freqs = [float(f) for f in freqs]
        if rot_dim is not None and rot_dim != 2 * len(freqs):
            raise self._bad(f"Rotary: {len(freqs)} frequencies for rot_dim {rot_dim}")
        if layout not in ("half", "interleaved"):
            raise self._bad(f"Rotary: layout {layout!r}")
        if not freqs or 2 * len(freqs) > d_h:
            raise self._bad(f"Rotary: {len(freqs)} pairs in {d_h} components")
        st, turns = B.saf_rotary_turns(freqs)
        _check(st, "saf_rotary_turns")
        self.d_h, self.rot_dim, self.layout, self.scale = d_h, 2 * len(freqs), layout, scale
        self._flags = B.SAF_ROTARY_INTERLEAVED if layout == "interleaved" else 0
        self.turns = torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).to(
            self.device)

    def apply(self, q, k=None, *, positions=None, cu_seqlens=None, seq_len=None, n_new=None,
              out=None, inverse=False):
        """q [total, H, d_h] (packed rows) or [B, H, T, d_h] (as the layer and the cache take
        them), k the same with its own heads or None, bf16 or fp32, rows in any order.  Row t of
        a sequence is at position t; or as ``positions`` ([total] or [B, T] int32) says; or
        counted from its sequence's start in ``cu_seqlens`` [n + 1] (packed rows); or at
        seq_len - n_new + t as in PagedCache.append.  Returns (q, k) turned, in new tensors or in
        ``out`` (a pair; (q, k) itself for in place).  Rows of no sequence and rows behind n_new
        are left as they were in ``out``, 0 in new tensors.  ``inverse`` turns back: applied to
        the gradients of the results it gives those of q and k."""
        shape, dtype = q.shape, q.dtype
        packed = len(shape) == 3
        if not packed and len(shape) != 4:
            raise self._bad("apply: q is neither [total, H, d_h] nor [B, H, T, d_h]")
        if dtype is torch.bfloat16:
            code = B.SAF_BF16
        elif dtype is torch.float32:
            code = B.SAF_F32
        else:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "apply: q is neither bf16 nor fp32")
        d = self.d_h
        if packed:
            B_, (T, H, last) = 1, shape
        else:
            B_, H, T, last = shape
        if last != d:
            raise self._bad(f"apply: rows of {last} components, d_h is {d}")
        self._counts("apply: rows", B_, T, H)
        rq = self._rows(q, shape, dtype, "apply: q")
        rk = k_shape = None
        H_k = 0
        if k is not None:
            k_shape = k.shape
            if len(k_shape) != len(shape):
                raise self._bad("apply: k has another number of dimensions than q")
            H_k = k_shape[1]
            rk = self._rows(k, (T, H_k, d) if packed else (B_, H_k, T, d), dtype, "apply: k")
        flags = self._flags | B.SAF_ROTARY_INVERSE if inverse else self._flags
        ok = None
        if out is None:
            flags |= B.SAF_CLEAR_REST
            new_q, new_k = torch.empty(shape, dtype=dtype, device=self.device), None
            if k is not None:
                new_k = torch.empty(k_shape, dtype=dtype, device=self.device)
            # (rows of new tensors need no checks: they are a third of the call's host part)
            if packed:
                oq = B.saf_rows(new_q.data_ptr(), 0, H * d, d)
                if k is not None:
                    ok = B.saf_rows(new_k.data_ptr(), 0, H_k * d, d)
            else:
                oq = B.saf_rows(new_q.data_ptr(), H * T * d, d, T * d)
                if k is not None:
                    ok = B.saf_rows(new_k.data_ptr(), H_k * T * d, d, T * d)
            out = new_q, new_k
        elif (out[1] is None) != (k is None):
            raise self._bad("apply: out is not a pair like (q, k)")
        else:
            oq = self._rows(out[0], shape, dtype, "apply: out")
            if k is not None:
                ok = self._rows(out[1], k_shape, dtype, "apply: out")
        at = cu = lens = new = None
        n = 0
        if positions is not None:
            if cu_seqlens is not None or seq_len is not None:
                raise self._bad("apply: positions are given in more than one way")
            at = self._need(positions, (T,) if packed else (B_, T), torch.int32,
                            "apply: positions")
        elif cu_seqlens is not None:
            if seq_len is not None:
                raise self._bad("apply: positions are given in more than one way")
            cu_shape = cu_seqlens.shape
            if not packed or len(cu_shape) != 1 or cu_shape[0] < 1:
                raise self._bad("apply: cu_seqlens [n + 1] goes with packed rows")
            n = cu_shape[0] - 1
            self._counts("apply: sequences", n)
            cu = self._need(cu_seqlens, cu_shape, torch.int32, "apply: cu_seqlens")
        elif seq_len is not None:
            lens = self._need(seq_len, (B_,), torch.int32, "apply: seq_len")
        if n_new is not None:
            new = self._need(n_new, (B_,), torch.int32, "apply: n_new")
        self._call(B.saf_rotary, B.saf_rotary_dims(B_, T, H, H_k, d, self.rot_dim, code), rq, rk,
                   oq, ok, self.turns.data_ptr(), self.scale, at, cu, n, lens, new, flags)
        return out


class PackedAttention(_OnDevice):
    """The hybrid causal attention layer on sequences of different lengths laid end to end.

    Rows cu_seqlens[s] <= i < cu_seqlens[s + 1] (int32 [n + 1] on the GPU) of q [total, H, d_h]
    and k, v [total, H_kv, d_h] (bf16, rows in any order: views of one projection's output will
    do) are sequence s; frozen heads (``head_is_static``, host booleans) count their pattern's
    positions from its first row.  A call has at most ``max_total`` rows and ``max_seqs``
    sequences of at most ``max_len`` rows; with ``backward`` the workspace has room for the
    gradients' sums.  Every call makes the frozen heads' tables for ``max_len`` rows, so it had
    better be near the longest sequence (with it at 4096 they take 2 us beside the rest; at 131072 a
    call on short prompts takes 0.3 ms, and 33 where alpha + rho range over more than 80).
    Nothing synchronises, and every call can be captured in a CUDA graph.
    Calls share the object's workspace, so they belong on one stream at a time.
    """

    def __init__(self, H: int, d_h: int, head_is_static, *, max_total: int, max_seqs: int,
                 max_len: int, H_kv=None, backward: bool = True, device="cuda"):
        self._place(device)
        self.H, self.d_h, self.H_kv = H, d_h, H if H_kv is None else H_kv
        self._counts("PackedAttention", max_total, max_seqs, max_len, H, self.H_kv, d_h)
        self.max_total, self.max_seqs, self.max_len = max_total, max_seqs, max_len
        self.head_is_static = bytes(int(bool(x)) for x in head_is_static)
        if len(self.head_is_static) != H:
            raise self._bad(f"PackedAttention: a mask of {len(self.head_is_static)} heads")
        self._frozen = any(self.head_is_static)
        self.ws_bytes = B.saf_packed_attn_workspace_size(
            B.saf_packed_dims(max_total, max_seqs, max_len, H, self.H_kv, d_h, max_len), backward)
        if self.ws_bytes == 0:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "saf_packed_attn_workspace_size")
        self._backward = backward
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.workspace[:256].zero_()  # the status before the first call

    def _common(self, q, cu_seqlens, alpha, rho):
        """(dims, cu_seqlens, alpha, rho) as the C entries take them."""
        shape, n = q.shape, cu_seqlens.shape
        if len(shape) != 3 or shape[0] > self.max_total:
            raise self._bad(f"PackedAttention: q is not [total, H, d_h], total <= {self.max_total}")
        if len(n) != 1 or not 1 <= n[0] <= self.max_seqs + 1:
            raise self._bad(f"PackedAttention: want cu_seqlens [n + 1], n <= {self.max_seqs}")
        cu = self._need(cu_seqlens, n, torch.int32, "PackedAttention: cu_seqlens")
        pa = pr = None
        T = 0
        if self._frozen:
            if alpha is None or rho is None:
                raise self._bad("PackedAttention: frozen heads need alpha and rho")
            T = alpha.shape[-1] if alpha.dim() == 2 else -1
            if not self.max_len <= T < 1 << 31:
                raise self._bad(f"PackedAttention: {T} columns of alpha, max_len {self.max_len}")
            pa = self._need(alpha, (self.H, T), torch.float32, "PackedAttention: alpha")
            pr = self._need(rho, (self.H, T), torch.float32, "PackedAttention: rho")
        return B.saf_packed_dims(shape[0], n[0] - 1, self.max_len, self.H, self.H_kv, self.d_h,
                                 T), cu, pa, pr

    def forward(self, q, k, v, cu_seqlens, alpha=None, rho=None, out=None, lse=None):
        """(out [total, H, d_h], lse [H, total] fp32).  Rows of no sequence are left as they were
        in buffers that are given, 0 and -inf in those that the call makes.  alpha, rho
        [H, >= max_len] fp32 are needed where heads are frozen."""
        dims, cu, pa, pr = self._common(q, cu_seqlens, alpha, rho)
        total, bf16 = dims.total, torch.bfloat16
        wide, narrow = (total, self.H, self.d_h), (total, self.H_kv, self.d_h)
        flags = 0
        if out is None and lse is None:
            # both are new: the call itself clears what it does not work on
            flags = B.SAF_CLEAR_REST
            out, po = self._fresh(wide)
            lse = torch.empty((self.H, total), dtype=torch.float32, device=self.device)
            pl = lse.data_ptr()
        else:
            if out is None:
                out = torch.zeros(wide, dtype=bf16, device=self.device)
            if lse is None:
                lse = torch.full((self.H, total), -math.inf, device=self.device)
            po = self._rows(out, wide, bf16, "forward: out")
            pl = self._need(lse, (self.H, total), torch.float32, "forward: lse")
        rows = self._rows
        self._call(B.saf_packed_attn_fwd, dims, rows(q, wide, bf16, "forward: q"),
                   rows(k, narrow, bf16, "forward: k"), rows(v, narrow, bf16, "forward: v"), cu,
                   pa, pr, self.head_is_static, po, pl, flags, self.workspace.data_ptr(),
                   self.ws_bytes)
        return out, lse

    def backward(self, q, k, v, out, lse, dout, cu_seqlens, alpha=None, rho=None, grads=None):
        """(dq, dk, dv) for the gradient dout of out; out and lse are the forward's.  Written to
        ``grads`` (a triple; rows of no sequence are left as they were) or to new tensors."""
        if not self._backward:
            raise B.SafError(B.SAF_ERR_STATE, "backward: made with backward=False")
        dims, cu, pa, pr = self._common(q, cu_seqlens, alpha, rho)
        total, bf16 = dims.total, torch.bfloat16
        wide, narrow = (total, self.H, self.d_h), (total, self.H_kv, self.d_h)
        rows, flags = self._rows, 0
        if grads is None:
            flags = B.SAF_CLEAR_REST
            (dq, pq), (dk, pk), (dv, pv) = self._fresh(wide), self._fresh(narrow), self._fresh(narrow)
        else:
            dq, dk, dv = grads
            pq = rows(dq, wide, bf16, "backward: dq")
            pk = rows(dk, narrow, bf16, "backward: dk")
            pv = rows(dv, narrow, bf16, "backward: dv")
        self._call(B.saf_packed_attn_bwd, dims, rows(q, wide, bf16, "backward: q"),
                   rows(k, narrow, bf16, "backward: k"), rows(v, narrow, bf16, "backward: v"),
                   rows(out, wide, bf16, "backward: out"),
                   self._need(lse, (self.H, total), torch.float32, "backward: lse"),
                   rows(dout, wide, bf16, "backward: dout"), cu, pa, pr, self.head_is_static,
                   pq, pk, pv, flags, self.workspace.data_ptr(), self.ws_bytes)
        return dq, dk, dv

    def device_status(self):
        return B.saf_get_device_status(_ptr(self.workspace), 0, _stream(self.device))


class BeamSearch(_OnDevice):
    """Beam search over ``n_groups`` sequences with ``beams`` slots each (slot g * beams + b).

        parent, token, scores, finished, history = search.step(
            logits, scores, finished, history=history, n_tokens=n)
        cache.fork(parent)

    ``end`` is the token that ends a sequence (None: no token does).  Calls share the object's
    workspace, so they belong on one stream at a time.
    """

    def __init__(self, n_groups: int, beams: int, vocab: int, *, end=None, device="cuda"):
        self._place(device)
        self.n_groups, self.beams, self.vocab = n_groups, beams, vocab
        self.end, self.slots = end, n_groups * beams
        self._counts("BeamSearch", n_groups, beams, vocab, 0 if end is None else end)
        if n_groups < 1:
            raise self._bad(f"BeamSearch: {n_groups} groups")
        with torch.cuda.device(self.device):
            self.ws_bytes = B.saf_beam_workspace_size(
                B.saf_beam_dims(n_groups, beams, vocab, vocab, B.SAF_F32,
                                -1 if end is None else end, 0))
        if self.ws_bytes == 0:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "saf_beam_workspace_size")
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._whole = torch.empty(self.slots, dtype=torch.int32, device=self.device)  # a shape

    def step(self, logits, scores, finished=None, *, history=None, n_tokens=None,
             history_out=None):
        """logits [slots, vocab] (bf16 or fp32, rows any distance apart), scores [slots] fp32,
        finished [slots] bool or None, history [slots, columns] int32 with ``n_tokens`` [1] int32
        columns filled.  Returns (parent, token, scores, finished, history): the new slots, best
        first in each group; finished is None without an ending token, history None without one.
        The history is written to ``history_out`` (not the same tensor), as far as it is filled."""
        slots, dtype, st = self.slots, logits.dtype, logits.stride()
        n = (slots,)
        if dtype is torch.float32:
            code = B.SAF_F32
        elif dtype is torch.bfloat16:
            code = B.SAF_BF16
        else:
            raise B.SafError(B.SAF_ERR_UNSUPPORTED, "step: logits are neither bf16 nor fp32")
        if (logits.shape != (slots, self.vocab) or logits.get_device() != self._index
                or (st[1] != 1 and self.vocab > 1) or (st[0] < self.vocab and slots > 1)):
            raise self._bad(f"step: want logits [{slots}, {self.vocab}] on {self.device} whose "
                            "rows are contiguous and apart")
        ps = self._need(scores, n, torch.float32, "step: scores")
        pf = None
        if finished is not None:
            if self.end is None:
                raise self._bad("step: finished slots without an ending token")
            pf = self._need(finished, n, torch.bool, "step: finished")
        ph = pn = po = None
        columns = 0
        if history is not None:
            shape = history.shape
            if n_tokens is None or len(shape) != 2 or shape[0] != slots:
                raise self._bad("step: history [slots, columns] needs n_tokens")
            columns = shape[1]
            self._counts("step: columns", columns)
            if history_out is None:
                history_out = torch.full_like(history, -1)
            ph = self._need(history, shape, torch.int32, "step: history")
            po = self._need(history_out, shape, torch.int32, "step: history_out")
            pn = self._need(n_tokens, (1,), torch.int32, "step: n_tokens")
        elif history_out is not None:
            raise self._bad("step: history_out without a history")
        parent, token = torch.empty_like(self._whole), torch.empty_like(self._whole)
        score = torch.empty_like(scores)
        done = pd = None
        end = -1
        if self.end is not None:
            end = self.end
            done = torch.empty(n, dtype=torch.bool, device=self.device)
            pd = done.data_ptr()
        dims = B.saf_beam_dims(self.n_groups, self.beams, self.vocab,
                               st[0] if slots > 1 else self.vocab, code, end, columns)
        self._call(B.saf_beam_step, dims, logits.data_ptr(), ps, pf, ph, pn, parent.data_ptr(),
                   token.data_ptr(), score.data_ptr(), pd, po, self.workspace.data_ptr(),
                   self.ws_bytes)
        return parent, token, score, done, history_out


def fit_compact(A_hat, candidates, k, kl_max=0.2, steps=400, lr=1e-2):
    """Fit alpha/rho to A_hat [num_heads, T, T] for each candidate head (device
    int32, priority order) and select the first k that pass the KL gate.
    Returns (alpha [n, T], rho [n, T], kl [n], selected [n_selected])."""
    num_heads, T, _ = A_hat.shape
    n = candidates.numel()
    dev = A_hat.device
    alpha = torch.empty((n, T), dtype=torch.float32, device=dev)
    rho = torch.empty((n, T), dtype=torch.float32, device=dev)
    kl = torch.empty(n, dtype=torch.float32, device=dev)
    sel = torch.empty(max(k, 1), dtype=torch.int32, device=dev)
    n_sel = torch.zeros(1, dtype=torch.int32, device=dev)
    st = B.saf_fit_compact(_ptr(A_hat), num_heads, T, _ptr(candidates), n, k, kl_max, steps, lr,
                           _ptr(alpha), _ptr(rho), _ptr(kl), _ptr(sel), _ptr(n_sel),
                           _stream(dev))
    _check(st, "saf_fit_compact")
    return alpha, rho, kl, sel[: int(n_sel.item())]


def num_select(r: float, num_heads: int) -> int:
    return B.saf_calib_num_select(r, num_heads)
