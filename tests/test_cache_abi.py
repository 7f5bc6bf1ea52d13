"""The paged cache's calls refuse what they cannot take before any CUDA work, and the layout of
a record is what the header says (no GPU needed)."""

import os

import numpy as np
import pytest

import cache_reference as ref


@pytest.fixture(scope="module")
def B():
    from dynamic_causal_attention_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from dynamic_causal_attention_gb300 import _binding
    return _binding


def dims(B, n_seqs=2, max_pages=4, n_pages=8, page_size=64, H=4, H_kv=2, d_h=64,
         page_stride=1 << 20):
    return B._cache_dims(n_seqs, max_pages, n_pages, page_size, H, H_kv, d_h, page_stride)


MASK = bytes([0, 0, 1, 0])
BAD_DIMS = [(dict(n_seqs=-1), 1), (dict(max_pages=0), 1), (dict(n_pages=0), 1),
            (dict(page_size=0), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(H_kv=0), 1),
            (dict(d_h=0), 1), (dict(page_stride=1 << 20 | 8), 1),
            (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(d_h=48), 2),
            (dict(d_h=256), 2), (dict(H=512, H_kv=2), 2), (dict(n_seqs=40000), 2),
            (dict(max_pages=1 << 25), 2)]


def calls(B, d):
    """Each entry point with arguments that pass every check but those of `d`."""
    return {
        "append": lambda: B.saf_cache_append(d, MASK, 16, 16, 16, 0, 1, 16, 16, 16, None),
        "attn": lambda: B.saf_cache_attn(d, MASK, 16, 16, 16, 16, 8, 1, 16, 16, 16, 16, 16, 256,
                                         1 << 40, None),
        "fork": lambda: B.saf_cache_fork(d, 16, 16, 16, 16, 16, 16, 16, None),
        "grow": lambda: B.saf_cache_grow(d, 16, 1024, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16,
                                         1 << 40, None),
        "compact": lambda: B.saf_cache_compact(d, 16, 1024, 16, 16, 16, 16, 16, 16, 1 << 40, None),
    }


@pytest.mark.parametrize("bad,status", BAD_DIMS)
def test_bad_dims_are_refused_by_every_call(B, bad, status):
    d = dims(B, **bad)
    for name, call in calls(B, d).items():
        assert call() == status, name
    assert B.saf_cache_layer_layout(d, MASK)[0] == status
    assert B.saf_cache_attn_workspace_size(d, 1) == 0
    assert B.saf_cache_pages_workspace_size(d) == 0


def test_attn_refusals(B):
    ok = dict(mask=MASK, layer=16, Q=16, alpha=16, rho=16, T=8, n_q=1, n_new=16, seq_len=16,
              table=16, out=16, lse=16, ws=256, ws_bytes=1 << 40)

    def call(d=None, **kw):
        a = {**ok, **kw}
        return B.saf_cache_attn(d or dims(B), a["mask"], a["layer"], a["Q"], a["alpha"], a["rho"],
                                a["T"], a["n_q"], a["n_new"], a["seq_len"], a["table"], a["out"],
                                a["lse"], a["ws"], a["ws_bytes"], None)
    for bad in (dict(mask=None), dict(layer=None), dict(layer=8), dict(Q=None), dict(Q=24),
                dict(alpha=None), dict(rho=None), dict(rho=20), dict(T=-1), dict(n_q=-1),
                dict(n_new=18), dict(seq_len=None), dict(seq_len=2), dict(table=None),
                dict(out=None), dict(out=24), dict(lse=8), dict(ws=None), dict(ws=128),
                dict(ws_bytes=16)):
        assert call(**bad) == B.SAF_ERR_INVALID_ARG, bad
    # a record longer than the distance between pages
    assert call(dims(B, page_stride=1024)) == B.SAF_ERR_INVALID_ARG
    # rows beyond 31 bits
    assert call(n_q=1 << 30) == B.SAF_ERR_UNSUPPORTED
    assert call(dims(B, H=1, H_kv=1), mask=b"\0", n_q=(1 << 30) + 1) == B.SAF_ERR_UNSUPPORTED
    # nothing to do: no pointer is looked at
    none = {k: None for k in ok if k not in ("T", "n_q", "ws_bytes", "mask")}
    assert call(dims(B, n_seqs=0), **none) == B.SAF_OK
    assert call(n_q=0, **none) == B.SAF_OK
    assert B.saf_last_launch_count() == 0


def test_append_refusals(B):
    ok = dict(mask=MASK, layer=16, K=16, V=16, dtype=0, n_q=1, n_new=16, seq_len=16, table=16)

    def call(d=None, **kw):
        a = {**ok, **kw}
        return B.saf_cache_append(d or dims(B), a["mask"], a["layer"], a["K"], a["V"], a["dtype"],
                                  a["n_q"], a["n_new"], a["seq_len"], a["table"], None)
    for bad in (dict(mask=None), dict(layer=None), dict(layer=40), dict(K=None), dict(K=8),
                dict(V=None), dict(V=24), dict(dtype=2), dict(n_q=-1), dict(n_new=17),
                dict(seq_len=None), dict(table=None), dict(table=6)):
        assert call(**bad) == B.SAF_ERR_INVALID_ARG, bad
    assert call(dims(B, page_stride=1024)) == B.SAF_ERR_INVALID_ARG
    assert call(n_q=1 << 30) == B.SAF_ERR_UNSUPPORTED
    none = dict(layer=None, K=None, V=None, n_new=None, seq_len=None, table=None)
    assert call(dims(B, n_seqs=0), **none) == B.SAF_OK
    assert call(n_q=0, **none) == B.SAF_OK


def test_page_call_refusals(B):
    d = dims(B)
    g = [16, 1024, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 1 << 40, None]
    for at, bad in [(0, None), (0, 8), (1, 1000), (1, (1 << 20) + 16), (2, None), (3, None),
                    (4, 8), (5, None), (6, 24), (7, None), (8, 8), (9, None), (10, None),
                    (11, None), (11, 8), (12, 16)]:
        a = list(g)
        a[at] = bad
        assert B.saf_cache_grow(d, *a) == B.SAF_ERR_INVALID_ARG, (at, bad)
    f = [16] * 7 + [None]
    for at in range(7):
        for bad in (None, 8):
            a = list(f)
            a[at] = bad
            assert B.saf_cache_fork(d, *a) == B.SAF_ERR_INVALID_ARG, (at, bad)
    c = [16, 1024, 16, 16, 16, 16, 16, 16, 1 << 40, None]
    for at, bad in [(0, None), (1, 8), (1, (1 << 20) + 16), (2, None), (3, 8), (4, None), (5, None),
                    (6, None), (7, None), (8, 16)]:
        a = list(c)
        a[at] = bad
        assert B.saf_cache_compact(d, *a) == B.SAF_ERR_INVALID_ARG, (at, bad)
    empty = dims(B, n_seqs=0)
    assert B.saf_cache_fork(empty, *([None] * 8)) == B.SAF_OK
    assert B.saf_cache_grow(empty, None, 1024, *([None] * 10), 0, None) == B.SAF_OK


def test_layout(B):
    for H, H_kv, page, d, frozen in [(4, 2, 64, 64, ()), (4, 2, 16, 32, (2, 3)),
                                     (12, 4, 128, 128, (0, 1, 2, 5)), (3, 3, 32, 64, (0, 1, 2))]:
        mask = bytes(int(h in frozen) for h in range(H))
        st, L = B.saf_cache_layer_layout(dims(B, H=H, H_kv=H_kv, page_size=page, d_h=d), mask)
        assert st == B.SAF_OK
        g = H // H_kv
        h_k = sum(any(not mask[h] for h in range(k * g, k * g + g)) for k in range(H_kv))
        assert L.H_k == h_k and L.v == h_k * page * d
        assert L.k_scale == L.v + H_kv * page * d and L.v_scale == L.k_scale + 4 * h_k
        end = L.v_scale + 4 * H_kv
        assert end <= L.bytes < end + 128 and L.bytes % 128 == 0


def test_reference_codes():
    """The test reference's own e4m3 rounding, against torch's."""
    import torch
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0 ** e
                        for e in range(-12, 10)] + [ref.E4M3[:127], -ref.E4M3[:127],
                                                    (ref.E4M3[:126] + ref.E4M3[1:127]) / 2,
                                                    [0.0, np.nan, np.inf, -np.inf]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x), want)
    for v in (0.0, 448.0, 448.1, 447.9, 1.75, 1.76, 1e-30, 3e38):
        s = ref.block_scale(np.array([v], np.float32))
        assert 448 * s >= np.float32(v) and (s == 2.0 ** -64 or 224 * s < np.float32(v))
