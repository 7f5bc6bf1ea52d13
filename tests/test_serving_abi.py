"""Rotary positions, the beam step and the packed attention refuse what they cannot take before any
CUDA work, and what runs on the host alone is right (no GPU needed)."""

import math
import os
from fractions import Fraction

import numpy as np
import pytest


@pytest.fixture(scope="module")
def B():
    from dynamic_causal_attention_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from dynamic_causal_attention_gb300 import _binding
    return _binding


@pytest.fixture(scope="module")
def api(B):
    from dynamic_causal_attention_gb300 import api
    return api


# ------------------------------------------------------------------ rotary positions
def test_turns_are_fractions_of_a_turn_to_53_bits(B):
    radians = [1.0, 0.5, 1e-4, 1e-12, 2 * math.pi, 7.0, -0.25, 0.0, 500000.0 ** -0.5]
    st, turns = B.saf_rotary_turns(radians)
    assert st == B.SAF_OK
    for r, t in zip(radians, turns):
        # what a double holds of r / 2 pi, modulo 1
        want = Fraction(r / 6.283185307179586) % 1
        diff = (Fraction(t, 1 << 64) - want) % 1
        assert min(diff, 1 - diff) <= Fraction(1, 1 << 63) + abs(Fraction(r)) / (1 << 52), r
    assert B.saf_rotary_turns([])[0] == B.SAF_OK
    for bad in (math.nan, math.inf):
        assert B.saf_rotary_turns([1.0, bad])[0] == B.SAF_ERR_INVALID_ARG


def test_frequencies(api):
    f = api.rotary_frequencies(64, 10000.0)
    assert f[0] == 1.0 and np.allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert np.array_equal(api.rotary_frequencies(64, kind="linear", stretch=4.0), f / 4)
    g = api.rotary_frequencies(64, kind="base", stretch=4.0)
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    r = api.rotary_frequencies(64, kind="ramp", stretch=8.0, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(r[turns >= 32], f[turns >= 32])
    assert np.allclose(r[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    assert np.all(np.diff(r) < 0)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(base=0.0), dict(stretch=-1.0),
                dict(kind="other"), dict(fast=1.0), dict(rot_dim=2, kind="base", stretch=2.0)):
        with pytest.raises(api.SafError):
            api.rotary_frequencies(**{"rot_dim": 64, **bad})


def test_rotary_refusals(B):
    rows = lambda **kw: B.saf_rows(**{**dict(p=16, seq=4096, row=256, head=64), **kw})
    ok = dict(dims=dict(B=2, T=8, H=4, H_k=2, d_h=64, rot=64, dtype=0), q=rows(), k=rows(),
              q_out=rows(p=1 << 20), k_out=rows(p=1 << 21), turns=16, scale=1.0, positions=None,
              cu=None, n_seqs=0, seq_len=None, n_new=None, flags=0)

    def call(**kw):
        a = {**ok, **kw}
        d = None if a["dims"] is None else B.saf_rotary_dims(**{**ok["dims"], **a["dims"]})
        return B.saf_rotary(d, a["q"], a["k"], a["q_out"], a["k_out"], a["turns"], a["scale"],
                            a["positions"], a["cu"], a["n_seqs"], a["seq_len"], a["n_new"],
                            a["flags"], None)
    for bad in (dict(dims=None), dict(dims=dict(rot=63)), dict(dims=dict(rot=66)),
                dict(dims=dict(rot=0)), dict(dims=dict(B=-1)), dict(dims=dict(dtype=7)),
                dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(turns=None),
                dict(turns=12), dict(scale=math.nan), dict(flags=8), dict(q=rows(p=None)),
                dict(q=rows(p=17)), dict(q=rows(row=-64)), dict(q_out=rows(row=0)),
                dict(k_out=rows(head=32)), dict(q_out=rows(seq=8)),
                dict(q=rows(p=1 << 20, row=512)),         # in place with other strides
                dict(positions=16, seq_len=16), dict(positions=16, cu=16), dict(n_new=16),
                dict(positions=18), dict(seq_len=16, n_new=17), dict(cu=16, n_seqs=1),
                dict(n_seqs=-1)):
        assert call(**bad) == B.SAF_ERR_INVALID_ARG, bad
    for bad in (dict(d_h=512), dict(H=300), dict(H_k=257), dict(B=1 << 20, T=1 << 12)):
        assert call(dims=bad) == B.SAF_ERR_UNSUPPORTED, bad
    # nothing to do: no pointer is looked at
    for d in (dict(B=0), dict(T=0), dict(H=0, H_k=0)):
        assert call(dims=d, q=None, k=None, q_out=None, k_out=None, turns=None) == B.SAF_OK


def test_rotary_outputs_must_not_run_into_themselves(B):
    rows = lambda **kw: B.saf_rows(**{**dict(p=1 << 20, seq=4096, row=256, head=64), **kw})
    dims = B.saf_rotary_dims(2, 8, 4, 0, 64, 64, 0)
    call = lambda out: B.saf_rotary(dims, rows(p=16), None, out, None, 16, 1.0, None, None, 0, None,
                                    None, 0, None)
    for bad in (dict(row=64), dict(row=192), dict(head=256), dict(seq=64), dict(seq=1984),
                dict(row=64, head=448), dict(seq=64, row=128, head=1023), dict(row=1 << 62, seq=1 << 62)):
        assert call(rows(**bad)) == B.SAF_ERR_INVALID_ARG, bad


def test_counts_beyond_an_int_are_refused(api):
    big = (1 << 32) + 8
    for bad in (dict(max_total=big), dict(max_seqs=big), dict(max_len=big), dict(max_total=-1)):
        with pytest.raises(api.SafError, match="out of range"):
            api.PackedAttention(2, 64, [0, 0], **{**dict(max_total=8, max_seqs=1, max_len=8), **bad},
                                device="cpu")
    for n in ((big, 1, 100), (1, big, 100), (1, 1, big)):
        with pytest.raises(api.SafError, match="out of range"):
            api.BeamSearch(*n, device="cpu")
    with pytest.raises(api.SafError, match="out of range"):
        api.BeamSearch(1, 1, 100, end=big, device="cpu")
    import torch
    turn = api.Rotary(2, device="cpu")
    with pytest.raises(api.SafError, match="out of range"):
        turn.apply(torch.zeros(1, 1, 2).expand(big, 1, 2))


def test_rotary_objects_refuse(api):
    for bad in (dict(layout="pairs"), dict(freqs=[]), dict(freqs=[1.0] * 40), dict(rot_dim=62, freqs=[1.0]),
                dict(freqs=[math.inf])):
        with pytest.raises(api.SafError):
            api.Rotary(64, device="cpu", **bad)


# ------------------------------------------------------------------ beam step
BEAM = dict(n_groups=3, beams=4, vocab=1000, row_stride=1000, dtype=1, end=2, max_tokens=16)


def test_beam_refusals(B):
    ok = dict(logits=16, scores=16, finished=16, history=16, n_tokens=16, parent=16, token=16,
              score_out=16, finished_out=16, history_out=64, ws=256, ws_bytes=1 << 40)

    def call(dims=None, **kw):
        a = {**ok, **kw}
        return B.saf_beam_step(B.saf_beam_dims(**{**BEAM, **(dims or {})}), *[a[k] for k in ok], None)
    for bad in (dict(n_groups=-1), dict(beams=0), dict(vocab=0), dict(row_stride=999),
                dict(dtype=5), dict(end=1000), dict(end=-2), dict(max_tokens=-1)):
        assert call(bad) == B.SAF_ERR_INVALID_ARG, bad
        assert B.saf_beam_workspace_size(B.saf_beam_dims(**{**BEAM, **bad})) == 0
    for bad in (dict(beams=33), dict(vocab=(1 << 22) + 1, row_stride=1 << 23),
                dict(n_groups=1 << 28)):
        assert call(bad) == B.SAF_ERR_UNSUPPORTED, bad
        assert B.saf_beam_workspace_size(B.saf_beam_dims(**{**BEAM, **bad})) == 0
    for bad in (dict(logits=None), dict(logits=18), dict(scores=None), dict(scores=2),
                dict(parent=None), dict(token=None), dict(token=6), dict(score_out=None),
                dict(history=None), dict(history_out=None), dict(n_tokens=None),
                dict(history_out=16), dict(n_tokens=3), dict(ws=None), dict(ws=128),
                dict(ws_bytes=64)):
        assert call(**bad) == B.SAF_ERR_INVALID_ARG, bad
    assert call(dict(end=-1)) == B.SAF_ERR_INVALID_ARG       # finished slots without an end
    assert call(dict(max_tokens=0)) == B.SAF_ERR_INVALID_ARG  # a history without columns
    assert call(dict(n_groups=0), **{k: None for k in ok if k != "ws_bytes"}) == B.SAF_OK


# ------------------------------------------------------------------ packed attention
PACKED = dict(total=500, n_seqs=3, max_len=300, H=4, H_kv=2, d_h=64, T_pat=300)
MASK = bytes([0, 0, 1, 0])


class Statuses:
    """The forward's status [0] and the backward's [1].  A call is made when its status is asked
    for: one that is not to be refused would, with a GPU at hand, run on addresses that are none."""

    def __init__(self, B, fwd, bwd):
        self.calls, self.launched = (fwd, bwd), B.SAF_ERR_CUDA

    def __getitem__(self, i):
        status = self.calls[i]()
        assert status != self.launched, "not refused: a launch was tried"
        return status

    def __eq__(self, other):
        return (self[0], self[1]) == other


def packed_calls(B, dims=None, rows=None, **kw):
    d = None if dims is None and kw.pop("no_dims", False) else \
        B.saf_packed_dims(**{**PACKED, **(dims or {})})
    r = lambda name: (rows or {}).get(name, B.saf_rows(p=16, seq=0, row=512, head=64))
    ok = dict(cu=16, alpha=16, rho=16, mask=MASK, lse=16, flags=0, ws=256, ws_bytes=1 << 45)
    a = {**ok, **kw}
    return Statuses(
        B,
        lambda: B.saf_packed_attn_fwd(d, r("q"), r("k"), r("v"), a["cu"], a["alpha"], a["rho"],
                                      a["mask"], r("out"), a["lse"], a["flags"], a["ws"],
                                      a["ws_bytes"], None),
        lambda: B.saf_packed_attn_bwd(d, r("q"), r("k"), r("v"), r("out"), a["lse"], r("dout"),
                                      a["cu"], a["alpha"], a["rho"], a["mask"], r("dq"), r("dk"),
                                      r("dv"), a["flags"], a["ws"], a["ws_bytes"], None))


def test_packed_refusals(B):
    for bad, status in ((dict(total=-1), 1), (dict(n_seqs=-1), 1), (dict(max_len=-1), 1),
                        (dict(H=0), 1), (dict(H_kv=3), 1), (dict(H_kv=0), 1), (dict(d_h=0), 1),
                        (dict(d_h=48), 2), (dict(d_h=256), 2), (dict(H=512), 2),
                        (dict(n_seqs=1 << 21), 2), (dict(max_len=131073), 2),
                        (dict(total=1 << 30), 2)):
        assert packed_calls(B, bad) == (status, status), bad
        for back in (0, 1):
            assert B.saf_packed_attn_workspace_size(B.saf_packed_dims(**{**PACKED, **bad}), back) == 0
    both = (B.SAF_ERR_INVALID_ARG,) * 2
    for bad in (dict(cu=None), dict(cu=18), dict(alpha=None), dict(rho=None), dict(rho=6),
                dict(mask=None), dict(flags=1), dict(flags=8), dict(ws=None), dict(ws=64),
                dict(ws_bytes=1000), dict(lse=2), dict(dims=dict(T_pat=299)), dict(no_dims=True)):
        assert packed_calls(B, **bad) == both, bad
    assert packed_calls(B, lse=None)[1] == B.SAF_ERR_INVALID_ARG
    R = lambda **kw: B.saf_rows(**{**dict(p=16, seq=0, row=512, head=64), **kw})
    for bad in (None, R(p=None), R(p=24), R(row=500), R(row=32), R(head=68), R(head=0)):
        for name in ("q", "k", "v"):
            assert packed_calls(B, rows={name: bad}) == both, (name, bad)
        for name in ("dout", "dq", "dk", "dv"):
            assert packed_calls(B, rows={name: bad})[1] == B.SAF_ERR_INVALID_ARG, (name, bad)
        assert packed_calls(B, rows={"out": bad})[0] == B.SAF_ERR_INVALID_ARG
    # rows of an output that run into one another
    for name in ("dq", "dk", "dv"):
        assert packed_calls(B, rows={name: R(row=64, head=128)})[1] == B.SAF_ERR_INVALID_ARG
    assert packed_calls(B, rows={"out": R(row=128, head=64)})[0] == B.SAF_ERR_INVALID_ARG
    # nothing to do
    none = dict(cu=None, alpha=None, rho=None, mask=None, lse=None, ws=None)
    rows = dict.fromkeys(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))
    assert packed_calls(B, dict(total=0), rows, **none) == (B.SAF_OK,) * 2


def test_packed_workspace_never_grows_with_less(B):
    size = lambda back, **kw: B.saf_packed_attn_workspace_size(
        B.saf_packed_dims(**{**PACKED, "total": 5000, "n_seqs": 40, "max_len": 3000, **kw}), back)
    for back in (0, 1):
        full = size(back)
        assert 0 < size(0) <= full
        for less in (dict(total=4999), dict(total=100), dict(n_seqs=39), dict(n_seqs=0),
                     dict(max_len=2872), dict(max_len=1), dict(total=0)):
            assert 0 < size(back, **less) <= full, less


def test_rotary_outputs_in_the_place_of_the_other_tensor(B):
    """q_out where k or k_out lies, and the other way round: threads of other heads would read what
    is written."""
    rows = lambda p: B.saf_rows(p, 4096, 256, 64)
    q, k, a, b = rows(1 << 20), rows(1 << 21), rows(1 << 22), rows(1 << 23)
    dims = B.saf_rotary_dims(2, 8, 4, 4, 64, 64, 0)
    for out_q, out_k in ((a, a), (q, q), (k, q), (k, k), (k, b), (a, q)):
        assert B.saf_rotary(dims, q, k, out_q, out_k, 16, 1.0, None, None, 0, None, None, 0,
                            None) == B.SAF_ERR_INVALID_ARG
    # one tensor for both, each in its own place
    assert B.saf_rotary(dims, q, q, q, q, 16, 1.0, None, None, 0, None, None, 0,
                        None) == B.SAF_ERR_INVALID_ARG
