"""Packed attention at its limits: a backward of seconds."""

import math

import pytest
import torch

import packed_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def test_a_short_sequence_behind_seconds_of_work(api):
    """Whole tiles pass the warp that clears the ends of sequences by: behind three sequences of 1024
    whole tiles under 256 heads it waits for the last one's single row for as long as the others
    take, some seconds, and no wait may run out over that.

    Q = K = 0, V = dO = 1, so P = 1 / (i + 1), out = 1, dS = 0, and dV(j) is 256 times the sum of
    P over i >= j, of which the last tile's rows have up to 128 terms a head (checked: P rounded to
    bf16, 2^-8, the result rounded, 2^-8, up to 2048 x 16 terms added in fp32, 2^-9 of their sum)."""
    H, d, n = 256, 32, 131072
    lens = [n, n, n, 1]
    total = sum(lens)
    cu = torch.tensor([0, n, 2 * n, 3 * n, total], dtype=torch.int32, device="cuda")
    base = lambda v: torch.full(((total + H) * d,), v, dtype=torch.bfloat16, device="cuda")
    # heads that overlap rows: inputs may
    wide = lambda v: base(v).as_strided((total, H, d), (d, d, 1))
    zeros, ones = wide(0.0), wide(1.0)
    k = torch.zeros((total, 1, d), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    lse = torch.log(pos.double() + 1).float()[None].expand(H, total).contiguous()
    layer = api.PackedAttention(H, d, [0] * H, max_total=total, max_seqs=4, max_len=n, H_kv=1)
    dq, dk, dv = layer.backward(zeros, k, v, ones, lse, ones, cu)
    assert layer.device_status() == (0, 0)
    assert not dq.any() and not dk.any()
    assert torch.isfinite(dv).all()
    assert (dv[-1] == H).all()
    back = torch.arange(n - 128, n, dtype=torch.float64, device="cuda")
    want = H * (1 / (back + 1)).flip(0).cumsum(0).flip(0)
    for s in range(3):
        got = dv[s * n + n - 128:s * n + n, 0].double()
        assert ((got - want[:, None]).abs() <= (2 * ref.U + 2.0 ** -9) * want[:, None]).all()
