"""Packed attention at its limits: a backward of seconds, the longest sequences, a hundred thousand
of them."""

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


def sampled(q, k, v, do, alpha, rho, frozen, at, chunk=1024):
    """{name: (value, bound)} of rows ``at`` of one sequence in 64 bits (packed_reference's formulas and
    bounds), a chunk of rows at a time."""
    n, H, d = q.shape
    c, U = 1 / math.sqrt(d), ref.U
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")
    m = len(at)
    sel = torch.tensor(at, device="cuda")
    out, e_out, lse, e_lse, dq, eq = z(m, H, d), z(m, H, d), z(m, H), z(m, H), z(m, H, d), z(m, H, d)
    dk, ek, dv, ev = (z(m, 1, d) for _ in range(4))
    K, V = k[:, 0].double(), v[:, 0].double()
    j = torch.arange(n, device="cuda")
    for h in range(H):
        for r0 in range(0, n, chunk):
            i = torch.arange(r0, min(n, r0 + chunk), device="cuda")
            w = i[-1] + 1                              # keys that any row of the chunk sees
            Q, dO = q[i, h].double(), do[i, h].double()
            if frozen[h]:
                x = alpha[h, :w].double()[None] + rho[h][(i[:, None] - j[:w]).clamp(min=0)].double()
            else:
                x = Q @ K[:w].T * c
            x.masked_fill_(j[:w] > i[:, None], -math.inf)
            s = torch.logsumexp(x, 1)
            p = x.sub_(s[:, None]).exp_()
            o = p @ V[:w]
            eo = 1.1 * (2 * U * (p @ V[:w].abs()) + U * o.abs()) + 1e-6
            lost = (dO.abs() * eo).sum(1)              # of D, from the rounded out
            D = (dO * o).sum(1)
            inside = sel < w
            cols = sel[inside]
            pc = p[:, cols]
            dv[inside, 0] += pc.T @ dO
            ev[inside, 0] += U * (pc.T @ dO.abs())
            if not frozen[h]:
                ds = pc * (dO @ V[cols].T - D[:, None])
                dk[inside, 0] += ds.T @ Q * c
                ek[inside, 0] += (U * ds.abs() + pc * lost[:, None]).T @ Q.abs() * c
            for a, row in enumerate(at):
                if not r0 <= row < r0 + chunk:
                    continue
                b = row - r0
                out[a, h], e_out[a, h], lse[a, h] = o[b], eo[b], s[b]
                size = 0 if frozen[h] else float((Q[b].abs() @ K[:w].abs().T).max()) * c
                e_lse[a, h] = 2.0 ** -24 * ((d + 8) * size + 16 * (1 + abs(float(s[b]))) + row + 1)
                if frozen[h]:
                    continue
                ds = p[b] * (V[:w] @ dO[b] - D[b])
                es = U * ds.abs() + p[b] * lost[b]
                dq[a, h] = ds @ K[:w] * c
                eq[a, h] = es @ K[:w].abs() * c
    got = {"out": (out, e_out), "lse": (lse, e_lse)}
    for name, x, e in (("dq", dq, eq), ("dk", dk, ek), ("dv", dv, ev)):
        got[name] = (x, 1.1 * (e + U * x.abs()) + 1e-6)
    return got


@pytest.mark.parametrize("d,n,other", [(64, 131072, 131071), (32, 40001, 5), (128, 40064, 129)])
def test_longest_sequences(api, d, n, other):
    H, frozen = 2, [0, 1]
    gen = torch.Generator(device="cuda").manual_seed(d)
    total = n + other
    q, do = (torch.randn((total, H, d), device="cuda", generator=gen).bfloat16() for _ in range(2))
    k, v = (torch.randn((total, 1, d), device="cuda", generator=gen).bfloat16() for _ in range(2))
    alpha = torch.randn((H, n), device="cuda", generator=gen)
    rho = (0.3 * torch.randn((H, n), device="cuda", generator=gen)
           - torch.log1p(torch.arange(n, device="cuda", dtype=torch.float32)))
    cu = torch.tensor([0, n, total], dtype=torch.int32, device="cuda")
    layer = api.PackedAttention(H, d, frozen, max_total=total, max_seqs=2, max_len=n, H_kv=1)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    grads = layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    assert layer.device_status() == (0, 0)
    at = [0, 1, 2, 127, 128, 5000, n // 2 - 1, n // 2, n - 129, n - 128, n - 2, n - 1]
    want = sampled(q[:n], k[:n], v[:n], do[:n], alpha, rho, frozen, at)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse.T, *grads)):
        ref.check(name, t[at], *want[name])
    # the other one is as if it were alone
    one = [t[n:].contiguous() for t in (q, k, v, do)]
    cu1 = torch.tensor([0, other], dtype=torch.int32, device="cuda")
    out1, lse1 = layer.forward(*one[:3], cu1, alpha, rho)
    assert torch.equal(out[n:, 0], out1[:, 0]) and torch.equal(lse[0, n:], lse1[0])


def test_a_hundred_thousand_sequences(api):
    """Of one row or none: the row's weight is 1, so out = V, lse its logit, dV = dO, dQ = dK = 0
    up to what test_first_rows_see_themselves_only allows."""
    H, d, n = 2, 64, 100003
    gen = torch.Generator(device="cuda").manual_seed(0)
    lens = (torch.arange(n, device="cuda") % 3 > 0).int()
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).int()])
    total = int(cu[-1])
    q, k, v, do = (torch.randn((total, H, d), device="cuda", generator=gen).bfloat16() for _ in range(4))
    layer = api.PackedAttention(H, d, [0, 1], max_total=total, max_seqs=n, max_len=1)
    alpha, rho = torch.zeros((H, 1), device="cuda"), torch.zeros((H, 1), device="cuda")
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    dq, dk, dv = layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    assert layer.device_status() == (0, 0)
    assert torch.equal(out, v) and torch.equal(dv, do)
    s = (q[:, 0].double() * k[:, 0].double()).sum(1) / 8
    size = (q[:, 0].double().abs() * k[:, 0].double().abs()).sum(1) / 8
    assert ((lse[0].double() - s).abs() <= 2.0 ** -24 * (72 * size + 16 * (1 + s.abs()))).all()
    assert not lse[1].any()
    left = 1.01 * 2.0 ** -15 * (do.double().abs() * v.double().abs()).sum(-1, keepdim=True)[:, :1] / 8
    assert (dq[:, :1].double().abs() <= left * k[:, :1].double().abs()).all()
    assert (dk[:, :1].double().abs() <= left * q[:, :1].double().abs()).all()
    assert not dq[:, 1].any() and not dk[:, 1].any()
