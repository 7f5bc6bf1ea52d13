"""The packed attention from its definition in 64 bits (torch, one head of one sequence at a
time), with a bound on what an implementation may be off.

A rounding to bf16 is off by at most u = finfo(bf16).eps / 2 = 2^-8 of the value.  The
implementation rounds the weights (for P V), P and dS (for the gradients) and every result
once, and forms D = rowsum(dO o O) from the rounded O; products and sums are fp32.  With
A = sum_j p_j |v_j|:

* out:  weights off by u each, and (frozen heads) their sum by u:  2 u A + u |out|
* dV:   u sum_i p_ij |dO_i| + u |dV|
* dS:   u |dS| + p (sum_c |dO_c| E_out_c)   with E_out the bound of out
* dQ, dK: the bound of dS times |K|, |Q|, + u of the result

times 1.1 for the fp32 parts (at most 2^-14 of the terms), plus 1e-6.
"""

import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
MASKED = -2.3e38


def weights(q, k, alpha, rho, frozen):
    """log weights [n, n] of one head, -inf where a row does not look."""
    n = q.shape[0]
    i = torch.arange(n, device=q.device)
    if frozen:
        x = alpha.double()[:n][None] + rho.double()[(i[:, None] - i[None]).clamp(min=0)]
        x = torch.where((alpha[:n][None] < MASKED) | (rho[(i[:, None] - i[None]).clamp(min=0)] < MASKED),
                        -math.inf, x)
    else:
        x = q.double() @ k.double().T / math.sqrt(q.shape[1])
    return torch.where(i[None] > i[:, None], -math.inf, x)


def packed(q, k, v, lens, starts, frozen, alpha=None, rho=None, dout=None):
    """{name: (value, bound)} of out, lse (bound relative to 1) and, with dout, dq, dk, dv; rows of
    no sequence 0 and -inf."""
    total, H, d = q.shape
    Hkv, g = k.shape[1], H // k.shape[1]
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)
    out, e_out, lse = z(total, H, d), z(total, H, d), torch.full_like(z(H, total), -math.inf)
    e_lse = z(H, total)
    dq, dk, dv = z(total, H, d), z(total, Hkv, d), z(total, Hkv, d)
    eq, ek, ev = torch.zeros_like(dq), torch.zeros_like(dk), torch.zeros_like(dv)
    for a, n in zip(starts, lens):
        b = a + n
        for h in range(H if n else 0):
            kv = h // g
            Q, K, V = q[a:b, h].double(), k[a:b, kv].double(), v[a:b, kv].double()
            x = weights(q[a:b, h], k[a:b, kv], None if alpha is None else alpha[h],
                        None if rho is None else rho[h], frozen[h])
            s = torch.logsumexp(x, 1)
            lse[h, a:b] = s
            p = torch.exp(x - torch.where(s > -math.inf, s, 0.0)[:, None])
            # fp32 sums of products and of up to n exponentials
            size = z(n) if frozen[h] else (Q.abs() @ K.abs().T).amax(1) / math.sqrt(d)
            e_lse[h, a:b] = 2.0 ** -24 * ((d + 8) * size + 16 * (1 + torch.nan_to_num(s).abs()) + n)
            o = p @ V
            out[a:b, h] = o
            eo = 1.1 * (2 * U * (p @ V.abs()) + U * o.abs()) + 1e-6
            e_out[a:b, h] = eo
            if dout is None:
                continue
            do = dout[a:b, h].double()
            dv[a:b, kv] += p.T @ do
            ev[a:b, kv] += U * (p.T @ do.abs())
            if frozen[h]:
                continue
            dp = do @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            es = U * ds.abs() + p * (do.abs() * eo).sum(1, keepdim=True)
            c = 1 / math.sqrt(d)
            dq[a:b, h] = ds @ K * c
            eq[a:b, h] = es @ K.abs() * c
            dk[a:b, kv] += ds.T @ Q * c
            ek[a:b, kv] += es.T @ Q.abs() * c
    got = {"out": (out, e_out), "lse": (lse, e_lse)}
    if dout is not None:
        for name, x, e in (("dq", dq, eq), ("dk", dk, ek), ("dv", dv, ev)):
            got[name] = (x, 1.1 * (e + U * x.abs()) + 1e-6)
    return got


def check(name, got, want, bound):
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), name
    assert not torch.isnan(got).any(), f"{name}: NaN"
    over = torch.where(inf, 0.0, (got - want).abs() - bound)
    assert (over <= 0).all(), (f"{name}: off by {float((got - want)[~inf].abs().max()):.3e}, "
                               f"{float(over.max()):.3e} over its bound at "
                               f"{[int(i) for i in torch.nonzero(over == over.max())[0]]}")
