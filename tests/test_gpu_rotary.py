"""Rotary positions against complex rotations in 64 bits.

An angle is off by at most 2^-32 of a turn from the cut of its phase and, in fp32, by 2^-24 of at
most half a turn from its conversion: 2^-22.3 radians.  A sine or cosine is off by that, by 2 units
in the last place of CUDA's function (2^-23 each) and by half a one from the scale; a turned
component is two products and a sum, each off by half a unit: so by at most
2^-20 * scale * (|x1| + |x2|), and by u |y| more when it is rounded to its type."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def turned(x, pos, freqs, layout, scale, inverse, axis=1):
    """(value, bound) in 64 bits; pos [rows ...] without the heads' axis."""
    n = 2 * len(freqs)
    f = torch.tensor([float(v) for v in freqs], dtype=torch.float64, device=x.device)
    a = (pos.double()[..., None] * f).unsqueeze(axis)
    if inverse:
        a = -a
    y = x.double().clone()
    p, q = (y[..., :n // 2], y[..., n // 2:n]) if layout == "half" else (y[..., 0:n:2], y[..., 1:n:2])
    r0 = (p * torch.cos(a) - q * torch.sin(a)) * scale
    r1 = (q * torch.cos(a) + p * torch.sin(a)) * scale
    e = 2.0 ** -20 * abs(scale) * (p.abs() + q.abs())
    bound = torch.zeros_like(y)
    if layout == "half":
        y[..., :n // 2], y[..., n // 2:n] = r0, r1
        bound[..., :n // 2], bound[..., n // 2:n] = e, e
    else:
        y[..., 0:n:2], y[..., 1:n:2] = r0, r1
        bound[..., 0:n:2], bound[..., 1:n:2] = e, e
    u = torch.finfo(x.dtype).eps / 2
    bound[..., :n] += u * (y[..., :n].abs() + bound[..., :n])
    return y, bound


def check(got, want):
    value, bound = want
    assert not torch.isnan(got).any()
    over = (got.double() - value).abs() - bound
    assert (over <= 0).all(), float(over.max())


def rows(gen, dtype, *shape):
    return torch.randn(shape, device="cuda", generator=gen).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (128, 128), (128, 26), (32, 2), (80, 80),
                                   (256, 64), (6, 4), (7, 6)])
@pytest.mark.parametrize("inverse", [False, True])
def test_types_layouts_and_parts(api, dtype, layout, d, rot, inverse):
    gen = torch.Generator(device="cuda").manual_seed(d * rot)
    q, k = rows(gen, dtype, 2, 3, 37, d), rows(gen, dtype, 2, 1, 37, d)
    r = api.Rotary(d, rot_dim=rot, layout=layout, scale=1.25)
    freqs = api.rotary_frequencies(rot)
    pos = torch.arange(37, device="cuda").expand(2, 37)
    for x, y in zip((q, k), r.apply(q, k, inverse=inverse)):
        check(y, turned(x, pos, freqs, layout, 1.25, inverse))
        assert torch.equal(y[..., rot:], x[..., rot:])
    # without k, and in place
    alone, none = r.apply(q, inverse=inverse)
    assert none is None and torch.equal(alone, r.apply(q, k, inverse=inverse)[0])
    own_q, own_k = q.clone(), k.clone()
    got = r.apply(own_q, own_k, inverse=inverse, out=(own_q, own_k))
    assert got[0] is own_q and torch.equal(own_q, alone)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_given_positions_far_and_negative(api, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = api.Rotary(64, base=500000.0)
    freqs = api.rotary_frequencies(64, 500000.0)
    q = rows(gen, dtype, 2, 4, 9, 64)
    at = torch.tensor([0, 1, -1, 131072, 1000003, 2 ** 31 - 1, -2 ** 31, 16777217, 5],
                      dtype=torch.int32, device="cuda")
    pos = torch.stack([at, at.flip(0)])
    # 2^31 radians: the definition's own angle is off by 2^-23 there; frequencies that are
    # exact in few bits keep it exact
    exact = [2.0 ** -i for i in range(32)]
    for use in (freqs, exact):
        r = api.Rotary(64, freqs=use)
        far = pos if use is exact else pos.clamp(-2 ** 21, 2 ** 21)
        y, _ = r.apply(q, positions=far)
        check(y, turned(q, far, use, "half", 1.0, False))


def test_turning_back_is_the_gradient(api):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = api.Rotary(64, rot_dim=32, layout="interleaved", scale=0.75)
    q, dy = rows(gen, torch.float32, 1, 2, 50, 64), rows(gen, torch.float32, 1, 2, 50, 64)
    freqs, pos = api.rotary_frequencies(32), torch.arange(50, device="cuda")[None]
    dx, _ = r.apply(dy, inverse=True)
    check(dx, turned(dy, pos, freqs, "interleaved", 0.75, True))
    # against differences of <dy, y> in 64 bits (y is linear in q)
    way = torch.randn_like(q)
    up, down = (turned(q + s * way, pos, freqs, "interleaved", 0.75, False)[0] for s in (1.0, -1.0))
    slope = ((up - down) * dy.double()).sum() / 2
    bound = (turned(dy, pos, freqs, "interleaved", 0.75, True)[1] * way.double().abs()).sum()
    assert abs((dx.double() * way.double()).sum() - slope) <= bound + 1e-5 * abs(slope)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_packed_rows(api, layout):
    gen = torch.Generator(device="cuda").manual_seed(3)
    lens, head, tail = [5, 0, 1, 130, 0, 64], 3, 4
    cu = [head]
    for n in lens:
        cu.append(cu[-1] + n)
    total = cu[-1] + tail
    x = rows(gen, torch.bfloat16, total, 4 + 2 + 2, 64)
    x[:head], x[cu[-1]:] = math.nan, math.nan
    q, k = x[:, :4], x[:, 4:6]                        # views of one projection
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pos = torch.zeros(total, dtype=torch.int64, device="cuda")
    for a, n in zip(cu, lens):
        pos[a:a + n] = torch.arange(n, device="cuda")
    freqs = api.rotary_frequencies(64)
    r = api.Rotary(64, layout=layout)
    live = slice(head, cu[-1])
    for src, y in zip((q, k), r.apply(q, k, cu_seqlens=cut)):
        check(y[live], turned(src[live], pos[live], freqs, layout, 1.0, False))
        assert not y[:head].any() and not y[cu[-1]:].any()
    given = tuple(torch.full((total, h, 64), 9.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    r.apply(q, k, cu_seqlens=cut, out=given)
    for src, y in zip((q, k), given):
        check(y[live], turned(src[live], pos[live], freqs, layout, 1.0, False))
        assert (y[:head] == 9).all() and (y[cu[-1]:] == 9).all()
    # no sequence at all, and heads-major rows
    none = torch.tensor([7], dtype=torch.int32, device="cuda")
    assert not r.apply(q, cu_seqlens=none)[0].any()
    major = q[live].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(r.apply(major, cu_seqlens=cut - head)[0], r.apply(q[live], cu_seqlens=cut - head)[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_positions_of_the_cache(api, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = 6
    q, k = rows(gen, dtype, 4, 3, n, 32), rows(gen, dtype, 4, 3, n, 32)
    seq_len = torch.tensor([6, 100, 4096, 2], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([6, 1, 9, -3], dtype=torch.int32, device="cuda")  # cut to 0..n
    fresh = n_new.clamp(0, n).long()
    t = torch.arange(n, device="cuda")
    pos = (seq_len.long() - fresh)[:, None] + t
    live = (t < fresh[:, None])[:, None, :, None]
    r, freqs = api.Rotary(32), api.rotary_frequencies(32)
    for x, y in zip((q, k), r.apply(q, k, seq_len=seq_len, n_new=n_new)):
        v, b = turned(x, pos, freqs, "half", 1.0, False)
        check(y, (v * live, b * live))
    old = tuple(x.clone() for x in (q, k))
    r.apply(q, k, seq_len=seq_len, n_new=n_new, out=(q, k))
    for x, was in zip((q, k), old):
        v, b = turned(was, pos, freqs, "half", 1.0, False)
        check(x, (torch.where(live, v, was.double()), b * live))
    # n_new None: all rows
    y, _ = r.apply(old[0], seq_len=seq_len)
    check(y, turned(old[0], seq_len.long()[:, None] - n + t, freqs, "half", 1.0, False))


def test_many_rows_and_broadcast_input(api):
    gen = torch.Generator(device="cuda").manual_seed(5)
    r, freqs = api.Rotary(64), api.rotary_frequencies(64)
    x = rows(gen, torch.bfloat16, 1, 1, 5000, 64).expand(3, 5, 5000, 64)
    pos = torch.arange(5000, device="cuda").expand(3, 5000)
    y, _ = r.apply(x)
    check(y, turned(x, pos, freqs, "half", 1.0, False))
    # rows that are not 16 bytes apart
    odd = rows(gen, torch.bfloat16, 700, 3 * 64 + 1)[:, 1:].unflatten(1, (3, 64))
    y, _ = r.apply(odd)
    check(y, turned(odd, pos[0, :700], freqs, "half", 1.0, False))


def test_graph_stream_and_refusals(api):
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = api.Rotary(64)
    q = rows(gen, torch.bfloat16, 2, 4, 1, 64)
    lens = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    r.apply(q, seq_len=lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = r.apply(q, seq_len=lens)
    lens.copy_(torch.tensor([600, 77], dtype=torch.int32))
    graph.replay()
    assert torch.equal(y, r.apply(q, seq_len=lens)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z, _ = r.apply(q, seq_len=lens)
    side.synchronize()
    assert torch.equal(y, z)
    bad = [dict(q=q[0, 0]), dict(q=q.half()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q=q, k=q[0]),
           dict(q=q, k=q.float()), dict(q=q, out=(q, q)), dict(q=q, positions=lens),
           dict(q=q, cu_seqlens=lens), dict(q=q, seq_len=lens.long()), dict(q=q, n_new=lens),
           dict(q=q, seq_len=lens, positions=lens.view(2, 1)),
           dict(q=torch.empty(2, 4, 64, 2, device="cuda").transpose(2, 3).bfloat16())]
    for kw in bad[:-1]:
        with pytest.raises(api.SafError):
            r.apply(kw.pop("q"), kw.pop("k", None), **kw)
    with pytest.raises(api.SafError):  # rows that are not contiguous
        r.apply(torch.empty((2, 4, 64, 2), dtype=torch.bfloat16, device="cuda").transpose(2, 3))
