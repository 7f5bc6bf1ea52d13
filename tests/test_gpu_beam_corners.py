"""The beam step where a part of a row is gone through twice: more logits than places reach the first
tile's threshold, or NaN, infinities and logits beyond 2^20 are among them."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def best(logits, scores, K):
    """(parent, token, score in 64 bits) by score, slot, logit and token, on the GPU."""
    x = logits.double()
    x = torch.where((x >= -2.3e38) & (x < math.inf), x, -math.inf)
    lse = torch.logsumexp(x, 1, keepdim=True)
    lse = torch.where(lse == -math.inf, 0.0, lse)
    # a slot's K best: by logit, then token (sorting keeps the order of equal ones)
    top, token = torch.sort(x, dim=1, descending=True, stable=True)
    top, token = top[:, :K], token[:, :K]
    s = scores.double()
    s = torch.where((s >= -2.3e38) & (s < math.inf), s, -math.inf)
    score = torch.where(top == -math.inf, -math.inf, s[:, None] + (top - lse))
    # (no offer: the fp32 score is none)
    score = torch.where(score.float() < -2.3e38, -math.inf, score)
    wide = score.shape[1]
    score = score.view(-1, K * wide)
    score, at = torch.sort(score, dim=1, descending=True, stable=True)
    score, at = score[:, :K], at[:, :K]
    slot = at // wide + torch.arange(score.shape[0], device=x.device)[:, None] * K
    token = token.reshape(score.shape[0], -1).gather(1, at)
    none = score == -math.inf
    out = (torch.where(none, -1, slot), torch.where(none, -1, token), score)
    if wide < K:
        pad = lambda t, v: torch.nn.functional.pad(t, (0, K - t.shape[1]), value=v)
        out = tuple(pad(t, v) for t, v in zip(out, (-1, -1, -math.inf)))
    return tuple(t.flatten() for t in out)


def rows(kind, G, K, V):
    gen = torch.Generator().manual_seed(G + K)
    ramp = torch.arange(V, dtype=torch.float32) / V
    x = 30 * ramp + torch.randn((G * K, V), generator=gen)
    if kind == "equal":
        x = torch.zeros_like(x)
    elif kind == "nan":
        x[:, 5::4097] = math.nan
        x[:, 7::9001] = math.inf
    elif kind == "far":
        x = torch.round(4 * x) / 4 + 2.0 ** 21
    # (scores of different slots are 4e-6 apart or more for these seeds, but for equal rows)
    return x.cuda(), (-7.0 * torch.arange(G * K) / K).cuda()


@pytest.mark.parametrize("kind", ["rising", "equal", "nan", "far"])
@pytest.mark.parametrize("G,K,V", [(64, 8, 128003), (8, 2, 50001), (16, 32, 70001)])
def test_a_second_pass_gives_the_same_bits_every_time(api, kind, G, K, V):
    x, s = rows(kind, G, K, V)
    search = api.BeamSearch(G, K, V)
    parent, token, score = search.step(x, s)[:3]
    wp, wt, ws = best(x, s, K)
    assert torch.equal(parent.long(), wp)
    assert torch.equal(token.long(), wt)
    assert ((score.double() - ws).abs() <= 2.0 ** -24 * ws.abs() + 2.0 ** -19.3).all()
    for i in range(60):
        again = search.step(x, s)
        for a, b in zip((parent, token, score), again):
            assert torch.equal(a, b), i


def collapse(kind, K, V):
    gen = torch.Generator(device="cuda").manual_seed(K + V)
    x = torch.rand((3 * K, V), device="cuda", generator=gen)
    s = torch.full((3 * K,), -math.inf, device="cuda")
    if kind == "far scores":          # 64 bits hold multiples of 128 there
        s[:] = -1e18
    elif kind == "one slot":
        s[::K] = -1e18
    else:                             # logits that vanish beside their log sum
        x *= 1e-20
        s[::K] = -1.0
    return x, s


@pytest.mark.parametrize("kind", ["far scores", "one slot", "tiny logits"])
@pytest.mark.parametrize("K,V", [(1, 500), (4, 1000), (8, 40000), (32, 3001)])
def test_offers_of_a_slot_go_by_their_logits(api, kind, K, V):
    """Also where 64 bits give them the same score: the larger logit first, then the lower token."""
    x, s = collapse(kind, K, V)
    for y in (x, x.flip(1).contiguous(), x.bfloat16()):
        parent, token, score = api.BeamSearch(3, K, V).step(y, s)[:3]
        wp, wt, ws = best(y, s, K)
        assert torch.equal(parent.long(), wp)
        assert torch.equal(token.long(), wt)
        assert ((score.double() - ws).abs() <= 2.0 ** -24 * ws.abs() + 2.0 ** -19.3).all()


def test_sums_of_a_second_pass_are_as_exact(api):
    """Rows of equal logits with a NaN: a thread adds 128 terms of the same value, whose roundings
    go the same way (one after another they would add up to 2^-19).  In sixteens: 15 roundings of
    2^-24, the function's 2^-22, its argument's 1.4 x 2^-24; scores near 0 add nothing."""
    n, V = 1900, 32768                # one part of eight tiles a row
    gen = torch.Generator(device="cuda").manual_seed(1)
    c = 6 * torch.rand((n, 1), device="cuda", generator=gen) - 3
    x = c.expand(n, V).contiguous()
    x[:, 777] = math.nan
    want = math.log(V - 1)            # of the row without its logit's value
    s = torch.full((n,), want, device="cuda")
    parent, token, score = api.BeamSearch(n, 1, V).step(x, s)[:3]
    assert torch.equal(parent.long(), torch.arange(n, device="cuda")) and not token.any()
    off = (score.double() - (s.double() - want)).abs()
    assert off.max() <= 2.0 ** -22 + 16.5 * 2.0 ** -24, float(off.max())
    # beyond 2^20, against the largest logit
    step = 0.25 * (1 + torch.arange(n, device="cuda") % 12)
    x = (2.0 ** 21 - step)[:, None].expand(n, V).contiguous()
    x[:, 0] = 2.0 ** 21
    want = torch.log1p((V - 1) * torch.exp(-step.double()))
    s = want.float()
    _, token, score = api.BeamSearch(n, 1, V).step(x, s)[:3]
    assert not token.any()
    off = (score.double() - (s.double() - want)).abs()
    assert off.max() <= 2.0 ** -22 + 16.5 * 2.0 ** -24, float(off.max())


def test_scores_that_leave_the_type_are_no_offers(api):
    """An offer whose score would be -inf in fp32, or below what a score counts from, is none: the
    slot would have a parent but never go on."""
    x = torch.tensor([[0.0, -1e37, -2e38, -1e38], [0.0, -2.2e38, -2e38, -2e38]], device="cuda")
    s = torch.tensor([-2e38, -2.25e38], device="cuda")
    parent, token, score = api.BeamSearch(1, 2, 4).step(x, s)[:3]
    assert parent.tolist() == [0, 0] and token.tolist() == [0, 1]
    x[0, 1] = -1.5e38
    parent, token, score = api.BeamSearch(1, 2, 4).step(x, s)[:3]
    assert parent.tolist() == [0, 1] and token.tolist() == [0, 0]
    s[1] = -math.inf
    parent, token, score = api.BeamSearch(1, 2, 4).step(x, s)[:3]
    assert parent.tolist() == [0, -1] and token.tolist() == [0, -1]
    assert score[1] == -math.inf
    x = torch.where(x == 0, 0.0, -2.2e38)
    K = 4
    x, s = x[:1].expand(2 * K, 4).contiguous(), torch.full((2 * K,), -2e38, device="cuda")
    parent, token, score = api.BeamSearch(2, K, 4).step(x, s)[:3]
    wp, wt, ws = best(x, s, K)
    assert torch.equal(parent.long(), wp) and torch.equal(token.long(), wt)
    assert torch.equal(score == -math.inf, wp < 0)


# ---- limits
@pytest.mark.parametrize("G,K,V,dtype", [(1, 32, 1 << 22, torch.bfloat16), (2, 2, 1 << 22, torch.float32),
                                         (1, 1, 1 << 22, torch.float32), (3, 23, (1 << 21) + 5, torch.float32),
                                         (30000, 3, 40, torch.float32), (100000, 1, 7, torch.bfloat16)])
def test_largest_vocabulary_and_many_groups(api, G, K, V, dtype):
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((G * K, V), device="cuda", generator=gen).to(dtype)
    s = -40.0 * (torch.arange(G * K, device="cuda") % K)   # (the slots' offers do not meet)
    x[:, V // 2] += 3.0
    search = api.BeamSearch(G, K, V)
    for i in range(2):
        parent, token, score = search.step(x, s)[:3]
    wp, wt, ws = best(x, s, K)
    assert torch.equal(parent.long(), wp)
    assert torch.equal(token.long(), wt)
    assert ((score.double() - ws).abs() <= 2.0 ** -24 * ws.abs() + 2.0 ** -19.3).all()
