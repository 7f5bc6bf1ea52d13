"""The beam step against a sort of all offers in 64 bits.

Which offers win and in which order has to be the same: the scores here are apart by more than what
64 bits and the kernel's sums can differ by, or equal bit for bit in a way that the definition's
ties decide.  An exponential 2^t is off by 2^-22 of itself from the function and by
2 |t| 2^-24 ln 2 from its argument, which weighted with 2^t is at most 2^-24; a thread adds up to 136 of
them in fp32, in pairs and tiles of 16, off by at most 24 roundings of 2^-24: 2^-19.3 of the sum in all,
and so much in its logarithm.  A score is then rounded to fp32 once: 2^-24 of itself."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.bfloat16).min


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def step(logits, scores, finished, K, end):
    """(parent, token, score in 64 bits) from the definition, on the host."""
    x, s = logits.double().cpu(), scores.double().cpu()
    n, V = x.shape
    x = torch.where((x >= -2.3e38) & (x < math.inf), x, -math.inf)
    parent, token, score = [], [], []
    for g in range(n // K):
        ways = []
        for b in range(g * K, g * K + K):
            if not (s[b] >= -2.3e38 and s[b] < math.inf):
                continue
            if finished is not None and bool(finished[b]):
                ways.append((float(s[b]), 0.0, b, end))
                continue
            row = x[b]
            if not (row > -math.inf).any():
                continue
            lse = torch.logsumexp(row, 0)
            top = torch.topk(row, min(V, 4 * K)).values[-1]
            for v in torch.nonzero((row >= top) & (row > -math.inf))[:, 0].tolist():
                ways.append((float(s[b] + (row[v] - lse)), float(row[v]), b, v))
        ways.sort(key=lambda w: (-w[0], w[2], w[3]))
        ways = ways[:K]
        parent += [w[2] for w in ways] + [-1] * (K - len(ways))
        token += [w[3] for w in ways] + [-1] * (K - len(ways))
        score += [w[0] for w in ways] + [-math.inf] * (K - len(ways))
    return torch.tensor(parent), torch.tensor(token), torch.tensor(score, dtype=torch.float64)


def check(api, logits, scores, finished=None, end=None, K=4, search=None):
    n, V = logits.shape
    search = search or api.BeamSearch(n // K, K, V, end=end)
    parent, token, score, done, none = search.step(logits, scores, finished)
    assert none is None
    wp, wt, ws = step(logits, scores, finished, K, end)
    assert torch.equal(parent.cpu().long(), wp), (parent, wp)
    assert torch.equal(token.cpu().long(), wt), (token, wt)
    got = score.double().cpu()
    inf = torch.isinf(ws)
    assert torch.equal(got[inf], ws[inf])
    off = (got - ws)[~inf].abs()
    assert (off <= 2.0 ** -24 * ws[~inf].abs() + 2.0 ** -19.3).all(), float(off.max())
    assert (done is None) == (end is None)
    if end is not None:
        assert torch.equal(done.cpu(), (wp >= 0) & (wt == end))
    return search


def inputs(G, K, V, dtype=torch.float32, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (spread * torch.randn((G * K, V), device="cuda", generator=gen)).to(dtype)
    return x, -10 * torch.rand(G * K, device="cuda", generator=gen)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,K,V", [(1, 1, 1), (1, 1, 2), (2, 3, 2), (1, 4, 5), (3, 2, 257), (1, 1, 4097),
                                   (2, 8, 1000), (1, 32, 3001), (1, 32, 40000), (40, 5, 2048),
                                   (2, 31, 9973), (1, 4, 200001), (150, 2, 5000), (40, 16, 30001)])
def test_sizes(api, G, K, V, dtype):
    x, s = inputs(G, K, V, dtype)
    search = check(api, x, s, K=K)
    check(api, x.flip(1).contiguous(), s, K=K, search=search)   # the counters are zero again


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_at_any_distance_and_alignment(api, dtype):
    for V in (1000, 5003):
        for shift in (0, 1, 3, 5):
            for gap in (0, 1, 2, 7):
                big = torch.full((9, V + gap + shift), math.nan, dtype=dtype, device="cuda")
                x, s = inputs(2, 4, V, dtype, seed=V + shift)
                view = big[:8, shift:shift + V]
                view.copy_(x)
                check(api, view, s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_and_odd_logits(api, dtype):
    K, V = 4, 20011
    x, s = inputs(9, K, V, dtype)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x[0, ::2] = -math.inf
    x[1, ::3] = math.nan
    x[2, 5::7] = math.inf                     # counts as masked
    x[3] = torch.where(torch.rand(V, device="cuda", generator=gen) < 0.99, LOWEST, x[3])
    x[4] = -math.inf                          # no way on
    x[5] = LOWEST
    x[6] = math.nan
    x[7] = -1e9                               # a mask that is finite: every token equally likely
    x[8, 10:] = -1e9
    x[9, :-3] = -math.inf
    x[10] += 5e6 if dtype == torch.float32 else 3e7   # beyond 2^20
    x[11] = torch.where(torch.arange(V, device="cuda") == 17, x[11] + 3e6, x[11])
    x[12:16] = -math.inf                      # a whole group without a way on
    x[16, 1:] = -math.inf
    x[17:20] = -math.inf                      # a group with a single one
    s[20:24] = torch.tensor([-math.inf, math.nan, torch.finfo(torch.float32).min, -3.0])
    check(api, x, s)


def test_equal_scores_go_to_the_lowest(api):
    K, V = 8, 30000
    x = torch.zeros((K, V), device="cuda")
    s = torch.zeros(K, device="cuda")
    check(api, x, s, K=K)                     # everything equal
    x[:, 1000:] = 1.0
    check(api, x, s, K=K)
    x = torch.randn((1, V), device="cuda").bfloat16().expand(K, V).contiguous()
    check(api, x, s, K=K)                     # the same row in every beam
    x = torch.arange(V, device="cuda", dtype=torch.float32).expand(K, V).contiguous() / 1000
    check(api, x, -s - torch.arange(K, device="cuda") / 7, K=K)   # rising all the way
    check(api, x.flip(1).contiguous(), s, K=K)
    x = torch.zeros((K, V), device="cuda")
    x[:, ::2] = -0.0
    check(api, x, s, K=K)                     # -0 is 0


@pytest.mark.parametrize("K,V", [(8, 128003), (32, 70001), (1, 200000), (16, 33000)])
def test_parts_whose_first_logits_are_the_smallest(api, K, V):
    """Far more logits above the first tile's than the places for them: rising along the vocabulary,
    in steps of 4096, in bf16's coarse steps, with NaN and infinities on the way."""
    G = max(1, 512 // K)
    gen = torch.Generator(device="cuda").manual_seed(K)
    ramp = torch.arange(V, device="cuda", dtype=torch.float32) / V
    noise = torch.randn((G * K, V), device="cuda", generator=gen)
    s = -10 * torch.rand(G * K, device="cuda", generator=gen)
    search = check(api, 30 * ramp + noise, s, K=K)
    check(api, 5 * torch.floor(ramp * V / 4096) + noise, s, K=K, search=search)
    check(api, (30 * ramp + noise).bfloat16(), s, K=K, search=search)
    x = 30 * ramp + noise
    x[:, 5::4097] = math.nan
    x[:, 7::9001] = math.inf
    check(api, x, s, K=K, search=search)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_finished_slots_stand_still(api, dtype):
    K, V, end = 4, 5000, 7
    x, s = inputs(6, K, V, dtype)
    done = torch.tensor([1, 0, 0, 0, 1, 1, 1, 1, 0, 0, 0, 0, 0, 1, 0, 1] + [0] * 8, device="cuda").bool()
    x[0], x[5] = math.nan, math.nan           # rows of finished slots are not read
    x[8:12, end] = 30.0                       # the ending token is the likely one
    s[13] = s[15]                             # equal scores of two finished slots
    s[4] = -math.inf
    check(api, x, s, done, end)


def test_first_step_and_in_place_scores(api):
    K, V = 5, 9000
    x, s = inputs(3, K, V, seed=3)
    s = torch.where(torch.arange(3 * K, device="cuda") % K == 0, 0.0, -math.inf)
    x = x[::K].repeat_interleave(K, 0).contiguous()
    check(api, x, s, K=K)


def test_scores_in_their_own_place(api):
    from dynamic_causal_attention_gb300 import _binding as B
    G, K, V = 7, 4, 3000
    x, s = inputs(G, K, V, seed=4)
    done = (torch.arange(G * K, device="cuda") % 5 == 0)
    search = api.BeamSearch(G, K, V, end=2)
    want = search.step(x, s, done)
    parent, token = (torch.zeros(G * K, dtype=torch.int32, device="cuda") for _ in range(2))
    dims = B.saf_beam_dims(G, K, V, V, B.SAF_F32, 2, 0)
    st = B.saf_beam_step(dims, x.data_ptr(), s.data_ptr(), done.data_ptr(), None, None,
                         parent.data_ptr(), token.data_ptr(), s.data_ptr(), done.data_ptr(), None,
                         search.workspace.data_ptr(), search.ws_bytes,
                         torch.cuda.current_stream().cuda_stream)
    assert st == B.SAF_OK
    for a, b in zip((parent, token, s, done), want):
        assert torch.equal(a, b)


def test_histories_follow_their_parents(api):
    G, K, V, cols = 5, 3, 4000, 70
    search = api.BeamSearch(G, K, V, end=1)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for n in (0, 1, 33, 69, 70, 500, -4):
        x, s = inputs(G, K, V, seed=n + 10)
        s[3:6] = -math.inf                    # a group that is free
        x[6:8], s[8] = -math.inf, -math.inf   # and one with a single way on
        x[6, 9] = 0.0
        h = torch.randint(0, V, (G * K, cols), device="cuda", generator=gen).int()
        out = torch.full_like(h, -7)
        count = torch.tensor([n], dtype=torch.int32, device="cuda")
        parent, token, _, _, got = search.step(x, s, history=h, n_tokens=count, history_out=out)
        assert got is out
        m = min(max(n, 0), cols)
        for i in range(G * K):
            p = int(parent[i])
            want = torch.full((cols,), -7, dtype=torch.int32, device="cuda")
            want[:m] = h[p, :m] if p >= 0 else -1
            if m < cols:
                want[m] = token[i]
            assert torch.equal(out[i], want), (n, i)
        fresh = search.step(x, s, history=h, n_tokens=count)[4]
        assert torch.equal(fresh[:, :m], out[:, :m])


def test_graph_stream_and_same_bits(api):
    K, V = 4, 50001
    x, s = inputs(12, K, V)
    search = api.BeamSearch(12, K, V)
    first = search.step(x, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taped = search.step(x, s)
    for i in range(20):
        graph.replay()
    for a, b in zip(first[:3], taped[:3]):
        assert torch.equal(a, b)
    y, _ = inputs(12, K, V, seed=5)
    x.copy_(y)
    graph.replay()
    want = search.step(x, s)
    for a, b in zip(want[:3], taped[:3]):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = search.step(x, s)
    side.synchronize()
    assert torch.equal(other[2], want[2])


def test_refusals(api):
    search = api.BeamSearch(2, 2, 100, end=3)
    x, s = inputs(2, 2, 100)
    done = torch.zeros(4, dtype=torch.bool, device="cuda")
    h = torch.zeros((4, 8), dtype=torch.int32, device="cuda")
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    for a, kw in (((x[:3], s), {}), ((x[:, :99], s), {}), ((x.half(), s), {}), ((x.cpu(), s), {}),
                  ((x, s.double()), {}), ((x, s[:3]), {}), ((x, s, done.int()), {}),
                  ((x, s), dict(history=h)), ((x, s), dict(history=h, n_tokens=n, history_out=h)),
                  ((x, s), dict(history_out=h)), ((x, s), dict(history=h.long(), n_tokens=n)),
                  ((x, s), dict(history=h, n_tokens=n.long())), ((x.t().contiguous().t(), s), {}),
                  ((x[:1].expand(4, 100), s), {})):
        with pytest.raises(api.SafError):
            search.step(*a, **kw)
    with pytest.raises(api.SafError):
        api.BeamSearch(2, 2, 100).step(x, s, done)
    for bad in (dict(n_groups=0), dict(beams=0), dict(beams=33), dict(vocab=0), dict(end=100)):
        with pytest.raises(api.SafError):
            api.BeamSearch(**{**dict(n_groups=2, beams=2, vocab=100), **bad})
