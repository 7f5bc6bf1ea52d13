"""Prompts of different lengths from the first row to beams: rotary positions, the packed layer, the
cache, the beam step and the cache's fork, one after another as a serving program calls them.

What the cache's attention gives for a beam's newest token is held against the packed layer on the
beam's whole text.  The cache rounds K and V to e4m3, off by at most w = 2^-4 of each value (and
2^-10 of the block's scale's step below its normal range: less than 2^-13 of the largest): so a
logit is off by at most D = (w + 2^-13) sum |q| |k|max / sqrt(d) and the output by
(exp(2 D) - 1) max|v| + 2 w max|v|, the bf16 roundings of either side inside the second w."""

import math

import pytest
import torch

import packed_reference as ref
from test_gpu_beam import step as beam_reference

pytestmark = pytest.mark.gpu

H, HKV, D, V, PAGE, FROZEN = 4, 2, 64, 500, 16, [0, 1, 0, 0]


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def test_prompts_to_beams(api):
    gen = torch.Generator(device="cuda").manual_seed(11)
    lens, K, steps = [5, 40, 130], 2, 4
    G, T = len(lens), max(lens) + steps
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)
    # a one-layer model without trained weights: token -> q, k, v; heads' outputs -> logits
    table, head = (0.7 * rnd(V, H + 2 * HKV, D)).bfloat16(), 0.2 * rnd(H * D, V)
    alpha, rho = rnd(H, T), -torch.log1p(torch.arange(T, device="cuda").float()).repeat(H, 1)
    rotary = api.Rotary(D, rot_dim=32)
    packed = api.PackedAttention(H, D, FROZEN, max_total=4 * T * G * K, max_seqs=G * K, max_len=T,
                                 H_kv=HKV)
    slots = G * K
    cache = api.PagedCache([FROZEN], H, D, H_kv=HKV, n_seqs=slots, max_pages=-(-T // PAGE),
                           n_pages=slots * -(-T // PAGE), page_size=PAGE, max_new=max(lens))
    search = api.BeamSearch(G, K, V, end=0)
    i32 = dict(dtype=torch.int32, device="cuda")

    def split(tokens):  # rows of q, k, v
        x = table[tokens]
        return x[..., :H, :], x[..., H:H + HKV, :], x[..., H + HKV:, :]

    def run_packed(texts):
        cu = [0]
        for t in texts:
            cu.append(cu[-1] + len(t))
        q, k, v = split(torch.cat(texts))
        cu_t = torch.tensor(cu, **i32)
        q, k = rotary.apply(q, k, cu_seqlens=cu_t)
        out, lse = packed.forward(q, k, v, cu_t, alpha, rho)
        return q, k, v, out, lse, cu

    prompts = [torch.randint(1, V, (n,), device="cuda", generator=gen) for n in lens]
    q, k, v, out, lse, cu = run_packed(prompts)
    want = ref.packed(q, k, v, lens, cu[:-1], FROZEN, alpha, rho)
    ref.check("out", out, *want["out"])
    # the first beam of each group takes the prompt into the cache, the others fork it
    n_new = torch.zeros(slots, **i32)
    n_new[::K] = torch.tensor(lens, **i32)
    granted, short = cache.grow(n_new)
    new_k, new_v = (torch.zeros((slots, HKV, max(lens), D), dtype=torch.bfloat16, device="cuda")
                    for _ in range(2))
    for g, n in enumerate(lens):
        new_k[g * K, :, :n] = k[cu[g]:cu[g + 1]].transpose(0, 1)
        new_v[g * K, :, :n] = v[cu[g]:cu[g + 1]].transpose(0, 1)
    cache.append(0, new_k, new_v, n_new=granted)
    cache.fork(torch.arange(slots, **i32) // K * K)
    assert int(short) == 0
    last = torch.stack([out[c - 1] for c in cu[1:]])
    logits = (last.float().flatten(1) @ head).repeat_interleave(K, 0).contiguous()
    scores = torch.where(torch.arange(slots, device="cuda") % K == 0, 0.0, -math.inf)
    finished = torch.zeros(slots, dtype=torch.bool, device="cuda")
    history, n_tokens = torch.zeros((slots, steps), **i32), torch.zeros(1, **i32)
    texts = [prompts[s // K] for s in range(slots)]

    for t in range(steps):
        wp, wt, _ = beam_reference(logits, scores, finished, K, 0)
        parent, token, scores, finished, history = search.step(
            logits, scores, finished, history=history, n_tokens=n_tokens)
        n_tokens += 1
        assert torch.equal(parent.cpu().long(), wp) and torch.equal(token.cpu().long(), wt)
        cache.fork(parent)
        texts = [torch.cat([texts[p], x[None]]) for p, x in zip(parent.tolist(), token.long())]
        for s in range(slots):
            assert torch.equal(history[s, :t + 1].long(), texts[s][lens[s // K]:])
        # the new tokens through the cache
        granted, short = cache.grow(torch.ones(slots, **i32))
        assert int(short) == 0 and (granted == 1).all()
        q1, k1, v1 = (x[:, :, None].contiguous() for x in split(token.long()))
        q1, k1 = rotary.apply(q1, k1, seq_len=cache.seq_len, n_new=granted)
        cache.append(0, k1, v1, n_new=granted)
        got, _ = cache.attend(0, q1, alpha, rho, n_new=granted)
        # and the whole texts through the packed layer
        q, k, v, out, lse, cu = run_packed(texts)
        for s in range(slots):
            a, b = cu[s], cu[s + 1]
            for h in range(H):
                kv = h * HKV // H
                top = v[a:b, kv].float().abs().max()
                size = 0.0 if FROZEN[h] else float(
                    q[b - 1, h].float().abs().sum() * k[a:b, kv].float().abs().max()) / math.sqrt(D)
                slack = (2.0 ** -4 + 2.0 ** -13) * size
                bound = (math.expm1(2 * slack) + 2 * 2.0 ** -4) * float(top)
                off = (got[s, h, 0].float() - out[b - 1, h].float()).abs().max()
                assert float(off) <= bound, (t, s, h)
        # (frozen heads see K in neither: only V is rounded there)
        assert cache.device_status() == (0, 0) and packed.device_status() == (0, 0)
        logits = (got[:, :, 0].float().flatten(1) @ head).contiguous()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_wait_for_what_writes_their_inputs(api, captured):
    """Inputs written by a long kernel just before the call, and right behind it overwritten: the
    same bits as with synchronised ones (behind a join of two streams too, and that in a graph)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(s, device="cuda", generator=gen)
    total, H, d, cu = 700, 4, 64, torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    turn = api.Rotary(d)
    layer = api.PackedAttention(H, d, [0, 1, 0, 0], max_total=total, max_seqs=2, max_len=400)
    search = api.BeamSearch(2, 4, 50000)
    big = draw(4096, 4096)
    ints = lambda *s: torch.randint(0, 400, s, device="cuda", generator=gen, dtype=torch.int32)
    # every input, and what the calls see until it is written
    src = dict(x=draw(total, 3 * H, d).bfloat16(), cu=cu, alpha=draw(H, 400), rho=draw(H, 400),
               at=ints(total), logits=draw(8, 50000), scores=torch.zeros(8, device="cuda"),
               history=ints(8, 20), n=torch.tensor([7], dtype=torch.int32, device="cuda"))
    now = {k: torch.zeros_like(t) for k, t in src.items()}

    def fill(slow):
        # 4096^3 products ahead of the copies keep the calls' predecessors running
        z = (big @ big @ big)[0, 0] * 0 if slow else torch.zeros((), device="cuda")
        z = z.nan_to_num(0.0)
        for k, t in src.items():
            now[k].copy_(t + z.to(t.dtype))

    def calls(slow, behind=None):
        res, w = [], now
        q, k, v = w["x"][:, :H], w["x"][:, H:2 * H], w["x"][:, 2 * H:]
        for call in (lambda: turn.apply(q, k, cu_seqlens=w["cu"]),
                     lambda: turn.apply(q, k, positions=w["at"]),
                     lambda: layer.forward(q, k, v, w["cu"], w["alpha"], w["rho"]),
                     lambda: search.step(w["logits"], w["scores"], history=w["history"],
                                         n_tokens=w["n"])):
            fill(slow)
            if behind is not None:
                behind.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(behind):
                    w["logits"].add_(0.0)
                torch.cuda.current_stream().wait_stream(behind)
            res += [t for t in call() if t is not None]
            for t in w.values():
                t.zero_()
        # (and the kernels of the backward one another)
        fill(slow)
        out, lse = layer.forward(q, k, v, w["cu"], w["alpha"], w["rho"])
        res += layer.backward(q, k, v, out, lse, out, w["cu"], w["alpha"], w["rho"])[1:]
        return res
    want = calls(False)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    if not captured:
        got = calls(True)
        want, got = want + want, got + calls(True, other)
    else:
        calls(True, other)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls(True, other)
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
