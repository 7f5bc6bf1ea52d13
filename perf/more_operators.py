"""Measured cases of three operators around the hybrid layer, each next to its plain form.

* ``prefill``, ``train``  the hybrid layer on sequences of different lengths laid end to end:
  rows cu[s] <= i < cu[s + 1] of [total, heads, d] are sequence s; dynamic heads run causal
  softmax attention inside a sequence, frozen heads mix V by softmax(alpha(j) + rho(i - j)),
  i and j counted from the sequence's first row.  ``train`` is the forward and its backward.
* ``rotary``  turns pairs of Q's and K's components by position times frequency (and back: the
  gradient), in both layouts, over a part of the head, at positions given in any of the ways in
  which the layer's callers have them
* ``beam``  one step of beam search: the best beams of each group over beams x vocabulary by
  accumulated log probability, their parents (what a fork of the cache takes), tokens, and the
  histories of tokens reordered
"""

import math
import random

import torch

own = False

DEV = "cuda"
MASKED = -2.3e38  # values below count as -inf (a mask of the type's lowest value)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short prompts that arrive together, 124M-shaped layer: the smallest call
        dict(name="prefill_short", op="prefill", seqs=6, longest=100, heads=12, kv_heads=12, dim=64,
             frozen=3, layout="fused", tail=0, masked=False, empty=False),
        # a batch of prompts of every length up to the training length, with rows of padding
        # behind the last and a slot without tokens
        dict(name="prefill_124m", op="prefill", seqs=16, longest=4096, heads=12, kv_heads=12,
             dim=64, frozen=3, layout="fused", tail=77, masked=True, empty=True),
        # two long prompts and two short ones, 1B shape with grouped K/V
        dict(name="prefill_1b", op="prefill", seqs=4, longest=8192, heads=16, kv_heads=4, dim=128,
             frozen=4, layout="rows", tail=0, masked=False, empty=False),
        # many short documents of a fine-tuning set, small heads
        dict(name="train_short", op="train", seqs=40, longest=300, heads=4, kv_heads=2, dim=32,
             frozen=1, layout="heads", tail=5, masked=True, empty=True),
        # a training batch of the 124M shape, packed documents instead of rows of 4096
        dict(name="train_124m", op="train", seqs=16, longest=4096, heads=12, kv_heads=12, dim=64,
             frozen=3, layout="fused", tail=0, masked=False, empty=False),
        # a training batch of the 1B shape with grouped K/V
        dict(name="train_1b", op="train", seqs=3, longest=8192, heads=16, kv_heads=8, dim=128,
             frozen=4, layout="fused", tail=0, masked=False, empty=False),
        # one token for each of 64 sequences on its way into the cache
        dict(name="rotary_token", op="rotary", seqs=64, longest=4096, new=1, heads=12, kv_heads=12,
             dim=64, turned=64, layout="half", where="cache", wide=False, back=False, base=10000.0,
             stretch=1.0, far=0),
        # Q and K of a packed training batch, parts of one projection's output
        dict(name="rotary_124m", op="rotary", seqs=16, longest=4096, new=0, heads=12, kv_heads=12,
             dim=64, turned=64, layout="half", where="packed", wide=False, back=False,
             base=10000.0, stretch=1.0, far=0),
        # the gradient for half-turned heads of long contexts, positions given token by token
        dict(name="rotary_far_grad", op="rotary", seqs=2, longest=8190, new=8190, heads=16,
             kv_heads=4, dim=128, turned=64, layout="interleaved", where="given", wide=True,
             back=True, base=500000.0, stretch=8.0, far=1000000),
        # the first step of one search, only one beam alive
        dict(name="beam_first", op="beam", groups=1, beams=4, vocab=32000, wide=False, first=True,
             finished=False, masked=False, history=128, step=0),
        # a step of the 12 sequences with 4 beams each that the cache forks
        dict(name="beam_step", op="beam", groups=12, beams=4, vocab=50001, wide=True, first=False,
             finished=True, masked=False, history=512, step=311),
        # a large batch of wide beams over a large vocabulary, some tokens forbidden
        dict(name="beam_wide", op="beam", groups=64, beams=8, vocab=128003, wide=True, first=False,
             finished=True, masked=True, history=1024, step=1000),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng: random.Random):
    op = rng.choice(["prefill", "prefill", "train", "train", "rotary", "rotary", "beam", "beam"])
    if op == "beam":
        while True:
            groups, beams, vocab = _spread(rng, 1, 128), rng.randint(1, 16), _spread(rng, 1000, 200000)
            if groups * beams * vocab <= 64 * 8 * 128003:
                break
        history = _spread(rng, 1, 1500)
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, wide=rng.random() < 0.5,
                    first=rng.random() < 0.3, finished=rng.random() < 0.5,
                    masked=rng.random() < 0.4, history=history, step=rng.randint(0, history - 1))
    dim, kv = rng.choice([32, 64, 64, 128, 128]), rng.choice([1, 2, 3, 4, 8, 12])
    heads = kv * rng.choice([1, 1, 2, 3, 4, 8])
    if op == "rotary":
        while True:
            seqs, longest = _spread(rng, 1, 64), _spread(rng, 1, 16384)
            where = rng.choice(["packed", "cache", "given", "plain"])
            new = 0 if where == "packed" else min(longest, rng.choice([1, _spread(rng, 1, 8192)]))
            rows = seqs * (new or longest)
            if rows * (heads + kv) * dim <= 65536 * 24 * 64:
                break
        return dict(op=op, seqs=seqs, longest=longest, new=new, heads=heads, kv_heads=kv, dim=dim,
                    turned=rng.choice([dim, dim, dim // 2, dim // 4, dim - 6]),
                    layout=rng.choice(["half", "interleaved"]), where=where,
                    wide=rng.random() < 0.4, back=rng.random() < 0.4,
                    base=rng.choice([10000.0, 500000.0]), stretch=rng.choice([1.0, 1.0, 4.0, 8.0]),
                    far=rng.choice([0, 0, 100000, 1000000]))
    while True:
        case = dict(op=op, seqs=_spread(rng, 1, 64), longest=_spread(rng, 1, 8192), heads=heads,
                    kv_heads=kv, dim=dim, frozen=rng.choice([0, heads // 4, rng.randint(0, heads)]),
                    layout=rng.choice(["fused", "rows", "heads"]),
                    tail=rng.choice([0, 0, rng.randint(1, 300)]), masked=rng.random() < 0.4,
                    empty=rng.random() < 0.4)
        lens = _lengths(case)
        if (heads * dim * sum(n * n for n in lens) <= 16 * 128 * 2.2 * 8192 ** 2
                and (sum(lens) + case["tail"]) * (heads + 2 * kv) * dim <= 2 ** 27):
            return case


def _lengths(case):
    """Tokens of each sequence: the first is the longest, the others spread below it."""
    n, t = case["seqs"], case["longest"]
    lens = [t if b == 0 else 1 + int((b * 0.6180339887) % 1.0 * t) for b in range(n)]
    if case.get("empty"):
        lens = [0 if b % 5 == 3 else x for b, x in enumerate(lens)]
    return lens


def _frozen(case):
    """Host list: 1 for each frozen query head."""
    h, n = case["heads"], case["frozen"]
    at = {i * h // n for i in range(n)} if n else set()
    return [int(i in at) for i in range(h)]


def _frequencies(case):
    """Frequency of each turned pair in radians a token, in 64 bits.  A context ``stretch`` times
    longer than the trained one (4096) keeps the fast pairs as they are and slows the slow ones
    down, with a ramp between one and 32 turns over the trained context."""
    n = case["turned"] // 2
    out = [case["base"] ** (-2.0 * p / case["turned"]) for p in range(n)]
    if case["stretch"] == 1.0:
        return out
    full = []
    for f in out:
        turns = 4096 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        full.append(f * keep + f / case["stretch"] * (1.0 - keep))
    return full


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "beam":
        _prepare_beam(s, case, gen)
    elif case["op"] == "rotary":
        _prepare_rotary(s, case, gen)
    else:
        _prepare_packed(s, case, gen)
    return s


def _normal(gen, *shape):
    return torch.randn(shape, device=DEV, generator=gen)


def _starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _prepare_packed(s, case, gen):
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    s["lens"], s["frozen"] = _lengths(case), _frozen(case)
    cu = _starts(s["lens"])
    total = cu[-1] + case["tail"]
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    # the rows behind the last sequence hold what was there before: anything
    if case["layout"] == "heads":
        x = _normal(gen, H + 2 * Hkv, total, d).to(torch.bfloat16).transpose(0, 1)
    else:
        x = _normal(gen, total, H + 2 * Hkv, d).to(torch.bfloat16)
    x[cu[-1]:] = torch.nan
    s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if case["layout"] == "rows":
        s["q"], s["k"], s["v"] = (s[n].contiguous() for n in "qkv")
    T = case["longest"]
    dist = torch.arange(T, device=DEV, dtype=torch.float32)
    s["alpha"] = _normal(gen, H, T)
    s["rho"] = 0.3 * _normal(gen, H, T) - torch.log1p(dist)
    if case["masked"]:
        # every second head looks back over a window, every third does not see the first tokens
        s["rho"][::2, 200:] = torch.finfo(torch.float32).min
        s["alpha"][::3, :5] = -torch.inf
    if case["op"] == "train":
        s["dout"] = _normal(gen, total, H, d).to(torch.bfloat16)
        s["dout"][cu[-1]:] = torch.nan
    if own:
        from dynamic_causal_attention_gb300 import api
        s["layer"] = api.PackedAttention(H, d, s["frozen"], max_total=total, max_seqs=case["seqs"],
                                         max_len=T, H_kv=Hkv, backward=case["op"] == "train",
                                         device=DEV)


def _prepare_rotary(s, case, gen):
    H, Hkv, d, n = case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    t = torch.float32 if case["wide"] else torch.bfloat16
    lens = _lengths(case)
    i32 = dict(dtype=torch.int32, device=DEV)
    s["freqs"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV)
    if case["where"] == "packed":
        s["lens"] = lens
        s["cu"] = torch.tensor(_starts(lens), **i32)
        x = _normal(gen, sum(lens), H + 2 * Hkv, d).to(t)  # a projection's output: Q, K and V
        s["q"], s["k"] = x[:, :H], x[:, H:H + Hkv]
    else:
        new = case["new"]
        s["q"], s["k"] = _normal(gen, n, H, new, d).to(t), _normal(gen, n, Hkv, new, d).to(t)
        if case["where"] == "cache":
            # tokens of each slot, the new ones among them; a chunk that some slots do not fill
            s["lens"] = torch.tensor([case["far"] + max(new, x) for x in lens], **i32)
            s["news"] = torch.tensor([new if b % 3 == 0 else (b * 7919) % (new + 1)
                                      if new > 1 else 1 for b in range(n)], **i32)
        elif case["where"] == "given":
            first = torch.randint(0, case["far"] + 1, (n, 1), device=DEV, generator=gen)
            s["pos"] = (first + torch.arange(new, device=DEV)).to(torch.int32)
    if own:
        from dynamic_causal_attention_gb300 import api
        s["rotary"] = api.Rotary(d, freqs=_frequencies(case), layout=case["layout"], device=DEV)


def _prepare_beam(s, case, gen):
    G, K, V = case["groups"], case["beams"], case["vocab"]
    n = G * K
    x = 2.0 * _normal(gen, n, V)
    # a few tokens that the model thinks likely
    at = torch.randint(0, V, (n, 20), device=DEV, generator=gen)
    x.scatter_add_(1, at, 6.0 * torch.rand((n, 20), device=DEV, generator=gen))
    if case["masked"]:
        x = torch.where(torch.rand((n, V), device=DEV, generator=gen) < 0.05, -torch.inf, x)
        x[:, ::97] = torch.finfo(torch.bfloat16).min
    s["logits"] = x if case["wide"] else x.to(torch.bfloat16)
    s["scores"] = -30.0 * torch.rand(n, device=DEV, generator=gen) / K - 20.0
    if case["first"]:
        s["scores"] = torch.where(torch.arange(n, device=DEV) % K == 0, 0.0, -torch.inf)
    done = torch.rand(n, device=DEV, generator=gen) < 0.2
    s["finished"] = done if case["finished"] else torch.zeros_like(done)
    s["history"] = torch.randint(0, V, (n, case["history"]), device=DEV, generator=gen).to(torch.int32)
    s["history_out"] = torch.zeros_like(s["history"])
    s["step"] = torch.tensor([case["step"]], dtype=torch.int32, device=DEV)
    s["end"] = 2  # the token that ends a sequence
    if own:
        from dynamic_causal_attention_gb300 import api
        s["search"] = api.BeamSearch(G, K, V, end=s["end"], device=DEV)


# ------------------------------------------------------------------ run
def run(s):
    op = s["case"]["op"]
    return (_OWN if own else _PLAIN)[op](s)


def _own_prefill(s):
    return s["layer"].forward(s["q"], s["k"], s["v"], s["cu"], s["alpha"], s["rho"])


def _own_train(s):
    out, lse = s["layer"].forward(s["q"], s["k"], s["v"], s["cu"], s["alpha"], s["rho"])
    grads = s["layer"].backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["cu"], s["alpha"],
                                s["rho"])
    return (out, lse, *grads)


def _own_rotary(s):
    where = {"packed": lambda: dict(cu_seqlens=s["cu"]), "plain": dict,
             "cache": lambda: dict(seq_len=s["lens"], n_new=s["news"]),
             "given": lambda: dict(positions=s["pos"])}[s["case"]["where"]]()
    return s["rotary"].apply(s["q"], s["k"], inverse=s["case"]["back"], **where)


def _own_beam(s):
    return s["search"].step(s["logits"], s["scores"], s["finished"], history=s["history"],
                            n_tokens=s["step"], history_out=s["history_out"])


def _weights(s, a, n, heads, g):
    """Logits [heads, n, n] of one sequence's heads, -inf where a row does not look."""
    i = torch.arange(n, device=DEV)
    out = []
    for h in heads:
        if s["frozen"][h]:
            x = s["alpha"][h, :n][None] + s["rho"][h][(i[:, None] - i[None]).clamp(min=0)]
            x = torch.where(x < MASKED, -torch.inf, x)
        else:
            x = s["q"][a:a + n, h].float() @ s["k"][a:a + n, h // g].float().T
            x *= s["case"]["dim"] ** -0.5
        out.append(x.masked_fill_(i[None] > i[:, None], -torch.inf))
    return torch.stack(out)


def _plain_packed(s, back):
    """Sequence by sequence, K/V head by K/V head, in 32 bits."""
    c = s["case"]
    H, Hkv, d = c["heads"], c["kv_heads"], c["dim"]
    g, total = H // Hkv, s["q"].shape[0]
    out = torch.zeros((total, H, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((H, total), -torch.inf, device=DEV)
    dq, dk, dv = (torch.zeros((total, h, d), dtype=torch.bfloat16, device=DEV) for h in (H, Hkv, Hkv))
    a = 0
    for n in s["lens"]:
        for kv in range(Hkv if n else 0):
            heads = list(range(kv * g, kv * g + g))
            x = _weights(s, a, n, heads, g)
            top = x.amax(-1, keepdim=True)
            top = torch.where(top == -torch.inf, 0.0, top)
            p = torch.exp(x - top)
            sums = p.sum(-1, keepdim=True)
            lse[heads, a:a + n] = (top + torch.log(sums))[..., 0]
            p /= torch.where(sums > 0, sums, 1.0)
            v = s["v"][a:a + n, kv].float()
            out[a:a + n, heads] = (p @ v).transpose(0, 1).to(torch.bfloat16)
            if not back:
                continue
            do = s["dout"][a:a + n, heads].float().transpose(0, 1)            # [g, n, d]
            dv[a:a + n, kv] = (p.transpose(1, 2) @ do).sum(0).to(torch.bfloat16)
            live = [h for h in heads if not s["frozen"][h]]
            if live:
                at = [h - kv * g for h in live]
                dp = do[at] @ v.T
                ds = p[at] * (dp - (p[at] * dp).sum(-1, keepdim=True)) * d ** -0.5
                key = s["k"][a:a + n, kv].float()
                dq[a:a + n, live] = (ds @ key).transpose(0, 1).to(torch.bfloat16)
                q = s["q"][a:a + n, live].float().transpose(0, 1)
                dk[a:a + n, kv] = (ds.transpose(1, 2) @ q).sum(0).to(torch.bfloat16)
        a += n
    return (out, lse, dq, dk, dv) if back else (out, lse)


def _positions(s):
    """(position of each row, which rows are turned)."""
    c = s["case"]
    if c["where"] == "packed":
        i = torch.arange(s["q"].shape[0], device=DEV)
        return i - s["cu"].long()[torch.searchsorted(s["cu"].long(), i, right=True) - 1], None
    t = torch.arange(c["new"], device=DEV)
    if c["where"] == "cache":
        return (s["lens"] - s["news"])[:, None] + t, t < s["news"][:, None]
    if c["where"] == "given":
        return s["pos"], None
    return t.expand(c["seqs"], -1), None


def _plain_rotary(s):
    c = s["case"]
    pos, live = _positions(s)
    angle = pos.double()[..., None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["back"]:
        sin = -sin
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)  # the heads' axis of Q and K
    n = c["turned"]

    def turn(x):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :n // 2], y[..., n // 2:n]
            new = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:n:2], y[..., 1:n:2]
            new = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        y = torch.cat([new, y[..., n:]], -1).to(x.dtype)
        return y if live is None else torch.where(live[:, None, :, None], y, torch.zeros_like(y))
    return turn(s["q"]), turn(s["k"])


def _plain_beam(s):
    c = s["case"]
    G, K, V = c["groups"], c["beams"], c["vocab"]
    x = s["logits"].double()
    x = torch.where((x >= MASKED) & (x < torch.inf), x, -torch.inf)
    top = x.amax(1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    x -= top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    x = torch.where(torch.isnan(x), -torch.inf, x)
    x += s["scores"].double()[:, None]
    # a finished beam has one way on: the ending token again, at no cost
    still = torch.full_like(x[:1], -torch.inf)
    x = torch.where(s["finished"][:, None], still, x)
    x[:, s["end"]] = torch.where(s["finished"], s["scores"].double(), x[:, s["end"]])
    x = x.view(G, K * V)
    parent, token, score = [], [], []
    place = torch.arange(K * V, device=DEV)
    for _ in range(K):
        best = x.amax(1, keepdim=True)
        at = torch.where(x == best, place, K * V).amin(1)              # ties: the lowest
        alive = best[:, 0] > -torch.inf
        parent.append(torch.where(alive, torch.arange(G, device=DEV) * K + at // V, -1))
        token.append(torch.where(alive, at % V, -1))
        score.append(best[:, 0])
        x.scatter_(1, at[:, None], -torch.inf)
    parent, token = (torch.stack(t, 1).flatten().to(torch.int32) for t in (parent, token))
    score = torch.stack(score, 1).flatten().float()
    finished = (parent >= 0) & (token == s["end"])
    col, n = torch.arange(c["history"], device=DEV), s["step"]
    rows = torch.where((parent >= 0)[:, None], s["history"][parent.clamp(min=0).long()], -1)
    rows = torch.where(col < n, rows, token[:, None])
    return parent, token, score, finished, torch.where(col <= n, rows, s["history_out"])


_OWN = {"prefill": _own_prefill, "train": _own_train, "rotary": _own_rotary, "beam": _own_beam}
_PLAIN = {"prefill": lambda s: _plain_packed(s, False), "train": lambda s: _plain_packed(s, True),
          "rotary": _plain_rotary, "beam": _plain_beam}


# ------------------------------------------------------------------ work
def work(case):
    """Bytes that the call cannot do without (each input read once, each output written once),
    and the products' operations."""
    if case["op"] == "beam":
        n = case["groups"] * case["beams"]
        size = n * case["vocab"] * (4 if case["wide"] else 2)
        return {"bytes": size + n * 22 + 4 * n * (2 * case["step"] + 1),
                "flops": 4 * n * case["vocab"]}
    H, Hkv, d, lens = case["heads"], case["kv_heads"], case["dim"], _lengths(case)
    if case["op"] == "rotary":
        n, new = case["seqs"], case["new"]
        rows = sum(lens) if case["where"] == "packed" else n * new
        turned = rows
        if case["where"] == "cache":
            turned = sum(new if b % 3 == 0 else (b * 7919) % (new + 1) if new > 1 else 1
                         for b in range(n))
        size = (H + Hkv) * d * (4 if case["wide"] else 2)
        return {"bytes": (rows + turned) * size + 4 * (rows if case["where"] == "given" else n),
                "flops": turned * (H + Hkv) * case["turned"] * 3}
    m, g = _frozen(case), H // Hkv
    ice, dyn = sum(m), H - sum(m)
    keyed = sum(1 for kv in range(Hkv) if not all(m[kv * g:kv * g + g]))  # K heads that are read
    rows, pairs = sum(lens) + case["tail"], sum(n * (n + 1) // 2 for n in lens)
    live = sum(lens)
    size = 2 * d * (live * (dyn + keyed + Hkv) + rows * H) + 4 * H * rows
    size += 8 * ice * max(lens) + 4 * len(lens)
    flops = pairs * d * (4 * dyn + 2 * ice)
    if case["op"] == "train":
        size += 2 * d * (live * H + rows * (H + 2 * Hkv))
        flops += pairs * d * (8 * dyn + 2 * ice)
    return {"bytes": size, "flops": flops}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The outputs from their definition in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "beam":
        return _exact_beam(case, s)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    return _exact_packed(case, s)


def _exact_packed(case, s):
    """One head of one sequence at a time; the gradients by automatic differentiation."""
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    back, total, g = case["op"] == "train", s["q"].shape[0], H // Hkv
    f64 = dict(dtype=torch.float64, device=DEV)
    out, lse = torch.zeros((total, H, d), **f64), torch.full((H, total), -torch.inf, **f64)
    grads = [torch.zeros((total, h, d), **f64) for h in (H, Hkv, Hkv)]
    a = 0
    for n in s["lens"]:
        b = a + n
        for h in range(H if n else 0):
            kv = h // g
            q, k, v = (t[a:b].double().detach().requires_grad_(back)
                       for t in (s["q"][:, h], s["k"][:, kv], s["v"][:, kv]))
            with torch.set_grad_enabled(back):
                j = torch.arange(n, device=DEV)
                if s["frozen"][h]:
                    table = torch.nn.functional.pad(s["rho"][h, :n].double().flip(0), (0, n - 1),
                                                    value=-torch.inf)
                    x = s["alpha"][h, :n].double()[None] + table.unfold(0, n, 1).flip(0)[:n]
                    x = torch.where(x < MASKED, -torch.inf, x)
                else:
                    x = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
                    x = x + torch.where(j[:, None] >= j, 0.0, -torch.inf)
                z = torch.logsumexp(x, 1)
                y = torch.exp(x - torch.where(z > -torch.inf, z, 0.0)[:, None]) @ v
            out[a:b, h], lse[h, a:b] = y.detach(), z.detach()
            if back:
                wanted = (v,) if s["frozen"][h] else (q, k, v)
                got = torch.autograd.grad(y, wanted, s["dout"][a:b, h].double())
                grads[2][a:b, kv] += got[-1]
                if len(got) > 1:
                    grads[0][a:b, h] = got[0]
                    grads[1][a:b, kv] += got[1]
            del x, z, y
        a = b
    return (out, lse, *grads) if back else (out, lse)


def _exact_rotary(case, s):
    """The pairs as complex numbers."""
    n = case["turned"]
    pos, live = _positions(s)
    turn = torch.polar(torch.ones_like(pos[..., None] * s["freqs"]), pos.double()[..., None] * s["freqs"])
    if case["back"]:
        turn = turn.conj()

    def one(x):
        y = x.double()
        w = turn.unsqueeze(1)
        if case["layout"] == "half":
            z = torch.complex(y[..., :n // 2], y[..., n // 2:n]) * w
            y = torch.cat([z.real, z.imag, y[..., n:]], -1)
        else:
            z = torch.view_as_complex(y[..., :n].unflatten(-1, (n // 2, 2)).contiguous()) * w
            y = torch.cat([torch.view_as_real(z).flatten(-2), y[..., n:]], -1)
        return y if live is None else y * live[:, None, :, None]
    return one(s["q"]), one(s["k"])


def _exact_beam(case, s):
    """The scores alone: the group's candidates sorted."""
    G, K, V = case["groups"], case["beams"], case["vocab"]
    score = torch.empty((G, K), dtype=torch.float64, device=DEV)
    for g in range(G):
        ways = []
        for b in range(g * K, g * K + K):
            if bool(s["finished"][b]):
                ways.append(s["scores"][b:b + 1].double())
                continue
            x = s["logits"][b].double()
            x = x[(x >= MASKED) & (x < torch.inf)]
            ways.append(s["scores"][b].double() + torch.log_softmax(x, 0))
        best = torch.sort(torch.cat(ways), descending=True).values[:K]
        score[g] = -torch.inf
        score[g, :best.numel()] = best
    return None, None, score.flatten(), None, None
