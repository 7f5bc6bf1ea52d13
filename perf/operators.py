"""Measured cases of the paged 8-bit cache: the calls a serving program makes of it, each next
to its plain form.

A page of the cache holds ``page`` tokens of every layer.  One layer's record in a page is

    K codes [H_k, page, d] | V codes [H_kv, page, d] | K scales [H_k] | V scales [H_kv]

(codes: e4m3, one byte; scales: fp32, one for each block of ``page`` tokens and head), padded
to a multiple of 128 bytes.  H_k counts the K/V heads that serve at least one dynamic query
head: a frozen head's weights come from its alpha/rho vectors, so its K is never stored.  A
page table row lists the pages of one sequence; ``ref`` counts how many rows hold a page.

Operators (the ``op`` of a case):

* ``append``   quantises new K/V rows into the pages (power-of-two block scales)
* ``attend``   the hybrid layer over the cache: dynamic heads run softmax attention over the
               dequantised K/V, frozen heads mix V by softmax(alpha(j) + rho(i - j))
* ``grow``     pages for the tokens to come; a shared last page is copied first
* ``fork``     rows take over the pages of their parents' rows (fork, reorder, free)
* ``compact``  used pages move into the lowest page numbers
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence of the 124M-shaped layer, a few words in: the smallest serving call
        dict(name="token_alone", op="attend", seqs=1, heads=12, kv_heads=12, dim=64, page=64,
             tokens=100, new=1, frozen=3, packed=False, ragged=False),
        # a decode step of the 124M-shaped layer with grouped K/V, sequences of every age up to
        # its training length
        dict(name="tokens_124m", op="attend", seqs=48, heads=12, kv_heads=4, dim=64, page=32,
             tokens=4096, new=1, frozen=3, packed=False, ragged=True),
        # a decode step of the 1B-shaped layer, a full batch at its training length
        dict(name="tokens_1b", op="attend", seqs=32, heads=16, kv_heads=16, dim=128, page=64,
             tokens=8192, new=1, frozen=4, packed=False, ragged=False),
        # a prompt's next chunk over what the cache holds already, 1B shape with grouped K/V
        dict(name="chunk_1b", op="attend", seqs=2, heads=16, kv_heads=4, dim=128, page=128,
             tokens=8192, new=2000, frozen=4, packed=True, ragged=False),
        # what precedes every decode step: one token for each of 64 sequences
        dict(name="append_tokens", op="append", seqs=64, heads=12, kv_heads=12, dim=64, page=64,
             tokens=1500, new=1, frozen=3, packed=False, ragged=True, wide=True),
        # four prompts written at once, the first page of each already begun
        dict(name="append_prompts", op="append", seqs=4, heads=16, kv_heads=16, dim=128, page=64,
             tokens=8190, new=1999, frozen=4, packed=False, ragged=False, wide=False),
        # pages for the next token of 64 sequences that were forked from 16: shared last pages
        # are copied for all 12 layers
        dict(name="grow_step", op="grow", seqs=64, columns=64, pages=2048, layers=12, kv_heads=4,
             dim=64, page=64, tokens=3001, new=1, shared=4),
        # 200 prompts admitted at once into a cache of small pages
        dict(name="grow_prompts", op="grow", seqs=200, columns=512, pages=65536, layers=1,
             kv_heads=4, dim=64, page=16, tokens=500, new=4001, shared=1),
        # a beam step of 12 sequences with 4 beams each
        dict(name="fork_beams", op="fork", seqs=48, columns=64, pages=2048, page=64, tokens=4001,
             beams=4),
        # a round of forks and releases over a large batch of long sequences
        dict(name="fork_many", op="fork", seqs=1000, columns=1024, pages=200000, page=64,
             tokens=60001, beams=5),
        # a small cache after a few releases
        dict(name="compact_small", op="compact", seqs=20, columns=40, pages=512, layers=1,
             kv_heads=4, dim=64, page=32, used=301, moved=40),
        # a 12-layer cache whose owner wants a quarter of its memory back
        dict(name="compact_large", op="compact", seqs=100, columns=128, pages=8192, layers=12,
             kv_heads=2, dim=64, page=128, used=5801, moved=1700),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng: random.Random):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "grow", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([32, 64, 64, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 12, 16])
    if op in ("attend", "append"):
        heads = kv * rng.choice([1, 1, 2, 3, 4, 8])
        frozen = rng.choice([0, rng.randint(0, heads), rng.randint(0, heads), heads // 4])
        while True:
            seqs, tokens = _spread(rng, 1, 64), _spread(rng, 1, 32768)
            kind = rng.random()
            new = 1 if kind < 0.5 else min(tokens, rng.randint(2, 8)) if kind < 0.7 \
                else min(tokens, _spread(rng, 9, 2000))
            cost = seqs * tokens * kv * dim
            rows = seqs * heads * new
            if cost <= 32 * 8192 * 16 * 128 and rows * tokens <= 2 * 16 * 2000 * 8192 \
                    and rows * dim <= 2 * 16 * 2000 * 128 and seqs * kv * new * dim <= 4 * 16 * 1999 * 128:
                break
        case = dict(op=op, seqs=seqs, heads=heads, kv_heads=kv, dim=dim, page=page, tokens=tokens,
                    new=new, frozen=frozen, packed=rng.random() < 0.5, ragged=rng.random() < 0.6)
        if op == "append":
            case["wide"] = rng.random() < 0.3
        return case
    layers = rng.choice([1, 2, 12])
    record = _record(kv, kv, page, dim)[-1] * layers
    if op == "compact":
        pages = min(_spread(rng, 16, 60000), max(16, (2 << 30) // record))
        used = rng.randint(1, pages)
        moved = min(rng.randint(0, used), pages - used, max(1, (600 << 20) // record))
        columns = _spread(rng, 8, 256)
        return dict(op=op, seqs=-(-used // columns) + rng.randint(0, 9), columns=columns, pages=pages,
                    layers=layers, kv_heads=kv, dim=dim, page=page, used=used, moved=moved)
    seqs, columns = _spread(rng, 1, 600), _spread(rng, 2, 600)
    tokens = rng.randint(1, columns * page)
    if op == "fork":
        return dict(op=op, seqs=seqs, columns=columns, pages=seqs * columns + rng.randint(1, 999),
                    page=page, tokens=tokens, beams=rng.randint(1, 8))
    new = 1 if rng.random() < 0.6 else _spread(rng, 2, columns * page)
    pages = max(64, min(seqs * columns + rng.randint(0, 999), (1 << 30) // record))
    seqs = max(1, min(seqs, pages // (2 * columns), max(1, (400 << 20) // record)))
    if seqs * columns * 2 > pages:
        columns = max(1, pages // (2 * seqs))
        tokens, new = min(tokens, columns * page), min(new, columns * page)
    return dict(op=op, seqs=seqs, columns=columns, pages=pages, layers=layers, kv_heads=kv,
                dim=dim, page=page, tokens=tokens, new=new, shared=rng.randint(1, 4))


# ------------------------------------------------------------------ layout
def _record(h_k, h_kv, page, dim):
    """Byte offsets of (V codes, K scales, V scales) in a layer's record, and its length."""
    v = h_k * page * dim
    ks = v + h_kv * page * dim
    vs = ks + 4 * h_k
    return v, ks, vs, (vs + 4 * h_kv + 127) // 128 * 128


def _frozen(case):
    """Host list: 1 for each frozen query head."""
    h, n = case["heads"], case["frozen"]
    at = range(n) if case["packed"] else [i * h // n for i in range(n)]
    return [int(i in set(at)) for i in range(h)]


def _k_heads(case):
    """The K/V heads whose K is stored: those with a dynamic query head."""
    m, g = _frozen(case), case["heads"] // case["kv_heads"]
    return [k for k in range(case["kv_heads"]) if not all(m[k * g:(k + 1) * g])]


def _lengths(case):
    """Tokens of each sequence, the new ones among them."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [t] * n
    return [max(case["new"], t if b == 0 else 1 + int((b * 0.6180339887) % 1.0 * t)) for b in range(n)]


def _news(case):
    """New tokens of each sequence: a ragged step leaves some sequences out or short."""
    n, new = case["seqs"], case["new"]
    if not case["ragged"] or new == 1:
        return [new] * n
    return [new if b % 3 == 0 else (b * 7919) % (new + 1) for b in range(n)]


def _views(pool, h_k, h_kv, page, dim):
    """(K codes, V codes, K scales, V scales) of a one-layer pool [n_pages, record bytes]."""
    n, (v, ks, vs, _) = pool.shape[0], _record(h_k, h_kv, page, dim)
    return (pool[:, :v].view(n, h_k, page, dim), pool[:, v:ks].view(n, h_kv, page, dim),
            pool[:, ks:vs].view(torch.float32), pool[:, vs:vs + 4 * h_kv].view(torch.float32))


def _pow2(e):
    """2^e as fp32, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e >= -64 with 448 * 2^e >= amax (448 = 0.875 * 2^9: the largest e4m3 value)."""
    m, x = torch.frexp(amax)
    return (x - 9 + (m > 0.875)).clamp(min=-64)


def _encode(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


# ------------------------------------------------------------------ prepare
def _tokens(gen, n, heads, page, dim):
    """K or V rows as a model makes them: normal, heads of different size, some large tokens."""
    x = torch.randn((n, heads, page, dim), device=DEV, generator=gen)
    x *= torch.exp(0.4 * torch.randn((1, heads, 1, 1), device=DEV, generator=gen))
    big = torch.rand((n, 1, page, 1), device=DEV, generator=gen) < 0.01
    return torch.where(big, 4.0 * x, x)


def _fill(part, scale, gen, dim_heads):
    """Fill a pool's codes and scales with quantised rows (every page: recycled pages hold the
    rows of the sequences that had them before)."""
    n, heads, page, dim = part.shape
    step = max(1, (1 << 27) // max(1, heads * page * dim))
    for a in range(0, n if heads else 0, step):
        b = min(n, a + step)
        x = _tokens(gen, b - a, heads, page, dim)
        e = _exponent(x.abs().amax(dim=(2, 3)))
        part[a:b] = _encode(x * _pow2(-e)[:, :, None, None])
        scale[a:b] = _pow2(e)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] in ("attend", "append"):
        B, H, Hkv, P, d, new = (case[k] for k in ("seqs", "heads", "kv_heads", "page", "dim", "new"))
        lens, kh = _lengths(case), _k_heads(case)
        cols = -(-case["tokens"] // P)
        need = [-(-n // P) for n in lens]
        n_pages = sum(need) + 3
        ids = torch.randperm(n_pages, device=DEV, generator=gen).to(torch.int32)
        table = torch.full((B, cols), -1, **i32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        pool = torch.zeros((n_pages, _record(len(kh), Hkv, P, d)[-1]), dtype=torch.uint8, device=DEV)
        kc, vc, ks, vs = _views(pool, len(kh), Hkv, P, d)
        _fill(kc, ks, gen, d)
        _fill(vc, vs, gen, d)
        s.update(pool=pool, table=table, lens=torch.tensor(lens, **i32), width=max(lens),
                 news=torch.tensor(_news(case), **i32), frozen=_frozen(case), k_heads=kh)
        if case["op"] == "attend":
            s["q"] = torch.randn((B, H, new, d), device=DEV, generator=gen).to(torch.bfloat16)
            s["alpha"] = torch.randn((H, cols * P), device=DEV, generator=gen)
            dist = torch.arange(cols * P, device=DEV, dtype=torch.float32)
            s["rho"] = 0.3 * torch.randn((H, cols * P), device=DEV, generator=gen) - torch.log1p(dist)
            s["out"] = torch.zeros((B, H, new, d), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros((B, H, new), device=DEV)
        else:
            t = torch.float32 if case["wide"] else torch.bfloat16
            make = lambda: _tokens(gen, B, Hkv, new, d).to(t)  # noqa: E731
            s["k"], s["v"] = make(), make()
        s["n_seqs"], s["columns"], s["n_pages"] = B, cols, n_pages
        layers = [s["frozen"]]
    else:
        S, cols, n_pages, P = (case[k] for k in ("seqs", "columns", "pages", "page"))
        ids = torch.randperm(n_pages, device=DEV, generator=gen)
        col = torch.arange(cols, device=DEV)[None, :]
        slot = torch.arange(S, device=DEV)[:, None]
        if case["op"] == "compact":
            used, moved = case["used"], case["moved"]
            low = torch.randperm(used, device=DEV, generator=gen)[:used - moved]
            high = used + torch.randperm(n_pages - used, device=DEV, generator=gen)[:moved]
            held = torch.cat([low, high])[torch.randperm(used, device=DEV, generator=gen)]
            flat = torch.full((S * cols,), -1, dtype=torch.int64, device=DEV)
            flat[:used] = held
            table = flat.view(S, cols)
        else:
            # groups of sequences that were forked: the same pages, the last one too
            many = case["shared"] if case["op"] == "grow" else case["beams"]
            lens = [1 + (case["tokens"] - 1) * (b // many + 1) // (-(-S // many)) for b in range(S)]
            if case["op"] == "grow":
                lens = [min(n, cols * P) for n in lens]
            s["lens"] = torch.tensor(lens, **i32)
            need = (s["lens"].long()[:, None] + P - 1) // P
            head = slot // many * many
            first = torch.cumsum(torch.where(slot == head, need, 0).flatten(), 0)[:, None] - need[head[:, 0]]
            k = first[head[:, 0]] + col
            table = torch.where(col < need, ids[k.clamp(max=n_pages - 1)], -1)
            if case["op"] == "grow":
                s["news"] = torch.tensor([min(case["new"], cols * P - n) for n in lens], **i32)
            else:
                # each group keeps one beam and refills from it; every seventh group is released
                keep = head + torch.randint(0, many, (S, 1), device=DEV, generator=gen)
                keep = torch.where(torch.rand((S, 1), device=DEV, generator=gen) < 0.5, keep, slot)
                parent = torch.where(slot // many % 7 == 6, -1, keep.clamp(max=S - 1))
                s["parent"] = parent.flatten().to(torch.int32)
        table = table.to(torch.int32)
        ref = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
        ref.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0], dtype=torch.int64))
        s.update(table=table, ref=ref.to(torch.int32), table_out=torch.zeros_like(table),
                 ref_out=torch.zeros(n_pages, **i32), lens_out=torch.zeros(S, **i32))
        heads, n = case.get("kv_heads", 1), case.get("layers", 1)
        stride = _record(heads, heads, P, case.get("dim", 32))[-1] * n
        if case["op"] == "fork":  # touches no page
            s["pool"] = torch.zeros((n_pages, stride), dtype=torch.uint8, device=DEV)
        else:
            s["pool"] = torch.randint(0, 256, (n_pages, stride), dtype=torch.uint8, device=DEV, generator=gen)
        s["n_seqs"], s["columns"], s["n_pages"] = S, cols, n_pages
        layers = [[0] * heads] * n
    if own:
        from dynamic_causal_attention_gb300 import api
        s["cache"] = api.PagedCache(
            layers, case.get("heads", case.get("kv_heads", 1)), case.get("dim", 32),
            H_kv=case.get("kv_heads", 1), n_seqs=s["n_seqs"], max_pages=s["columns"],
            n_pages=s["n_pages"], page_size=case["page"], max_new=case.get("new", 1), device=DEV,
            pool=s["pool"], page_table=s["table"], seq_len=s.get("lens"), ref=s.get("ref"))
    return s


# ------------------------------------------------------------------ run
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_attend(s):
    return s["cache"].attend(0, s["q"], s["alpha"], s["rho"], n_new=s["news"], out=s["out"], lse=s["lse"])


def _own_append(s):
    s["cache"].append(0, s["k"], s["v"], n_new=s["news"])
    return _appended(s)


def _own_grow(s):
    granted, short = s["cache"].grow(s["news"], into=(s["table_out"], s["lens_out"], s["ref_out"]))
    return s["table_out"], s["lens_out"], s["ref_out"], granted, short, s["pool"]


def _own_fork(s):
    s["cache"].fork(s["parent"], into=(s["table_out"], s["lens_out"], s["ref_out"]))
    return s["table_out"], s["lens_out"], s["ref_out"]


def _own_compact(s):
    n = s["cache"].compact(into=(s["table_out"], s["ref_out"]))
    return s["table_out"], s["ref_out"], n, s["pool"]


def _appended(s):
    c = s["case"]
    kc, vc, ks, vs = _views(s["pool"], len(s["k_heads"]), c["kv_heads"], c["page"], c["dim"])
    e4m3 = torch.float8_e4m3fn
    return {"k": kc.view(e4m3), "v": vc.view(e4m3), "k_scale": ks, "v_scale": vs}


def _plain_attend(s):
    c = s["case"]
    B, H, P, d, new, g = c["seqs"], c["heads"], c["page"], c["dim"], c["new"], c["heads"] // c["kv_heads"]
    kc, vc, ks, vs = _views(s["pool"], len(s["k_heads"]), c["kv_heads"], P, d)
    j = torch.arange(s["width"], device=DEV)
    page = s["table"][:, j // P].long()                                   # [B, L]
    there = (page >= 0) & (page < s["n_pages"]) & (j < s["lens"][:, None])
    page = page.clamp(0, s["n_pages"] - 1)
    e4m3 = torch.float8_e4m3fn
    v = vc[page, :, (j % P)[None]].view(e4m3).float() * vs[page][..., None]  # [B, L, H_kv, d]
    v = torch.where(there[:, :, None, None], v, 0.0)
    t = torch.arange(new, device=DEV)
    pos = (s["lens"] - s["news"])[:, None] + t                            # [B, new]
    seen = there[:, None, :] & (j <= pos[:, :, None])                     # [B, new, L]
    logits = torch.empty((B, H, new, s["width"]), device=DEV)
    dyn = [h for h in range(H) if not s["frozen"][h]]
    if dyn:
        k = kc[page, :, (j % P)[None]].view(e4m3).float() * ks[page][..., None]  # [B, L, H_k, d]
        mine = torch.tensor([s["k_heads"].index(h // g) for h in dyn], device=DEV)
        logits[:, dyn] = s["q"][:, dyn].float() @ k[:, :, mine].permute(0, 2, 3, 1) * d ** -0.5
    ice = [h for h in range(H) if s["frozen"][h]]
    if ice:
        dist = (pos[:, :, None] - j).clamp(0, s["rho"].shape[1] - 1)      # [B, new, L]
        logits[:, ice] = (s["alpha"][ice][None, :, None, :s["width"]]
                          + s["rho"][ice][:, dist].transpose(0, 1))
    logits = torch.where(seen[:, None], logits, -torch.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    of = torch.arange(H, device=DEV) // g
    out = p @ v[:, :, of].transpose(1, 2) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    live = (t < s["news"][:, None])[:, None]                              # [B, 1, new]
    return (torch.where(live[..., None], out.to(torch.bfloat16), s["out"]),
            torch.where(live, lse, s["lse"]))


def _plain_append(s):
    c = s["case"]
    P, d, B, new, Hkv = c["page"], c["dim"], c["seqs"], c["new"], c["kv_heads"]
    kc, vc, ks, vs = _views(s["pool"], len(s["k_heads"]), Hkv, P, d)
    cols = (new + P - 2) // P + 1                 # pages that new rows can touch, at most
    first = s["lens"] - s["news"]                 # position of the first new token
    col = (first // P)[:, None] + torch.arange(cols, device=DEV)           # [B, cols]
    pos = col[:, :, None] * P + torch.arange(P, device=DEV)                # [B, cols, P]
    fresh = (pos >= first[:, None, None]) & (pos < s["lens"][:, None, None])
    old = pos < first[:, None, None]
    at = torch.nonzero(fresh.any(-1) & (col < s["table"].shape[1]))
    page = s["table"][at[:, 0], col[at[:, 0], at[:, 1]]].long()
    at, page = at[page >= 0], page[page >= 0]
    fresh, old = fresh[at[:, 0], at[:, 1]][:, None], old[at[:, 0], at[:, 1]][:, None]  # [n, 1, P]
    row = (pos[at[:, 0], at[:, 1]] - first[at[:, 0]][:, None]).clamp(0, new - 1)       # [n, P]
    pairs = [(vc, vs, s["v"])] + ([(kc, ks, s["k"][:, s["k_heads"]])] if s["k_heads"] else [])
    return _plain_pages(s, pairs, at, page, fresh, old, row)


def _plain_pages(s, pairs, at, page, fresh, old, row):
    def write(codes, scales, x):
        x = x.float()[at[:, 0][:, None], :, row].transpose(1, 2)                       # [n, heads, P, d]
        size = torch.where(torch.isfinite(x) & fresh[..., None], x.abs(), 0.0).amax((2, 3))
        kept = codes[page]
        before = torch.where(old.any(-1), scales[page], 0.0)
        scale = torch.maximum(_pow2(_exponent(size)), before)
        again = _encode(kept.view(torch.float8_e4m3fn).float() * (before / scale)[:, :, None, None])
        again = torch.where(old[..., None], again, kept)
        x = _encode(x / scale[:, :, None, None])
        codes[page] = torch.where(fresh[..., None], x, again)
        scales[page] = scale
    write(*pairs[0])
    if len(pairs) > 1:
        write(*pairs[1])
    return _appended(s)


def _plain_grow(s):
    c = s["case"]
    P, table, lens, ref, news = c["page"], s["table"], s["lens"].long(), s["ref"], s["news"].long()
    cols, n_pages = table.shape[1], ref.shape[0]
    n = torch.where((news > 0) & (lens + news <= cols * P), news, 0)
    begin, end = (lens + P - 1) // P, (lens + n + P - 1) // P
    tail = (lens // P).clamp(max=cols - 1)
    held = table.gather(1, tail[:, None])[:, 0].long()
    copy = (n > 0) & (lens % P != 0) & (held >= 0) & (held < n_pages)
    copy = copy & (ref[held.clamp(0, n_pages - 1)] > 1)
    end = torch.where(n > 0, end, begin)
    needs = end - begin + copy
    base = torch.cumsum(needs, 0) - needs
    total = needs.sum()
    free = ref <= 0
    order = torch.argsort(free.logical_not().to(torch.uint8), stable=True)  # free pages first, ascending
    short = (total - free.sum()).clamp(min=0)
    ok = short == 0
    col = torch.arange(cols, device=DEV)
    k = (base + copy)[:, None] + col - begin[:, None]
    taken = ok & (col >= begin[:, None]) & (col < end[:, None])
    table = torch.where(taken, order[k.clamp(0, n_pages - 1)].to(torch.int32), table)
    copy = copy & ok
    to = order[base.clamp(max=n_pages - 1)]
    table = torch.where(copy[:, None] & (col == tail[:, None]), to[:, None].to(torch.int32), table)
    rank = torch.cumsum(free, 0) - 1
    ref = torch.where(free & (rank < total) & ok, 1, ref)
    ref = ref.index_add(0, torch.where(copy, held, 0), -copy.to(torch.int32))
    at = torch.nonzero(copy)[:, 0]
    s["pool"][to[at]] = s["pool"][held[at]]
    granted = torch.where(ok, n, 0).to(torch.int32)
    return table, (lens + granted).to(torch.int32), ref.to(torch.int32), granted, short.to(torch.int32).view(1), s["pool"]


def _plain_fork(s):
    table, ref, n = s["table"], s["ref"], s["n_seqs"]
    parent = s["parent"].long()
    alive = (parent >= 0) & (parent < n)
    parent = parent.clamp(0, n - 1)
    rows = torch.where(alive[:, None], table[parent], -1)
    lens = torch.where(alive, s["lens"][parent], 0)

    def count(t):
        held = (t >= 0) & (t < ref.shape[0])
        return torch.zeros_like(ref).index_add(0, torch.where(held, t, 0).flatten(), held.flatten().to(torch.int32))
    return rows, lens, ref + count(rows) - count(table)


def _plain_compact(s):
    table, ref, n_pages = s["table"], s["ref"], s["n_pages"]
    used = ref > 0
    n = used.sum()
    ids = torch.arange(n_pages, device=DEV)
    source = torch.nonzero(used & (ids >= n))[:, 0]
    target = torch.nonzero(~used & (ids < n))[:, 0]
    s["pool"][target] = s["pool"][source]
    place = ids.clone()
    place[source] = target
    out = torch.where((table >= 0) & (table < n_pages), place[table.clamp(0, n_pages - 1)].to(torch.int32), table)
    ref = ref.clone()
    ref[target] = ref[source]
    ref[source] = 0
    return out, ref, n.to(torch.int32).view(1), s["pool"]


_OWN = {"attend": _own_attend, "append": _own_append, "grow": _own_grow, "fork": _own_fork, "compact": _own_compact}
_PLAIN = {"attend": _plain_attend, "append": _plain_append, "grow": _plain_grow, "fork": _plain_fork,
          "compact": _plain_compact}


# ------------------------------------------------------------------ work
def work(case):
    """Bytes that the call cannot do without (each input read once, each output written once),
    and the products' operations."""
    op, P = case["op"], case["page"]
    if op in ("attend", "append"):
        B, H, Hkv, d, new = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "new"))
        lens, news, m = _lengths(case), _news(case), _frozen(case)
        Hk, dyn = len(_k_heads(case)), m.count(0)
        rows = sum(news)
        if op == "append":
            pages = sum((n - 1) // P - (n - k) // P + 1 for n, k in zip(lens, news) if k)
            # new rows in, their codes out, scales in and out, a table entry for each page
            size = rows * (Hk + Hkv) * d * ((4 if case["wide"] else 2) + 1) + pages * ((Hk + Hkv) * 8 + 4)
            return {"bytes": size + 8 * B, "flops": rows * (Hk + Hkv) * d * 2}
        live = [(n, k) for n, k in zip(lens, news) if k]
        size = sum(n * (Hk + Hkv) * d + -(-n // P) * (4 * (Hk + Hkv) + 4) for n, _ in live)
        size += rows * (dyn + H) * d * 2 + rows * H * 4 + 8 * B
        # the vectors of the frozen heads, as far as the longest sequence reaches
        size += (H - dyn) * 8 * max((n for n, _ in live), default=0)
        seen = sum(n * k - k * (k - 1) // 2 for n, k in live)
        return {"bytes": size, "flops": seen * d * 2 * (2 * dyn + (H - dyn))}
    S, cols, pages = case["seqs"], case["columns"], case["pages"]
    size = 2 * 4 * S * cols + 2 * 4 * pages
    if op == "fork":
        return {"bytes": size + 12 * S, "flops": 0}
    record = _record(case["kv_heads"], case["kv_heads"], P, case["dim"])[-1] * case["layers"]
    if op == "compact":
        return {"bytes": size + 4 + 2 * case["moved"] * record, "flops": 0}
    many = case["shared"]
    lens = [min(1 + (case["tokens"] - 1) * (b // many + 1) // (-(-S // many)), cols * P) for b in range(S)]
    last = S % many == 1 and S - 1  # a group of one: its last page is its own
    copies = sum(1 for b, n in enumerate(lens) if many > 1 and b != last and n % P and n < cols * P)
    return {"bytes": size + 16 * S + 4 + 2 * copies * record, "flops": 0}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The outputs from their definition in 64 bits (attend, append); None for whole numbers."""
    if case["op"] == "attend":
        return _exact_attend(case, prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    return None


def _e4m3_values():
    """The value of each of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    out = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append((-x if c & 128 else x) if c & 127 != 127 else math.nan)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _exact_attend(case, s):
    B, H, P, d, new = (case[k] for k in ("seqs", "heads", "page", "dim", "new"))
    g, values = H // case["kv_heads"], _e4m3_values()
    kc, vc, ks, vs = _views(s["pool"], len(s["k_heads"]), case["kv_heads"], P, d)
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, k) in enumerate(zip(_lengths(case), _news(case))):
        pages = s["table"][b, :-(-n // P)].long()

        def rows(codes, scales, h):
            return (values[codes[pages, h].long()] * scales[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
        at = torch.arange(n - k, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        for kv in range(case["kv_heads"] if k else 0):
            v = rows(vc, vs, kv)
            key = rows(kc, ks, s["k_heads"].index(kv)) if kv in s["k_heads"] else None
            for h in range(kv * g, kv * g + g):
                if s["frozen"][h]:
                    x = s["alpha"][h, :n].double()[None] + s["rho"][h].double()[(at - j).clamp(min=0)]
                else:
                    x = s["q"][b, h, :k].double() @ key.T / math.sqrt(d)
                x = x.masked_fill(j > at, -math.inf)
                lse[b, h, :k] = torch.logsumexp(x, 1)
                out[b, h, :k] = torch.softmax(x, 1) @ v
    return out, lse


def _exact_append(case, s):
    P, d = case["page"], case["dim"]
    values = _e4m3_values()
    kc, vc, ks, vs = _views(s["pool"], len(s["k_heads"]), case["kv_heads"], P, d)

    def nearest(x):
        a = x.abs().clamp(max=448.0)
        step = torch.exp2((torch.floor(torch.log2(a.clamp(min=2.0 ** -20)))).clamp(min=-6.0) - 3.0)
        return torch.copysign(torch.round(a / step) * step, x)
    got = {}
    for name, codes, scales, x in (("k", kc, ks, s["k"][:, s["k_heads"]]), ("v", vc, vs, s["v"])):
        val, sc = values[codes.long()], scales.double()
        for b, (n, k) in enumerate(zip(_lengths(case), _news(case))):
            first = n - k
            for c in range(first // P, (n - 1) // P + 1 if k and codes.shape[1] else 0):
                lo, hi = max(first, c * P), min(n, c * P + P)
                p = int(s["table"][b, c])
                new = x[b, :, lo - first:hi - first].double()
                # a whole logarithm may come out a few units of the last place above itself; the
                # next larger fp32 value lies 8e-8 above
                want = torch.ceil(torch.log2(new.abs().amax((1, 2)) / 448.0) - 1e-12).clamp(min=-64.0)
                scale = torch.exp2(want)
                if lo > c * P:
                    scale = torch.maximum(scale, sc[p])
                    val[p, :, :lo - c * P] = nearest(val[p, :, :lo - c * P] * (sc[p] / scale)[:, None, None])
                val[p, :, lo - c * P:hi - c * P] = nearest(new / scale[:, None, None])
                sc[p] = scale
        got[name], got[name + "_scale"] = val, sc
    return got
