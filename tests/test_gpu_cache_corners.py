"""Corners of the paged 8-bit cache: inputs at the ends of their ranges, rows whose sum is
empty, tokens taken back, tensors that change under the cache."""

import numpy as np
import pytest
import torch

import cache_reference as ref
from test_gpu_cache import DEV, Case, host, i32, mask_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api as _api
    return _api


KERNELS = [(3, "cache_attn"), (70, "cache_chunk")]


@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("e_q,e_k", [(-80, -64), (-30, -126), (-110, -10)])
def test_small_queries_against_small_scales(api, d, e_q, e_k, n_q, kernel):
    # the factor of a logit underflows: the weights are equal, keys behind a row weigh nothing
    c = Case(api, mask_of(4, (1,)), 2, d, 16, [200, n_q + 13], n_q, seed=d, kernel=kernel)
    c.k_scales = np.where(np.isfinite(c.k_scales), 2.0 ** e_k, c.k_scales).astype(np.float32)
    c.q = (c.q.float() * 2.0 ** e_q).to(torch.bfloat16)
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("page,tail", [(64, 1), (16, 3), (32, 1)])
def test_nan_in_a_table_that_ends_inside_a_tile(api, page, tail):
    # seq_len lies far behind the table, whose keys are no multiple of 128: every row sees all
    # of them, the NaN among them too
    cols = 2 ** 18 // page + tail
    length = cols * page + 1000
    holes = [(0, j) for j in range(2, cols - 3)]
    c = Case(api, mask_of(4, (1,)), 1, 32, page, [length], 80, holes=holes, cols=cols, seed=page)
    c.kernel = "cache_chunk"
    c.v_codes[c.table[0, cols - 1], 0, page - 5, 3] = 0x7F
    c.v_codes[c.table[0, cols - 1], 0, 0, 30] = 0xFF
    c.put()
    out, lse = c.run()
    assert bool(torch.isnan(out[0, :, :, [3, 30]].float()).all())
    c.check(out, lse)


@pytest.mark.parametrize("n_q,kernel,slots", [(1, "cache_attn", 1), (1, "cache_attn", 500),
                                              (64, "cache_chunk", 1), (64, "cache_chunk", 80)])
@pytest.mark.parametrize("nats,keys,at", [(16.0, 2 ** 15, 0), (17.5, 2 ** 17, 0),
                                          (17.5, 2 ** 20, 5), (19.0, 2 ** 20, -100)])
def test_many_keys_far_below_the_largest(api, nats, keys, at, n_q, kernel, slots):
    """One key `nats` above all others, whose V is zero: out is their share.  With many slots (all
    on the same pages) a warp or CTA has a long run of keys, with one the keys are cut into parts.

    Tolerance: 2^-8 for bf16; the approximate exponential and the fp32 logits (2^-18); the f16
    weight of a key, 2^-25 of at least 2^(11 - nats / ln 2), or 2^-11; two fp32 sums with 16 keys to
    an addition.  That of the products grows evenly, and each addition is off by at most 2^-23 of
    the sum so far: keys / 16 * 2^-24.  That of the weights holds the large one from its key on,
    and each addition rounds by up to 2^-24 of the whole: keys / 16 * 2^-24 as well."""
    d, page = 32, 128
    at %= keys - n_q
    cols = max(keys, 2 ** 18) // page
    n_pages = keys // page
    cache = api.PagedCache([[0, 1]], 2, d, H_kv=1, n_seqs=slots, max_pages=cols, n_pages=n_pages,
                           page_size=page, max_new=n_q, device=DEV)
    cache.page_table[:, :n_pages] = torch.arange(n_pages, device=DEV)
    cache.seq_len.fill_(keys)
    kc, vc, ks, vs = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
                      for x in cache.views(0))
    kc.zero_(), vc.fill_(0x38), ks.fill_(1.0), vs.fill_(1.0)   # 0x38: 1.0
    kc[at // page, 0, at % page, 0] = 0x38
    vc[at // page, 0, at % page] = 0
    q = torch.zeros((slots, 2, n_q, d), dtype=torch.bfloat16, device=DEV)
    q[:, 0, :, 0] = nats * d ** 0.5
    alpha, rho = torch.zeros((2, keys), device=DEV), torch.zeros((2, keys), device=DEV)
    alpha[1, at] = nats
    from dynamic_causal_attention_gb300 import _binding as B
    B.saf_trace_enable(1)
    out, lse = cache.attend(0, q, alpha, rho)
    names = [B.saf_trace_get(i)[1] for i in range(B.saf_trace_count())]
    B.saf_trace_enable(0)
    assert kernel in names
    n = keys - n_q + np.arange(n_q)                    # the other keys that row t sees
    for h, x in ((0, float(q[0, 0, 0, 0]) / d ** 0.5), (1, nats)):
        total = n + np.exp(x)
        got = host(out[:, h].double())
        rel = 2.0 ** -8 + 2.0 ** -18 + keys * 2.0 ** -27 + max(2.0 ** -11, 2.0 ** (-36 + nats / np.log(2)))
        err = np.abs(got / (n / total)[None, :, None] - 1)
        assert err.max() <= rel, (h, err.max(), rel)
        err = np.abs(host(lse[:, h].double()) - np.log(total))
        assert err.max() <= 2.0 ** -15 + keys * 2.0 ** -28, err.max()


@pytest.mark.parametrize("n_q,kernel,lens", [(3, "cache_attn", [150, 40]), (70, "cache_chunk", [150, 75]),
                                             (2, "cache_attn", [5003, 40]),
                                             (70, "cache_chunk", [5003, 75])])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (32, 64)])
def test_rows_without_weight_that_see_nan(api, d, page, n_q, kernel, lens):
    # out = 0 and lse = -inf where every weight is zero, whatever V holds; a row with weight
    # takes the NaN as 0 * NaN does
    c = Case(api, mask_of(6, (0, 1, 2, 3, 4)), 3, d, page, lens, n_q, T_pat=max(lens), seed=d,
             kernel=kernel)
    c.alpha[0] = -np.inf
    c.rho[1] = -np.inf
    c.alpha[2, :30] = -np.inf
    for s, j in [(0, 3), (0, lens[0] // 2), (0, lens[0] - 1), (1, 20), (1, lens[1] - 2)]:
        c.v_codes[c.table[s, j // page], :, j % page, 5] = 0x7F
    c.put()
    out, lse = c.run()
    assert bool((out[:, :2] == 0).all()) and bool((lse[:, :2] == -np.inf).all())
    c.check(out, lse)


@pytest.mark.parametrize("n_q,kernel", KERNELS)
def test_patterns_shorter_than_the_distance_and_nan(api, n_q, kernel):
    # keys behind the vectors' end weigh nothing: rows that see only such keys are empty
    c = Case(api, mask_of(4, (0, 1, 2, 3)), 2, 64, 16, [260, 75], n_q, T_pat=2, seed=1, kernel=kernel)
    c.alpha[:2, :] = -np.inf
    c.v_codes[c.table[0, 1], :, 3, 7] = 0xFF
    c.v_codes[c.table[0, 15], :, 9, 7] = 0xFF
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("times", [30.0, 300.0, 1000.0, 30000.0])
def test_queries_with_an_outlying_channel(api, d, times, n_q, kernel):
    # a channel of q far above the others, whose K is small: the others make the logits
    c = Case(api, mask_of(4, ()), 2, d, 16, [200, n_q + 60], n_q, seed=d, kernel=kernel)
    with np.errstate(invalid="ignore"):
        small = ref.encode(ref.E4M3[c.k_codes[..., 3]] / times)
    c.k_codes[..., 3] = np.where((c.k_codes[..., 3] & 0x7F) == 0x7F, c.k_codes[..., 3], small)
    c.q[..., 3] *= times
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_queries_of_every_size(api, d, n_q, kernel):
    # components 2^-16 to 2^0 of the largest, each with 8 bits, against K of the inverse sizes
    # as far as a code reaches
    c = Case(api, mask_of(4, ()), 4, d, 32, [150, n_q + 7], n_q, seed=d, kernel=kernel)
    rng = np.random.default_rng(d)
    e = rng.integers(0, 17, d)
    q = rng.uniform(0.5, 1.0, c.q.shape) * rng.choice([-1.0, 1.0], c.q.shape) * 2.0 ** -e
    c.q = torch.tensor(q, dtype=torch.bfloat16, device=DEV)
    k = rng.uniform(0.5, 1.0, c.k_codes.shape) * rng.choice([-1.0, 1.0], c.k_codes.shape) * 2.0 ** (e - 8.0)
    c.k_codes, c.k_scales = ref.encode(k), np.ones_like(c.k_scales)
    c.put()
    c.check(*c.run())


@pytest.mark.filterwarnings("ignore::RuntimeWarning")  # (the reference's sums of infinities)
@pytest.mark.parametrize("n_q,kernel", [(3, "cache_attn"), (70, "cache_chunk"), (300, "cache_chunk")])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_queries_that_are_not_finite(api, d, n_q, kernel):
    # NaN reaches the rows that see a key, and only those; of an infinite component against K of
    # one sign the logits are all -inf (no weight) or +inf (NaN)
    lens = [n_q + 90, n_q + 90, n_q + 90, n_q, n_q + 90]
    holes = [(0, j) for j in range(40)] + [(1, 1), (1, 2), (2, 0), (2, 3)]
    holes = [(s, j) for s, j in holes if j < -(-lens[s] // 16)]
    c = Case(api, mask_of(4, (3,)), 2, d, 16, lens, n_q, holes=holes, seed=d, kernel=kernel)
    rng = np.random.default_rng(d)
    fin = (c.k_codes[..., 2] & 0x7F) != 0x7F
    down = ref.encode(-rng.uniform(1.0, 100.0, c.k_codes.shape[:-1]))
    c.k_codes[..., 2] = np.where(fin, down, c.k_codes[..., 2])
    c.put()
    c.q[0] = float("nan")                        # a slot without a page
    c.q[1, :, 0, 1] = float("nan")
    c.q[1, 0, n_q - 1] = float("nan")
    c.q[2, :, 1, 2] = float("inf")
    c.q[2, 1, n_q - 1, 2] = float("-inf")
    c.q[3, 0, 0, 2] = float("inf")
    c.q[3, 1, n_q // 2, 2] = float("inf")
    c.q[4] = 3.38e38                             # bf16's largest are finite
    c.q[4, :, :, 1::2] = 0.0
    c.q[4, :, :, 2] = 0.0
    c.k_codes[:] = np.where(((c.k_codes & 0x7F) != 0x7F) & (np.arange(d) % 2 == 0) & (np.arange(d) != 2),
                            0, c.k_codes)        # ... against K of zeros
    c.put()
    out, lse = c.run()
    assert bool((out[0, :3] == 0).all()) and bool((lse[0, :3] == -np.inf).all())
    assert bool((out[2, :3, 1] == 0).all()) and bool((lse[2, :3, 1] == -np.inf).all())
    assert bool(torch.isnan(out[2, 1, n_q - 1].float()).all())
    c.check(out, lse)


@pytest.mark.filterwarnings("ignore::RuntimeWarning")
@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 128])
def test_patterns_that_are_not_finite(api, d, n_q, kernel):
    # an alpha of NaN or +inf reaches the rows that see its key, not those that have a hole there
    # or stand before it
    holes = [(0, 1), (0, 2), (1, 2)]
    c = Case(api, mask_of(4, (0, 2, 3)), 2, d, 16, [n_q + 90, n_q + 60, n_q + 2], n_q, holes=holes,
             seed=d, kernel=kernel)
    c.alpha[0, 16:48] = np.nan
    c.alpha[2, 33] = np.inf
    c.alpha[3, n_q + 50] = np.nan
    out, lse = c.run()
    assert not bool(torch.isnan(out[0, 0].float()).any()) and bool(torch.isnan(out[1, 0].float()).all())
    c.check(out, lse)


def grow_over_held(table, seq_len, counts, n_new, page):
    """cache_reference.grow for rows that hold pages behind their length: those that no other
    row holds, from the first new column on, are used again; behind them, and where a page is
    shared, the row gives its page up and takes a free one."""
    S, cols = table.shape
    n = len(counts)
    keep = np.zeros(S, dtype=int)
    lens = np.maximum(seq_len, 0)
    for s in range(S):
        if n_new[s] <= 0 or lens[s] + int(n_new[s]) > cols * page:
            continue
        begin, end = -(-int(lens[s]) // page), -(-(int(lens[s]) + int(n_new[s])) // page)
        while begin + keep[s] < end:
            t = table[s, begin + keep[s]]
            if not 0 <= t < n or counts[t] != 1:
                break
            keep[s] += 1
    free = [p for p in range(n) if counts[p] <= 0]
    out, out_ref, out_len = table.copy(), counts.copy(), lens.copy()
    granted, copies, at = np.zeros(S, dtype=np.int32), [], 0

    def take():
        nonlocal at
        at += 1
        if at > len(free):
            return -1
        out_ref[free[at - 1]] = 1
        return free[at - 1]
    for s in range(S):
        k = int(n_new[s])
        if k <= 0 or lens[s] + k > cols * page:
            continue
        granted[s] = k
        if lens[s] % page:
            held = table[s, lens[s] // page]
            if 0 <= held < n and counts[held] > 1:
                new = take()
                copies.append((held, new))
                out_ref[held] -= 1
                out[s, lens[s] // page] = new
        begin, end = -(-int(lens[s]) // page), -(-(int(lens[s]) + k) // page)
        for c in range(begin + keep[s], end):
            t = table[s, c]
            out[s, c] = take()
            if 0 <= t < n and counts[t] > 0:
                out_ref[t] -= 1
        out_len[s] += k
    if at > len(free):
        return table, seq_len, counts, np.zeros(S, dtype=np.int32), at - len(free), []
    return out, out_len, out_ref, granted, 0, copies


TAKEN_BACK = [(1, 4, 9, 16), (6, 9, 90, 16), (40, 30, 2600, 16), (300, 12, 9001, 16),
              (2000, 6, 30000, 16), (3, 700, 9000, 16)]


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("S,cols,n_pages,page", TAKEN_BACK)
def test_grow_after_tokens_were_taken_back(api, S, cols, n_pages, page, into):
    from test_gpu_cache import page_cache, random_tables
    rng = np.random.default_rng(S + cols)
    for seed, most in enumerate((1, 2 * page, cols * page)):
        table, lens = random_tables(rng, S, cols, n_pages, page, 0.3)
        # lengths go down, pages stay; some entries behind are holes or no pages
        lens = (lens * rng.random(S) ** 0.5).astype(np.int32)
        lens[rng.random(S) < 0.1] = 0
        counts = np.bincount(table[table >= 0].flatten(), minlength=n_pages).astype(np.int32)
        cache, got_counts, pool = page_cache(api, table, lens, n_pages, page, seed)
        assert np.array_equal(counts, got_counts)
        n_new = rng.integers(-1, most + 1, S).astype(np.int32)
        before = host(pool)
        w_table, w_lens, w_ref, granted, short, copies = grow_over_held(table, lens, counts, n_new, page)
        to = tuple(torch.full_like(t, -7) for t in (cache.page_table, cache.seq_len, cache.ref)) \
            if into else None
        got_granted, got_short = cache.grow(i32(n_new), into=to)
        got = [host(t) for t in (to or (cache.page_table, cache.seq_len, cache.ref))]
        assert int(got_short) == short and np.array_equal(host(got_granted), granted)
        for g, w in zip(got, (w_table, w_lens, w_ref)):
            assert np.array_equal(g, w)
        # nothing is lost: every page is counted as often as it is held
        held = np.bincount(got[0][got[0] >= 0].flatten(), minlength=n_pages)
        assert np.array_equal(held, got[2])
        for a, b in copies:
            before[b] = before[a]
        assert np.array_equal(host(pool), before)


def test_drafts_taken_back_again_and_again(api):
    # a pool with no page to spare: every draft fits into the pages that the row holds already
    cache = api.PagedCache([[0, 0]], 2, 32, n_seqs=2, max_pages=4, n_pages=7, page_size=16,
                           max_new=20, device=DEV)
    cache.grow(i32([45, 45]))
    for i in range(12):
        granted, short = cache.grow(i32([19, 3]))
        assert int(short) == 0 and host(granted).tolist() == [19, 3]
        cache.seq_len.sub_(i32([18, 3]) if i % 2 else i32([19, 3]))
        if i == 5:
            cache.seq_len.copy_(i32([45, 45]))
        held = host(cache.page_table)
        assert np.array_equal(np.bincount(held[held >= 0], minlength=7), host(cache.ref))
        cache.seq_len.clamp_(max=45)
    assert int((cache.ref > 0).sum()) == 7


@pytest.mark.parametrize("into", [False, True])
def test_entries_that_no_count_knows_are_overwritten(api, into):
    # a caller that starts over by clearing lengths and counts, not the table
    cache = api.PagedCache([[0, 0]], 2, 32, n_seqs=3, max_pages=4, n_pages=12, page_size=16,
                           device=DEV)
    cache.grow(i32([64, 64, 64]))
    cache.seq_len.zero_()
    cache.ref.zero_()
    cache.page_table.copy_(cache.page_table.flip(0))
    to = tuple(torch.zeros_like(t) for t in (cache.page_table, cache.seq_len, cache.ref)) if into else None
    granted, short = cache.grow(i32([40, 64, 16]), into=to)
    table, lens, counts = to or (cache.page_table, cache.seq_len, cache.ref)
    assert int(short) == 0 and host(granted).tolist() == [40, 64, 16]
    got = host(table)
    assert got[0, :3].tolist() == [0, 1, 2] and got[1].tolist() == [3, 4, 5, 6] and got[2, 0] == 7
    assert host(counts).tolist() == [1] * 8 + [0] * 4


def test_tensors_that_change_under_the_cache(api):
    # the cache looks at its tensors on every call: new storage is used, another shape refused
    c = Case(api, mask_of(4, (2,)), 2, 64, 16, [40, 25], 2, seed=6)
    k = c.cache
    out, lse = c.run()
    old = [k.page_table.data, k.seq_len.data, k.pool.data]   # (the old memory stays alive)
    pool = torch.zeros((k.n_pages, old[2].stride(0)), dtype=torch.uint8, device=DEV)
    pool[:, :k.page_bytes].copy_(old[2])
    k.pool.data = pool[:, :k.page_bytes]
    k.page_table.data = old[0].clone()
    k.seq_len.data = old[1].clone()
    for t in old:
        t.zero_()
    out2, lse2 = c.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    table, lens = k.page_table.clone(), k.seq_len.clone()
    k.grow(i32([0, 0]))
    k.fork(i32([1, 0]))
    assert torch.equal(k.page_table, table.flip(0)) and torch.equal(k.seq_len, lens.flip(0))
    v = torch.zeros((2, 2, 1, 64), device=DEV)
    q = c.q[:, :, :1].contiguous()
    pat = torch.zeros((4, 64), device=DEV)
    calls = [lambda: k.append(0, v, v), lambda: k.attend(0, q, pat, pat), lambda: k.grow(i32([1, 1])),
             lambda: k.fork(i32([0, 1])), lambda: k.compact()]
    for name in ("page_table", "seq_len", "ref", "pool"):
        t = getattr(k, name)
        was = t.data
        for other in (was[:-1].clone(), was.float(), was.cpu()):
            t.data = other if other.dtype == t.dtype else other.to(torch.int64)
            for i, call in enumerate(calls):
                if name == "ref" and i < 2 or name == "seq_len" and i == 4 or name == "pool" and i == 3:
                    continue                                  # these do not look at it
                with pytest.raises(api.SafError):
                    call()
                    pytest.fail(f"{name}: call {i} was taken")
            t.data = was
    for call in calls:
        call()


def test_outputs_that_the_call_makes_hold_no_old_memory(api):
    # rows behind n_new of buffers that attend itself allocates: no token, so out = 0, lse = -inf
    for n_q, kernel in KERNELS:
        c = Case(api, mask_of(4, (2,)), 2, 64, 16, [120, n_q, 90], n_q, n_new=[n_q, 0, 2], seed=6,
                 kernel=kernel)
        want, want_lse = c.run()
        a, r = (torch.from_numpy(x).to(DEV) for x in (c.alpha, c.rho))
        for _ in range(3):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                    for n in (c.q.nbytes, want_lse.nbytes) for _ in range(8)]
            del junk  # (what the allocator hands out next holds NaN)
            out, lse = c.cache.attend(0, c.q, a, r, n_new=i32(c.n_new))
            for s, n in enumerate(c.n_new):
                assert torch.equal(out[s, :, :n], want[s, :, :n])
                assert torch.equal(lse[s, :, :n], want_lse[s, :, :n])
                assert bool((out[s, :, n:] == 0).all()) and bool((lse[s, :, n:] == -np.inf).all())


@pytest.mark.parametrize("n_q,kernel", KERNELS)
def test_masks_of_the_lowest_value_are_masks_of_minus_infinity(api, n_q, kernel):
    c = Case(api, mask_of(6, (0, 1, 2, 3)), 3, 64, 32, [150, 75], n_q, seed=2, kernel=kernel)
    got = []
    for low in (-np.inf, np.finfo(np.float32).min):
        c.alpha[0, ::3] = low
        c.rho[1, 2:50] = low
        c.alpha[2] = low
        c.rho[3] = low
        got.append(c.run())
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool((got[1][0][:, 2:4] == 0).all()) and bool((got[1][1][:, 2:4] == -np.inf).all())


@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 128])
def test_scales_of_v_at_the_ends_of_their_range(api, d, n_q, kernel):
    # blocks of zeros (scale 2^-64) beside large ones: their keys count in the sums all the same
    c = Case(api, mask_of(4, (1,)), 2, d, 16, [300, n_q + 40], n_q, seed=d, kernel=kernel)
    rng = np.random.default_rng(d)
    small = rng.random(c.v_scales.shape) < 0.5
    fin = np.isfinite(c.v_scales)
    c.v_scales = np.where(fin, np.where(small, 2.0 ** -64, 2.0 ** 36), c.v_scales).astype(np.float32)
    zero = np.broadcast_to((small & fin)[:, :, None, None], c.v_codes.shape)
    c.v_codes = np.where(zero & ((c.v_codes & 0x7F) != 0x7F), 0, c.v_codes)
    c.put()
    c.check(*c.run())
