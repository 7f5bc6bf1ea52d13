"""The paged 8-bit cache against a float64 / integer reference: quantising append, attention
over the pages, page tables, and a serving run of all of them together."""

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api as _api
    return _api


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def host(t):
    return t.detach().cpu().numpy()


def bits(t):
    """Codes of an e4m3 view as host bytes."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


def k_heads_of(mask, H_kv):
    g = len(mask) // H_kv
    return [k for k in range(H_kv) if not all(mask[k * g:(k + 1) * g])]


class Case:
    """A one-layer cache whose pages hold random quantised rows (NaN codes where `dirt` lies
    behind a slot's tokens), with host copies of everything."""

    def __init__(self, api, mask, H_kv, d, page, lens, n_q, seed=0, n_new=None, spare=3, holes=(),
                 T_pat=None, wide_stride=0, cols=None, dirt=True, max_new=None, kernel=None):
        # kernel: the one that attends.  The library chooses by sizes, the page table's width
        # among them: wide tables (2^18 keys) make small calls take the one for many rows
        self.kernel = kernel
        if kernel == "cache_chunk":
            T_pat = T_pat or max(1, -(-max(lens) // page)) * page
            cols = 2 ** 18 // page
        rng = np.random.default_rng(seed)
        H, S = len(mask), len(lens)
        self.mask, self.H, self.H_kv, self.d, self.page = list(mask), H, H_kv, d, page
        self.k_heads = k_heads_of(mask, H_kv)
        cols = cols or max(1, -(-max(lens) // page))
        need = [min(cols, -(-max(n, 0) // page)) for n in lens]
        n_pages = sum(need) + spare
        ids = rng.permutation(n_pages)
        table = np.full((S, cols), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = ids[at:at + n]
            at += n
        self.held = table.copy()
        for s, c in holes:
            table[s, c] = [-1, n_pages, 2 ** 31 - 1][(s + c) % 3]
        self.table, self.lens = table, np.asarray(lens, dtype=np.int32)
        self.n_new = np.full(S, n_q, dtype=np.int32) if n_new is None else np.asarray(n_new, np.int32)
        probe = api.PagedCache([mask], H, d, H_kv=H_kv, n_seqs=S, max_pages=cols, n_pages=n_pages,
                               page_size=page, max_new=max_new or max(n_q, 1), device=DEV)
        pool = torch.zeros((n_pages, probe.page_bytes + wide_stride), dtype=torch.uint8, device=DEV)
        self.cache = api.PagedCache([mask], H, d, H_kv=H_kv, n_seqs=S, max_pages=cols,
                                    n_pages=n_pages, page_size=page, max_new=max_new or max(n_q, 1),
                                    device=DEV, pool=pool[:, :probe.page_bytes],
                                    page_table=i32(table), seq_len=i32(lens))
        self.q = torch.tensor(rng.standard_normal((S, H, n_q, d)), dtype=torch.bfloat16, device=DEV)
        T = cols * page if T_pat is None else T_pat
        self.alpha = rng.standard_normal((H, T)).astype(np.float32)
        self.rho = (-np.log1p(np.arange(T)) + 0.3 * rng.standard_normal((H, T))).astype(np.float32)
        kc, vc, ks, vs = self.cache.views(0)
        self.k_codes, self.k_scales = self._rows(rng, n_pages, len(self.k_heads))
        self.v_codes, self.v_scales = self._rows(rng, n_pages, H_kv)
        if dirt:
            for s in range(S):
                for c in range(min(cols, -(-max(int(lens[s]), 1) // page))):
                    p = self.held[s, c]
                    free = page - (max(int(lens[s]), 0) - c * page)
                    if p >= 0 and free > 0:
                        self.k_codes[p, :, page - min(free, page):] = 0x7F
                        self.v_codes[p, :, page - min(free, page):] = 0xFF
            for p in set(range(n_pages)) - set(self.held[self.held >= 0].tolist()):
                self.k_codes[p], self.v_codes[p] = 0xFF, 0x7F
                self.k_scales[p], self.v_scales[p] = np.nan, np.inf
        self.put()

    def _rows(self, rng, n, heads):
        x = rng.standard_normal((n, heads, self.page, self.d)) * np.exp(
            rng.standard_normal((n, heads, 1, 1)))
        s = np.array([[ref.block_scale(x[p, h]) for h in range(heads)] for p in range(n)])
        s = s.reshape(n, heads)
        return ref.encode(x / s[:, :, None, None]), s.astype(np.float32)

    def put(self):
        kc, vc, ks, vs = self.cache.views(0)
        kc.copy_(torch.from_numpy(self.k_codes).to(DEV).view(torch.float8_e4m3fn))
        vc.copy_(torch.from_numpy(self.v_codes).to(DEV).view(torch.float8_e4m3fn))
        ks.copy_(torch.from_numpy(self.k_scales))
        vs.copy_(torch.from_numpy(self.v_scales))

    def run(self, **kw):
        a, r = (torch.from_numpy(x).to(DEV) for x in (self.alpha, self.rho))
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:3], 7.0, device=DEV)
        from dynamic_causal_attention_gb300 import _binding as B
        if self.kernel:
            B.saf_trace_enable(1)
        self.cache.attend(0, self.q, a, r, n_new=i32(self.n_new), out=out, lse=lse, **kw)
        if self.kernel:
            names = [B.saf_trace_get(i)[1] for i in range(B.saf_trace_count())]
            B.saf_trace_enable(0)
            assert self.kernel in names
        return out, lse

    def check(self, out, lse, slots=slice(None)):
        want, want_lse, tol, lse_tol = ref.attend(
            host(self.q[slots].double()), self.k_codes, self.k_scales, self.v_codes, self.v_scales,
            self.k_heads, self.alpha, self.rho, self.mask, self.table[slots], self.lens[slots],
            self.n_new[slots], self.page)
        out, lse = host(out[slots].double()), host(lse[slots].double())
        n_q = self.q.shape[2]
        live = np.arange(n_q)[None, :] < np.clip(self.n_new[slots], 0, n_q)[:, None]
        live = np.broadcast_to(live[:, None], lse.shape)
        assert np.all(out[~live] == 7.0) and np.all(lse[~live] == 7.0), "rows behind n_new changed"
        got, want, tol = out[live], want[live], tol[live]
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(got)), "NaN at other places"
        err = np.abs(got - want)[~nan]
        assert np.all(err <= tol[~nan]), (err - tol[~nan]).max()
        a, w, t = lse[live], want_lse[live], lse_tol[live]
        empty = w == -np.inf
        assert np.array_equal(a == -np.inf, empty)
        ok = ~empty & ~np.isnan(w)
        assert np.array_equal(np.isnan(a), np.isnan(w))
        assert np.all(np.abs(a[ok] - w[ok]) <= t[ok]), (np.abs(a[ok] - w[ok]) - t[ok]).max()


def mask_of(H, frozen):
    return [int(h in frozen) for h in range(H)]


# ------------------------------------------------------------------ attend
SHAPES = [  # H, H_kv, frozen, d, page
    (4, 4, (1,), 64, 64),
    (12, 4, (0, 4, 8), 64, 32),
    (16, 16, (0, 5, 15), 128, 64),
    (16, 4, (0, 1, 2, 3), 128, 128),   # one group frozen whole: its K is not stored
    (8, 1, (), 32, 16),
    (24, 8, tuple(range(24)), 32, 32),  # no K at all
    (20, 2, (3, 11), 64, 16),           # ten heads to a K/V head
    (48, 2, (0, 47), 128, 32),          # 24 heads to a K/V head
    (3, 3, (), 128, 16),
]


@pytest.mark.parametrize("H,H_kv,frozen,d,page", SHAPES)
def test_single_tokens(api, H, H_kv, frozen, d, page):
    lens = [1, 0, page - 1, page, page + 1, 5 * page + 7, 300, 17]
    c = Case(api, mask_of(H, frozen), H_kv, d, page, lens, 1, seed=H + d)
    c.check(*c.run())


@pytest.mark.parametrize("H,H_kv,frozen,d,page", SHAPES)
@pytest.mark.parametrize("n_q,kernel", [(2, "cache_attn"), (7, "cache_attn"), (50, None),
                                        (50, "cache_chunk")])
def test_several_tokens(api, H, H_kv, frozen, d, page, n_q, kernel):
    # as many new tokens as there are, fewer tokens than new ones, none, one, all but one
    lens = [n_q, max(0, n_q - 3), 77, 2 * page + 1, 260, 4]
    n_new = [n_q, n_q, 0, 1, n_q - 1, -2]
    c = Case(api, mask_of(H, frozen), H_kv, d, page, lens, n_q, n_new=n_new, seed=n_q + d,
             kernel=kernel)
    c.check(*c.run())


@pytest.mark.parametrize("d,page,g", [(64, 64, 1), (128, 32, 4), (32, 16, 3)])
@pytest.mark.parametrize("n_q,kernel", [(1, "cache_attn"), (150, None),
                                        (150, "cache_chunk")])
def test_long_sequences_are_cut_and_joined(api, d, page, g, n_q, kernel):
    # one long sequence next to short ones: its keys are split over many CTAs
    c = Case(api, mask_of(2 * g, (0,)), 2, d, page, [5003, 150, 900], n_q,
             n_new=[min(n_q, 2), min(n_q, 140), n_q], seed=3, kernel=kernel)
    c.check(*c.run())


@pytest.mark.parametrize("kernel", [None, "cache_chunk"])
@pytest.mark.parametrize("d,page", [(128, 128), (64, 16)])
def test_prompt_chunks(api, d, page, kernel):
    # the first chunk of a prompt (nothing before it), and chunks behind a context
    c = Case(api, mask_of(8, (2, 3)), 4, d, page, [257, 700, 391], 257, n_new=[257, 130, 255], seed=9,
             kernel=kernel)
    c.check(*c.run())


@pytest.mark.parametrize("d", [32, 64, 128])
def test_many_short_prompts(api, d):
    # several whole units of 64 rows for each CTA: half of a tile's warps have none
    c = Case(api, mask_of(4, ()), 4, d, 64, [128 - (s * 7) % 64 for s in range(160)], 64, seed=5,
             kernel="cache_chunk")
    out, lse = c.run()
    c.check(out, lse, slice(0, 160, 3))


def test_frozen_heads_behind_short_units(api):
    # 260 rows of the dynamic heads: a row of units of 256, then one of 4, whose second tile of
    # rows is empty, then the frozen heads' units with both
    c = Case(api, mask_of(24, range(2, 24, 3)), 8, 32, 64, [600 - 3 * s for s in range(16)], 130,
             seed=6, kernel="cache_chunk")
    out, lse = c.run()
    c.check(out, lse, slice(0, 16, 3))


@pytest.mark.parametrize("n_q", [64, 128, 129, 300])
@pytest.mark.parametrize("frozen", [(0, 1, 2), (1, 3, 4, 5, 6)])
def test_row_tiles_of_frozen_heads_come_in_pairs(api, n_q, frozen):
    # odd and even numbers of tiles; the two of a unit are of one head or of two
    lens = [n_q + 70, 333, n_q, 20]
    c = Case(api, mask_of(8, frozen), 1, 64, 32, lens, n_q, n_new=[n_q, min(n_q, 201), n_q - 1, 30],
             seed=n_q, kernel="cache_chunk")
    for s, j in [(0, n_q + 65), (2, n_q - 3)]:
        c.v_codes[c.table[s, j // 32], :, j % 32, 3] = 0x7F
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", [(1, "cache_attn"), (3, "cache_attn"), (40, None),
                                        (40, "cache_chunk")])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16), (32, 128)])
def test_holes_and_dirty_pages(api, d, page, n_q, kernel):
    lens = [6 * page + 3, 2 * page, 5 * page - 1]
    holes = [(0, 0), (0, 3), (1, 0), (1, 1), (2, 4)]  # slot 1 has no page left
    c = Case(api, mask_of(6, (1, 4)), 2, d, page, lens, n_q, holes=holes, seed=21,
             kernel=kernel)
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", [(5, "cache_attn"), (40, None),
                                        (40, "cache_chunk"), (200, "cache_chunk")])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_nan_rows_reach_only_the_rows_that_see_them(api, d, n_q, kernel):
    page = 32
    c = Case(api, mask_of(4, (0,)), 2, d, page, [n_q + 90, n_q], n_q, seed=5,
             kernel=kernel)
    for s, j in [(0, 90 + n_q // 2), (1, n_q - 2)]:
        p = c.table[s, j // page]
        c.v_codes[p, :, j % page, 3] = 0x7F
        c.v_codes[p, 0, j % page, d - 1] = 0xFF
        c.k_codes[p, 1, j % page, 5] = 0x7F
    c.put()
    c.check(*c.run())


def test_lengths_behind_the_page_table(api):
    # seq_len beyond max_pages * page_size: the keys that exist still count
    c = Case(api, mask_of(4, (2,)), 2, 64, 16, [40, 100, 64], 3, cols=4, T_pat=200, seed=8)
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", [(4, "cache_attn"), (60, "cache_chunk")])
def test_frozen_patterns(api, n_q, kernel):
    # vectors shorter than the sequence, entries of -inf, rows whose every weight is zero
    for T in (1, 50, 200):
        c = Case(api, mask_of(6, (0, 1, 2, 3, 4)), 3, 64, 32, [150, 33, 1], n_q, T_pat=T, seed=T,
                 kernel=kernel)
        c.alpha[1, ::2] = -np.inf
        c.rho[2, :] = -np.inf
        c.alpha[3] = -np.inf
        c.rho[4, min(5, T - 1):] = -np.inf
        c.alpha[0] *= 20
        c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", [(3, "cache_attn"), (60, "cache_chunk")])
def test_scales_of_any_size(api, n_q, kernel):
    # block scales far apart within a sequence; queries far outside f16's range
    c = Case(api, mask_of(4, (1,)), 2, 64, 16, [200, 130], n_q, seed=4, kernel=kernel)
    rng = np.random.default_rng(0)
    e = rng.integers(-30, 20, size=c.v_scales.shape)
    fin = np.isfinite(c.v_scales)
    c.v_scales = np.where(fin, 2.0 ** e * 1.37, c.v_scales).astype(np.float32)
    c.k_scales = np.where(np.isfinite(c.k_scales), c.k_scales * 2.0 ** -40, c.k_scales).astype(np.float32)
    c.q = (c.q.float() * 2.0 ** 40).to(torch.bfloat16)
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("n_q,kernel", [(2, "cache_attn"), (70, "cache_chunk")])
def test_pages_far_apart_and_layers_behind_one_another(api, n_q, kernel):
    # page_stride * page beyond 2^32 bytes; the layer is not the first of its page
    n_pages, page, d = 300, 16, 64
    masks = [[0, 0], [1, 0], [0, 0]]
    small = Case(api, masks[1], 2, d, page, [70, 16], n_q, seed=2, kernel=kernel)
    n, cols = small.cache.n_pages, small.table.shape[1]
    probe = api.PagedCache(masks, 2, d, n_seqs=2, max_pages=cols, n_pages=2, page_size=page, device=DEV)
    stride = 16 << 20
    pool = torch.zeros((n_pages, stride), dtype=torch.uint8, device=DEV)
    big = api.PagedCache(masks, 2, d, n_seqs=2, max_pages=cols, n_pages=n_pages, page_size=page,
                         max_new=n_q, device=DEV, pool=pool[:, :probe.page_bytes])
    place = np.linspace(n_pages - 1, 1, n).astype(np.int32)
    big.seq_len.copy_(i32(small.lens))
    big.page_table.copy_(i32(np.where(small.table >= 0, place[small.table], -1)))
    for dst, src in zip(big.views(1), small.cache.views(0)):
        for a, b in enumerate(place):
            dst[int(b)].copy_(src[a])
    a, r = (torch.from_numpy(x).to(DEV) for x in (small.alpha, small.rho))
    out, lse = big.attend(1, small.q, a, r, n_new=i32(small.n_new))
    small.check(out, lse)
    k, v = (torch.randn((2, 2, n_q, d), device=DEV) for _ in range(2))
    big.append(1, k, v)
    small.cache.append(0, k, v)
    for dst, src in zip(big.views(1), small.cache.views(0)):
        for x, y in zip(dst[torch.from_numpy(place).long().to(DEV)], src):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    others = torch.ones(n_pages, dtype=torch.bool)
    others[torch.from_numpy(place).long()] = False
    assert int(pool[others.to(DEV)].max()) == 0 and int(pool[:, probe.page_bytes:].max()) == 0


@pytest.mark.parametrize("n_q,lens,kernel", [
    (1, [3000, 10, 1200], "cache_attn"), (64, [3000, 64, 1200], None),
    (64, [3000, 64, 1200], "cache_chunk")])
def test_same_bits_again_and_on_another_stream(api, n_q, lens, kernel):
    c = Case(api, mask_of(8, (1, 6)), 2, 128, 64, lens, n_q, seed=12, kernel=kernel)
    out, lse = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, lse2 = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert c.cache.device_status() == (0, 0)


def test_attend_without_lse_or_counts(api):
    from dynamic_causal_attention_gb300 import _binding as B
    c = Case(api, mask_of(4, ()), 2, 64, 32, [90, 33], 2, seed=1)
    out, _ = c.run()
    again = torch.zeros_like(out)
    k = c.cache
    st = B.saf_cache_attn(k.dims, bytes(4), k.pool.data_ptr(), c.q.data_ptr(), None, None, 0, 2,
                          None, k.seq_len.data_ptr(), k.page_table.data_ptr(), again.data_ptr(),
                          None, k.workspace.data_ptr(), k.ws_bytes,
                          torch.cuda.current_stream().cuda_stream)
    assert st == B.SAF_OK and torch.equal(out, again)


# ------------------------------------------------------------------ append
def check_append(api, mask, H_kv, d, page, dtype, lens, n_q, n_new, seed=0, spoil=None):
    c = Case(api, mask, H_kv, d, page, lens, n_q, n_new=n_new, seed=seed, dirt=False,
             holes=[(0, 1)] if len(c_pages(lens, page)) and c_pages(lens, page)[0] > 2 else [])
    rng = np.random.default_rng(seed + 1)
    x = [rng.standard_normal((len(lens), H_kv, n_q, d)) * np.exp(
        2 * rng.standard_normal((len(lens), H_kv, n_q, 1))) for _ in range(2)]
    k, v = (torch.tensor(a, dtype=torch.float32, device=DEV).to(dtype) for a in x)
    if spoil:
        spoil(k, v)
    kc, vc, ks, vs = (a.copy() for a in (c.k_codes, c.v_codes, c.k_scales, c.v_scales))
    n = np.full(len(lens), n_q) if n_new is None else n_new
    ref.append(kc, ks, host(k.double())[:, c.k_heads], c.table, c.lens, n, page)
    ref.append(vc, vs, host(v.double()), c.table, c.lens, n, page)
    for _ in range(2):  # the second time changes nothing
        c.cache.append(0, k, v, n_new=None if n_new is None else i32(n_new))
        got = c.cache.views(0)
        for name, a, b in (("K", got[0], kc), ("V", got[1], vc)):
            a = bits(a)
            nan = (a & 0x7F) == 0x7F
            assert np.array_equal(nan, (b & 0x7F) == 0x7F), name
            assert np.array_equal(a[~nan], b[~nan]), name
        assert np.array_equal(host(got[2]), ks) and np.array_equal(host(got[3]), vs)


def c_pages(lens, page):
    return [-(-max(n, 0) // page) for n in lens]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,H_kv,frozen,d,page", SHAPES)
def test_append_single_tokens(api, H, H_kv, frozen, d, page, dtype):
    lens = [1, 0, page, page + 1, 3 * page - 1, 2 * page + 9, 0]
    check_append(api, mask_of(H, frozen), H_kv, d, page, dtype, lens, 1, None, seed=d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,H_kv,frozen,d,page", SHAPES[:5])
def test_append_rows(api, H, H_kv, frozen, d, page, dtype):
    lens = [4 * page, 3 * page + 5, 20, 2 * page + 1, page]
    n_new = [2 * page + 3, 3 * page + 9, 40, 0, 1]  # the second and third: more than the length
    check_append(api, mask_of(H, frozen), H_kv, d, page, dtype, lens, 3 * page + 9, n_new, seed=page)


def test_append_odd_values(api):
    def spoil(k, v):
        k[0, 0, 0] = 0.0
        k[0, :, 1, 3] = float("nan")
        k[1, :, :, 7] = float("inf")
        v[0, :, 0, 0] = float("-inf")
        v[1, 1] = 0.0           # a block of nothing: the smallest scale
        v[2] *= 2.0 ** 100
        k[2] *= 2.0 ** -90
        v[3, :, :, 1] = 448.0   # exactly the largest value of a scale
        v[4] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        check_append(api, mask_of(4, ()), 2, 64, 16, dtype, [2, 19, 50, 17, 33], 2, None, spoil=spoil)


def test_append_without_k(api):
    c = Case(api, [1, 1], 2, 64, 16, [5], 5, seed=3)
    v = torch.randn((1, 2, 5, 64), device=DEV)
    c.cache.append(0, None, v)
    ref.append(c.v_codes, c.v_scales, host(v.double()), c.table, c.lens, [5], 16)
    got = c.cache.views(0)
    assert np.array_equal(bits(got[1]), c.v_codes) and np.array_equal(host(got[3]), c.v_scales)


# ------------------------------------------------------------------ pages
def page_cache(api, table, lens, n_pages, page, seed=0, stride_extra=0):
    S, cols = table.shape
    ref_counts = np.bincount(table[table >= 0].flatten(), minlength=n_pages).astype(np.int32)
    probe = api.PagedCache([[0, 0], [1, 0]], 2, 32, n_seqs=S, max_pages=cols, n_pages=n_pages,
                           page_size=page, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pool = torch.randint(0, 256, (n_pages, probe.page_bytes + stride_extra), dtype=torch.uint8,
                         device=DEV, generator=gen)
    cache = api.PagedCache([[0, 0], [1, 0]], 2, 32, n_seqs=S, max_pages=cols, n_pages=n_pages,
                           page_size=page, device=DEV, pool=pool[:, :probe.page_bytes],
                           page_table=i32(table), seq_len=i32(lens), ref=i32(ref_counts))
    return cache, ref_counts, pool


def random_tables(rng, S, cols, n_pages, page, share):
    table = np.full((S, cols), -1, dtype=np.int32)
    lens = np.zeros(S, dtype=np.int32)
    free = list(rng.permutation(n_pages))
    for s in range(S):
        if s and rng.random() < share:
            q = rng.integers(0, s)
            table[s], lens[s] = table[q], lens[q]
            continue
        n = int(rng.integers(0, cols * page + 1))
        need = -(-n // page)
        if need > len(free) // 2:
            n = need = 0
        table[s, :need] = [free.pop() for _ in range(need)]
        lens[s] = n
    return table, lens


PAGES = [(1, 1, 1, 16), (5, 7, 40, 16), (33, 9, 203, 32), (300, 5, 1021, 64), (64, 40, 5000, 16),
         (7000, 3, 9001, 16), (90, 1100, 140003, 16)]


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("S,cols,n_pages,page", PAGES)
def test_fork(api, S, cols, n_pages, page, into):
    rng = np.random.default_rng(S)
    for seed in range(2):
        table, lens = random_tables(rng, S, cols, n_pages, page, 0.5)
        cache, counts, _ = page_cache(api, table, lens, n_pages, page)
        parent = np.where(rng.random(S) < 0.4, np.arange(S), rng.integers(-1, S + 1, S))
        parent[rng.random(S) < 0.05] = -2 ** 31
        want = ref.fork(table, lens, counts, parent)
        keep = [t.clone() for t in (cache.page_table, cache.seq_len, cache.ref)]
        to = tuple(torch.full_like(t, -7) for t in keep) if into else None
        cache.fork(i32(parent), into=to)
        for got, w in zip(to or (cache.page_table, cache.seq_len, cache.ref), want):
            assert np.array_equal(host(got), w)
        if into:
            for got, k in zip((cache.page_table, cache.seq_len, cache.ref), keep):
                assert torch.equal(got, k)


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("S,cols,n_pages,page", PAGES)
def test_grow(api, S, cols, n_pages, page, into):
    rng = np.random.default_rng(S + 1)
    for seed, most in enumerate((1, 2 * page, cols * page)):
        table, lens = random_tables(rng, S, cols, n_pages, page, 0.5)
        cache, counts, pool = page_cache(api, table, lens, n_pages, page, seed, stride_extra=64)
        n_new = rng.integers(-1, most + 1, S).astype(np.int32)
        n_new[rng.random(S) < 0.02] = 2 ** 31 - 1
        before = host(pool)
        w_table, w_lens, w_ref, granted, short, copies = ref.grow(table, lens, counts, n_new, page)
        if short:
            w_table, w_lens, w_ref = table, lens, counts
        to = tuple(torch.full_like(t, -7) for t in (cache.page_table, cache.seq_len, cache.ref)) \
            if into else None
        got_granted, got_short = cache.grow(i32(n_new), into=to)
        for got, w in zip(to or (cache.page_table, cache.seq_len, cache.ref), (w_table, w_lens, w_ref)):
            assert np.array_equal(host(got), w)
        assert int(got_short) == short and np.array_equal(host(got_granted), granted)
        for a, b in copies:
            before[b, :cache.page_bytes] = before[a, :cache.page_bytes]
        assert np.array_equal(host(pool), before)


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("S,cols,n_pages,page", PAGES)
def test_compact(api, S, cols, n_pages, page, into):
    rng = np.random.default_rng(S + 2)
    for seed, share in enumerate((0.3, 0.9)):
        table, lens = random_tables(rng, S, cols, n_pages, page, share)
        cache, counts, pool = page_cache(api, table, lens, n_pages, page, seed, stride_extra=16)
        before = host(pool)
        w_table, w_ref, n, moves = ref.compact(table, counts)
        to = (torch.full_like(cache.page_table, -7), torch.full_like(cache.ref, -7)) if into else None
        used = cache.compact(into=to)
        for got, w in zip(to or (cache.page_table, cache.ref), (w_table, w_ref)):
            assert np.array_equal(host(got), w)
        assert int(used) == n
        for a, b in moves:
            before[b, :cache.page_bytes] = before[a, :cache.page_bytes]
        assert np.array_equal(host(pool), before)


def test_full_and_empty_pools(api):
    cache, counts, _ = page_cache(api, np.arange(6, dtype=np.int32).reshape(2, 3), [48, 48], 6, 16)
    assert int(cache.compact()) == 6
    granted, short = cache.grow(i32([1, 0]))     # past the end of the table: left alone
    assert host(granted).tolist() == [0, 0] and int(short) == 0
    cache.fork(i32([-1, -1]))
    assert int(cache.compact()) == 0 and int(cache.ref.abs().max()) == 0
    granted, short = cache.grow(i32([48, 48]))
    assert host(granted).tolist() == [48, 48] and int(short) == 0
    assert host(cache.page_table).tolist() == [[0, 1, 2], [3, 4, 5]]


# ------------------------------------------------------------------ together
def test_serving_run(api):
    """Two layers, prompts, single tokens, forks, releases and a compaction; each step's
    attention against a reference that keeps every sequence's rows by itself."""
    rng = np.random.default_rng(77)
    masks = [mask_of(6, (0, 3)), mask_of(6, (2, 3))]
    H, H_kv, d, page, S, cols, n_pages = 6, 3, 64, 16, 5, 8, 30
    cache = api.PagedCache(masks, H, d, H_kv=H_kv, n_seqs=S, max_pages=cols, n_pages=n_pages,
                           page_size=page, max_new=40, device=DEV)
    T = cols * page
    alpha = rng.standard_normal((H, T)).astype(np.float32)
    rho = (-np.log1p(np.arange(T)) + 0.3 * rng.standard_normal((H, T))).astype(np.float32)
    a_dev, r_dev = torch.from_numpy(alpha).to(DEV), torch.from_numpy(rho).to(DEV)
    # the reference: each slot's own pages, never shared
    own = [[{"kc": np.zeros((cols, len(k_heads_of(m, H_kv)), page, d), np.uint8),
             "ks": np.zeros((cols, len(k_heads_of(m, H_kv))), np.float32),
             "vc": np.zeros((cols, H_kv, page, d), np.uint8),
             "vs": np.zeros((cols, H_kv), np.float32)} for m in masks] for _ in range(S)]
    lens = np.zeros(S, dtype=np.int32)
    row = np.arange(cols, dtype=np.int32)[None]

    def step(n_new):
        n_q = max(1, int(max(n_new)))
        granted, short = cache.grow(i32(n_new))
        assert int(short) == 0 and host(granted).tolist() == list(n_new)
        lens[:] += np.asarray(n_new, np.int32)
        for layer, mask in enumerate(masks):
            k, v, q = (torch.tensor(rng.standard_normal((S, h, n_q, d)), dtype=torch.bfloat16,
                                    device=DEV) for h in (H_kv, H_kv, H))
            cache.append(layer, k, v, n_new=granted)
            out = torch.full_like(q, 7.0)
            lse = torch.full(q.shape[:3], 7.0, device=DEV)
            cache.attend(layer, q, a_dev, r_dev, n_new=granted, out=out, lse=lse)
            kh = k_heads_of(mask, H_kv)
            for s in range(S):
                o = own[s][layer]
                one = slice(s, s + 1)
                ref.append(o["kc"], o["ks"], host(k.double())[one][:, kh], row, lens[one], n_new[s:s + 1], page)
                ref.append(o["vc"], o["vs"], host(v.double())[one], row, lens[one], n_new[s:s + 1], page)
                want, want_lse, tol, lse_tol = ref.attend(
                    host(q.double())[one], o["kc"], o["ks"], o["vc"], o["vs"], kh, alpha, rho, mask,
                    row, lens[one], n_new[s:s + 1], page)
                n = n_new[s]
                assert np.all(np.abs(host(out.double())[s, :, :n] - want[0, :, :n]) <= tol[0, :, :n])
                assert np.all(np.abs(host(lse.double())[s, :, :n] - want_lse[0, :, :n]) <= lse_tol[0, :, :n])
                assert np.all(host(out.double())[s, :, n:] == 7.0)

    def fork(parent):
        nonlocal own
        cache.fork(i32(parent))
        import copy
        own = [copy.deepcopy(own[p]) if p >= 0 else copy.deepcopy(own[s]) for s, p in enumerate(parent)]
        lens[:] = [lens[p] if p >= 0 else 0 for p in parent]

    step([21, 0, 40, 1, 0])
    step([1, 0, 1, 1, 0])
    fork([0, 0, 2, 3, 2])        # slots 1 and 4 take over begun pages
    step([1, 1, 1, 1, 1])        # ... and each gets a copy before it writes
    step([3, 17, 1, 15, 2])
    fork([1, -1, 4, 4, -1])      # reorder and release
    n = int(cache.compact())
    assert n == int((cache.ref > 0).sum()) and int((cache.ref[n:]).abs().sum()) == 0
    step([1, 5, 30, 1, 0])
    counts = np.bincount(host(cache.page_table)[host(cache.page_table) >= 0], minlength=n_pages)
    assert np.array_equal(counts, host(cache.ref))
    # slot 2 would pass the end of its row: the others grow
    granted, short = cache.grow(i32([60, 60, 60, 60, 60]))
    assert int(short) == 0 and host(granted).tolist() == [60, 60, 0, 60, 60]
    # more than the pool holds: nothing happens, and the step after it writes nothing
    before = [t.clone() for t in (cache.page_table, cache.seq_len, cache.ref, cache.pool)]
    granted, short = cache.grow(i32([20, 20, 20, 20, 20]))
    want_short = ref.grow(*[host(t) for t in before[:3]], np.full(5, 20), page)[4]
    assert int(short) == want_short > 0 and int(granted.abs().max()) == 0
    k = torch.randn((S, H_kv, 40, d), device=DEV)
    cache.append(0, k, k, n_new=granted)
    for t, b in zip((cache.page_table, cache.seq_len, cache.ref, cache.pool), before):
        assert torch.equal(t, b)


def test_captured_step_replays(api):
    """A captured step (grow, append, attend) replayed token after token, and a second graph on
    the same cache, against the same calls made one by one on another cache."""
    masks = [mask_of(4, (1,))]
    kw = dict(n_seqs=3, max_pages=6, n_pages=18, page_size=16, max_new=2, device=DEV)
    one, two = (api.PagedCache(masks, 4, 64, H_kv=2, **kw) for _ in range(2))
    T = 96
    alpha, rho = torch.randn((4, T), device=DEV), torch.randn((4, T), device=DEV)
    q = torch.zeros((3, 4, 2, 64), dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros((3, 2, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    want = i32([1, 2, 0])

    def step(cache, out, lse):
        granted, _ = cache.grow(want)
        cache.append(0, k, v, n_new=granted)
        cache.attend(0, q, alpha, rho, n_new=granted, out=out, lse=lse)
        return granted

    outs = [(torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV)) for _ in range(2)]
    graphs, side = [], torch.cuda.Stream()
    step(two, *outs[1])           # warm up on the other cache, then start over
    two.fork(i32([-1, -1, -1]))
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            keep = step(one, *outs[0])
        graphs.append((g, keep))
    gen = torch.Generator(device=DEV).manual_seed(1)
    for i in range(24):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device=DEV, generator=gen))
        want.copy_(i32([[1, 2, 0], [2, 1, 1], [0, 1, 2]][i % 3]))
        graphs[i % 2][0].replay()
        step(two, *outs[1])
        torch.cuda.synchronize()
        for a, b in zip(outs[0], outs[1]):
            assert torch.equal(a, b), i
        assert torch.equal(one.seq_len, two.seq_len) and torch.equal(one.page_table, two.page_table)
    assert one.device_status() == (0, 0)


def test_two_caches_on_two_streams(api):
    # calls of both kernels and a pool's calls at once, against the same ones one by one
    kw = [dict(n_q=1, seed=1, kernel="cache_attn"), dict(n_q=120, seed=2, kernel="cache_chunk")]
    cases = [Case(api, mask_of(8, (1, 6)), 2, 64, 64, [1900, 700], **k) for k in kw]
    alone = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run())
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
        assert c.cache.device_status() == (0, 0)


def test_status_of_a_fresh_cache(api):
    junk = torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV)
    del junk  # (what the allocator hands out next holds no zeros)
    cache = api.PagedCache([[0, 1]], 2, 64, n_seqs=2, max_pages=2, n_pages=4, device=DEV)
    assert cache.device_status() == (0, 0)


def test_refusals(api):
    cache = api.PagedCache([[0, 1]], 2, 64, n_seqs=2, max_pages=2, n_pages=4, page_size=16, device=DEV)
    q = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16, device=DEV)
    pat = torch.zeros((2, 32), device=DEV)
    bad = [
        lambda: cache.attend(0, q.float(), pat, pat),
        lambda: cache.attend(0, q),                              # frozen head, no pattern
        lambda: cache.attend(0, q, pat, pat[:, :16].contiguous()),
        lambda: cache.attend(0, q, pat, pat[:, ::2]),
        lambda: cache.attend(0, q.transpose(0, 1), pat, pat),    # strides
        lambda: cache.attend(0, q.expand(2, 2, 3, 64).contiguous(), pat, pat),  # over max_new
        lambda: cache.attend(0, q, pat, pat, n_new=torch.ones(2, dtype=torch.int64, device=DEV)),
        lambda: cache.attend(0, q, pat, pat, n_new=torch.ones(3, dtype=torch.int32, device=DEV)),
        lambda: cache.attend(0, q.cpu(), pat, pat),
        lambda: cache.attend(0, q, pat, pat, out=torch.zeros_like(q).float()),
        lambda: cache.append(0, q, q.half()),
        lambda: cache.append(0, q.float(), q),
        lambda: cache.append(0, None, q),
        lambda: cache.append(0, q[..., :32], q),
        lambda: cache.grow(torch.ones(3, dtype=torch.int32, device=DEV)),
        lambda: cache.fork(torch.ones(2, device=DEV)),
        lambda: cache.compact(into=(cache.ref, cache.ref)),
        lambda: api.PagedCache([[0, 1]], 2, 64, n_seqs=0, max_pages=2, n_pages=4, device=DEV),
        lambda: api.PagedCache([[0]], 2, 64, n_seqs=2, max_pages=2, n_pages=4, device=DEV),
        lambda: api.PagedCache([[0, 1]], 2, 48, n_seqs=2, max_pages=2, n_pages=4, device=DEV),
        lambda: api.PagedCache([[0, 1]], 2, 64, n_seqs=2, max_pages=2, n_pages=4, device=DEV,
                               pool=torch.zeros((4, 64), dtype=torch.uint8, device=DEV)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(api.SafError):
            call()
            pytest.fail(f"call {i} was taken")
