"""The hybrid layer on sequences of different lengths laid end to end against its definition in
64 bits (packed_reference has the bounds and their derivation)."""

import math

import pytest
import torch

import packed_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api
    return api


def inputs(lens, H, Hkv, d, seed=0, head=0, tail=0, layout="rows", T=None, fill=math.nan):
    """Q, K, V, dout with ``head`` rows before the first and ``tail`` behind the last sequence."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    total = head + sum(lens) + tail
    heads = H + 2 * Hkv
    if layout == "heads":
        x = torch.randn((heads, total, d), device="cuda", generator=gen).bfloat16().transpose(0, 1)
    else:
        x = torch.randn((total, heads, d), device="cuda", generator=gen).bfloat16()
    do = torch.randn((total, H, d), device="cuda", generator=gen).bfloat16()
    for t in (x, do):
        t[:head] = fill
        t[head + sum(lens):] = fill
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if layout == "rows":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    T = T or max([1, *lens])
    alpha = torch.randn((H, T), device="cuda", generator=gen)
    rho = (0.3 * torch.randn((H, T), device="cuda", generator=gen)
           - torch.log1p(torch.arange(T, device="cuda", dtype=torch.float32)))
    cu = [head]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, do, alpha, rho, torch.tensor(cu, dtype=torch.int32, device="cuda"), cu[:-1]


def run(api, lens, H, Hkv, d, frozen, back=True, change=None, **kw):
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, Hkv, d, **kw)
    if change:
        change(q, k, v, alpha, rho)
    layer = api.PackedAttention(H, d, frozen, max_total=q.shape[0], max_seqs=max(1, len(lens)),
                                max_len=max([1, *lens]), H_kv=Hkv)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    got = {"out": out, "lse": lse}
    if back:
        got.update(zip(("dq", "dk", "dv"), layer.backward(q, k, v, out, lse, do, cu, alpha, rho)))
    assert layer.device_status() == (0, 0)
    want = ref.packed(q, k, v, lens, starts, frozen, alpha, rho, do if back else None)
    for name, t in got.items():
        ref.check(name, t, *want[name])
    return got


LENS = [[1], [2, 1], [128], [129], [127, 1], [300], [5, 0, 260, 1, 128, 64], [0, 0, 77, 0],
        [384, 256, 130], [1] * 40, [513, 40, 200, 385]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_lengths(api, lens, d):
    run(api, lens, 4, 4, d, [0, 1, 0, 1])


@pytest.mark.parametrize("H,Hkv,frozen", [(1, 1, [0]), (1, 1, [1]), (4, 2, [0, 0, 1, 1]),
                                          (6, 2, [1, 0, 0, 0, 1, 1]), (8, 1, [0, 1] * 4),
                                          (4, 4, [0] * 4), (4, 2, [1] * 4), (3, 3, [1, 0, 1])])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_heads(api, H, Hkv, frozen, d):
    run(api, [200, 300, 50], H, Hkv, d, frozen, head=3, tail=9)


@pytest.mark.parametrize("layout", ["rows", "fused", "heads"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_layouts_and_rows_of_no_sequence(api, layout, d):
    got = run(api, [150, 257], 4, 2, d, [0, 1, 0, 0], layout=layout, head=130, tail=133)
    n = 130 + 150 + 257
    for name in ("out", "dq", "dk", "dv"):
        assert not got[name][:130].any() and not got[name][n:].any()
    assert (got["lse"][:, n:] == -math.inf).all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_given_buffers_keep_the_other_rows(api, d):
    lens, H, Hkv, frozen = [100, 31], 4, 2, [0, 1, 0, 0]
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, Hkv, d, head=2, tail=70)
    layer = api.PackedAttention(H, d, frozen, max_total=q.shape[0], max_seqs=2, max_len=100,
                                H_kv=Hkv)
    full = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")
    total = q.shape[0]
    # outputs in an order of their own
    out = full(H, total, d).transpose(0, 1)
    lse = torch.full((H, total), 5.0, device="cuda")
    layer.forward(q, k, v, cu, alpha, rho, out=out, lse=lse)
    grads = (full(total, H, d), full(Hkv, total, d).transpose(0, 1), full(total, Hkv, d))
    layer.backward(q, k, v, out, lse, do, cu, alpha, rho, grads=grads)
    want = ref.packed(q, k, v, lens, starts, frozen, alpha, rho, do)
    live = slice(2, 133)
    for name, t in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        ref.check(name, t[live], want[name][0][live], want[name][1][live])
        assert (t[:2] == 7).all() and (t[133:] == 7).all(), name
    assert (lse[:, 133:] == 5).all() and (lse[:, :2] == 5).all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_patterns_with_empty_rows_masks_and_wide_ranges(api, d):
    def change(q, k, v, alpha, rho):
        alpha[0, :5] = -math.inf                     # the first rows see nothing
        rho[1, 60:] = torch.finfo(torch.float32).min  # a window, masked by the lowest value
        alpha[2] *= 60                               # a range that needs the exact exponentials
        alpha[2, :3] = -math.inf
        rho[3, 1:] = -math.inf                       # the identity
        rho[4] = -math.inf                           # nothing at all
        alpha[5, ::2] = torch.finfo(torch.float32).min
    for lens in ([140, 3, 260], [4, 1, 2]):
        got = run(api, lens, 6, 6, d, [1] * 6, change=change)
        assert not got["out"][:, 4].any() and (got["lse"][4] == -math.inf).all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_other_sequences_infinities_stay_theirs(api, d):
    """Infinities and NaN in one sequence's K, V, Q reach no other one's results."""
    lens, H, frozen = [140, 100, 300], 4, [0, 1, 0, 1]
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, H, d)
    layer = api.PackedAttention(H, d, frozen, max_total=540, max_seqs=3, max_len=300)

    def both():
        out, lse = layer.forward(q, k, v, cu, alpha, rho)
        return out, lse.T, *layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    clean = [t.clone() for t in both()]
    q[140:240:7], k[141:240:5], v[140:240:3], do[150] = math.nan, math.inf, -math.inf, math.nan
    for a, b in zip(clean, both()):
        for part in (slice(0, 140), slice(240, 540)):
            if a is clean[2]:  # dQ: parts are added in the order in which they arrive
                ref.check("dq", b[part], a[part].double(), 2 * ref.U * a[part].double().abs() + 1e-6)
            else:
                assert torch.equal(a[part], b[part])


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_and_items(api, d):
    lens = [(37 * i) % 290 for i in range(60)]
    run(api, lens, 8, 4, d, [0, 1, 0, 0, 1, 1, 0, 0])


@pytest.mark.parametrize("Hkv", [256, 1])
@pytest.mark.parametrize("dynamic", [(), (255,), (0,), (7, 8)])
def test_as_many_heads_as_there_can_be(api, Hkv, dynamic):
    run(api, [130, 3], 256, Hkv, 32, [h not in dynamic for h in range(256)])


# more work items than the GPU has SMs, so that sequences share a frozen head's weights
SHARED = [[384] * 6, [700, 1, 130, 0, 129, 385, 384, 128, 257, 40], [900, 520, 512, 641, 300],
          [2, 1] * 45]


@pytest.mark.parametrize("lens", SHARED, ids=str)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_sequences_share_weights(api, lens, d):
    def change(q, k, v, alpha, rho):
        alpha[0, :5] = -math.inf                    # the first rows see nothing
        alpha[1] *= 60                              # exact exponentials
        rho[2, 60:] = torch.finfo(torch.float32).min
        rho[3, 1:] = -math.inf
    got = run(api, lens, 20, 20, d, [1] * 19 + [0], head=1, tail=5, change=change)
    # sequences that share agree with one alone to the bit (with the same longest length: the
    # tables are against the largest entries up to it)
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, 20, 20, d, head=1, tail=5)
    change(q, k, v, alpha, rho)
    b = max(range(len(lens)), key=lambda i: (lens[i] % 128, lens[i]))
    rows = slice(starts[b], starts[b] + lens[b])
    layer = api.PackedAttention(20, d, [1] * 19 + [0], max_total=lens[b], max_seqs=1,
                                max_len=max(lens), H_kv=20)
    one = [t[rows].contiguous() for t in (q, k, v, do)]
    cu1 = torch.tensor([0, lens[b]], dtype=torch.int32, device="cuda")
    out, lse = layer.forward(*one[:3], cu1, alpha, rho)
    dv = layer.backward(*one[:3], out, lse, one[3], cu1, alpha, rho)[2]
    assert torch.equal(got["out"][rows, :19], out[:, :19])
    assert torch.equal(got["lse"][:19, rows], lse[:19])
    assert torch.equal(got["dv"][rows, :19], dv[:, :19])


def test_long_sequence(api):
    run(api, [4000, 3, 1100], 2, 1, 128, [0, 1])


def test_fewer_rows_than_the_object_has_room_for(api):
    d, H, frozen = 64, 3, [0, 0, 1]
    layer = api.PackedAttention(H, d, frozen, max_total=5000, max_seqs=30, max_len=700)
    for seed, lens in enumerate(([700, 3], [], [0], [12] * 30, [699, 128, 500])):
        q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, H, d, seed=seed, T=800, tail=1)
        out, lse = layer.forward(q, k, v, cu, alpha, rho)
        grads = layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
        want = ref.packed(q, k, v, lens, starts, frozen, alpha, rho, do)
        for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(name, t, *want[name])


def test_bad_offsets_stay_in_bounds(api):
    """Offsets that fall, lie outside or are longer than max_len: no row is in two sequences, and
    the last good one is right."""
    d, H = 64, 2
    q, k, v, do, alpha, rho, _, _ = inputs([400], H, H, d)
    layer = api.PackedAttention(H, d, [0, 1], max_total=400, max_seqs=5, max_len=100)
    cu = torch.tensor([-5, 60, 20, 500, 90, 7], dtype=torch.int32, device="cuda")
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    assert layer.device_status() == (0, 0)
    want = ref.packed(q, k, v, [60], [0], [0, 1], alpha, rho)
    ref.check("out", out[:60], want["out"][0][:60], want["out"][1][:60])


@pytest.mark.parametrize("d", [32, 64, 128])
def test_same_bits_again_and_from_a_graph(api, d):
    lens, H, Hkv, frozen = [300, 40, 129, 700], 4, 2, [0, 0, 1, 0]
    q, k, v, do, alpha, rho, cu, _ = inputs(lens, H, Hkv, d)
    layer = api.PackedAttention(H, d, frozen, max_total=q.shape[0], max_seqs=4, max_len=700, H_kv=Hkv)

    def both():
        out, lse = layer.forward(q, k, v, cu, alpha, rho)
        return (out, lse, *layer.backward(q, k, v, out, lse, do, cu, alpha, rho))
    first, again = both(), both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taped = both()
    for t in taped:
        t.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    for other in (again, taped):
        for i, (a, b) in enumerate(zip(first, other)):
            if i == 2:
                ref.check("dq", b, a.double(), 2 * ref.U * a.double().abs() + 1e-6)
            else:
                assert torch.equal(a, b), i
    # other lengths, same graph
    cu.copy_(torch.tensor([0, 500, 500, 600, 1169], dtype=torch.int32))
    graph.replay()
    new = both()
    for i, (a, b) in enumerate(zip(new, taped)):
        if i == 2:
            ref.check("dq", b, a.double(), 2 * ref.U * a.double().abs() + 1e-6)
        else:
            assert torch.equal(a, b), i


def test_equals_the_layer_of_one_length(api):
    """B sequences of equal length: what HybridAttention computes."""
    B, H, T, d, frozen = 3, 4, 256, 64, [0, 1, 0, 0]
    q, k, v, do, alpha, rho, cu, starts = inputs([T] * B, H, H, d)
    layer = api.PackedAttention(H, d, frozen, max_total=B * T, max_seqs=B, max_len=T)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    dense = api.HybridAttention(B, H, T, d, frozen)
    b = lambda t: t.view(B, T, H, d).transpose(1, 2).contiguous()
    want, _ = dense.forward(b(q), b(k), b(v), alpha, rho)
    assert torch.equal(b(out), want)


def test_gradients_against_differences(api):
    """<dout, out(x + h) - out(x - h)> / 2h in 64 bits along random directions."""
    lens, H, Hkv, d, frozen = [70, 40], 2, 1, 32, [0, 1]
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, Hkv, d)
    layer = api.PackedAttention(H, d, frozen, max_total=110, max_seqs=2, max_len=70, H_kv=Hkv)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    grads = layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    bounds = ref.packed(q, k, v, lens, starts, frozen, alpha, rho, do)
    x = [t.double() for t in (q, k, v)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i, name in enumerate(("dq", "dk", "dv")):
        way = torch.randn(x[i].shape, dtype=torch.float64, device="cuda", generator=gen)
        f = []
        for h in (1e-5, -1e-5):
            y = [t + h * way if j == i else t for j, t in enumerate(x)]
            o = ref.packed(*y, lens, starts, frozen, alpha, rho)["out"][0]
            f.append((o * do.double()).sum())
        slope = (f[0] - f[1]) / 2e-5
        got = (grads[i].double() * way).sum()
        assert abs(got - slope) <= (bounds[name][1] * way.abs()).sum() + 1e-6 * abs(slope) + 1e-6


def test_other_stream_and_strided_inputs(api):
    lens, H, d, frozen = [130, 200], 2, 64, [0, 1]
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, H, d, layout="fused")
    layer = api.PackedAttention(H, d, frozen, max_total=330, max_seqs=2, max_len=200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = layer.forward(q, k, v, cu, alpha, rho)
    side.synchronize()
    want = ref.packed(q, k, v, lens, starts, frozen, alpha, rho)
    ref.check("out", out, *want["out"])


def test_more_items_than_are_shared_out(api):
    """Short sequences by the thousand: the backward's items go by the fixed order then."""
    lens = [(7 * i) % 12 for i in range(1400)]
    run(api, lens, 8, 8, 32, [0] * 8)


@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_are_ranked_or_listed(api, d):
    """Up to 48 rounds of items are ranked by cost, up to 192 listed in shared memory (48 at 128)."""
    lens = [(7 * i) % 12 for i in range(1300)] + [150, 300]
    run(api, lens, 8, 8, d, [0] * 7 + [1])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("layout", ["rows", "fused", "heads"])
def test_first_rows_see_themselves_only(api, d, layout):
    """dQ of a sequence's first row is zero: its weight is 1 whatever Q is.  What is left of
    P (dP - D) are fp32 sums of d products on either side (d 2^-24 of their sizes each, d <= 128)
    and exp's 2^-20: less than 2^-15 of sum |dO| |V|, times |K| / sqrt(d) and a bf16 rounding."""
    lens, H, Hkv = [1, 3, 200, 1, 2, 130], 4, 2
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, Hkv, d, layout=layout)
    layer = api.PackedAttention(H, d, [0] * H, max_total=sum(lens), max_seqs=6, max_len=200,
                                H_kv=Hkv)
    out, lse = layer.forward(q, k, v, cu)
    dq = layer.backward(q, k, v, out, lse, do, cu)[0]
    kk, vv = (t[starts].double().repeat_interleave(2, 1) for t in (k, v))
    size = (do[starts].double().abs() * vv.abs()).sum(-1, keepdim=True)
    assert (dq[starts].double().abs() <= 1.01 * 2.0 ** -15 * size * kk.abs() / math.sqrt(d)).all()


def test_rows_behind_the_longest_length(api):
    """A sequence longer than max_len: its first max_len rows are as if it ended there, the rest is
    left alone in given buffers and cleared in new ones."""
    d, H, n = 64, 2, 200
    q, k, v, do, alpha, rho, cu, _ = inputs([n, 90], H, H, d)
    layer = api.PackedAttention(H, d, [0, 1], max_total=290, max_seqs=2, max_len=130)
    want = ref.packed(q, k, v, [130, 90], [0, n], [0, 1], alpha, rho, do)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    grads = layer.backward(q, k, v, out, lse, do, cu, alpha, rho)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(name, t, *want[name])
    given = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    layer.forward(q, k, v, cu, alpha, rho, out=given[0], lse=given[1])
    assert (given[0][130:n] == 7).all() and (given[1][:, 130:n] == 7).all()
    assert torch.equal(given[0][:130], out[:130]) and torch.equal(given[0][n:], out[n:])


def test_gradients_into_one_projection(api):
    """dq, dk, dv as views of one tensor, as a projection's backward wants them."""
    lens, H, Hkv, d, frozen = [77, 200], 4, 2, 64, [0, 1, 0, 0]
    q, k, v, do, alpha, rho, cu, starts = inputs(lens, H, Hkv, d, layout="fused", tail=3)
    layer = api.PackedAttention(H, d, frozen, max_total=280, max_seqs=2, max_len=200, H_kv=Hkv)
    out, lse = layer.forward(q, k, v, cu, alpha, rho)
    whole = torch.full((280, H + 2 * Hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    parts = whole[:, :H], whole[:, H:H + Hkv], whole[:, H + Hkv:]
    layer.backward(q, k, v, out, lse, do, cu, alpha, rho, grads=parts)
    want = ref.packed(q, k, v, lens, starts, frozen, alpha, rho, do)
    for name, t in zip(("dq", "dk", "dv"), parts):
        ref.check(name, t[:277], want[name][0][:277], want[name][1][:277])
    assert (whole[277:] == 5).all()


def test_refusals(api):
    d, H = 64, 4
    q, k, v, do, alpha, rho, cu, _ = inputs([50, 14], H, 2, d, layout="fused")
    layer = api.PackedAttention(H, d, [0, 0, 0, 1], max_total=64, max_seqs=2, max_len=50, H_kv=2,
                                backward=False)
    ok = dict(q=q, k=k, v=v, cu_seqlens=cu, alpha=alpha, rho=rho)
    layer.forward(**ok)
    more = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[0]), dict(k=q), dict(v=v[:63]),
                dict(k=k.cpu()), dict(cu_seqlens=cu.long()), dict(cu_seqlens=more),
                dict(cu_seqlens=cu[:0]), dict(cu_seqlens=cu.cpu()), dict(alpha=None),
                dict(rho=rho[:, :49]), dict(alpha=alpha[:, :49], rho=rho[:, :49]),
                dict(alpha=alpha[0]), dict(rho=rho.double()), dict(out=q[:, :, :32]),
                dict(lse=torch.empty(64, H, device="cuda")),
                dict(q=torch.zeros((H, d, 64), device="cuda").bfloat16().permute(2, 0, 1)),
                dict(q=torch.zeros((65, H, d), device="cuda").bfloat16()),
                # rows that lie on no 16-byte boundary, and all in one place
                dict(q=torch.zeros((64, H * d + 1), device="cuda").bfloat16()[:, 1:].unflatten(1, (H, d))),
                dict(k=k[:1].expand(64, 2, d))):
        with pytest.raises(api.SafError):
            layer.forward(**{**ok, **bad})
    with pytest.raises(api.SafError):
        layer.backward(q, k, v, *layer.forward(**ok), do, cu, alpha, rho)
    for bad in (dict(d_h=48), dict(H_kv=3), dict(max_len=200000), dict(head_is_static=[0])):
        with pytest.raises(api.SafError):
            api.PackedAttention(**{**dict(H=4, d_h=64, head_is_static=[0] * 4, max_total=64, max_seqs=2,
                                          max_len=64), **bad})
