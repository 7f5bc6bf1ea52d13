"""A plain float64 / integer reference of the paged 8-bit cache (test infrastructure).

NumPy on the host, loops over slots, heads and pages; shares no code with the library.
"""

import math

import numpy as np

E4M3 = np.array([(-1.0 if c & 128 else 1.0)
                 * ((c & 7) / 8 * 2.0 ** -6 if (c >> 3 & 15) == 0
                    else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                 if c & 127 != 127 else np.nan for c in range(256)])
_POSITIVE = E4M3[:127]  # ascending


def encode(x):
    """Nearest e4m3 code (ties to even, saturating at 448; NaN -> 0x7f) of float64 values."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    bad = np.isnan(a)
    a = np.where(bad, 0.0, a)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(_POSITIVE[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(bad, 0x7F, code).astype(np.uint8)


def block_scale(values):
    """The least power of two s >= 2^-64 with 448 s >= |x| for every finite x."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    v = v[np.isfinite(v)]
    amax = v.max() if v.size else 0.0
    if amax == 0.0:
        return 2.0 ** -64
    m, e = math.frexp(amax)
    return 2.0 ** max(-64, e - 9 + (m > 0.875))


def append(codes, scales, x, table, seq_len, n_new, page):
    """One tensor (K or V): codes [n_pages, heads, page, d] uint8, scales [n_pages, heads],
    x [n_seqs, heads, n_q, d]; updated in place."""
    n_pages, heads = codes.shape[:2]
    for s in range(len(seq_len)):
        n = min(max(int(n_new[s]), 0), x.shape[2])
        end = max(int(seq_len[s]), 0)
        first = end - n
        end = min(end, table.shape[1] * page)
        for c in range(max(first, 0) // page, (end - 1) // page + 1 if end > max(first, 0) else 0):
            p = int(table[s, c])
            if not 0 <= p < n_pages:
                continue
            lo, hi = max(first, 0, c * page), min(end, (c + 1) * page)
            for h in range(heads):
                new = x[s, h, lo - first:hi - first].astype(np.float64)
                scale = block_scale(new)
                k = lo - c * page
                if k > 0:
                    old = float(scales[p, h])
                    if old > scale:
                        scale = old
                    elif old < scale:
                        codes[p, h, :k] = encode(E4M3[codes[p, h, :k]] * (old / scale))
                scales[p, h] = scale
                codes[p, h, k:k + hi - lo] = encode(new / scale)


def attend(q, k_codes, k_scales, v_codes, v_scales, k_heads, alpha, rho, frozen, table, seq_len,
           n_new, page):
    """(out, lse, bound on |out - computed|, bound on |lse - computed|); rows behind n_new hold
    NaN in all four.

    The bounds: a dot product of d terms summed in fp32 in any order, each addition off by at
    most 2^-23 of the sum of magnitudes; a few fp32 roundings of the logit and an approximate
    exponential (2^-20 together); weights rounded to f16 relative to the largest contribution
    (2^-11 of each, and at most 2^-25 of it where the weight is subnormal); one rounding of the
    result to bf16 (2^-8).
    """
    B, H, n_q, d = q.shape
    g, n_pages, cap = H // v_codes.shape[1], v_codes.shape[0], table.shape[1] * page
    out = np.full((B, H, n_q, d), np.nan)
    lse = np.full((B, H, n_q), np.nan)
    tol, lse_tol = out.copy(), lse.copy()
    for b in range(B):
        n = min(max(int(n_new[b]), 0), n_q)
        length = max(int(seq_len[b]), 0)
        keys = [j for j in range(min(length, cap)) if 0 <= table[b, j // page] < n_pages]
        keys = np.array(keys, dtype=np.int64)
        pg, sl = table[b, keys // page], keys % page
        for h in range(H if n else 0):
            kv = h // g
            sv = v_scales[pg, kv].astype(np.float64)
            v = E4M3[v_codes[pg, kv, sl]] * sv[:, None]
            if not frozen[h]:
                kh = k_heads.index(kv)
                k = E4M3[k_codes[pg, kh, sl]] * k_scales[pg, kh].astype(np.float64)[:, None]
            for t in range(n):
                i = length - n + t
                see = keys <= i
                if frozen[h]:
                    x = np.full(len(keys), -np.inf)
                    T = alpha.shape[1]
                    ok = see & (keys < T) & (i - keys < T)
                    x[ok] = (alpha[h, keys[ok]].astype(np.float64)
                             + rho[h, i - keys[ok]].astype(np.float64))
                    fin = np.isfinite(x)
                    mag = (np.abs(alpha[h, keys[fin]]) + np.abs(rho[h, i - keys[fin]])).max() \
                        if fin.any() else 0.0
                    delta = 2.0 ** -21 * (1 + mag) + 2.0 ** -20
                else:
                    with np.errstate(invalid="ignore"):
                        x = np.where(see, k @ q[b, h, t] / math.sqrt(d), -np.inf)
                        mag = np.abs(k[see]) @ np.abs(q[b, h, t]) / math.sqrt(d)
                    mag = np.nanmax(mag) if see.any() else 0.0
                    delta = 2.0 ** -23 * (d + 8) * mag + 2.0 ** -20
                top = x[see].max() if see.any() else -np.inf
                if top == -np.inf:
                    out[b, h, t], lse[b, h, t], tol[b, h, t], lse_tol[b, h, t] = 0, -np.inf, 0, 0
                    continue
                w = np.where(see, np.exp(x - top), 0.0)
                total = w.sum()
                w = w / total
                live = see
                out[b, h, t] = w[live] @ v[live]
                lse[b, h, t] = top + np.log(total)
                mean = w[live] @ np.abs(v[live])
                floor = len(keys) * 2.0 ** -25 * 448.0 * (w[live] * sv[live]).max()
                tol[b, h, t] = (2.0 ** -8 * np.abs(out[b, h, t])
                                + (2.0 ** -11 * 1.02 + 2 * delta) * mean + floor + 1e-37)
                lse_tol[b, h, t] = delta + 2.0 ** -20 * (1 + abs(lse[b, h, t]))
    return out, lse, tol, lse_tol


def fork(table, seq_len, ref, parent):
    n = len(seq_len)
    new = np.full_like(table, -1)
    lens = np.zeros_like(seq_len)
    for s, p in enumerate(parent):
        if 0 <= p < n:
            new[s], lens[s] = table[p], seq_len[p]
    ref = ref.copy()
    for old, now in zip(table.flatten(), new.flatten()):
        if old != now:
            if 0 <= old < len(ref):
                ref[old] -= 1
            if 0 <= now < len(ref):
                ref[now] += 1
    return new, lens, ref


def grow(table, seq_len, ref, n_new, page):
    """(table, seq_len, ref, granted, n_short, [(from, to) page copies])."""
    S, cols = table.shape
    free = [p for p in range(len(ref)) if ref[p] <= 0]
    table, lens, out_ref = table.copy(), seq_len.copy(), ref.copy()
    granted = np.zeros(S, dtype=np.int32)
    copies, at = [], 0

    def take():
        nonlocal at
        at += 1
        if at > len(free):
            return -1
        out_ref[free[at - 1]] = 1
        return free[at - 1]
    for s in range(S):
        length, n = max(int(seq_len[s]), 0), int(n_new[s])
        if n <= 0 or length + n > cols * page:
            continue
        granted[s] = n
        if length % page:
            held = int(table[s, length // page])
            if 0 <= held < len(ref) and ref[held] > 1:
                new = take()
                copies.append((held, new))
                out_ref[held] -= 1
                table[s, length // page] = new
        for c in range(-(-length // page), -(-(length + n) // page)):
            table[s, c] = take()
        lens[s] = length + n
    if at > len(free):
        return None, None, None, np.zeros(S, dtype=np.int32), at - len(free), []
    return table, lens, out_ref, granted, 0, copies


def compact(table, ref):
    """(table, ref, n_used, [(from, to)])."""
    n = int((ref > 0).sum())
    src = [p for p in range(n, len(ref)) if ref[p] > 0]
    dst = [p for p in range(n) if ref[p] <= 0]
    place = dict(zip(src, dst))
    new = np.array([[place.get(int(p), int(p)) for p in row] for row in table],
                   dtype=table.dtype).reshape(table.shape)
    out = ref.copy()
    for a, b in place.items():
        out[b], out[a] = ref[a], 0
    return new, out, n, list(place.items())
