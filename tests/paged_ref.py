"""Plain float64 forms of the operators of include/mha_paged.h, and the errors
that the stored types and fp32 arithmetic allow (numpy only)."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a rounding step, relative
U = 2.0 ** -24                                 # the same of the fp32 arithmetic


def rotate(x, pos, inv_freq, interleaved, sign=1.0):
    """x [..., d] float64, pos broadcastable to x.shape[:-1]."""
    y = x.copy()
    r = 2 * len(inv_freq)
    if r == 0:
        return y
    ang = np.asarray(pos, dtype=np.float64)[..., None] * inv_freq.astype(np.float64)
    c, s = np.cos(ang), sign * np.sin(ang)
    ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def pair_size(x, rotary, interleaved):
    """|a| + |b| over each element's pair (|x| where nothing is rotated)."""
    m = np.abs(x).copy()
    ia = np.arange(0, rotary, 2) if interleaved else np.arange(rotary // 2)
    ib = ia + 1 if interleaved else ia + rotary // 2
    both = m[..., ia] + m[..., ib]
    m[..., ia] = m[..., ib] = both
    return m


def norm_rope(x, w, pos, inv_freq, interleaved, eps):
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(n, pos, inv_freq, interleaved)


def norm_rope_tol(x, w, pos, inv_freq, interleaved, eps, dtype):
    """fp32: a sum of d squares (d/2 half steps on average of a tree; d at most),
    rsqrt, two products, the rotation (angle to 2^-25 turn = 3.2 half steps of
    fp32 at 1, sincospi 2, three operations), then one rounding."""
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y = rotate(n, pos, inv_freq, interleaved)
    d = x.shape[-1]
    return HALF[dtype] * np.abs(y) + (d + 16) * U * pair_size(n, 2 * len(inv_freq), interleaved)


def norm_rope_bwd(x, w, dy, pos, inv_freq, interleaved, eps):
    """(dx, dw or None)."""
    g = rotate(dy, pos, inv_freq, interleaved, sign=-1.0)
    if w is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, gw = x * r, g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdims=True))
    return dx, (g * n).reshape(-1, x.shape[-1]).sum(0)


def norm_rope_bwd_tol(x, w, dy, pos, inv_freq, interleaved, eps, dtype, chain):
    """As norm_rope_tol, the sums' errors relative to the sums of magnitudes;
    ``chain``: additions behind one another in the weight's gradient."""
    d = x.shape[-1]
    r2 = 2 * len(inv_freq)
    g = rotate(dy, pos, inv_freq, interleaved, sign=-1.0)
    gs = pair_size(dy, r2, interleaved)  # bounds |g|, and scales its error
    if w is None:
        return HALF[dtype] * np.abs(g) + 16 * U * gs, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dx = norm_rope_bwd(x, w, dy, pos, inv_freq, interleaved, eps)[0]
    aw = gs * np.abs(w)
    size = r * (aw + np.abs(n) * (aw * np.abs(n)).mean(-1, keepdims=True))
    tol_dw = (chain + d + 32) * U * (gs * np.abs(n)).reshape(-1, d).sum(0)
    return HALF[dtype] * np.abs(dx) + 3 * (d + 16) * U * size, tol_dw


def positions(cache, table_row, n, page, pages, layout):
    """Rows of positions 0 .. n - 1 of a cache: ([n, heads, d], present [n])."""
    j = np.arange(n)
    inside = j // page < len(table_row)
    ids = np.where(inside, np.asarray(table_row)[np.minimum(j // page, len(table_row) - 1)], -1) \
        if len(table_row) else np.full(n, -1)
    ok = (ids >= 0) & (ids < pages)
    i = np.where(ok, ids, 0)
    rows = cache[i, j % page] if layout == "bshd" else cache[i, :, j % page]
    return rows, ok


def paged_attention(q, kc, vc, starts, lens, table, out, *, page, layout, causal, scale, dtype):
    """(out, tolerance) of paged attention; q [T,H,d], caches in their layout, all
    float64; ``out``: what the rows of no sequence hold.

    Tolerance per element, A = sum w |v| the weighted mean magnitude: every
    softmax weight is off by its score's fp32 error (d products and sums of
    magnitude scale * |q|.|k|, the exponent's own rounding, exp2) and, in bf16, by
    half a step of bf16; the sums over the keys by at most one fp32 half step per
    key; the result by half a step of its type."""
    o, tol = out.copy(), np.zeros_like(out)
    T, H, d = q.shape
    pages = kc.shape[0]
    Hkv = kc.shape[2 if layout == "bshd" else 1]
    cap = table.shape[1] * page
    for b in range(len(lens)):
        lo = min(max(int(starts[b]), 0), T)
        hi = min(max(int(starts[b + 1]), lo), T)
        full = max(int(lens[b]), 0)
        n, ln = hi - lo, min(full, cap)
        if n == 0:
            continue
        K, ok = positions(kc, table[b], ln, page, pages, layout)
        V, _ = positions(vc, table[b], ln, page, pages, layout)
        K, V = np.where(ok[:, None, None], K, 0), np.where(ok[:, None, None], V, 0)
        j = np.arange(ln)[None, :]
        see = np.broadcast_to(ok[None, :], (n, ln))
        if causal:
            see = see & (j <= full - n + np.arange(n)[:, None])
        for h in range(H):
            g = h // (H // Hkv)
            qh = q[lo:hi, h]
            x = np.where(see, scale * (qh @ K[:, g].T), -np.inf)
            size = np.where(see, abs(scale) * (np.abs(qh) @ np.abs(K[:, g]).T), 0.0)
            m = x.max(-1, keepdims=True, initial=-np.inf)
            e = np.exp(x - np.where(np.isfinite(m), m, 0))
            l = e.sum(-1, keepdims=True)
            w = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
            res = w @ V[:, g]
            A = w @ np.abs(V[:, g])
            score = size.max(-1, keepdims=True, initial=0.0)
            weight = (d + 8) * U * score + 2.0 ** -20 + 2 * ln * U
            if dtype == "bf16":
                weight = weight + HALF["bf16"]
            o[lo:hi, h] = res
            tol[lo:hi, h] = 2.0 * weight * A if dtype == "f32" else \
                weight * A + ((d + 8) * U * score + 2.0 ** -20 + 2 * ln * U) * A
            tol[lo:hi, h] += HALF[dtype] * np.abs(res)
    return o, tol
