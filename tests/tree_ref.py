"""Plain float64 form of the attention of drafted trees over a paged cache, and the errors
that the stored types and fp32 arithmetic allow (numpy only)."""
import numpy as np

from paged_ref import HALF, U, positions


def bits(mask_row):
    """The number whose bit m says whether the row's token sees new token m."""
    return sum((int(w) & 0xffffffff) << (32 * i) for i, w in enumerate(mask_row))


def ancestors(parents, words):
    """Mask rows of one tree: a token sees its ancestors and itself."""
    sees = []
    for i, p in enumerate(parents):
        sees.append(1 << i | (sees[p] if p >= 0 else 0))
    rows = np.array([[s >> (32 * w) & 0xffffffff for w in range(words)] for s in sees],
                    dtype=np.uint32).reshape(len(parents), words)
    return rows.view(np.int32)


def tree_attention(q, kc, vc, mask, starts, lens, table, out, *, page, layout, scale, dtype):
    """(out, tolerance); q [T,H,d], caches in their layout, all float64; ``out``: what the
    rows of no sequence hold.  The tolerance is that of paged_ref.paged_attention: which
    positions a row sees changes neither the products nor the sums' lengths."""
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
        see = np.zeros((n, ln), dtype=bool)
        for i in range(n):
            number = bits(mask[lo + i])
            for j in range(ln):
                m = j - (full - n)
                see[i, j] = ok[j] and (m < 0 or number >> m & 1)
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
            o[lo:hi, h] = res
            tol[lo:hi, h] = (2.0 * weight + (HALF["bf16"] if dtype == "bf16" else 0.0)) * A
            tol[lo:hi, h] += HALF[dtype] * np.abs(res)
    return o, tol
