"""The page pool's operators as a program on the host would do them (numpy, one row and one
page after another)."""
import numpy as np


def reserve(table, lens, new, parents, refs, page):
    """(table, lengths, refs, moves, counts) of mha_paged_reserve."""
    (old, width), rows, pool = table.shape, len(new), len(refs)
    cap = width * page
    lens, new = np.clip(lens.astype(np.int64), 0, cap), np.clip(new.astype(np.int64), 0, cap)
    refs = refs.astype(np.int64).copy()
    there = lambda p: 0 <= p < pool  # noqa: E731
    for b in range(old):
        for p in table[b, :-(-lens[b] // page)]:
            if there(p):
                refs[p] -= 1
    kept, last = [], []
    for i in range(rows):
        par = i if parents is None else int(parents[i])
        n = min(lens[par], new[i]) if 0 <= par < old else 0
        pages = [int(p) if there(p) else -1 for p in table[par, :-(-n // page)]] if n else []
        part = n % page != 0
        for p in pages[:len(pages) - part]:
            if p >= 0:
                refs[p] += 1
        kept.append(pages)
        last.append(pages[-1] if part else -1)
    own = set()
    for p in sorted(set(last) - {-1}):
        if refs[p] <= 0:
            refs[p] += 1
            own.add(last.index(p))
    free = [p for p in range(pool) if refs[p] <= 0]
    n_free, used = len(free), 0
    out = np.full((rows, width), -1, dtype=np.int32)
    lengths, moves = np.zeros(rows, dtype=np.int32), np.full((rows, 2), -1, dtype=np.int32)
    for i in range(rows):
        pages = list(kept[i])
        copied = last[i] >= 0 and i not in own
        # places that need a page, in order
        places = ([len(pages) - 1] if copied else []) + list(range(len(pages), -(-new[i] // page)))
        pages += [-1] * (-(-new[i] // page) - len(pages))
        reach = new[i]
        if copied:
            pages[places[0]] = -1
        for x in places:
            if used == n_free:
                reach = min(reach, x * page)
                continue
            pages[x] = free[used]
            refs[free[used]] = 1
            if copied and x == places[0]:
                moves[i] = last[i], free[used]
            used += 1
        out[i, :len(pages)] = pages
        lengths[i] = reach
    return out, lengths, refs.astype(np.int32), moves, np.array([used, n_free - used], np.int32)


def stands(keep, count, start, length):
    """How many of a list's entries stand."""
    n = 0
    for i in range(max(0, min(int(count), len(keep)))):
        if keep[i] <= (keep[i - 1] if i else -1) or keep[i] >= length - start:
            break
        n += 1
    return n


def compact(caches, keep, counts, starts, lens, src, dst, page, layout):
    """New contents of the caches [layers, pages, ...] and the new lengths."""
    pool = caches[0].shape[1]
    before = [c.copy() for c in caches]
    after = [c.copy() for c in caches]
    out = np.zeros(len(lens), dtype=np.int32)
    for b in range(len(lens)):
        length = max(int(lens[b]), 0)
        start = 0 if starts is None else min(max(int(starts[b]), 0), length)
        n = stands(keep[b], counts[b], start, length)
        out[b] = start + n
        for i in range(n):
            p, q = start + int(keep[b][i]), start + i
            if max(p, q) // page >= src.shape[1]:
                continue
            x, y = src[b, p // page], dst[b, q // page]
            if not (0 <= x < pool and 0 <= y < pool):
                continue
            for old, new in zip(before, after):
                if layout == "bshd":
                    new[:, y, q % page] = old[:, x, p % page]
                else:
                    new[:, y, :, q % page] = old[:, x, :, p % page]
    return after, out
