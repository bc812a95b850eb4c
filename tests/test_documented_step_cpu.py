"""The generation step that the project's overview shows, on the plain forms of the page
pool's operators."""
import types

import numpy as np
import pytest

import documented_step
import pages_ref

LAYERS, D = 2, 4


def plain():
    """The operators of the step, on numpy arrays; an append writes the keys as they are."""
    def reserve(table, lengths, new, refs, *, page_size, parents=None):
        return pages_ref.reserve(table, lengths, new, parents, refs, page_size)

    def copy(k, v, moves):
        for a, b in moves:
            if a >= 0 and b >= 0:
                k[:, b], v[:, b] = k[:, a], v[:, a]

    def append_at(q, k, v, kc, vc, positions, q_out, *, inv_freq, q_starts, kv_lengths, block_table,
                  layout):
        page, holders = kc.shape[1], {}
        for b, ln in enumerate(kv_lengths):
            for p in block_table[b, :-(-ln // page)]:
                holders.setdefault(int(p), set()).add(b)
        for b, ln in enumerate(kv_lengths):
            n = q_starts[b + 1] - q_starts[b]
            for i in range(n):
                at = ln - n + i
                p = int(block_table[b, at // page])
                assert holders[p] == {b}, "a page that is written is another row's too"
                kc[p, at % page], vc[p, at % page] = k[q_starts[b] + i], v[q_starts[b] + i]

    def compact(k, v, keep, counts, *, starts, kv_lengths, block_table, layout):
        page = k.shape[2]
        (k[:], v[:]), lengths = pages_ref.compact([k, v], keep, counts, starts, kv_lengths, block_table,
                                                  block_table, page, layout)
        return lengths

    return types.SimpleNamespace(mha_paged_reserve=reserve, mha_paged_copy=copy,
                                 mha_paged_append_at=append_at, mha_paged_compact=compact,
                                 mha_paged_tree_fwd=lambda *a, **kw: None)


@pytest.mark.parametrize("forks", [False, True, None], ids=["same_rows", "forks", "one_call"])
def test_steps_lose_no_page(forks):
    B, pages = 4, 200
    caches = [np.zeros((LAYERS, pages, 64, 1, D), np.int64) for _ in range(2)]

    def fill(tokens):
        rows = np.repeat(tokens[:, None, None], D, 2)
        return rows, rows, -rows

    pool = documented_step.Pool(plain(), lambda a: a, lambda a: a, caches,
                                lambda k: k[0, :, :, 0, 0], fill, None, B, 40, pages)
    documented_step.run(pool, 36, 3, forks)
