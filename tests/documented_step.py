"""The generation step that the project's overview shows, taken from there and run over and
over, with the page pool watched: every page's references are those of the rows that reach it,
no row writes to a page that another one holds, and the cache holds what the accepted tokens
left."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def shown_step() -> str:
    """The overview's block with a step of drafted trees."""
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    (block,) = [b for b in blocks if "mha_paged_reserve" in b]
    return block


# the same where no row forks: one call for the tables of a step, by how far the old ones reach
ONE_CALL = """
table, reach, refs, moves, _ = mha.mha_paged_reserve(table, reach, lengths + n, refs, page_size=64)
mha.mha_paged_copy(k_caches, v_caches, moves)
batch = dict(q_starts=starts, kv_lengths=reach, block_table=table, layout="bshd")
mha.mha_paged_append_at(q, k, v, k_caches[0], v_caches[0], positions, q, inv_freq=freq, **batch)
out = mha.mha_paged_tree_fwd(q, k_caches[0], v_caches[0], mask, max_q=n, **batch)
lengths = mha.mha_paged_compact(k_caches, v_caches, accepted, counts, starts=base,
                                kv_lengths=reach, block_table=table, layout="bshd")
"""


class Pool:
    """B sequences over a pool of pages; `up` and `down` take arrays to where mha computes and
    back, `fill` makes a step's q, k and v from the tokens' numbers, `read` tells from the keys
    the number of the token that each cell of layer 0 holds, [pages, page]."""

    def __init__(self, mha, up, down, caches, read, fill, freq, B, width, pool, page=64):
        self.up, self.down, self.read, self.fill = up, down, read, fill
        self.B, self.page, self.next = B, page, 1
        k_caches, v_caches = caches
        self.space = dict(mha=mha, k_caches=k_caches, v_caches=v_caches, freq=freq,
                          table=up(np.full((B, width), -1, np.int32)), refs=up(np.zeros(pool, np.int32)),
                          lengths=up(np.zeros(B, np.int32)), reach=up(np.zeros(B, np.int32)))
        self.held = [[] for _ in range(B)]  # the tokens of each sequence
        self.used = []                      # pages in use after each step

    def live(self, lengths):
        table, refs = self.down(self.space["table"]), np.zeros(len(self.down(self.space["refs"])), int)
        for row, ln in zip(table, lengths):
            pages = row[:-(-ln // self.page)]
            assert (pages >= 0).all()
            np.add.at(refs, pages, 1)
        return refs

    def step(self, code, rng, n, parents=None, prompt=False):
        """One step of trees of n tokens; `prompt`: chains that are accepted whole."""
        B, s = self.B, self.space
        forked = list(range(B)) if parents is None else parents
        before = [list(self.held[p]) if p >= 0 else [] for p in forked]
        tokens = self.next + np.arange(B * n)
        self.next += B * n
        trees = [[i - 1 if prompt else int(rng.integers(-1, i)) for i in range(n)] for _ in range(B)]
        keep, counts = np.zeros((B, n), np.int32), np.zeros(B, np.int32)
        for b, tree in enumerate(trees):
            at, path = n - 1 if prompt else int(rng.integers(-1, n)), []
            while at >= 0:
                path.insert(0, at)
                at = tree[at]
            keep[b, :len(path)], counts[b] = path, len(path)
            self.held[b] = before[b] + [int(tokens[b * n + i]) for i in path]
        words = -(-n // 32)
        mask = np.zeros((B * n, words), np.int64)
        for b, tree in enumerate(trees):
            for i, p in enumerate(tree):
                mask[b * n + i] = mask[b * n + p] if p >= 0 else 0
                mask[b * n + i, i // 32] |= 1 << i % 32
        q, k, v = self.fill(tokens)
        s.update(n=n, parents=self.up(np.array(forked, np.int32)), q=q, k=k, v=v,
                 base=self.up(np.array([len(x) for x in before], np.int32)),
                 starts=self.up(np.arange(B + 1, dtype=np.int32) * n),
                 positions=self.up(np.zeros(B * n, np.int32)),  # (angles 0: the keys stay as they are)
                 mask=self.up(mask.astype(np.uint32).view(np.int32)), accepted=self.up(keep),
                 counts=self.up(counts))
        exec(code, s)
        lengths, table = self.down(s["lengths"]), self.down(s["table"])
        assert lengths.tolist() == [len(x) for x in self.held]
        cells = self.read(s["k_caches"])
        for b, row in enumerate(table):
            have = [int(cells[row[j // self.page], j % self.page]) for j in range(lengths[b])]
            assert have == self.held[b], b
        refs = self.down(s["refs"])
        reach = lengths if code is not ONE_CALL else self.down(s["reach"])
        assert np.array_equal(refs, self.live(reach)), "references that no row has"
        # the last page of each row, which it writes to next, is its own
        for row, ln in zip(table, reach):
            assert ln % self.page == 0 or refs[row[ln // self.page]] == 1
        self.used.append(int((refs > 0).sum()))


def run(pool, steps, seed, forks):
    rng = np.random.default_rng(seed)
    code = shown_step() if forks is not None else ONE_CALL
    pool.step(code, rng, 70, prompt=True)
    for i in range(steps):
        parents = None
        if forks:
            parents = [int(x) for x in rng.integers(0, pool.B, pool.B)]
            if i % 3 == 2:
                parents[int(rng.integers(0, pool.B))] = -1
        pool.step(code, rng, (64, 17, 130, 1)[i % 4], parents)
    # some dozens of steps take no more than the tokens that there are
    most = max(len(x) for x in pool.held)
    assert pool.used[-1] <= pool.B * (-(-most // pool.page) + (3 if forks is None else 0))
