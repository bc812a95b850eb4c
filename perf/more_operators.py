"""Workloads of speculative decoding and of the page pool under a paged key/value cache.

Five operators, each in a plain form (elementary torch operations) and as the calls
a user makes of the framework (``own = True``):

  tree       attention of a tree of drafted tokens over a paged cache: every drafted
             token sees what is cached and its own ancestors (serving)
  append_at  drafted tokens normed and rotated at positions given with them, into the
             cells behind what is cached (serving)
  compact    the tokens that stay: an accepted path of a drafted tree moved to the front
             of its cells, or what is left of long sequences written into other pages
  reserve    the page tables of the next step: sequences grow, shrink, end, begin and fork
  copy       the pages that forked sequences may no longer share, in all layers

A case is a dict of plain values; ``prepare`` makes what a program holds before the
call, ``run`` is one pass, ``exact`` the definition, in 64 bits where it computes.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _tree(op, B, H, Hkv, d, dtype, n_lo, n_hi, len_lo, len_hi, page, layout, behind=0, norm=False,
          rotary=0, interleaved=False):
    c = dict(op=op, B=B, H=H, Hkv=Hkv, d=d, dtype=dtype, n_lo=n_lo, n_hi=n_hi, len_lo=len_lo,
             len_hi=len_hi, page=page, layout=layout, behind=behind)
    if op == "append_at":
        c.update(norm=norm, rotary=rotary, interleaved=interleaved)
    return c


def _compact(how, layers, B, Hkv, d, dtype, n_hi, len_lo, len_hi, page, layout):
    return dict(op="compact", how=how, layers=layers, B=B, Hkv=Hkv, d=d, dtype=dtype, n_hi=n_hi,
                len_lo=len_lo, len_hi=len_hi, page=page, layout=layout)


def _reserve(how, B, page, len_lo, len_hi, grow, beams, spare):
    return dict(op="reserve", how=how, B=B, page=page, len_lo=len_lo, len_hi=len_hi, grow=grow,
                beams=beams, spare=spare)


def _copy(layers, pairs, none, Hkv, d, dtype, page):
    return dict(op="copy", layers=layers, pairs=pairs, none=none, Hkv=Hkv, d=d, dtype=dtype,
                page=page)


def listed():
    return [
        # one user, 16 drafted tokens behind a short dialogue: latency
        dict(name="tree_one_h8_d64",
             **_tree("tree", 1, 8, 8, 64, BF16, 16, 16, 300, 300, 16, "bshd")),
        # a serving batch whose draft trees differ in size, grouped key/value heads
        dict(name="tree_drafts_b16_h32_kv8_d128",
             **_tree("tree", 16, 32, 8, 128, BF16, 9, 25, 1000, 4096, 64, "bhsd", behind=19)),
        # a large batch with trees of 64 tokens over long caches
        dict(name="tree_wide_b64_h32_kv8_d128",
             **_tree("tree", 64, 32, 8, 128, BF16, 64, 64, 4096, 8192, 64, "bshd")),
        # small fp32 trees (parity runs, small models)
        dict(name="tree_f32_b8_h8_kv2_d64",
             **_tree("tree", 8, 8, 2, 64, F32, 5, 13, 90, 700, 32, "bshd")),
        # the drafted tokens of a small batch on their way into the cache
        dict(name="append_at_b16_h32_kv8_d128",
             **_tree("append_at", 16, 32, 8, 128, BF16, 9, 25, 1000, 4096, 64, "bhsd", behind=19,
                     norm=True, rotary=128)),
        # ... and of 256 sequences with trees of 64
        dict(name="append_at_b256_h8_d64",
             **_tree("append_at", 256, 8, 8, 64, BF16, 64, 64, 128, 1024, 16, "bshd", rotary=64)),
        # after verification: the accepted path of each tree, 16 layers at once, in place
        dict(name="compact_accept_l16_b64_kv8_d128",
             **_compact("accept", 16, 64, 8, 128, BF16, 64, 128, 1024, 64, "bshd")),
        # long sequences shortened to their first and last tokens, into pages of their own
        dict(name="compact_evict_l4_b8_kv8_d128",
             **_compact("evict", 4, 8, 8, 128, BF16, 0, 4096, 8192, 64, "bhsd")),
        # the tables of a generation step: every sequence a few tokens longer, some end or begin
        dict(name="reserve_step_b256_page16",
             **_reserve("step", 256, 16, 128, 1024, 17, 1, 0.1)),
        # beam search over long sequences, small pages: every beam forks from one of its group
        dict(name="reserve_beams_b1024_page16",
             **_reserve("beams", 1024, 16, 2048, 8192, 1, 8, 0.1)),
        # eight beams of a small model, one layer: latency
        dict(name="copy_few_l1_kv8_d64", **_copy(1, 8, 3, 8, 64, BF16, 16)),
        # 128 forked sequences, all layers
        dict(name="copy_forks_l16_kv8_d128", **_copy(16, 160, 32, 8, 128, BF16, 64)),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "append_at", "compact", "reserve", "reserve", "copy"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    d = rng.choice([64, 128])
    e = 2 if dtype == BF16 else 4
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    layout = rng.choice(["bshd", "bhsd"])
    page = rng.choice([16, 32, 64, 128, 256])
    layers = _log_int(rng, 1, 16)
    if op == "reserve":
        how = rng.choice(["step", "step", "beams"])
        page = rng.choice([16, 32, 64, 128])
        B = _log_int(rng, 1, 1024)
        len_hi = _log_int(rng, 1, 8192)
        return _reserve(how, B, page, rng.randint(0, len_hi), len_hi, _log_int(rng, 1, 300),
                        _log_int(rng, 2, 16) if how == "beams" else 1,
                        rng.choice([0.0, 0.02, 0.1, 0.5]))
    if op == "copy":
        pairs = _log_int(rng, 1, 512)
        while pairs > 1 and layers * pairs * Hkv * d * page * e > 1 << 28:
            pairs = max(1, pairs // 2)
            layers = max(1, layers // 2)
        return _copy(layers, pairs, rng.randint(0, pairs), Hkv, d, dtype, page)
    B = _log_int(rng, 1, 128)
    len_hi = _log_int(rng, 1, 8192)
    if op == "compact":
        while B > 1 and layers * B * len_hi * Hkv * d * e > 1 << 28:
            B //= 2
        while layers > 1 and layers * B * len_hi * Hkv * d * e > 1 << 28:
            layers //= 2
        how = rng.choice(["accept", "evict"])
        return _compact(how, layers, B, Hkv, d, dtype,
                        rng.randint(1, min(200, len_hi)) if how == "accept" else 0,
                        rng.randint(1, len_hi), len_hi, page, layout)
    group = rng.choice([1, 1, 2, 3, 4, 8])
    while Hkv * group > 32:
        group = rng.choice([1, 2])
    H = Hkv * group
    n_hi = min(len_hi, _log_int(rng, 1, 256))
    n_lo = rng.randint(1, n_hi)
    len_lo = rng.randint(n_hi, len_hi)
    most = 1 << 28 if dtype == BF16 else 1 << 26
    while B > 1 and (B * len_hi * Hkv * d > most or
                     B * n_hi * len_hi * H * d > (1 << 36 if dtype == BF16 else 1 << 32)):
        B //= 2
    behind = rng.choice([0, 0, rng.randint(1, 64)])
    return _tree(op, B, H, Hkv, d, dtype, n_lo, n_hi, len_lo, len_hi, page, layout, behind,
                 rng.random() < 0.5, rng.choice([d, d, d // 2]) if op == "append_at" else 0,
                 rng.random() < 0.5)


def _spread(lo, hi, B):
    return [lo + (hi - lo) * b // max(1, B - 1) if B > 1 else hi for b in range(B)]


def _lens(case):
    """Drafted tokens and cached length (these tokens among them) of each sequence, the
    same for every seed but for their order; the largest trees behind the shortest caches."""
    n = _spread(case["n_lo"], case["n_hi"], case["B"])
    ln = _spread(case["len_lo"], case["len_hi"], case["B"])[::-1]
    return [(min(a, b), b) for a, b in zip(n, ln)]


def _parents(n, r):
    """A drafted tree, its best chain first: node 0 is the root, nodes up to a depth of 8 form
    the chain, and every other node hangs below an earlier one, often a shallow one."""
    return [-1 if i == 0 else (i - 1 if i <= 8 else int(i * r.random() ** 2)) for i in range(n)]


def _visible(parents):
    """Ancestors of each node, itself among them, as the bits of a number; and its depth."""
    sees, depth = [], []
    for i, p in enumerate(parents):
        sees.append((1 << i) | (sees[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return sees, depth


def _trees(case):
    """Parents of the drafted trees, one list per sequence of ``_lens``, the same for every
    seed."""
    return [_parents(n, random.Random(b)) for b, (n, _) in enumerate(_lens(case))]


def _evicted(ln):
    """Tokens that stay of a long sequence: the first few, and the last three quarters."""
    first = min(4, ln)
    return list(range(first)) + list(range(max(first, ln // 4), ln))


def _accepted(n, b):
    """An accepted path of a tree of n tokens as ``_parents`` lays it out: some of the best
    chain, then, sometimes, a branch beside it."""
    chain = min(n, 9)
    stop = 1 + (5 * b + 3) % chain
    path = list(range(stop))
    if stop < chain and n > 9:  # branches lie behind the chain
        at = 9 + (7 * b) % (n - 9)
        while len(path) < chain and at < n:
            path.append(at)
            at += 1 + (3 * b) % 5
    return path


def _kept(case):
    """(cached length, position of the kept tokens' list, the list) of each sequence."""
    res = []
    for b, ln in enumerate(_spread(case["len_lo"], case["len_hi"], case["B"])):
        if case["how"] == "accept":
            n = min(case["n_hi"], ln)
            res.append((ln, ln - n, _accepted(n, b)))
        else:
            res.append((ln, 0, _evicted(ln)))
    return res


def _next_lengths(case):
    """(old length, parent or -1, new length) of each sequence of a table update."""
    B, grow = case["B"], case["grow"]
    old = _spread(case["len_lo"], case["len_hi"], B)
    if case["how"] == "beams":  # beams of a group are equally long
        w = case["beams"]
        old = [old[b // w * w] for b in range(B)]
        par = []
        for b in range(B):
            lo = b // w * w
            hi = min(lo + w, B)
            par.append(lo + (b * b + 3 * b) % 7 % (hi - lo))
        return [(old[b], par[b], old[par[b]] + grow) for b in range(B)]
    res = []
    for b, ln in enumerate(old):
        kind = b % 16
        if kind == 5:    # ended
            res.append((ln, -1, 0))
        elif kind == 9:  # ended, another one begins in its place
            res.append((ln, -1, 1 + ln // 2))
        elif kind == 12:  # drafted tokens were rejected
            res.append((ln, b, max(0, ln - 1 - grow)))
        else:
            res.append((ln, b, ln + 1 + (b * 7) % grow))
    return res


def _page_bytes(case):
    return case["page"] * case["Hkv"] * case["d"] * (2 if case["dtype"] == BF16 else 4)


def _pages(n, page):
    return -(-n // page)


def _table_width(case):
    rows = _next_lengths(case)
    return max(1, max(_pages(max(a, c), case["page"]) for a, _, c in rows))


def work(case):
    if case["op"] == "reserve":
        rows = _next_lengths(case)
        # entries that are read: those of sequences that do not simply go on, and what is written
        read = sum(_pages(ln, case["page"]) for ln, _, _ in rows)
        return {"bytes": 4 * (read + case["B"] * (_table_width(case) + 6) + 2 * _pool(case)),
                "flops": 0}
    e = 2 if case["dtype"] == BF16 else 4
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * (case["pairs"] - case["none"]) * _page_bytes(case) +
                8 * case["pairs"], "flops": 0}
    if case["op"] == "compact":
        # a kept token that stays in its place is not touched
        moved = sum(sum(case["how"] == "evict" or i != k for i, k in enumerate(keep))
                    for _, _, keep in _kept(case))
        return {"bytes": 4 * case["layers"] * moved * Hkv * d * e +
                4 * sum(len(k) for _, _, k in _kept(case)), "flops": 0}
    H = case["H"]
    lens = _lens(case)
    T = sum(n for n, _ in lens)
    if case["op"] == "append_at":
        return {"bytes": 2 * T * (H + 2 * Hkv) * d * e + 8 * T, "flops": 10 * T * (H + Hkv) * d}
    seen = sum(n * (ln - n) for n, ln in lens) + \
        sum(sum(_visible(t)[1]) + len(t) for t in _trees(case))
    words = _pages(case["n_hi"], 32)
    return {"bytes": 2 * T * H * d * e + sum(ln for _, ln in lens) * Hkv * 2 * d * e + 4 * T * words,
            "flops": 4 * H * d * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _inv_freq(rotary):
    i = torch.arange(rotary // 2, dtype=torch.float64)
    return (BASE ** (-2.0 * i / rotary)).float().cuda()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pool(case):
    """Pages of the pool of a table update: what is in use before it (beams share three
    quarters of their pages), and some to spare."""
    rows = _next_lengths(case)
    live = sum(_pages(ln, case["page"]) for ln, _, _ in rows)
    more = sum(max(0, _pages(c, case["page"]) - _pages(a, case["page"])) + 1 for a, _, c in rows)
    return live + int(more * (1 + case["spare"])) + 3


def _scattered(lens, page, pool, width, np_rng):
    """A block table with pages taken from the pool in no order."""
    ids = np_rng.permutation(pool).astype(np.int32)
    table = np.zeros((len(lens), width), dtype=np.int32)
    at = 0
    for b, ln in enumerate(lens):
        m = _pages(ln, page)
        table[b, :m] = ids[at:at + m]
        at += m
    return table, ids[at:]


def _prepare_reserve(case, seed):
    np_rng = np.random.default_rng(seed)
    page, rows = case["page"], _next_lengths(case)
    B, width, pool = case["B"], _table_width(case), _pool(case)
    old = [r[0] for r in rows]
    table, _ = _scattered(old, page, pool, width, np_rng)
    if case["how"] == "beams":
        for b in range(B):  # whole pages at the front are the group's first beam's
            first = b // case["beams"] * case["beams"]
            m = old[b] // page * 3 // 4
            table[b, :m] = table[first, :m]
    refs = np.zeros(pool, dtype=np.int32)
    for b, ln in enumerate(old):
        refs[table[b, :_pages(ln, page)]] += 1
    # a prefix that the program itself holds on to
    refs[table[0, :_pages(old[0], page) // 2]] += 1
    # sequences keep their rows for the whole run; their order is the seed's
    if case["how"] == "step":
        order = np_rng.permutation(B)
        where = np.argsort(order)
        table = table[order]
        rows = [rows[o] for o in order]
        parents = [-1 if p < 0 else int(where[p]) for _, p, _ in rows]
    else:
        parents = [p for _, p, _ in rows]
    s = dict(case=case, table=_i32(table), lens=_i32([r[0] for r in rows]), parents=_i32(parents),
             new=_i32([r[2] for r in rows]), refs=_i32(refs))
    s["table_out"] = torch.empty_like(s["table"])
    s["lens_out"], s["refs_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["refs"])
    s["moves"] = torch.empty(B, 2, dtype=torch.int32, device="cuda")
    s["counts"] = torch.empty(2, dtype=torch.int32, device="cuda")
    if own:
        from transformer_head_scaled_mha_gb300 import mha_paged_reserve_workspace_size
        s["ws"] = torch.empty(mha_paged_reserve_workspace_size(B, pool), dtype=torch.uint8,
                              device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "reserve":
        return _prepare_reserve(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    np_rng = np.random.default_rng(seed)
    dt = _dt(case)
    Hkv, d, page = case["Hkv"], case["d"], case["page"]

    def normal(*shape, amp=1.0, about=0.0):
        x = torch.randn(*shape, generator=g, device="cuda", dtype=dt)
        return x if amp == 1.0 and about == 0.0 else x * amp + about

    s = dict(case=case)
    if case["op"] == "copy":
        pairs, none = case["pairs"], case["none"]
        pool = 2 * pairs + 3
        ids = np_rng.permutation(pool)[:2 * pairs].reshape(pairs, 2)
        ids[np_rng.permutation(pairs)[:none]] = -1
        s["moves"] = _i32(ids)
        shape = (case["layers"], pool, page, Hkv, d)
        s["kc"], s["vc"] = normal(*shape), normal(*shape)
        return s
    B = case["B"]
    order = np_rng.permutation(B).tolist()
    if case["op"] == "compact":
        kept = [_kept(case)[b] for b in order]
        lens = [k[0] for k in kept]
        width = _pages(max(lens), page) + 1
        used = sum(_pages(ln, page) for ln in lens)
        into = 0 if case["how"] == "accept" else used
        table, rest = _scattered(lens, page, used + into + 3, width, np_rng)
        s["table"] = _i32(table)
        s["to"] = s["table"]
        if into:
            to, at = np.zeros_like(table), 0
            for b, ln in enumerate(lens):
                m = _pages(ln, page)
                to[b, :m] = rest[at:at + m]
                at += m
            s["to"] = _i32(to)
        most = max(len(k[2]) for k in kept)
        keep = np.zeros((B, most), dtype=np.int32)
        for b, k in enumerate(kept):
            keep[b, :len(k[2])] = k[2]
        s["keep"], s["count"] = _i32(keep), _i32([len(k[2]) for k in kept])
        s["from"], s["kvlen"] = _i32([k[1] for k in kept]), _i32(lens)
        s["lens_out"] = torch.empty_like(s["kvlen"])
        pages = used + into + 3
        shape = (case["layers"], pages) + ((page, Hkv) if case["layout"] == "bshd"
                                           else (Hkv, page)) + (d,)
        s["kc"], s["vc"] = normal(*shape), normal(*shape)
        return s
    # ragged sequences, in an order of their own, and pages taken from a pool in no order
    H = case["H"]
    lens = [_lens(case)[b] for b in order]
    trees = [_trees(case)[b] for b in order]
    T = sum(n for n, _ in lens)
    width = _pages(max(ln for _, ln in lens), page) + 1
    pool = sum(_pages(ln, page) for _, ln in lens) + 3
    s["table"] = _i32(_scattered([ln for _, ln in lens], page, pool, width, np_rng)[0])
    s["starts"] = _i32(np.concatenate([[0], np.cumsum([n for n, _ in lens])]))
    s["kvlen"] = _i32([ln for _, ln in lens])
    s["max_q"], s["max_k"] = max(n for n, _ in lens), max(ln for _, ln in lens)
    rows = T + case["behind"]  # rows behind the last sequence, as a captured batch has them
    words = _pages(s["max_q"], 32)
    mask, pos, at = np.zeros((rows, words), dtype=np.uint32), np.zeros(rows, dtype=np.int32), 0
    for (n, ln), tree in zip(lens, trees):
        sees, depth = _visible(tree)
        for i in range(n):
            for w in range(words):
                mask[at + i, w] = (sees[i] >> (32 * w)) & 0xffffffff
        pos[at:at + n] = ln - n + np.array(depth)
        at += n
    s["mask"], s["pos"] = _i32(mask.view(np.int32)), _i32(pos)
    shape = (pool, page, Hkv, d) if case["layout"] == "bshd" else (pool, Hkv, page, d)
    s["kc"], s["vc"] = normal(*shape), normal(*shape)
    s["q"] = normal(rows, H, d)
    s["out"] = torch.zeros_like(s["q"])
    if case["op"] == "append_at":
        s["k"], s["v"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
        s["inv_freq"] = _inv_freq(case["rotary"])
        # learned scales near one
        s["qw"] = normal(d, amp=0.1, about=1.0) if case["norm"] else None
        s["kw"] = normal(d, amp=0.1, about=1.0) if case["norm"] else None
        return s
    s["scale"] = d ** -0.5
    if own:
        from transformer_head_scaled_mha_gb300 import mha_paged_workspace_size
        s["ws"] = torch.empty(mha_paged_workspace_size(B, rows, H, Hkv, d, s["max_q"], dt),
                              dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import transformer_head_scaled_mha_gb300 as mha
    c = s["case"]
    if c["op"] == "reserve":
        table, lens, refs, moves, counts = mha.mha_paged_reserve(
            s["table"], s["lens"], s["new"], s["refs"], page_size=c["page"], parents=s["parents"],
            table_out=s["table_out"], lengths_out=s["lens_out"], refs_out=s["refs_out"],
            moves=s["moves"], counts=s["counts"], workspace=s["ws"])
        return {"table": table, "lens": lens, "refs": refs, "moves": moves, "counts": counts}
    if c["op"] == "copy":
        mha.mha_paged_copy(s["kc"], s["vc"], s["moves"])
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    if c["op"] == "compact":
        lens = mha.mha_paged_compact(
            s["kc"], s["vc"], s["keep"], s["count"], s["lens_out"], starts=s["from"],
            kv_lengths=s["kvlen"], block_table=s["to"],
            src_table=None if s["to"] is s["table"] else s["table"], layout=c["layout"])
        return {"lens": lens, "k_cache": s["kc"], "v_cache": s["vc"]}
    batch = dict(q_starts=s["starts"], kv_lengths=s["kvlen"], block_table=s["table"],
                 layout=c["layout"])
    if c["op"] == "append_at":
        q = mha.mha_paged_append_at(
            s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["out"], q_weight=s["qw"],
            k_weight=s["kw"], inv_freq=s["inv_freq"], interleaved=c["interleaved"], eps=EPS,
            **batch)
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    out = mha.mha_paged_tree_fwd(s["q"], s["kc"], s["vc"], s["mask"], s["out"], max_q=s["max_q"],
                                 scale=s["scale"], workspace=s["ws"], **batch)
    return {"out": out}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_reserve(s):
    """Integers throughout; lists of pages have one place more than the pool, for what is
    not there."""
    page = s["case"]["page"]
    table, lens, new = s["table"].long(), s["lens"].long(), s["new"].long()
    parents, B, width, pool = s["parents"].long(), len(s["new"]), s["table"].shape[1], len(s["refs"])
    cap = width * page
    lens, new = lens.clamp(0, cap), new.clamp(0, cap)
    idx = torch.arange(width, device="cuda")[None]

    def named(ids, where):  # page number, or `pool` for none
        return torch.where(where & (ids >= 0) & (ids < pool), ids, pool)

    refs = torch.cat((s["refs"].long(), s["refs"].new_zeros(1).long()))
    held = named(table, idx < ((lens + page - 1) // page)[:, None])
    refs.scatter_add_(0, held.flatten(), torch.full_like(held.flatten(), -1))
    some = (parents >= 0) & (parents < len(lens))
    p = torch.where(some, parents, 0)
    keep = torch.where(some, torch.minimum(lens[p], new), 0)
    full, part = keep // page, keep % page != 0
    mine = named(table[p], (idx < ((keep + page - 1) // page)[:, None]))
    whole = torch.where(idx < full[:, None], mine, pool)
    refs.scatter_add_(0, whole.flatten(), torch.ones_like(whole.flatten()))
    last = torch.where(part, mine.gather(1, full.clamp(max=width - 1)[:, None])[:, 0], pool)
    i = torch.arange(B, device="cuda")
    lowest = torch.full((pool + 1,), B, device="cuda").scatter_reduce(0, last, i, "amin")
    stays = (last < pool) & (lowest[last] == i) & (refs[last] <= 0)
    refs[pool] = 0
    refs.scatter_add_(0, torch.where(stays, last, pool), torch.ones_like(last))
    copied = (last < pool) & ~stays
    had, want = (keep + page - 1) // page, (new + page - 1) // page
    need = copied + want - had
    first = need.cumsum(0) - need
    refs[pool] = 1
    free = refs <= 0
    rank = free.long().cumsum(0) - 1
    n_free, total = free.sum(), need.sum()
    given = torch.full((pool + 1,), -1, device="cuda")
    given.scatter_(0, torch.where(free, rank, pool), torch.arange(pool + 1, device="cuda"))
    given[pool] = -1
    take = lambda k: given[k.clamp(0, pool)]  # noqa: E731
    refs = torch.where(free & (rank < total), 1, refs)[:pool]
    fresh = take((first + copied)[:, None] + idx - had[:, None])
    out = torch.where(idx < had[:, None], torch.where(mine < pool, mine, -1), -1)
    out = torch.where((idx >= had[:, None]) & (idx < want[:, None]), fresh, out)
    here = copied[:, None] & (idx == full[:, None])
    out = torch.where(here, take(first)[:, None], out)
    got = torch.minimum((n_free - first).clamp(min=0), need)
    length = torch.where(got == need, new,
                         torch.where(copied & (got == 0), full * page, (had + got - copied.long()) * page))
    dst = torch.where(copied, take(first), -1)
    moves = torch.stack((torch.where(dst >= 0, last, -1), dst), -1)
    taken = torch.minimum(n_free, total)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return {"table": i32(out), "lens": i32(length), "refs": i32(refs), "moves": i32(moves),
            "counts": i32(torch.stack((taken, n_free - taken)))}


def _rotate(x, cos, sin, interleaved):
    """x [..., d] in 32 bits; the first 2 * cos.shape[-1] dimensions are rotated."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, v = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((u, v), dim=-1).flatten(-2) if interleaved else torch.cat((u, v), dim=-1)
    return torch.cat((rot, x[..., r:]), dim=-1)


def _norm_rope(x, w, cos, sin, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, cos, sin, interleaved).to(x.dtype)


def _tokens(s):
    """Sequence, index within it, cell's position and validity of each row of q."""
    starts, kvlen = s["starts"].long(), s["kvlen"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = (torch.searchsorted(starts, t, right=True) - 1).clamp(0, len(kvlen) - 1)
    n = starts[1:] - starts[:-1]
    i = t - starts[seq]
    return seq, i, kvlen[seq] - n[seq] + i, t < starts[-1]


def _cells(case, cache):
    """The cache as [..., pages, page, heads, d], whatever its layout."""
    return cache if case["layout"] == "bshd" else cache.transpose(-2, -3)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "reserve":
        return _plain_reserve(s)
    if c["op"] == "copy":
        src, dst = s["moves"].long().unbind(-1)
        # a pair without pages copies a page that no pair writes onto itself
        some = (src >= 0) & (dst >= 0)
        unused = s["kc"].shape[1] - 1
        free = torch.ones(unused + 1, dtype=torch.bool, device="cuda")
        free[torch.where(some, dst, src.clamp(min=0))] = False
        spare = free.long().argmax()
        src, dst = torch.where(some, src, spare), torch.where(some, dst, spare)
        for cache in (s["kc"], s["vc"]):
            cache[:, dst] = cache[:, src]
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    page = c["page"]
    if c["op"] == "compact":
        i = torch.arange(s["keep"].shape[1], device="cuda")[None]
        count = s["count"].long()[:, None]
        # places behind a list's end repeat its last one
        i = torch.minimum(i, count - 1)
        src = s["from"].long()[:, None] + s["keep"].long().gather(1, i)
        dst = s["from"].long()[:, None] + i
        a = s["table"].long().gather(1, src // page), src % page
        b = s["to"].long().gather(1, dst // page), dst % page
        for cache in (s["kc"], s["vc"]):
            rows = _cells(c, cache)
            rows[:, b[0], b[1]] = rows[:, a[0], a[1]]
        return {"lens": s["from"] + s["count"], "k_cache": s["kc"], "v_cache": s["vc"]}
    seq, i, pos, valid = _tokens(s)
    if c["op"] == "append_at":
        angle = s["pos"].double()[:, None] * s["inv_freq"].double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        q = torch.where(valid[:, None, None],
                        _norm_rope(s["q"], s["qw"], cos, sin, c["interleaved"]), s["out"])
        k = _norm_rope(s["k"], s["kw"], cos, sin, c["interleaved"])
        # the rows behind the last sequence repeat the last token's write
        T = s["k"].shape[0] - c["behind"]
        row = torch.arange(s["k"].shape[0], device="cuda").clamp(max=T - 1)
        p = pos[row]
        slot = s["table"].long()[seq[row], p // page], p % page
        _cells(c, s["kc"])[slot] = k[row]
        _cells(c, s["vc"])[slot] = s["v"][row]
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    # every sequence's queries and keys side by side, padded to the longest
    starts, kvlen = s["starts"].long(), s["kvlen"].long()
    H, Hkv = c["H"], c["Hkv"]
    j = torch.arange(s["max_k"], device="cuda")
    slot = s["table"].long()[:, j // page], (j % page)[None, :]
    live = j[None, :] < kvlen[:, None]
    K = _cells(c, s["kc"])[slot].float()
    V = torch.where(live[:, :, None, None], _cells(c, s["vc"])[slot].float(), 0.0)
    row = (starts[:-1, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=len(s["q"]) - 1)
    q = s["q"][row].float().unflatten(2, (Hkv, H // Hkv))
    sc = torch.einsum("bnghd,bkgd->bghnk", q, K) * s["scale"]
    base = kvlen - (starts[1:] - starts[:-1])
    m = (j[None, :] - base[:, None])[:, None].expand(-1, s["max_q"], -1)  # drafted token of a key
    word = s["mask"].long()[row].gather(2, (m // 32).clamp(0, s["mask"].shape[1] - 1))
    allowed = ((m < 0) | ((word >> (m % 32)) & 1 == 1)) & live[:, None, :]
    sc = sc.masked_fill(~allowed[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    w = (sc - torch.where(top == -math.inf, 0.0, top)).exp()
    o = torch.einsum("bghnk,bkgd->bnghd", w, V)
    total = w.sum(-1).permute(0, 3, 1, 2)[..., None]
    o = torch.where(total > 0, o / total, 0.0).flatten(2, 3)
    o = o[seq, i.clamp(0, s["max_q"] - 1)].to(s["q"].dtype)
    return {"out": torch.where(valid[:, None, None], o, s["out"])}


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------
def _define_reserve(s):
    """Sequence after sequence, as a program on the host would do it."""
    page = s["case"]["page"]
    table, lens, new, parents, refs = (s[x].cpu().numpy() for x in
                                       ("table", "lens", "new", "parents", "refs"))
    B, width = table.shape
    refs = refs.copy()
    for b in range(B):
        np.subtract.at(refs, table[b, :_pages(int(lens[b]), page)], 1)
    rows, writes = [], {}
    for i in range(B):
        p = int(parents[i])
        keep = min(int(lens[p]), int(new[i])) if p >= 0 else 0
        whole = table[p, :keep // page].tolist() if keep else []
        np.add.at(refs, np.array(whole, dtype=np.int64), 1)
        last = int(table[p, keep // page]) if keep % page else -1
        if last >= 0:
            writes.setdefault(last, []).append(i)
        rows.append((whole, last))
    stays = {who[0] for last, who in writes.items() if refs[last] <= 0}
    for last, who in writes.items():
        refs[last] += who[0] in stays
    free = iter(np.flatnonzero(refs <= 0).tolist())
    n_free, taken = int((refs <= 0).sum()), 0
    out = np.full((B, width), -1, dtype=np.int64)
    length, moves = np.zeros(B, dtype=np.int64), np.full((B, 2), -1, dtype=np.int64)
    for i, (whole, last) in enumerate(rows):
        pages, short = list(whole), False
        if last >= 0 and i in stays:
            pages.append(last)
        elif last >= 0:
            to = next(free, None)
            short = to is None
            if not short:
                moves[i] = last, to
                pages.append(to)
        while not short and len(pages) < _pages(int(new[i]), page):
            to = next(free, None)
            short = to is None
            if not short:
                pages.append(to)
        out[i, :len(pages)] = pages
        length[i] = len(pages) * page if short else int(new[i])
        kept = len(whole) + (last >= 0 and i in stays)
        taken += len(pages) - kept
        refs[np.array(pages[kept:], dtype=np.int64)] = 1
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return {"table": dev(out), "lens": dev(length), "refs": dev(refs.astype(np.int64)),
            "moves": dev(moves), "counts": dev(np.array([taken, n_free - taken]))}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "reserve":
        return _define_reserve(s)
    to64 = lambda t: None if t is None else t.double()  # noqa: E731
    kc, vc = to64(s["kc"]), to64(s["vc"])
    if c["op"] == "copy":
        for src, dst in s["moves"].cpu().tolist():
            if src >= 0 and dst >= 0:
                kc[:, dst].copy_(kc[:, src])
                vc[:, dst].copy_(vc[:, src])
        return {"k_cache": kc, "v_cache": vc}
    page, kvlen = c["page"], s["kvlen"].cpu().tolist()
    table = s["table"].cpu().tolist()

    def cell(row, p):  # the cell of a position, as indices of a cache without its layers
        return (row[p // page], p % page) if c["layout"] == "bshd" else (row[p // page], slice(None), p % page)

    if c["op"] == "compact":
        to, keep, first = (s[x].cpu().tolist() for x in ("to", "keep", "from"))
        count = s["count"].cpu().tolist()
        for b in range(c["B"]):
            if c["how"] == "evict":  # a run of tokens at a time: those with the same page ends
                i = 0
                while i < count[b]:
                    p, q, n = keep[b][i], i, 1
                    while i + n < count[b] and keep[b][i + n] == p + n and (p + n) % page and (q + n) % page:
                        n += 1
                    i += n
                    x, y = p % page, q % page
                    for cache in (kc, vc):
                        src, dst = cache[:, table[b][p // page]], cache[:, to[b][q // page]]
                        if c["layout"] == "bshd":
                            dst[:, y:y + n] = src[:, x:x + n]
                        else:
                            dst[:, :, y:y + n] = src[:, :, x:x + n]
                continue
            for cache in (kc, vc):
                rows = [cache[(slice(None),) + cell(table[b], first[b] + k)].clone()
                        for k in keep[b][:count[b]]]
                for i, r in enumerate(rows):
                    cache[(slice(None),) + cell(to[b], first[b] + i)] = r
        lens = torch.tensor([f + n for f, n in zip(first, count)]).cuda()
        return {"lens": lens, "k_cache": kc, "v_cache": vc}
    starts = s["starts"].cpu().tolist()
    if c["op"] == "append_at":
        r, inter = c["rotary"], c["interleaved"]

        def define(x, w):  # each pair as a complex number times e^(i pos f)
            if w is not None:
                x = to64(w) * x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               s["pos"].double()[:, None, None] * to64(s["inv_freq"]))
            z, rest = x[..., :r], x[..., r:]
            z = z.unflatten(-1, (r // 2, 2)) if inter else z.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
            return torch.cat((z, rest), -1)

        q, new = to64(s["out"]), define(to64(s["k"]), s["kw"])
        T = starts[-1]
        q[:T] = define(to64(s["q"]), s["qw"])[:T]
        for b, ln in enumerate(kvlen):
            lo, n = starts[b], starts[b + 1] - starts[b]
            p = torch.arange(ln - n, ln, device="cuda")
            ids = s["table"][b][p // page].long()
            for cache, x in ((kc, new), (vc, to64(s["v"]))):
                if c["layout"] == "bshd":
                    cache[ids, p % page] = x[lo:lo + n]
                else:
                    for h in range(c["Hkv"]):
                        cache[ids, h, p % page] = x[lo:lo + n, h]
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if work(c)["flops"] > 4e12:
        return None
    out, bits = to64(s["out"]), s["mask"].cpu().tolist()
    for b, ln in enumerate(kvlen):
        lo, n = starts[b], starts[b + 1] - starts[b]
        ids = table[b][:_pages(ln, page)]
        K, V = (torch.cat([cache[i] if c["layout"] == "bshd" else cache[i].transpose(0, 1)
                           for i in ids])[:ln] for cache in (kc, vc))
        see = torch.ones(n, ln, dtype=torch.bool)
        for i in range(n):
            number = sum((w & 0xffffffff) << (32 * k) for k, w in enumerate(bits[lo + i]))
            see[i, ln - n:] = torch.tensor([bool(number >> k & 1) for k in range(n)])
        see = see.cuda()
        for kv in range(c["Hkv"]):
            g = c["H"] // c["Hkv"]
            x = to64(s["q"][lo:lo + n, kv * g:(kv + 1) * g]).transpose(0, 1)
            logits = s["scale"] * (x @ K[:, kv].T)
            w = torch.softmax(logits.masked_fill(~see, -math.inf), -1)
            out[lo:lo + n, kv * g:(kv + 1) * g] = (w @ V[:, kv]).transpose(0, 1)
    return {"out": out}
