"""The page pool: tables of the next step, copies of pages and the tokens that stay, against
the plain forms of pages_ref.py (integers and copies: equal bit for bit), and a program that
generates with drafted trees on top of them."""
import numpy as np
import pytest

import pages_ref

pytestmark = pytest.mark.gpu


def up(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def down(t):
    return t.cpu().numpy()


def run_reserve(table, lens, new, parents, refs, page, in_place=False, **kw):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    B, width = len(new), table.shape[1]
    r = up(refs)
    junk = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.full((mha.mha_paged_reserve_workspace_size(B, len(refs)),), 255, dtype=torch.uint8,
                    device="cuda")
    got = mha.mha_paged_reserve(up(table), up(lens), up(new), r, page_size=page,
                                parents=up(parents), table_out=junk(B, width), lengths_out=junk(B),
                                refs_out=r if in_place else junk(len(refs)), moves=junk(B, 2),
                                counts=junk(2), workspace=ws, **kw)
    torch.cuda.synchronize()
    return [down(t) for t in got]


def check_reserve(table, lens, new, parents, refs, page, **kw):
    want = pages_ref.reserve(table, lens, new, parents, refs, page)
    got = run_reserve(table, lens, new, parents, refs, page, **kw)
    for name, g, w in zip(("table", "lengths", "refs", "moves", "counts"), got, want):
        assert np.array_equal(g, w), (name, g, w)
    return want


def state(rng, B, page, width, spare, share=0.0, most=None):
    """Tables of B sequences of any length over a pool; rows share whole pages now and then."""
    lens = rng.integers(0, (width * page if most is None else most) + 1, B).astype(np.int32)
    need = -(-lens // page)
    pool = int(need.sum()) + spare
    ids = rng.permutation(pool)
    table = rng.integers(-5, pool + 5, (B, width)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        if b and rng.random() < share:
            a = int(rng.integers(0, b))
            n = min(lens[a] // page, lens[b] // page)
            table[b, :n] = table[a, :n]
    refs = np.zeros(pool, dtype=np.int32)
    for b in range(B):
        np.add.at(refs, table[b, :need[b]], 1)
    return table, lens, refs


SIZES = [
    # (sequences, page, width, spare): one CTA, one cluster, the whole GPU
    (1, 16, 1, 3), (1, 16, 0, 2), (5, 16, 4, 7), (7, 64, 3, 0), (33, 32, 9, 40), (64, 16, 60, 500),
    (3, 128, 700, 100), (300, 16, 20, 2000), (100, 16, 300, 30000), (1024, 16, 61, 3000),
    (300, 16, 400, 20000), (1500, 256, 44, 500), (9000, 16, 2, 1000),
]


@pytest.mark.parametrize("size", SIZES, ids=["B%d_p%d_w%d_%d" % s for s in SIZES])
@pytest.mark.parametrize("share", [0.0, 0.6])
def test_steps_forks_ends_and_beginnings(size, share):
    B, page, width, spare = size
    rng = np.random.default_rng(B + width)
    cap = width * page
    table, lens, refs = state(rng, B, page, width, spare, share)
    grow = np.minimum(lens + rng.integers(0, 2 * page, B), cap).astype(np.int32)
    check_reserve(table, lens, grow, None, refs, page)
    # beams: every row continues any row
    par = rng.integers(-1, B, B).astype(np.int32)
    new = np.where(par >= 0, lens[par], 0) + rng.integers(-page, page, B)
    check_reserve(table, lens, new.astype(np.int32), par, refs, page)
    check_reserve(table, lens, new.astype(np.int32), par, refs, page, in_place=True)
    # fewer and more rows than there were; pages that the caller holds on to
    held = refs + (rng.random(len(refs)) < 0.3).astype(np.int32)
    for rows in (max(1, B // 3), B + 9):
        par = rng.integers(-2, B + 2, rows).astype(np.int32)
        new = rng.integers(0, cap + 1, rows).astype(np.int32)
        check_reserve(table, lens, new, par, held, page)
    check_reserve(table, lens, np.zeros(B, np.int32), None, refs, page)  # all end


@pytest.mark.parametrize("seed", range(20))
def test_a_pool_that_runs_out(seed):
    rng = np.random.default_rng(seed)
    B, page, width = int(rng.integers(1, 40)), 16, int(rng.integers(1, 8))
    table, lens, refs = state(rng, B, page, width, int(rng.integers(0, 6)), 0.5)
    rows = int(rng.integers(1, 50))
    par = rng.integers(-1, B, rows).astype(np.int32)
    new = rng.integers(0, width * page + 1, rows).astype(np.int32)
    _, length, _, _, counts = check_reserve(table, lens, new, par, refs, page)
    assert counts[1] >= 0 and (length <= new).all()


@pytest.mark.parametrize("seed", range(20))
def test_tables_that_hold_anything(seed):
    """Entries, parents, lengths and reference counts that no program would have: nothing is
    touched outside the arrays, and the result is that of the definition."""
    rng = np.random.default_rng(100 + seed)
    B, page, width, pool = int(rng.integers(1, 30)), 32, int(rng.integers(1, 9)), 25
    wild = lambda a, lo, hi: np.where(rng.random(a.shape) < 0.2,  # noqa: E731
                                      rng.choice([-2 ** 31, -1, hi, 2 ** 31 - 1], a.shape), a)
    table = wild(rng.integers(0, pool, (B, width)), 0, pool).astype(np.int32)
    lens = wild(rng.integers(0, width * page + 1, B), 0, width * page + 5).astype(np.int32)
    new = wild(rng.integers(0, width * page + 1, B), 0, width * page + 5).astype(np.int32)
    par = wild(rng.integers(0, B, B), 0, B).astype(np.int32)
    refs = rng.integers(-2, 4, pool).astype(np.int32)
    check_reserve(table, lens, new, par, refs, page)
    check_reserve(table, lens, new, None, refs, page, in_place=True)


@pytest.mark.parametrize("B,width,pool", [(1500, 9, 12000), (60, 1300, 30000), (40, 3, 60000),
                                          (2500, 3, 900)])
def test_large_tables_that_hold_anything(B, width, pool):
    """The same, of the whole GPU's kernels; and pools that run out."""
    rng = np.random.default_rng(B)
    page = 16
    wild = lambda a, lo, hi: np.where(rng.random(a.shape) < 0.1,  # noqa: E731
                                      rng.choice([-2 ** 31, -1, hi, 2 ** 31 - 1], a.shape), a)
    table = wild(rng.integers(0, pool, (B, width)), 0, pool).astype(np.int32)
    lens = wild(rng.integers(0, width * page + 1, B), 0, width * page + 5).astype(np.int32)
    new = wild(rng.integers(0, width * page + 1, B), 0, width * page + 5).astype(np.int32)
    par = wild(rng.integers(0, B, B), 0, B).astype(np.int32)
    for least in (-2, 0, 1):
        refs = rng.integers(least, 4, pool).astype(np.int32)
        check_reserve(table, lens, new, par, refs, page)
        check_reserve(table, lens, new, None, refs, page, in_place=True)


def test_empty_problems():
    z = lambda *s: np.zeros(s, dtype=np.int32)  # noqa: E731
    table, lens, refs = np.array([[1, 0]], np.int32), np.array([20], np.int32), np.ones(5, np.int32)
    check_reserve(table, lens, z(0), None, refs, 16)            # no rows: all pages given back
    check_reserve(z(0, 2), z(0), np.array([30, 5], np.int32), None, z(5), 16)
    check_reserve(z(1, 2), z(1), np.array([30], np.int32), None, z(0), 16)  # no pages
    check_reserve(z(1, 0), z(1), np.array([30], np.int32), None, z(3), 16)  # tables without width


def test_reserve_on_streams_in_graphs_and_again():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(3)
    for B, width in ((20, 8), (300, 300)):
        table, lens, refs = state(rng, B, 16, width, 4000, 0.4, most=width * 16 // 2)
        tables = [up(table), torch.zeros(B, width, dtype=torch.int32, device="cuda")]
        lengths, counts = [up(lens), torch.zeros_like(up(lens))], [up(refs), up(refs)]
        news = [up((lens + 7 * (i + 1)).astype(np.int32)) for i in range(6)]
        new = news[0].clone()
        moves = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
        par = up(rng.integers(0, B, B).astype(np.int32))
        ws = torch.empty(mha.mha_paged_reserve_workspace_size(B, len(refs)), dtype=torch.uint8,
                         device="cuda")

        def step(i):
            return mha.mha_paged_reserve(
                tables[i % 2], lengths[i % 2], new, counts[i % 2], page_size=16, parents=par,
                table_out=tables[1 - i % 2], lengths_out=lengths[1 - i % 2],
                refs_out=counts[1 - i % 2], moves=moves, workspace=ws)
        step(0)
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(i)
            graphs.append(g)
        tables[0].copy_(up(table))
        lengths[0].copy_(up(lens))
        counts[0].copy_(up(refs))
        want = (table, lens, refs)
        for i, n in enumerate(news):
            new.copy_(n)
            graphs[i % 2].replay()
            want = pages_ref.reserve(want[0], want[1], down(n), down(par), want[2], 16)[:3]
            for g, w in zip((tables, lengths, counts), want):
                assert np.array_equal(down(g[1 - i % 2]), w)
        side = torch.cuda.Stream()
        outs = [mha.mha_paged_reserve(up(table), up(lens), new, up(refs), page_size=16, parents=par,
                                      stream=s) for s in (None, side, None, side)]
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------
def caches(rng, shape, dt):
    import torch
    bits = rng.integers(-2 ** 15 if dt == "bf16" else -2 ** 31, 2 ** 15 if dt == "bf16" else 2 ** 31,
                        (2, *shape)).astype(np.int16 if dt == "bf16" else np.int32)
    return bits, [up(b).view(torch.bfloat16 if dt == "bf16" else torch.float32) for b in bits]


def bits_of(t):
    import torch
    return down(t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("layers,pages,page,Hkv,d,n", [
    (1, 9, 16, 1, 64, 3), (3, 40, 32, 2, 128, 25), (2, 9, 256, 3, 64, 4), (1, 5000, 16, 1, 64, 2400),
    (7, 33, 64, 8, 128, 11), (0, 9, 16, 1, 64, 3), (2, 1, 16, 2, 64, 5)])
def test_pages_are_copied(dt, layers, pages, page, Hkv, d, n):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(n)
    want, (kc, vc) = caches(rng, (layers, pages, page, Hkv, d), dt)
    moves = np.full((n, 2), -1, np.int32)
    ids = rng.permutation(pages)
    m = min(n, pages // 2)
    moves[:m] = ids[:2 * m].reshape(m, 2)
    bad = rng.random(n) < 0.3
    moves[bad, rng.integers(0, 2)] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31])
    rng.shuffle(moves)
    if n > 2:
        moves[1] = moves[1, 0]  # a page onto itself
    for c in want:
        before = c.copy()
        for a, b in moves:
            if 0 <= a < pages and 0 <= b < pages:
                c[:, b] = before[:, a]
    mha.mha_paged_copy(kc, vc, up(moves))
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])
    if layers == 1:  # the same without the dimension of layers
        mha.mha_paged_copy(kc[0], vc[0], up(moves[:, ::-1].copy()))
        for c in want:
            before = c.copy()
            for a, b in moves:
                if 0 <= a < pages and 0 <= b < pages:
                    c[:, a] = before[:, b]
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


# ---------------------------------------------------------------------------
# tokens that stay
# ---------------------------------------------------------------------------
def lists(rng, B, most, lens, starts, broken):
    keep = rng.integers(-3, 5000, (B, max(most, 1))).astype(np.int32)[:, :most]
    counts = np.zeros(B, dtype=np.int32)
    for b in range(B):
        room = lens[b] - starts[b]
        n = int(rng.integers(0, min(most, max(room, 0)) + 1))
        keep[b, :n] = np.sort(rng.permutation(max(room, 0))[:n])
        counts[b] = n
        if broken and n and rng.random() < 0.6:
            i = int(rng.integers(0, n))
            keep[b, i] = rng.choice([-1, room, 2 ** 31 - 1, -2 ** 31, keep[b, max(i - 1, 0)]])
        if broken and rng.random() < 0.2:
            counts[b] = rng.choice([-4, most + 3, 2 ** 31 - 1])
    return keep, counts


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("layers,B,Hkv,d,page,width,most,layout", [
    (1, 1, 1, 64, 16, 3, 1, "bshd"), (3, 9, 2, 64, 16, 12, 9, "bshd"), (2, 5, 3, 128, 32, 9, 32, "bhsd"),
    (1, 4, 2, 128, 64, 6, 33, "bshd"), (2, 3, 1, 64, 16, 60, 900, "bhsd"), (1, 7, 4, 128, 128, 4, 200, "bshd"),
    (1, 2, 8, 128, 256, 10, 2500, "bshd"), (2, 40, 8, 64, 16, 5, 12, "bhsd"), (0, 3, 2, 64, 16, 5, 9, "bshd"),
    (1, 3, 2, 64, 16, 5, 0, "bshd")])
@pytest.mark.parametrize("how", ["in place", "elsewhere", "broken"])
def test_tokens_that_stay(dt, layers, B, Hkv, d, page, width, most, layout, how):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(most + B)
    pool = 2 * B * width + 2
    ids = rng.permutation(pool)[:2 * B * width].reshape(2, B, width).astype(np.int32)
    src, dst = ids[0], ids[1] if how == "elsewhere" else ids[0]
    lens = rng.integers(0, width * page + 1, B).astype(np.int32)
    starts = np.array([rng.integers(0, n + 1) for n in lens], dtype=np.int32)
    if B > 1:
        starts[0] = 0
    if most > 32:
        starts[::2] = 0
    keep, counts = lists(rng, B, most, lens, starts, how == "broken")
    if how == "broken":
        lens[-1], starts[-1] = 10 ** 6, 5
        starts[B // 2] = -9
        src = dst = np.where(rng.random(src.shape) < 0.1, rng.choice([-1, pool, 2 ** 31 - 1]),
                             src).astype(np.int32)
    shape = (layers, pool) + ((page, Hkv) if layout == "bshd" else (Hkv, page)) + (d,)
    start, (kc, vc) = caches(rng, shape, dt)
    want, length = pages_ref.compact(start, keep, counts, starts, lens, src, dst, page, layout)
    got = mha.mha_paged_compact(kc, vc, up(keep), up(counts), starts=up(starts), kv_lengths=up(lens),
                                block_table=up(dst), src_table=up(src) if how == "elsewhere" else None,
                                layout=layout)
    torch.cuda.synchronize()
    assert np.array_equal(down(got), length)
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


@pytest.mark.parametrize("most", [20, 4000])
def test_lists_from_the_first_position(most):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(0)
    lens = np.array([most + 900, most // 2, 0, most + 17], dtype=np.int32)
    width = int(-(-lens.max() // 64))
    table = rng.permutation(4 * width).reshape(4, width).astype(np.int32)
    keep, counts = lists(rng, 4, most, lens, np.zeros(4, int), False)
    keep[3, :17] = np.arange(17)  # the head stays where it is, the rest moves up
    keep[3, 17:] = np.arange(34, most + 17)[:most - 17]
    counts[3] = most - 17
    keep[3, most - 17:] = 0
    start, (kc, vc) = caches(rng, (2, 4 * width, 64, 2, 64), "bf16")
    want, length = pages_ref.compact(start, keep, counts, None, lens, table, table, 64, "bshd")
    got = mha.mha_paged_compact(kc, vc, up(keep), up(counts), kv_lengths=up(lens),
                                block_table=up(table), layout="bshd")
    torch.cuda.synchronize()
    assert np.array_equal(down(got), length)
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


def test_moves_beyond_32_bit_offsets():
    """Caches of 3.2e9 elements in two layers: their last pages."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page, Hkv, d, pages = 64, 8, 128, 24500
    g = torch.Generator(device="cuda").manual_seed(0)
    kc, vc = (torch.empty(2, pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    last = [pages - 1, pages - 2, pages - 3, 1]
    small = [torch.randn(2, 4, page, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    for c, s in zip((kc, vc), small):
        for i, p in enumerate(last):
            c[:, p] = s[:, i]
    copies = lambda ids: up(np.array([[ids[0], ids[3]]], np.int32))  # noqa: E731
    i32 = lambda *a: up(np.array(a, np.int32))  # noqa: E731
    for keep in (np.arange(3, 20), np.arange(50, 120)):
        for cs, ids in (((kc, vc), last), (small, [0, 1, 2, 3])):
            mha.mha_paged_copy(*cs, copies(ids))
            mha.mha_paged_compact(*cs, up(keep.astype(np.int32)[None]), i32(len(keep)),
                                  starts=i32(30), kv_lengths=i32(190),
                                  block_table=up(np.array([ids], np.int32)), layout="bshd")
        torch.cuda.synchronize()
        for c, s in zip((kc, vc), small):
            for i, p in enumerate(last):
                assert torch.equal(c[:, p], s[:, i])


def test_moves_on_streams_and_in_graphs():
    """A captured copy and compaction, replayed with other pairs and lists, and both at once on
    streams of their own, each on caches of its own."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(5)
    layers, pages, page, Hkv, d, B, width = 3, 40, 16, 2, 64, 4, 8
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    spare = np.setdiff1d(np.arange(pages), table).astype(np.int32)
    lens = np.array([100, 128, 7, 60], np.int32)
    starts = np.array([3, 0, 0, 50], np.int32)
    for most in (12, 90):
        want, (kc, vc) = caches(rng, (layers, pages, page, Hkv, d), "bf16")
        turns = []
        for _ in range(3):
            keep, counts = lists(rng, B, most, lens, starts, False)
            moves = np.stack([rng.permutation(table.ravel())[:4], rng.permutation(spare)[:4]], -1)
            turns.append((keep, counts, moves.astype(np.int32)))
        keep, counts, moves = (up(x) for x in turns[0])
        out, args = up(lens).clone(), dict(starts=up(starts), kv_lengths=up(lens), block_table=up(table),
                                           layout="bshd")
        other = [c.clone() for c in (kc, vc)]

        def both(c, stream=None):
            mha.mha_paged_copy(*c, moves, stream=stream)
            mha.mha_paged_compact(*c, keep, counts, out, stream=stream, **args)
        both([c.clone() for c in (kc, vc)])  # (warm)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both((kc, vc))
        side = torch.cuda.Stream()
        for turn in turns:
            for t, x in zip((keep, counts, moves), turn):
                t.copy_(up(x))
            torch.cuda.synchronize()
            graph.replay()
            both(other, side)
            torch.cuda.synchronize()
            for c in want:
                c[:, turn[2][:, 1]] = c[:, turn[2][:, 0]]
            want, length = pages_ref.compact(want, turn[0], turn[1], starts, lens, table, table, page,
                                             "bshd")
            assert np.array_equal(down(out), length)
            for c, o, w in zip((kc, vc), other, want):
                assert np.array_equal(bits_of(c), w) and torch.equal(c.view(torch.int16), o.view(torch.int16))


@pytest.mark.parametrize("most", [3, 40])
def test_thousands_of_sequences_and_none(most):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(6)
    B, width, page = 5000, 4, 16
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    lens = rng.integers(0, width * page + 1, B).astype(np.int32)
    starts = np.array([rng.integers(0, n + 1) for n in lens], np.int32)
    keep, counts = lists(rng, B, most, lens, starts, True)
    start, (kc, vc) = caches(rng, (1, B * width, page, 1, 64), "bf16")
    got = mha.mha_paged_compact(kc, vc, up(keep), up(counts), starts=up(starts), kv_lengths=up(lens),
                                block_table=up(table), layout="bshd")
    want, length = pages_ref.compact(start, keep, counts, starts, lens, table, table, page, "bshd")
    torch.cuda.synchronize()
    assert np.array_equal(down(got), length)
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])
    none = torch.zeros(0, most, dtype=torch.int32, device="cuda")
    got = mha.mha_paged_compact(kc, vc, none, none[:, 0], kv_lengths=none[:, 0].contiguous(),
                                block_table=none, layout="bshd")
    assert got.shape == (0,)
    mha.mha_paged_copy(kc, vc, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(kc), want[0])


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("B", [3, 90])
def test_long_lists_in_place(dt, d, B):
    """Few sequences, whose rows are split over CTAs, and so many that they are not; some
    rounds to a list."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(B + d)
    Hkv, page, width = 5, 32, 45
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    lens = rng.integers(width * page // 2, width * page + 1, B).astype(np.int32)
    starts = np.where(rng.random(B) < 0.5, 0, rng.integers(0, 400, B)).astype(np.int32)
    keep, counts = lists(rng, B, width * page, lens, starts, False)
    start, (kc, vc) = caches(rng, (1, B * width, page, Hkv, d), dt)
    got = mha.mha_paged_compact(kc, vc, up(keep), up(counts), starts=up(starts), kv_lengths=up(lens),
                                block_table=up(table), layout="bshd")
    want, length = pages_ref.compact(start, keep, counts, starts, lens, table, table, page, "bshd")
    torch.cuda.synchronize()
    assert np.array_equal(down(got), length)
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_generation_with_drafted_trees(dt, layout):
    """Sequences that fork, draft trees, accept paths of them, end and begin, for some steps;
    every token's key and value is known, and what the attention sees is checked against the
    sequence's own list of them."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    import tree_ref
    from helpers import from_device
    from test_qk_rope_gpu import check, f64, rnd
    rng = np.random.default_rng(7)
    layers, B, H, Hkv, d, page, width, pool = 2, 5, 4, 2, 64, 16, 14, 60
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    shape = (layers, pool) + ((page, Hkv) if layout == "bshd" else (Hkv, page)) + (d,)
    kc, vc = (torch.full(shape, float("nan"), dtype=tdt, device="cuda") for _ in range(2))
    raw = lambda *s: rnd(rng, s, dt)  # noqa: E731
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    own = [[[] for _ in range(B)] for _ in range(layers)]  # (key, value) of each sequence's tokens
    prompts = [40, 17, 0, 33, 16]
    parents = [-1] * B
    base = [0] * B
    for step in range(9):
        trees = [[-1 if i == 0 else int(rng.integers(-1, i)) for i in range(n)]
                 for n in (prompts if step == 0 else rng.integers(0, 12, B))]
        if step == 0:
            trees = [[i - 1 for i in range(n)] for n in prompts]
        n = [len(t) for t in trees]
        new = [base[p] + k if p >= 0 else k for p, k in zip(parents, n)]
        table, lens_now, refs, moves, counts = mha.mha_paged_reserve(
            table, lens, up(np.array(new, np.int32)), refs, page_size=page,
            parents=up(np.array(parents, np.int32)))
        mha.mha_paged_copy(kc, vc, moves)
        assert down(lens_now).tolist() == new  # the pool is large enough
        held = down(refs)
        live = np.zeros(pool, int)
        for row, ln in zip(down(table), new):
            np.add.at(live, row[:-(-ln // page)], 1)
        assert np.array_equal(held, live) and down(counts)[1] == (live == 0).sum()
        own = [[list(o[p]) if p >= 0 else [] for p in parents] for o in own]
        starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(starts[-1])
        words = max(1, -(-max(n) // 32))
        mask = np.concatenate([tree_ref.ancestors(t, words) for t in trees]) if T else \
            np.zeros((0, words), np.int32)
        batch = dict(q_starts=up(starts), kv_lengths=lens_now, block_table=table, layout=layout)
        for layer in range(layers):
            q, k, v = raw(T, H, d), raw(T, Hkv, d), raw(T, Hkv, d)
            as_t = lambda a: up(a.view(np.int16)).view(torch.bfloat16) if dt == "bf16" else up(a)  # noqa: E731
            pos = up(np.zeros(T, np.int32))  # (no rotation: what the cache holds stays known)
            qd = mha.mha_paged_append_at(as_t(q), as_t(k), as_t(v), kc[layer], vc[layer], pos, **batch)
            out = mha.mha_paged_tree_fwd(qd, kc[layer], vc[layer], up(mask), max_q=max(max(n), 1), **batch)
            for b in range(B):
                own[layer][b] += [(k[t], v[t]) for t in range(starts[b], starts[b + 1])]
            most = max(len(o) for o in own[layer])
            K, V = np.zeros((B, most, Hkv, d)), np.zeros((B, most, Hkv, d))
            for b, o in enumerate(own[layer]):
                for j, (x, y) in enumerate(o):
                    K[b, j], V[b, j] = f64(x, dt), f64(y, dt)
            one = 1 << max(4, int(most - 1).bit_length())
            pad = lambda a: np.concatenate([a, np.zeros((B, one - most, Hkv, d))], 1)  # noqa: E731
            want, tol = tree_ref.tree_attention(
                f64(q, dt), pad(K), pad(V), mask, starts, np.array(new), np.arange(B)[:, None],
                np.zeros(q.shape), page=one, layout="bshd", scale=d ** -0.5, dtype=dt)
            torch.cuda.synchronize()
            check(f64(from_device(out), dt), want, tol, "step %d" % step)
        # accept a path of each tree, or the whole prompt
        paths = []
        for t in trees:
            at, path = len(t) - 1 if step == 0 else int(rng.integers(-1, len(t))) if t else -1, []
            while at >= 0:
                path.insert(0, at)
                at = t[at]
            paths.append(path)
        before = [m - k for m, k in zip(new, n)]
        keep = np.zeros((B, max(1, max(len(p) for p in paths))), np.int32)
        for b, p in enumerate(paths):
            keep[b, :len(p)] = p
        lens = mha.mha_paged_compact(kc, vc, up(keep), up(np.array([len(p) for p in paths], np.int32)),
                                     starts=up(np.array(before, np.int32)), kv_lengths=lens_now,
                                     block_table=table, layout=layout)
        own = [[o[b][:before[b]] + [o[b][before[b] + i] for i in paths[b]] for b in range(B)] for o in own]
        # give back what the rejected tokens took
        table, lens, refs, moves, _ = mha.mha_paged_reserve(table, lens_now, lens, refs, page_size=page)
        mha.mha_paged_copy(kc, vc, moves)
        base = down(lens).tolist()
        assert base == [len(o) for o in own[0]] == [len(o) for o in own[1]]
        parents = [0, 1, 2, 3, 4]
        if step % 3 == 1:
            parents = [int(x) for x in rng.integers(0, B, B)]
        if step % 4 == 3:
            parents[2] = -1
    assert mha.mha_debug_status() == mha.MHA_OK
