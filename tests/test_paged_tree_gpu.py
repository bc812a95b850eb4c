"""Trees of drafted tokens: their way into the paged cache at given positions, and their
attention over it, against the plain float64 forms (errors derived in tree_ref.py and
paged_ref.py)."""
import numpy as np
import pytest

import paged_ref as ref
import tree_ref
from helpers import from_device, to_device
from test_paged_gpu import batch, cache_of, dev
from test_qk_rope_gpu import check, f64, freqs, rnd

pytestmark = pytest.mark.gpu


def masks(rng, b, how, words=None):
    """Mask rows of a batch: "tree" (a random tree in each sequence), "chain", "any" (random
    bits, some rows without any, bits behind the new tokens too)."""
    n = np.diff(b["starts"])
    words = max(1, -(-int(n.max(initial=1)) // 32)) if words is None else words
    m = rng.integers(-2 ** 31, 2 ** 31, (b["T"], words)).astype(np.int32)
    if how == "any":
        m[rng.random(b["T"]) < 0.2] = 0
        return m
    for lo, k in zip(b["starts"], n):
        parents = [-1 if i == 0 else (i - 1 if how == "chain" else int(rng.integers(-1, i)))
                   for i in range(k)]
        m[lo:lo + k] = tree_ref.ancestors(parents, max(words, -(-int(k) // 32)))[:, :words]
    return m


def run_tree(q, kc, vc, mask, b, *, dt, layout, scale, max_q, fill=3.0, **kw):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    qd = dev(q, dt)
    out = torch.full_like(qd, fill)
    mha.mha_paged_tree_fwd(qd, dev(kc, dt), dev(vc, dt), dev(mask), out, q_starts=dev(b["starts"]),
                           kv_lengths=dev(b["lens"]), block_table=dev(b["table"]), max_q=max_q,
                           layout=layout, scale=scale, **kw)
    torch.cuda.synchronize()
    assert mha.mha_debug_status() == mha.MHA_OK
    return from_device(out)


def check_tree(seqs, H, Hkv, d, dt, page, layout, how="tree", seed=0, scale=None, max_q=None,
               behind=0, before=0, change=None, words=None, spoil=None, mask_of=None,
               max_pages=None):
    rng = np.random.default_rng(seed)
    b = batch(rng, seqs, page, behind=behind, before=before, max_pages=max_pages)
    if change is not None:  # (before the caches, whose cells without a position hold NaN)
        change(b)
    kc, vc = cache_of(rng, b, Hkv, page, d, dt, layout)
    q = rnd(rng, (b["T"], H, d), dt)
    mask = masks(rng, b, how, words)
    if mask_of is not None:
        mask = mask_of(mask)
    scale = d ** -0.5 if scale is None else scale
    max_q = max(1, int(np.diff(b["starts"]).max())) if max_q is None else max_q
    want, tol = tree_ref.tree_attention(
        f64(q, dt), np.nan_to_num(f64(kc, dt)), np.nan_to_num(f64(vc, dt)), mask, b["starts"],
        b["lens"], b["table"], np.full(q.shape, 3.0), page=page, layout=layout, scale=scale,
        dtype=dt)
    if spoil is not None:
        kc = spoil(b, kc, mask)
    out = run_tree(q, kc, vc, mask, b, dt=dt, layout=layout, scale=scale, max_q=max_q)
    check(f64(out, dt), want, tol, "tree")
    zero = (want == 0).all(-1)
    assert np.all(out[zero] == 0)  # rows that see nothing are +0.0 bit for bit
    return out


CASES = [
    # (seqs, H, Hkv, d, page, layout)
    ([(1, 1)], 1, 1, 64, 16, "bshd"),
    ([(16, 300)], 8, 8, 64, 16, "bshd"),
    ([(n, n + k) for n, k in ((1, 0), (2, 126), (3, 125), (4, 127), (5, 128), (6, 60), (7, 500))],
     2, 2, 64, 16, "bhsd"),
    ([(4, 4 + k) for k in (0, 60, 124, 125, 126, 127, 128, 129, 252)], 4, 2, 128, 64, "bshd"),
    ([(2, 2), (1, 700), (0, 40), (2, 5000)], 8, 1, 64, 256, "bhsd"),
    ([(31, 31 + 97), (32, 32 + 96), (33, 33 + 95), (17, 400)], 4, 2, 64, 16, "bshd"),
    ([(64, 64), (63, 64 + 128), (9, 1000), (25, 300)], 8, 2, 128, 64, "bhsd"),
    ([(64, 6000), (50, 70)], 32, 8, 128, 64, "bshd"),        # keys split over CTAs
    ([(200, 500), (256, 256), (129, 1000), (0, 3)], 4, 1, 64, 32, "bshd"),
    ([(130, 900), (1, 1)], 3, 3, 128, 128, "bhsd"),
    ([(13, 90 + 61 * i) for i in range(8)], 8, 2, 64, 32, "bshd"),
    ([(5, 300), (30, 77)], 136, 1, 64, 16, "bshd"),          # more heads to a group than rows
    ([(9 + i % 17, 40 + 13 * i) for i in range(60)], 8, 4, 64, 16, "bhsd"),
]


@pytest.mark.parametrize("c", CASES, ids=["%d_H%dKV%dd%d_p%d_%s" % ((i,) + c[1:])
                                          for i, c in enumerate(CASES)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["tree", "any"])
@pytest.mark.parametrize("room", [None, 200000], ids=["small_tables", "large_tables"])
def test_tree_attention(c, dt, how, room):
    """Small tables have units of few rows, on the few-query kernel; with room for long
    sequences the units are the usual ones."""
    seqs, H, Hkv, d, page, layout = c
    check_tree(seqs, H, Hkv, d, dt, page, layout, how, seed=len(seqs) + H,
               max_pages=None if room is None else room // page)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 1), (18, 2), (12, 1), (40, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_larger_units_of_fp32(H, Hkv, d):
    """Trees of more rows than 16 to a key/value head, fp32: at d 128 units of 32 rows where
    that makes for fewer, with groups of heads that fill them and that do not; keys split over
    CTAs, too."""
    for seqs in ([(40, 700), (33, 33), (1, 129), (0, 50), (35, 128)], [(70, 3000), (64, 70)]):
        for how in ("tree", "any"):
            check_tree(seqs, H, Hkv, d, "f32", 32, "bshd", how, seed=H, max_pages=200000 // 32,
                       behind=3)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("words", [1, 2, 7])
def test_rows_of_fewer_or_more_words_than_tokens(dt, words):
    for d, layout in ((64, "bshd"), (128, "bhsd")):
        check_tree([(40, 300), (3, 3), (100, 228), (7, 1000)], 4, 2, d, dt, 16, layout, "any",
                   seed=words, words=words)
    check_tree([(3, 300), (4, 133)], 4, 2, 64, dt, 16, "bshd", "any", seed=words, words=words)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("max_q", [1, 4, 5000])
def test_the_expected_tokens_do_not_matter(dt, max_q):
    check_tree([(40, 300), (1, 10), (3, 3), (0, 9), (7, 1000)], 4, 2, 64, dt, 16, "bshd", seed=2,
               max_q=max_q)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 30])
def test_rows_of_no_sequence_stay(dt, n):
    out = check_tree([(n, 100), (n, 31)], 4, 2, 64, dt, 16, "bhsd", seed=4, behind=9, before=5)
    keep = from_device(to_device(np.full((1,), 3.0, np.float32), "f32").to(
        to_device(out[:1], dt).dtype))
    assert np.all(out[:5] == keep) and np.all(out[-9:] == keep)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 5, 40])
def test_places_that_are_not_there(dt, n):
    # new tokens before the first position, without pages, behind the table's end; a hole
    def change(b):
        b["lens"][0], b["lens"][1] = n // 2, 0
        b["table"][2, 0] = -1
        b["table"][3, :] = 2 ** 31 - 1
        b["lens"][4] = b["table"].shape[1] * 16 + n // 2
    check_tree([(n, n), (n, n), (n, 70), (n, 50), (n, 200)], 4, 2, 64, dt, 16, "bshd", "any", seed=5,
               change=change)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,d", [(3, 2, 64), (4, 4, 128), (40, 4, 64), (64, 8, 128)])
def test_what_a_key_that_nobody_sees_holds_does_not_matter(dt, n, H, d):
    """Keys of new tokens that no row of the sequence sees are NaN and infinite."""
    def spoil(b, kc, mask):
        kc = kc.copy()
        for s in range(len(b["lens"])):
            lo, hi, ln = b["starts"][s], b["starts"][s + 1], b["lens"][s]
            seen = 0
            for t in range(lo, hi):
                seen |= tree_ref.bits(mask[t])
            for m in range(hi - lo):
                if not seen >> m & 1:
                    p = ln - (hi - lo) + m
                    bad = np.nan if m % 2 else np.inf
                    kc[b["table"][s, p // 16], p % 16] = \
                        np.float32(bad) if dt == "f32" else np.uint16(0x7FC0 if m % 2 else 0x7F80)
        return kc

    hide = np.random.default_rng(n).integers(0, 2, 64)

    def some(mask):
        off = [sum(1 << i for i in range(32) if hide[(32 * w + i) % 64])
               for w in range(mask.shape[1])]
        return mask & ~np.array(off, dtype=np.uint32).view(np.int32)
    check_tree([(n, n + 200), (n, n), (n, n + 113)], H, 2, d, dt, 16, "bshd", "any", spoil=spoil,
               mask_of=some, seed=3)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 30, 100])
def test_a_chain_is_causal(dt, n):
    """A tree without branches gives what mha_paged_fwd's causal mask does."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(n)
    H, Hkv, d, page = 8, 2, 64, 16
    b = batch(rng, [(n, n), (n, 500 + n), (n, 127), (n, 1000)] if n < 100 else
              [(n, 300), (n, 1000)], page, behind=2)
    caches = cache_of(rng, b, Hkv, page, d, dt, "bshd")
    kc, vc = (dev(t, dt) for t in caches)
    qh = rnd(rng, (b["T"], H, d), dt)
    q, mask = dev(qh, dt), masks(rng, b, "chain")
    kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
              max_q=n, layout="bshd")
    a = mha.mha_paged_tree_fwd(q, kc, vc, dev(mask), **kw)
    want = mha.mha_paged_fwd(q, kc, vc, **kw)
    torch.cuda.synchronize()
    # each is as near to the formula as its rounding allows (units are cut elsewhere: here a
    # unit's keys count whole)
    formula, tol = tree_ref.tree_attention(
        f64(qh, dt), *(np.nan_to_num(f64(t, dt)) for t in caches), mask, b["starts"], b["lens"],
        b["table"], np.zeros(qh.shape), page=page, layout="bshd", scale=d ** -0.5, dtype=dt)
    check(f64(from_device(a), dt), formula, tol, "chain")
    assert (np.abs(f64(from_device(a), dt) - f64(from_device(want), dt)) <= 2 * tol).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 40])
def test_streams_and_captured_trees(dt, n):
    """On streams of their own, and captured and replayed with other trees and lengths."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(12)
    H, Hkv, d, page = 4, 2, 128, 64
    b = batch(rng, [(n, 2000), (n, 100), (n, 800)], page)
    kc, vc = (dev(t, dt) for t in cache_of(rng, b, Hkv, page, d, dt, "bhsd"))
    q = dev(rnd(rng, (b["T"], H, d), dt), dt)
    ms = [dev(masks(rng, b, how)) for how in ("tree", "any", "chain")]
    lens = [dev(b["lens"] - 9 * i) for i in range(3)]
    kw = dict(q_starts=dev(b["starts"]), block_table=dev(b["table"]), max_q=n, layout="bhsd")
    want = [mha.mha_paged_tree_fwd(q, kc, vc, m, kv_lengths=ln, **kw) for m, ln in zip(ms, lens)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [mha.mha_paged_tree_fwd(q, kc, vc, m, kv_lengths=ln, stream=side, **kw)
           for m, ln in zip(ms, lens)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    ws = torch.empty(mha.mha_paged_workspace_size(3, b["T"], H, Hkv, d, n, q.dtype),
                     dtype=torch.uint8, device="cuda")
    m, ln, out = ms[0].clone(), lens[0].clone(), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mha.mha_paged_tree_fwd(q, kc, vc, m, out, kv_lengths=ln, workspace=ws, **kw)
    for i in (1, 2, 0):
        m.copy_(ms[i])
        ln.copy_(lens[i])
        graph.replay()
        assert torch.equal(out, want[i])
    assert mha.mha_debug_status() == mha.MHA_OK


def test_masks_beyond_32_bit_offsets():
    """A mask of more than 2^31 words; rows of the last tokens."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    words, T, n, d = 1 << 17, (1 << 14) + 300, 40, 64
    assert words * (T - n) > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    mask = torch.empty(T, words, dtype=torch.int32, device="cuda")
    small = torch.randint(-2 ** 31, 2 ** 31, (n, 2), generator=g, device="cuda").int()
    mask[T - n:, :2] = small
    mask[T - n:, 2:] = -1
    q = torch.randn(T, 2, d, generator=g, device="cuda")
    for dt, H in ((torch.bfloat16, 2), (torch.float32, 2), (torch.bfloat16, 1)):
        x = q[:, :H].to(dt).contiguous()
        kc, vc = (torch.randn(8, 16, 1, d, generator=g, device="cuda").to(dt) for _ in range(2))
        kw = dict(kv_lengths=dev(np.array([100], np.int32)), layout="bshd",
                  block_table=dev(np.arange(8, dtype=np.int32)[None]),
                  max_q=n if dt == torch.float32 or H == 2 else 8)
        a = mha.mha_paged_tree_fwd(x, kc, vc, mask, q_starts=dev(np.array([T - n, T], np.int32)), **kw)
        c = mha.mha_paged_tree_fwd(x[T - n:].contiguous(), kc, vc, small,
                                   q_starts=dev(np.array([0, n], np.int32)), **kw)
        assert torch.equal(a[T - n:], c)


# ---------------------------------------------------------------------------
# appending at given positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,rotary,inter,layout", [(64, 64, False, "bshd"), (128, 128, True, "bhsd"),
                                                   (128, 64, False, "bshd"), (64, 0, False, "bhsd")])
@pytest.mark.parametrize("norm", [True, False])
def test_append_at_positions(dt, d, rotary, inter, layout, norm):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(d + rotary)
    H, Hkv, page = 6, 2, 16
    b = batch(rng, [(7, 50), (1, 1), (0, 33), (20, 20), (5, 200)], page, behind=3, before=2)
    T = b["T"]
    q, k, v = (rnd(rng, (T, h, d), dt) for h in (H, Hkv, Hkv))
    w = [rnd(rng, (d,), dt, 0.3, 1.0) if norm else None for _ in range(2)]
    pos = rng.integers(-2 ** 31, 2 ** 31, T).astype(np.int32)
    pos[::3] = rng.integers(0, 300, len(pos[::3]))
    freq = freqs(rotary)
    shape = (b["pool"], page, Hkv, d) if layout == "bshd" else (b["pool"], Hkv, page, d)
    kc, vc = (torch.full(shape, 5.0, dtype=dev(k, dt).dtype, device="cuda") for _ in range(2))
    qo = torch.full_like(dev(q, dt), 3.0)
    up = lambda a: None if a is None else dev(a, dt)  # noqa: E731
    mha.mha_paged_append_at(dev(q, dt), dev(k, dt), dev(v, dt), kc, vc, dev(pos), qo,
                            q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                            block_table=dev(b["table"]), q_weight=up(w[0]), k_weight=up(w[1]),
                            inv_freq=dev(freq) if rotary else None, layout=layout,
                            interleaved=inter)
    torch.cuda.synchronize()
    lo, hi = b["starts"][0], b["starts"][-1]
    want, tol = np.full(q.shape, 3.0), np.zeros(q.shape)
    args = (pos[:, None], freq, inter, 1e-6)
    want[lo:hi] = ref.norm_rope(f64(q, dt), f64(w[0], dt), *args)[lo:hi]
    tol[lo:hi] = ref.norm_rope_tol(f64(q, dt), f64(w[0], dt), *args, dt)[lo:hi]
    check(f64(from_device(qo), dt), want, tol, "q")
    want, tol = np.full(shape, 5.0), np.zeros(shape)
    rows = ref.norm_rope(f64(k, dt), f64(w[1], dt), *args)
    rtol = ref.norm_rope_tol(f64(k, dt), f64(w[1], dt), *args, dt)
    wantv = np.full(shape, 5.0)
    for s, (row, ln) in enumerate(zip(b["table"], b["lens"])):
        n = b["starts"][s + 1] - b["starts"][s]
        for i in range(n):
            p, t = ln - n + i, b["starts"][s] + i
            at = (row[p // page], p % page) if layout == "bshd" else \
                (row[p // page], slice(None), p % page)
            want[at], tol[at], wantv[at] = rows[t], rtol[t], f64(v, dt)[t]
    check(f64(from_device(kc), dt), want, tol, "k cache")
    assert np.array_equal(f64(from_device(vc), dt), wantv)


def test_append_at_its_own_positions_is_append():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(1)
    b = batch(rng, [(7, 50), (20, 20), (5, 200)], 16)
    q, k, v = (dev(rnd(rng, (b["T"], h, 64), "bf16"), "bf16") for h in (4, 2, 2))
    pos = np.concatenate([np.arange(ln - n, ln) for n, ln in ((7, 50), (20, 20), (5, 200))])
    kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
              inv_freq=dev(freqs(64)), layout="bshd")
    caches = [[torch.zeros(b["pool"], 16, 2, 64, dtype=torch.bfloat16, device="cuda")
               for _ in range(2)] for _ in range(2)]
    a = mha.mha_paged_append(q, k, v, *caches[0], **kw)
    c = mha.mha_paged_append_at(q, k, v, *caches[1], dev(pos.astype(np.int32)), **kw)
    assert torch.equal(a, c)
    assert all(torch.equal(x, y) for x, y in zip(*caches))


@pytest.mark.parametrize("room", [None, 200000], ids=["small_tables", "large_tables"])
@pytest.mark.parametrize("n,H,Hkv,d", [(3, 2, 2, 64), (4, 8, 2, 128), (40, 4, 2, 128)])
def test_a_wait_that_runs_out(room, n, H, Hkv, d):
    """As test_paged_give_up_gpu.py: an issuer (of whichever kernel the call takes) waits for
    what nothing signals, the kernel returns, the status tells, and the next call is right."""
    import transformer_head_scaled_mha_gb300 as mha
    from test_paged_give_up_gpu import STALL_FEW, STALL_MANY, stalled
    rng = np.random.default_rng(n)
    room = None if room is None else room // 64
    for seqs in ([(n, 128 * t) for t in (1, 2, 3, 4, 5)] * 40, [(n, 20000)]):
        b = batch(rng, seqs, 64, max_pages=room)
        kc, vc = (dev(x, "bf16") for x in cache_of(rng, b, Hkv, 64, d, "bf16", "bshd"))
        q, mask = dev(rnd(rng, (b["T"], H, d), "bf16"), "bf16"), dev(masks(rng, b, "tree"))
        kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
                  max_q=n, layout="bshd")
        stalled(STALL_FEW | STALL_MANY, lambda: mha.mha_paged_tree_fwd(q, kc, vc, mask, **kw))
    check_tree([(n, 128), (n, 700)], H, Hkv, d, "bf16", 64, "bshd", seed=n, max_pages=room)
