"""The paged cache: appending to it and attention over it against the plain
float64 forms, with the errors derived in paged_ref.py."""
import numpy as np
import pytest

import gen
import paged_ref as ref
from helpers import from_device, to_device
from test_qk_rope_gpu import check, f64, freqs, rnd

pytestmark = pytest.mark.gpu


def batch(rng, seqs, page, extra_pages=3, behind=0, before=0, max_pages=None):
    """seqs: (new tokens, cached length) each.  A pool with pages in no order; table
    entries that hold no position name no page."""
    need = [-(-ln // page) for _, ln in seqs]
    pool = sum(need) + extra_pages
    ids = rng.permutation(pool)
    mp = max(max(need), 1) + 1 if max_pages is None else max_pages
    table = np.full((len(seqs), mp), 2 ** 31 - 1, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        m = min(m, mp)
        table[b, :m] = ids[at:at + m]
        at += m
    starts = (before + np.concatenate([[0], np.cumsum([n for n, _ in seqs])])).astype(np.int32)
    T = int(starts[-1]) + behind
    return dict(pool=pool, table=table, starts=starts, T=T,
                lens=np.array([ln for _, ln in seqs], dtype=np.int32))


def cache_of(rng, b, Hkv, page, d, dt, layout, amp=1.0):
    """Caches whose cells without a position hold NaN."""
    shape = (b["pool"], page, Hkv, d) if layout == "bshd" else (b["pool"], Hkv, page, d)
    used = np.zeros((b["pool"], page), dtype=bool)
    for row, ln in zip(b["table"], b["lens"]):
        for j in range(min(int(ln), len(row) * page)):
            if 0 <= row[j // page] < b["pool"]:
                used[row[j // page], j % page] = True
    hole = ~used[:, :, None, None] if layout == "bshd" else ~used[:, None, :, None]
    res = []
    for _ in range(2):
        x = rnd(rng, shape, dt, amp)
        bad = np.uint16(0x7FC0) if dt == "bf16" else np.float32(np.nan)
        res.append(np.where(hole, bad, x).astype(x.dtype))
    return res


def dev(a, dt=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if dt is None else to_device(a, dt)


def run_paged(q, kc, vc, b, *, dt, layout, causal=True, scale=None, max_q=None, fill=3.0, **kw):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    n = np.diff(b["starts"])
    qd = dev(q, dt)
    out = torch.full_like(qd, fill)
    d = q.shape[-1]
    mha.mha_paged_fwd(qd, dev(kc, dt), dev(vc, dt), out, q_starts=dev(b["starts"]),
                      kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
                      max_q=max(1, int(n.max())) if max_q is None else max_q, layout=layout,
                      mask_kind=8 if causal else 0, scale=d ** -0.5 if scale is None else scale,
                      **kw)
    torch.cuda.synchronize()
    assert mha.mha_debug_status() == mha.MHA_OK
    return from_device(out)


def check_paged(seqs, H, Hkv, d, dt, page, layout, causal=True, seed=0, scale=None, max_q=None,
                behind=0, before=0, amp=1.0, change=None, max_pages=None):
    rng = np.random.default_rng(seed)
    b = batch(rng, seqs, page, behind=behind, before=before, max_pages=max_pages)
    kc, vc = cache_of(rng, b, Hkv, page, d, dt, layout, amp)
    q = rnd(rng, (b["T"], H, d), dt, amp)
    if change is not None:
        change(b)
    out = run_paged(q, kc, vc, b, dt=dt, layout=layout, causal=causal, scale=scale, max_q=max_q)
    want, tol = ref.paged_attention(
        f64(q, dt), np.nan_to_num(f64(kc, dt)), np.nan_to_num(f64(vc, dt)), b["starts"], b["lens"],
        b["table"], np.full(q.shape, 3.0), page=page, layout=layout, causal=causal,
        scale=d ** -0.5 if scale is None else scale, dtype=dt)
    got = f64(out, dt)
    check(got, want, tol, "paged")
    # rows without a key are +0.0 bit for bit
    zero = (want == 0).all(-1)
    assert np.all(out[zero] == 0)
    return q, kc, vc, b, out


EDGES = [(1, ln) for ln in (1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700)]
CASES = [
    # (seqs, H, Hkv, d, page, layout)
    ([(1, 1)], 1, 1, 64, 16, "bshd"),
    ([(1, 300)], 8, 8, 64, 16, "bhsd"),
    (EDGES, 4, 2, 64, 16, "bshd"),
    (EDGES, 8, 2, 128, 64, "bhsd"),
    (EDGES, 3, 3, 128, 128, "bshd"),
    ([(0, 50), (1, 5000), (0, 0), (1, 3)], 4, 1, 128, 32, "bhsd"),       # keys split over CTAs
    ([(1, 20000)], 2, 1, 64, 256, "bshd"),
    ([(2, 300), (5, 5), (3, 129), (5, 1000)], 6, 2, 64, 16, "bhsd"),     # drafted tokens
    ([(4, 400), (1, 90), (4, 4)], 4, 4, 128, 16, "bshd"),
    ([(16, 513), (7, 300)], 4, 4, 64, 64, "bshd"),
    ([(8, 300), (3, 129), (1, 700), (0, 40)], 8, 2, 64, 16, "bhsd"),     # up to 32 rows
    ([(7, 1000), (7, 7), (2, 5000)], 4, 1, 128, 64, "bshd"),
    ([(1, 333), (1, 129)], 32, 1, 128, 32, "bshd"),
    ([(3, 200), (1, 1)], 18, 2, 64, 128, "bhsd"),
    ([(17, 17), (40, 400), (1, 77), (130, 131)], 4, 2, 64, 16, "bshd"),  # chunks
    ([(200, 900), (0, 300), (1, 1000), (64, 64)], 8, 2, 128, 64, "bhsd"),
    ([(300, 300)], 3, 1, 128, 128, "bhsd"),
    ([(129, 700), (128, 2000)], 6, 1, 64, 32, "bshd"),
    ([(1, 200), (3, 500)], 20, 1, 64, 16, "bshd"),                       # more than 16 heads share
    ([(2, 300), (1, 150)], 128, 1, 128, 16, "bhsd"),
    ([(2, 200)], 136, 1, 64, 16, "bshd"),                                # more than 128
    ([(1, 40 + 13 * i) for i in range(70)], 8, 4, 64, 16, "bshd"),       # more units than CTAs
]


@pytest.mark.parametrize("c", CASES, ids=["%d_H%dKV%dd%d_p%d_%s" % ((i,) + c[1:])
                                          for i, c in enumerate(CASES)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_attention(c, dt, causal):
    seqs, H, Hkv, d, page, layout = c
    check_paged(seqs, H, Hkv, d, dt, page, layout, causal, seed=len(seqs) + H)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("max_q", [1, 4, 5000])
def test_the_expected_tokens_do_not_matter(dt, max_q):
    check_paged([(40, 300), (1, 10), (3, 3), (0, 9), (7, 1000)], 4, 2, 64, dt, 16, "bshd",
                seed=2, max_q=max_q)
    check_paged([(1, 300), (1, 10)], 8, 2, 128, dt, 32, "bhsd", seed=3, max_q=max_q)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 30])
def test_rows_of_no_sequence_stay(dt, n):
    q, kc, vc, b, out = check_paged([(n, 100), (n, 31)], 4, 2, 64, dt, 16, "bhsd", seed=4,
                                    behind=9, before=5)
    keep = from_device(to_device(np.full((1,), 3.0, np.float32), "f32").to(
        to_device(q[:1], dt).dtype))
    assert np.all(out[:5] == keep) and np.all(out[-9:] == keep)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_tokens_before_the_first_position_are_zero(dt, n):
    for causal in (True, False):
        check_paged([(n, n // 2), (n, 0), (n, 200)], 4, 2, 64, dt, 16, "bshd", causal, seed=5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 6, 50])
@pytest.mark.parametrize("causal", [True, False])
def test_pages_that_are_not_there(dt, n, causal):
    def change(b):
        t = b["table"]
        t[0, 1], t[0, 4] = -1, b["pool"]             # holes in a sequence
        t[1, :] = -7                                 # a sequence without any page
        t[2, 0] = 2 ** 31 - 1
        b["lens"][3] = 5000                          # longer than its table: positions cut off
    check_paged([(n, 400), (n, 300), (n, 129), (n, 704)], 4, 2, 64, dt, 32, "bshd", causal, seed=6,
                change=change)
    check_paged([(n, 400), (n, 300), (n, 129), (n, 700)], 4, 2, 128, dt, 128, "bhsd", causal,
                seed=7, change=lambda b: b["table"].__setitem__((0, 1), -1))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_pages_shared_by_sequences(dt, n):
    def share(b):
        b["table"][1, :8] = b["table"][0, :8]    # one prefix
        b["table"][2, :4] = b["table"][2, 0]     # one page again and again
        b["table"][3] = b["table"][0]            # a whole table
    check_paged([(n, 500), (n, 300), (n, 400), (n, 450)], 4, 2, 64, dt, 16, "bshd", change=share,
                seed=21)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_offsets_and_lengths_out_of_range(dt):
    def change(b):
        b["starts"][0], b["starts"][-1] = -4, b["T"] + 1000
        b["lens"][1] = -5
    check_paged([(3, 60), (2, 40), (2, 70)], 4, 2, 64, dt, 16, "bshd", seed=8, change=change)

    def no_table(b):
        b["table"] = np.zeros((3, 0), dtype=np.int32)
    check_paged([(3, 60), (1, 40), (2, 70)], 4, 2, 64, dt, 16, "bshd", seed=8, change=no_table)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 12, 90])
def test_output_at_any_16_bytes(dt, n):
    # the rows' stores may be wider than that: the same numbers whatever the address
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(3)
    H, d, page = 4, 64, 32
    b = batch(rng, [(n, 300), (0, 40), (2 * n, 5 * n + 7)], page, behind=2)
    kc, vc = (dev(x, dt) for x in cache_of(rng, b, 2, page, d, dt, "bshd"))
    q = dev(rnd(rng, (b["T"], H, d), dt), dt)
    outs = []
    for offset in (0, 16 // q.element_size(), 32 // q.element_size()):
        buf = torch.full((q.numel() + 64,), 3.0, dtype=q.dtype, device="cuda")
        out = buf[offset:offset + q.numel()].view(q.shape)
        mha.mha_paged_fwd(q, kc, vc, out, q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                          block_table=dev(b["table"]), max_q=2 * n, layout="bshd", mask_kind=8,
                          scale=0.1)
        torch.cuda.synchronize()
        assert (buf[:offset] == 3).all() and (buf[offset + q.numel():] == 3).all()
        assert (out[-2:] == 3).all()
        outs.append(out.clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("n", [1, 33])
def test_scales(dt, scale, n):
    check_paged([(n, 500), (n, 129)], 4, 2, 64, dt, 16, "bshd", seed=9, scale=scale, amp=0.7)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 12, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_climbing_scores(dt, n, d):
    # the running maximum moves tile after tile; then falls from the first key on
    import numpy as np_
    rng = np_.random.default_rng(10)
    page, H, Hkv = 32, 4, 2
    b = batch(rng, [(n, 1500), (n, 700)], page)
    q = np_.abs(rng.normal(size=(b["T"], H, d))) * 0.5 + 0.5
    for sign in (1.0, -1.0):
        kc = np_.zeros((b["pool"], page, Hkv, d))
        for row, ln in zip(b["table"], b["lens"]):
            for j in range(ln):
                at = j if sign > 0 else ln - j
                kc[row[j // page], j % page] = at / 64.0 * (64.0 / d) * \
                    (0.5 + 0.1 * rng.normal(size=(Hkv, d)))
        vc = rng.normal(size=kc.shape)
        enc = gen.f64_to_bf16_bits if dt == "bf16" else (lambda x: x.astype(np_.float32))
        qs, ks, vs = enc(q), enc(kc), enc(vc)
        out = run_paged(qs, ks, vs, b, dt=dt, layout="bshd")
        want, tol = ref.paged_attention(f64(qs, dt), f64(ks, dt), f64(vs, dt), b["starts"],
                                        b["lens"], b["table"], np_.full(q.shape, 3.0), page=page,
                                        layout="bshd", causal=True, scale=d ** -0.5, dtype=dt)
        check(f64(out, dt), want, tol, "climbing %g" % sign)


def test_cache_beyond_32_bit_offsets():
    # 3.2e9 elements per cache; the sequence lives in its last pages
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page, Hkv, d, pages = 64, 8, 128, 49000
    assert pages * page * Hkv * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    for layout in ("bshd", "bhsd"):
        shape = (pages, page, Hkv, d) if layout == "bshd" else (pages, Hkv, page, d)
        kc, vc = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ids = [pages - 1, pages - 3, 2, pages - 2]
        small = [torch.randn(4, *shape[1:], generator=g, device="cuda").bfloat16()
                 for _ in range(2)]
        for c, s in ((kc, small[0]), (vc, small[1])):
            for i, p in enumerate(ids):
                c[p] = s[i]
        for n in (1, 40):
            q = torch.randn(n, 32, d, generator=g, device="cuda").bfloat16()
            kw = dict(q_starts=dev(np.array([0, n], np.int32)),
                      kv_lengths=dev(np.array([250], np.int32)), max_q=n, layout=layout)
            a = mha.mha_paged_fwd(q, kc, vc, block_table=dev(np.array([ids], np.int32)), **kw)
            b = mha.mha_paged_fwd(q, *small, block_table=dev(np.array([[0, 1, 2, 3]], np.int32)),
                                  **kw)
            assert torch.equal(a, b)
            k, v = (torch.randn(n, Hkv, d, generator=g, device="cuda").bfloat16()
                    for _ in range(2))
            ap = dict(q_starts=kw["q_starts"], kv_lengths=kw["kv_lengths"], layout=layout)
            mha.mha_paged_append(None, k, v, kc, vc,
                                 block_table=dev(np.array([ids], np.int32)), **ap)
            mha.mha_paged_append(None, k, v, *small,
                                 block_table=dev(np.array([[0, 1, 2, 3]], np.int32)), **ap)
            for c, s in ((kc, small[0]), (vc, small[1])):
                for i, p in enumerate(ids):
                    assert torch.equal(c[p], s[i])
        del kc, vc
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 60])
def test_streams_graphs_and_repeats(dt, n):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(12)
    H, Hkv, d, page = 8, 2, 128, 64
    b = batch(rng, [(n, 3000), (n, 100), (n, 800)], page)
    kc, vc = (dev(t, dt) for t in cache_of(rng, b, Hkv, page, d, dt, "bshd"))
    q = dev(rnd(rng, (b["T"], H, d), dt), dt)
    kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
              max_q=n, layout="bshd")
    want = mha.mha_paged_fwd(q, kc, vc, **kw)
    size = mha.mha_paged_workspace_size(3, b["T"], H, Hkv, d, n, q.dtype)
    torch.cuda.synchronize()
    # the same bits again, whatever the workspace held
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(mha.mha_paged_fwd(q, kc, vc, workspace=ws, **kw), want)
    # two streams at once, a workspace each
    sides = [torch.cuda.Stream() for _ in range(2)]
    wss = [torch.empty_like(ws) for _ in sides]
    outs = [torch.zeros_like(q) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, w, o in zip(sides, wss, outs):
            mha.mha_paged_fwd(q, kc, vc, o, workspace=w, stream=st, **kw)
    for st in sides:  # and with tensors of its own
        outs.append(mha.mha_paged_fwd(q, kc, vc, stream=st, **kw))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    # two captured graphs that share a workspace, replayed one after the other with other lengths
    graphs, gouts = [], []
    lens = dev(b["lens"])
    for _ in range(2):
        o = torch.zeros_like(q)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            mha.mha_paged_fwd(q, kc, vc, o, workspace=ws, **{**kw, "kv_lengths": lens})
        graphs.append(gr)
        gouts.append(o)
    for ln in (b["lens"], np.maximum(b["lens"] // 2, n).astype(np.int32), b["lens"]):
        lens.copy_(torch.from_numpy(ln))
        ref_out = mha.mha_paged_fwd(q, kc, vc, **{**kw, "kv_lengths": lens})
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o in gouts:
            assert torch.equal(o, ref_out)
    assert mha.mha_debug_status() == mha.MHA_OK


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,rotary,inter,norm", [(64, 64, False, True), (128, 64, True, True),
                                                 (128, 128, False, False), (64, 0, False, False)])
def test_append(layout, dt, d, rotary, inter, norm):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    for seqs, H, Hkv, page in (([(1, 1), (1, 33), (0, 9), (1, 16)], 4, 2, 16),
                               ([(5, 5), (40, 100), (3, 64)], 6, 6, 32),
                               ([(700, 2000), (900, 900), (1100, 1100)], 3, 1, 64)):
        rng = np.random.default_rng(H)
        b = batch(rng, seqs, page, behind=7, before=2)
        b["table"][0, 0] = -1 if seqs[0][1] > page else b["table"][0, 0]
        shape = (b["pool"], page, Hkv, d) if layout == "bshd" else (b["pool"], Hkv, page, d)
        kc, vc = rnd(rng, shape, dt), rnd(rng, shape, dt)
        T = b["T"]
        q, k, v = rnd(rng, (T, H, d), dt), rnd(rng, (T, Hkv, d), dt), rnd(rng, (T, Hkv, d), dt)
        qw, kw_ = (rnd(rng, (d,), dt, 0.3, 1.0) for _ in range(2)) if norm else (None, None)
        fr = freqs(rotary)
        up = lambda a: None if a is None else dev(a, dt)  # noqa: E731
        kd, vd, qd = up(kc), up(vc), up(q)
        qo = torch.full_like(qd, 3.0)
        common = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                      block_table=dev(b["table"]), q_weight=up(qw), k_weight=up(kw_),
                      inv_freq=dev(fr) if rotary else None, layout=layout, interleaved=inter,
                      eps=1e-5)
        mha.mha_paged_append(qd, up(k), up(v), kd, vd, qo, **common)
        # the plain form
        seq = np.concatenate([np.full(n, i) for i, (n, _) in enumerate(seqs)]).astype(int)
        pos = np.concatenate([np.arange(ln - n, ln) for n, ln in seqs]).astype(int)
        row = 2 + np.arange(len(seq))
        args = (pos[:, None], fr, inter, 1e-5)
        want, tol = np.full((T, H, d), 3.0), np.zeros((T, H, d))
        a = (f64(q, dt)[row], f64(qw, dt))
        want[row], tol[row] = ref.norm_rope(*a, *args), ref.norm_rope_tol(*a, *args, dt)
        check(f64(from_device(qo), dt), want, tol, "q")
        wk, wv, tk = f64(kc, dt), f64(vc, dt), np.zeros(shape)
        a = (f64(k, dt)[row], f64(kw_, dt))
        nk, nt, nv = ref.norm_rope(*a, *args), ref.norm_rope_tol(*a, *args, dt), f64(v, dt)[row]
        page_id = b["table"][seq, np.maximum(pos, 0) // page]
        ok = (pos >= 0) & (page_id >= 0) & (page_id < b["pool"])
        i, o = page_id[ok], pos[ok] % page
        for c, new in ((wk, nk), (wv, nv), (tk, nt)):
            if layout == "bshd":
                c[i, o] = new[ok]
            else:
                c[i, :, o] = new[ok]
        check(f64(from_device(kd), dt), wk, tk, "k cache")
        np.testing.assert_array_equal(f64(from_device(vd), dt), wv)
        # keys and values alone; queries in place
        k2, v2 = up(kc), up(vc)
        mha.mha_paged_append(None, up(k), up(v), k2, v2, **{**common, "q_weight": None})
        assert torch.equal(k2, kd) and torch.equal(v2, vd)
        mha.mha_paged_append(qd, up(k), up(v), k2, v2, qd, **common)
        assert torch.equal(qd[row], qo[row]) and torch.equal(k2, kd)
        np.testing.assert_array_equal(from_device(qd)[:2], q[:2])


def test_append_and_attend_agree_on_positions_outside_the_rows():
    # offsets past the buffer are clamped alike by both
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    T, H, d, page = 6, 2, 64, 16
    k = torch.randn(T, H, d, device="cuda").bfloat16()
    kc, vc = (torch.zeros(4, page, H, d, device="cuda").bfloat16() for _ in range(2))
    b = dict(q_starts=dev(np.array([-3, 50], np.int32)), kv_lengths=dev(np.array([20], np.int32)),
             block_table=dev(np.array([[2, 0]], np.int32)), layout="bshd")
    mha.mha_paged_append(None, k, k, kc, vc, **b)
    assert torch.equal(kc[2, 14:], k[:2]) and torch.equal(kc[0, :4], k[2:])
    assert kc.float().abs().sum() == k.float().abs().sum()


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 700, 1500])
def test_every_row_finds_its_sequence(B):
    # ragged and empty sequences, rows of none: each key tells where it should lie
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(B)
    n = rng.integers(0, 4, B) * rng.integers(0, 2, B)
    n[rng.integers(0, B)] += 3
    starts = (2 + np.concatenate([[0], np.cumsum(n)])).astype(np.int32)
    T = int(starts[-1]) + 3
    lens = (n + rng.integers(0, 40, B)).astype(np.int32)
    table = rng.permutation(B * 4).reshape(B, 4).astype(np.int32)
    k = torch.arange(1, T + 1, device="cuda", dtype=torch.float32)[:, None, None].expand(T, 1, 64)
    k = k.contiguous()
    kc, vc = (torch.zeros(B * 4, 16, 1, 64, device="cuda") for _ in range(2))
    mha.mha_paged_append(None, k, k, kc, vc, q_starts=dev(starts), kv_lengths=dev(lens),
                         block_table=dev(table), layout="bshd")
    want = np.zeros((B * 4, 16))
    for b in range(B):
        for i in range(n[b]):
            p = lens[b] - n[b] + i
            want[table[b, p // 16], p % 16] = 1 + starts[b] + i
    for c in (kc, vc):
        c = c.cpu().numpy()
        assert np.all(c == c[..., :1]) and np.array_equal(c[:, :, 0, 0], want)


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,Hkv,d,layout", [(8, 8, 64, "bshd"), (8, 2, 128, "bhsd")])
def test_generation_in_chunks_equals_the_sublayer(H, Hkv, d, layout):
    """Projections, append, attention over the cache, output projection, chunk by
    chunk and token by token, against the causal sublayer over whole sequences."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    g = torch.Generator(device="cuda").manual_seed(1)
    dm, page, lens = 512, 16, [200, 77]
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = [mk(ln, dm).bfloat16() for ln in lens]
    w = [(mk(dm, n) / dm ** 0.5).bfloat16() for n in (H * d, Hkv * d, Hkv * d)]
    wo = (mk(H * d, dm) / (H * d) ** 0.5).bfloat16()
    want = [mha.mha_sublayer_fwd(t[None], *w, wo, H=H, H_kv=Hkv, mask_kind=mha.MHA_MASK_CAUSAL)[0]
            for t in x]
    shape = (40, page, Hkv, d) if layout == "bshd" else (40, Hkv, page, d)
    kc, vc = (torch.full(shape, float("nan"), device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(40, generator=g, device="cuda").view(2, 20).int()
    done, got = [0, 0], [[], []]
    for step in ([100, 30], [1, 1], [1, 1], [0, 40], [60, 1], [38, 4]):
        rows = torch.cat([t[a:a + n] for t, a, n in zip(x, done, step)])
        done = [a + n for a, n in zip(done, step)]
        q, k, v = (mha.mha_linear_fwd(rows, t).view(len(rows), -1, d) for t in w)
        b = dict(q_starts=torch.tensor([0, step[0], sum(step)], dtype=torch.int32).cuda(),
                 kv_lengths=torch.tensor(done, dtype=torch.int32).cuda(), block_table=table,
                 layout=layout)
        q = mha.mha_paged_append(q, k, v, kc, vc, **b)
        o = mha.mha_paged_fwd(q, kc, vc, max_q=max(step), **b)
        y = mha.mha_linear_fwd(o.view(len(rows), H * d), wo)
        got[0].append(y[:step[0]])
        got[1].append(y[step[0]:])
    assert done == lens and mha.mha_debug_status() == mha.MHA_OK
    for a, b in zip(got, want):
        a = torch.cat(a).double()
        b = b.double()
        # the same projections; attention twice within half a bf16 step of the exact
        # weights and results, summed over H d values with weights of 1 / sqrt(H d)
        # each: 4 sigma of 3 half steps of values of about 1
        assert (a - b).abs().max() < 4 * 3 * 2.0 ** -8 * 1.0 + 2.0 ** -8 * b.abs().max()


def test_rotated_scores_depend_on_distance_alone():
    """Norm and rotation on both sides: attention over a cache is the same when
    every position moves by the same amount."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    g = torch.Generator(device="cuda").manual_seed(2)
    H, Hkv, d, L = 4, 2, 64, 90
    q, k, v = (torch.randn(1, L, h, d, generator=g, device="cuda") for h in (H, Hkv, Hkv))
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    fr = mha.rope_inv_freq(d)
    outs = []
    for start in (0, 1000, 123456):
        pos = (start + torch.arange(L, device="cuda", dtype=torch.int32))[None]
        a, b = mha.mha_qk_norm_rope_fwd(q, k, q_weight=w, k_weight=w, positions=pos, inv_freq=fr,
                                        layout="bshd")
        outs.append(mha.mha_fwd_ex(a, b, v, layout="bshd", mask_kind=mha.MHA_MASK_CAUSAL))
    # scores of normed rows are below 64 * 2.25 / 8 = 18; each side's rotation is exact
    # to 2^-22, so a score to 36 * 2^-22 and a weight to twice that, 2^-15.8
    for o in outs[1:]:
        assert (o - outs[0]).abs().max() < 2.0 ** -15 * v.abs().max()
    # and equal to the same through the paged cache
    kc, vc = (torch.zeros(8, 16, Hkv, d, device="cuda") for _ in range(2))
    batch_ = dict(q_starts=dev(np.array([0, L], np.int32)), kv_lengths=dev(np.array([L], np.int32)),
                  block_table=dev(np.array([[3, 1, 7, 0, 5, 6]], np.int32)), layout="bshd")
    qo = mha.mha_paged_append(q[0], k[0], v[0], kc, vc, q_weight=w, k_weight=w, inv_freq=fr,
                              **batch_)
    o = mha.mha_paged_fwd(qo, kc, vc, max_q=L, **batch_)
    assert (o - outs[0][0]).abs().max() < 2.0 ** -15 * v.abs().max()
