"""Calls of the paged operators that the documentation allows: captured steps whose lengths
move on, a cache without pages, pages longer than a tile, thousands of sequences, and what
lies in rows of no sequence."""
import numpy as np
import pytest

import paged_ref as ref
from helpers import from_device
from test_paged_gpu import batch, cache_of, check_paged, dev
from test_qk_rope_gpu import check, f64, freqs, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,Hkv", [(1, 8, 2), (3, 4, 2), (20, 4, 2)])
def test_captured_generation_steps(dt, n, H, Hkv):
    """Append and attend in one graph, replayed as the sequences grow, against the same
    calls made one by one."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(n)
    B, d, page, steps = 3, 64, 16, 5
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    shape = (B * 40, page, Hkv, d)
    table = dev(rng.permutation(B * 40).reshape(B, 40).astype(np.int32))
    starts = dev((n * np.arange(B + 1)).astype(np.int32))
    lens = dev(np.array([0, 100, 300], np.int32))
    w = dev(rnd(rng, (d,), dt, 0.1, 1.0), dt)
    kw = dict(q_starts=starts, block_table=table, layout="bshd")
    rope = dict(q_weight=w, k_weight=w, inv_freq=mha.rope_inv_freq(d))
    qs, ks, vs = (dev(rnd(rng, (steps, B * n, h, d), dt), dt) for h in (H, Hkv, Hkv))
    ws = torch.empty(mha.mha_paged_workspace_size(B, B * n, H, Hkv, d, n, tdt),
                     dtype=torch.uint8, device="cuda")
    caches = [[torch.zeros(shape, dtype=tdt, device="cuda") for _ in range(2)] for _ in range(2)]
    q, k, v = (torch.zeros_like(t[0]) for t in (qs, ks, vs))
    qo, out = torch.zeros_like(q), torch.zeros_like(q)

    def step(c, lengths, q, k, v, qo, out):
        mha.mha_paged_append(q, k, v, *c, qo, kv_lengths=lengths, **rope, **kw)
        mha.mha_paged_fwd(qo, *c, out, max_q=n, kv_lengths=lengths, workspace=ws, **kw)
    step(caches[0], lens, q, k, v, qo, out)  # (warm; its rows are written again)
    for c in caches[0]:
        c.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(n)
        step(caches[0], lens, q, k, v, qo, out)
    lens.copy_(dev(np.array([0, 100, 300], np.int32)))
    now = lens.clone()
    for s in range(steps):
        for a, b in ((q, qs), (k, ks), (v, vs)):
            a.copy_(b[s])
        graph.replay()
        now = now + n
        o = torch.zeros_like(out)
        step(caches[1], now, qs[s], ks[s], vs[s], torch.zeros_like(qo), o)
        assert torch.equal(out, o)
    assert torch.equal(lens, now)
    for a, b in zip(*caches):
        assert torch.equal(a, b)
    assert mha.mha_debug_status() == mha.MHA_OK


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_a_cache_without_pages(dt, n, layout):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    H, Hkv, d, page = 4, 2, 64, 32
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    shape = (0, page, Hkv, d) if layout == "bshd" else (0, Hkv, page, d)
    kc, vc = (torch.zeros(shape, dtype=tdt, device="cuda") for _ in range(2))
    q, k = (torch.randn(2 * n, h, d, device="cuda").to(tdt) for h in (H, Hkv))
    kw = dict(q_starts=dev(np.array([0, n, 2 * n], np.int32)), layout=layout,
              kv_lengths=dev(np.array([300, 5000], np.int32)),
              block_table=dev(np.zeros((2, 20), np.int32)))
    qo = mha.mha_paged_append(q, k, k, kc, vc, **kw)
    assert torch.equal(qo, q)
    out = mha.mha_paged_fwd(q, kc, vc, torch.full_like(q, 3.0), max_q=n, **kw)
    assert (out == 0).all() and mha.mha_debug_status() == mha.MHA_OK


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("page", [512, 4096])
def test_pages_longer_than_a_tile(dt, layout, page):
    for n in (1, 5, 33):
        check_paged([(n, page + 77), (n, 130), (n, page), (n, 2 * page + 1)], 4, 2, 64, dt, page,
                    layout, seed=page + n)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (20, 1)])
def test_thousands_of_sequences(dt, H, Hkv):
    rng = np.random.default_rng(0)
    seqs = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 3, 5000), rng.integers(0, 60, 5000))]
    check_paged(seqs, H, Hkv, 64, dt, 16, "bshd", seed=8)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 50])
def test_rows_of_no_sequence_may_hold_anything(dt, n):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(1)
    H, Hkv, d, page = 4, 2, 128, 16
    b = batch(rng, [(n, 200), (n, 7 + n)], page, behind=30, before=30)
    kc, vc = (dev(c, dt) for c in cache_of(rng, b, Hkv, page, d, dt, "bhsd"))
    q = dev(rnd(rng, (b["T"], H, d), dt), dt)
    kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
              max_q=n, layout="bhsd")
    want = mha.mha_paged_fwd(q, kc, vc, **kw)
    k = dev(rnd(rng, (b["T"], Hkv, d), dt), dt)
    for bad in (float("nan"), float("inf")):
        q[:30] = q[30 + 2 * n:] = bad
        assert torch.equal(mha.mha_paged_fwd(q, kc, vc, **kw), want)
        k[:30] = k[30 + 2 * n:] = bad
        # ... and nothing of them goes into the cache
        a = [c.clone() for c in (kc, vc)]
        before = [torch.isnan(c).sum() for c in a]
        kw2 = {x: y for x, y in kw.items() if x != "max_q"}
        mha.mha_paged_append(None, k, k, *a, inv_freq=mha.rope_inv_freq(d), **kw2)
        for c, m in zip(a, before):
            assert torch.isnan(c).sum() == m and not torch.isinf(c).any()


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_appending_to_long_pages_and_sharing_the_rest(dt, layout):
    """Pages longer than a tile; sequences that share their first pages and append to
    their own."""
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(2)
    page, Hkv, d = 1024, 2, 64
    shape = (6, page, Hkv, d) if layout == "bshd" else (6, Hkv, page, d)
    kc, vc = rnd(rng, shape, dt), rnd(rng, shape, dt)
    table = np.array([[3, 1, -1], [3, 5, 2], [0, 4, 4]], np.int32)
    starts, lens = np.array([0, 40, 1065, 1067], np.int32), np.array([1300, 2500, 1500], np.int32)
    T = 1067
    k, v = rnd(rng, (T, Hkv, d), dt), rnd(rng, (T, Hkv, d), dt)
    fr = freqs(d)
    kd, vd = dev(kc, dt), dev(vc, dt)
    mha.mha_paged_append(None, dev(k, dt), dev(v, dt), kd, vd, q_starts=dev(starts),
                         kv_lengths=dev(lens), block_table=dev(table), inv_freq=dev(fr),
                         layout=layout)
    wk, wv, tk = f64(kc, dt), f64(vc, dt), np.zeros(shape)
    for s in range(3):
        lo, hi = starts[s], starts[s + 1]
        pos = np.arange(lens[s] - (hi - lo), lens[s])
        args = (f64(k, dt)[lo:hi], None, pos[:, None], fr, False, 1e-6)
        for c, new in ((wk, ref.norm_rope(*args)), (tk, ref.norm_rope_tol(*args, dt)),
                       (wv, f64(v, dt)[lo:hi])):
            if layout == "bshd":
                c[table[s][pos // page], pos % page] = new
            else:
                c[table[s][pos // page], :, pos % page] = new
    check(f64(from_device(kd), dt), wk, tk, "k")
    np.testing.assert_array_equal(f64(from_device(vd), dt), wv)
