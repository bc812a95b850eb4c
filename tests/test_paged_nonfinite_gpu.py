"""Infinities and NaN that a token sees go through paged attention as the formula
takes them: exactly the rows that see one carry it on, on every kernel, in units
that one CTA works on and in units that several share; rows with nothing to attend
to are +0.0 whatever their query holds."""
import numpy as np
import pytest

import gen
import paged_ref as ref
from helpers import from_device
from test_paged_gpu import batch, dev
from test_qk_rope_gpu import f64, rnd

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def defined(q, kc, vc, b, layout, scale, dt):
    """softmax(scale q k) v in 64 bits over the positions each token sees, and the
    error that paged_ref.paged_attention allows (finite elements)."""
    out, tol = np.zeros_like(q), np.zeros_like(q)
    T, H, d = q.shape
    Hkv = kc.shape[2 if layout == "bshd" else 1]
    page = kc.shape[1 if layout == "bshd" else 2]
    for s, ln in enumerate(b["lens"]):
        lo, hi = int(b["starts"][s]), int(b["starts"][s + 1])
        K, V = (ref.positions(c, b["table"][s], int(ln), page, b["pool"], layout)[0]
                for c in (kc, vc))
        for i, t in enumerate(range(lo, hi)):
            n = max(int(ln) - (hi - lo) + i + 1, 0)  # positions that it sees
            if n == 0:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                x = scale * (K[:n, g] @ q[t, h])
                w = np.exp(x - x.max())
                w = w / w.sum()
                out[t, h] = w @ V[:n, g]
                size = abs(scale) * (np.abs(K[:n, g]) @ np.abs(q[t, h]))
                score = size[np.isfinite(size)].max(initial=0.0)
                err = (d + 8) * ref.U * score + 2.0 ** -20 + 2 * n * ref.U
                weight = 2 * err + (ref.HALF["bf16"] if dt == "bf16" else 0.0)
                tol[t, h] = weight * (w @ np.abs(V[:n, g])) + ref.HALF[dt] * np.abs(out[t, h])
    return out, tol


def store(x, dt):
    """float64 -> what the device tensor holds."""
    x = np.asarray(x)
    if dt == "f32":
        return x.astype(np.float32)
    bits = gen.f64_to_bf16_bits(np.where(np.isfinite(x), x, 0.0))
    special = np.where(np.isnan(x), 0x7FC0, np.where(x > 0, 0x7F80, 0xFF80))
    return np.where(np.isfinite(x), bits, special).astype(np.uint16)


# (dt, query heads, key/value heads, new tokens, d): every form of each kernel
FORMS = [
    ("f32", 2, 2, 1, 64), ("f32", 4, 1, 1, 128), ("f32", 4, 2, 7, 64),
    ("bf16", 2, 2, 1, 64), ("bf16", 2, 2, 1, 128), ("bf16", 2, 1, 1, 64), ("bf16", 4, 1, 1, 64),
    ("bf16", 4, 1, 1, 128), ("bf16", 4, 2, 4, 64), ("bf16", 4, 2, 4, 128), ("bf16", 4, 1, 4, 64),
    ("bf16", 4, 1, 4, 128), ("bf16", 4, 2, 40, 64), ("bf16", 2, 2, 40, 128),
    ("bf16", 2, 1, 150, 128),
]


@pytest.mark.parametrize("cut", [False, True], ids=["whole", "cut"])
@pytest.mark.parametrize("dt,H,Hkv,n,d", FORMS)
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_what_a_row_sees_goes_on(dt, H, Hkv, n, d, cut):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page, layout, scale = 16, "bshd", d ** -0.5
    short = min(max(n, 100), 128) if n <= 128 else n
    ln = 2000 if cut else short
    rng = np.random.default_rng(n + H + d)
    # the last one: tokens before the first position, which see nothing
    b = batch(rng, [(n, ln)] * 9 + [(n, 0)], page)
    q = f64(rnd(rng, (b["T"], H, d), dt), dt)
    kc, vc = (f64(rnd(rng, (b["pool"], page, Hkv, d), dt), dt) for _ in range(2))

    def at(cache, s, pos, g):  # a position's row
        return cache[b["table"][s][pos // page], pos % page, g]
    end = [int(x) - 1 for x in b["starts"][1:]]  # last token of each sequence
    q[end[1], H - 1, 3] = NAN
    q[end[2], 0, 5] = INF
    at(kc, 3, 0, 0)[7] = NAN              # seen by every token
    at(kc, 4, ln - 1, Hkv - 1)[2] = NAN   # seen by the last token alone
    at(vc, 5, 0, 0)[9] = NAN              # one column of the output
    q[end[6], :, 0] = INF
    kc[b["table"][6][0], 0, :, 0] = 0.0   # 0 times infinity
    # every score of one row -infinity
    q[end[7], 0, 0] = INF
    for pos in range(ln):
        at(kc, 7, pos, 0)[0] = -1.0 - pos % 3
    # three quarters of the keys of a head score -infinity: no weight (the first tokens of
    # a chunk may see no other key)
    q[int(b["starts"][8]):end[8] + 1, :H // Hkv, 1] = 2.0
    for pos in range(ln * 3 // 4):
        at(kc, 8, pos, 0)[1] = -INF
    q[end[9], 0, 0] = NAN
    qs, ks, vs = (store(x, dt) for x in (q, kc, vc))
    want, tol = defined(f64(qs, dt), f64(ks, dt), f64(vs, dt), b, layout, scale, dt)
    size = mha.mha_paged_workspace_size(len(b["lens"]), b["T"], H, Hkv, d, n,
                                        torch.float32 if dt == "f32" else torch.bfloat16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    qd = dev(qs, dt)
    out = mha.mha_paged_fwd(qd, dev(ks, dt), dev(vs, dt), torch.full_like(qd, 3.0),
                            q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                            block_table=dev(b["table"]), max_q=n, layout=layout, scale=scale,
                            workspace=ws)
    torch.cuda.synchronize()
    # words that tell which parts of cut units a CTA holds
    assert bool((ws.view(torch.int32)[:192 * 8:8] != 0).any()) == cut
    got = f64(from_device(out), dt)
    for s in range(len(b["lens"])):
        r = slice(int(b["starts"][s]), int(b["starts"][s + 1]))
        np.testing.assert_array_equal(np.isnan(got[r]), np.isnan(want[r]), "NaN, sequence %d" % s)
        fin = np.isfinite(want[r])
        assert np.all(np.abs(got[r] - want[r])[fin] <= tol[r][fin]), "sequence %d" % s
    assert np.isnan(want).any() and np.isnan(want[end[7], 0]).all()
    assert np.isfinite(want[end[8]]).all()
    # nothing to attend to: +0.0, bit for bit
    raw = from_device(out)[b["starts"][9]:]
    assert np.all(np.ascontiguousarray(raw).view(np.uint16 if dt == "bf16" else np.uint32) == 0)


@pytest.mark.parametrize("dt,H,Hkv,n,d", FORMS)
def test_scores_past_the_range_of_fp32_are_nan(dt, H, Hkv, n, d):
    # 2^120 * 2^15: +infinity in 32 bits, and infinity less infinity
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page, ln = 16, max(n, 90)
    rng = np.random.default_rng(1)
    b = batch(rng, [(n, ln), (n, ln)], page)
    q = np.abs(f64(rnd(rng, (b["T"], H, d), dt), dt)) + 0.5
    kc, vc = (np.abs(f64(rnd(rng, (b["pool"], page, Hkv, d), dt), dt)) + 0.5 for _ in range(2))
    row = int(b["starts"][1]) - 1
    q[row, H - 1] *= 2.0 ** 120
    kc[b["table"][0][0], 0] *= 2.0 ** 15
    out = mha.mha_paged_fwd(dev(store(q, dt), dt), dev(store(kc, dt), dt), dev(store(vc, dt), dt),
                            q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                            block_table=dev(b["table"]), max_q=n, layout="bshd")
    bad = torch.isnan(out).all(-1).cpu().numpy()
    assert bad[row, H - 1] and bad.sum() == 1 and not torch.isnan(out[row + 1:]).any()


@pytest.mark.parametrize("cut", [False, True], ids=["whole", "cut"])
@pytest.mark.parametrize("dt,H,Hkv,n,d", FORMS)
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_infinite_values_are_infinite_outputs(dt, H, Hkv, n, d, cut):
    import transformer_head_scaled_mha_gb300 as mha
    page, ln, scale = 16, 2000 if cut else max(n, 100), d ** -0.5
    rng = np.random.default_rng(2)
    b = batch(rng, [(n, ln)] * 6, page)
    q = f64(rnd(rng, (b["T"], H, d), dt), dt)
    kc, vc = (f64(rnd(rng, (b["pool"], page, Hkv, d), dt), dt) for _ in range(2))
    for s, (pos, value) in enumerate(((0, INF), (0, -INF), (ln - n, INF), (ln - n, -INF))):
        vc[b["table"][s][pos // page], pos % page, s % Hkv, 5 + s] = value  # every token sees it
    vc[b["table"][4][0], 0, 0, d - 1] = INF
    vc[b["table"][4][0], min(1, ln - n), 0, d - 1] = -INF  # (a chunk from the start: one value)
    qs, ks, vs = (store(x, dt) for x in (q, kc, vc))
    want, tol = defined(f64(qs, dt), f64(ks, dt), f64(vs, dt), b, "bshd", scale, dt)
    out = mha.mha_paged_fwd(dev(qs, dt), dev(ks, dt), dev(vs, dt), q_starts=dev(b["starts"]),
                            kv_lengths=dev(b["lens"]), block_table=dev(b["table"]), max_q=n,
                            layout="bshd", scale=scale)
    got = f64(from_device(out), dt)
    fin = np.isfinite(want)
    assert np.isinf(want).any() and (n == ln or np.isnan(want).any())
    np.testing.assert_array_equal(np.where(fin, 0.0, got), np.where(fin, 0.0, want))
    assert np.all(np.abs(got - want)[fin] <= tol[fin])


@pytest.mark.parametrize("far", [25, 60, 120])
@pytest.mark.parametrize("dt,H,Hkv,n,d", FORMS)
def test_far_scores(dt, H, Hkv, n, d, far):
    # scores of one sign, 2^far and more: the largest one's value (the others are 2^far / 8
    # and more below it), whatever tile it is in
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page, ln = 16, max(n + 200, 500)
    rng = np.random.default_rng(3)
    b = batch(rng, [(n, ln)] * 3, page)
    sign = np.array([1.0, -1.0, 1.0])
    q, kc = np.zeros((b["T"], H, d)), np.zeros((b["pool"], page, Hkv, d))
    vc = f64(rnd(rng, (b["pool"], page, Hkv, d), dt), dt)
    best = []
    for s in range(3):
        q[b["starts"][s]:b["starts"][s + 1], :, 3] = sign[s]
        top = [ln - n, 3, 130][s]  # seen by every token
        best.append(top)
        for pos in range(ln):
            size = 1.0 if (pos == top) == (sign[s] < 0) else 2.0
            kc[b["table"][s][pos // page], pos % page, :, 3] = size * 2.0 ** far * d ** 0.5
    out = mha.mha_paged_fwd(dev(store(q, dt), dt), dev(store(kc, dt), dt), dev(store(vc, dt), dt),
                            q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                            block_table=dev(b["table"]), max_q=n, layout="bshd", scale=d ** -0.5)
    got = f64(from_device(out), dt)
    for s, top in enumerate(best):
        v = vc[b["table"][s][top // page], top % page]  # [Hkv, d], stored exactly
        want = np.repeat(v, H // Hkv, axis=0)
        assert np.array_equal(got[b["starts"][s]:b["starts"][s + 1]],
                              np.broadcast_to(want, (n, H, d)))


@pytest.mark.parametrize("mask_kind", [8, 0], ids=["causal", "all"])
@pytest.mark.parametrize("dt,H,Hkv,n,d", FORMS)
def test_rows_without_keys_are_plus_zero_bit_for_bit(dt, H, Hkv, n, d, mask_kind):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    page = 16
    rng = np.random.default_rng(7)
    b = batch(rng, [(n, 0), (n, 300), (n, n // 2), (n, 2000)], page)
    b["table"][1] = -1                     # no pages: nothing is there
    qs = rnd(rng, (b["T"], H, d), dt)
    ks, vs = (store(-np.abs(f64(rnd(rng, (b["pool"], page, Hkv, d), dt), dt)), dt)
              for _ in range(2))           # negative values: a sum of none of them times 0 is -0
    qd = dev(qs, dt)
    out = mha.mha_paged_fwd(qd, dev(ks, dt), dev(vs, dt), torch.full_like(qd, -3.0),
                            q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]),
                            block_table=dev(b["table"]), max_q=n, layout="bshd",
                            mask_kind=mask_kind)
    bits = np.ascontiguousarray(from_device(out)).view(np.uint16 if dt == "bf16" else np.uint32)
    none = np.zeros(b["T"], dtype=bool)
    none[:2 * n] = True
    # tokens before the first position (without a mask they see what there is)
    none[2 * n:2 * n + (n - n // 2 if mask_kind == 8 else n if n // 2 == 0 else 0)] = True
    assert np.all(bits[none] == 0)
    assert np.all((bits[~none] != 0).any(-1))
