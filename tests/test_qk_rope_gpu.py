"""Per-head norm and position rotation of queries and keys and their gradients
against the plain float64 forms, with the errors derived in paged_ref.py."""
import numpy as np
import pytest

import gen
import paged_ref as ref
from helpers import from_device, to_device

pytestmark = pytest.mark.gpu


def rnd(rng, shape, dt, amp=1.0, about=0.0):
    x = rng.normal(size=shape) * amp + about
    return gen.f64_to_bf16_bits(x) if dt == "bf16" else x.astype(np.float32)


def freqs(rotary, base=10000.0):
    return (base ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))).astype(np.float32)


def make(B, H, Hkv, L, d, dt, layout, rotary, seed, norm=(True, True), far=0):
    rng = np.random.default_rng(seed)
    shape = lambda h: (B, L, h, d) if layout == "bshd" else (B, h, L, d)  # noqa: E731
    s = dict(q=rnd(rng, shape(H), dt), k=rnd(rng, shape(Hkv), dt), gq=rnd(rng, shape(H), dt),
             gk=rnd(rng, shape(Hkv), dt),
             qw=rnd(rng, (d,), dt, 0.3, 1.0) if norm[0] else None,
             kw=rnd(rng, (d,), dt, 0.3, 1.0) if norm[1] else None,
             pos=(rng.integers(0, far + 1, (B, 1)) + np.arange(L)).astype(np.int32),
             freq=freqs(rotary), axis=2 if layout == "bshd" else 1)
    return s


def on_gpu(s, dt):
    import torch
    up = lambda a: None if a is None else to_device(a, dt)  # noqa: E731
    g = {x: up(s[x]) for x in ("q", "k", "gq", "gk", "qw", "kw")}
    g["pos"] = torch.from_numpy(s["pos"]).cuda()
    g["freq"] = torch.from_numpy(s["freq"]).cuda() if len(s["freq"]) else None
    return g


def f64(a, dt):
    return None if a is None else gen.as_f64(a, dt)


def check(got, want, tol, label):
    assert np.isfinite(got).all(), label
    bad = np.abs(got - want) > tol
    assert not bad.any(), (label, float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()))


CASES = [
    # (B, H, Hkv, L, d, dtype, layout, rotary, interleaved)
    (1, 1, 1, 1, 64, "bf16", "bhsd", 64, False),
    (2, 8, 8, 32, 64, "f32", "bhsd", 64, True),
    (3, 4, 2, 7, 128, "bf16", "bshd", 128, False),
    (2, 6, 3, 33, 128, "bf16", "bhsd", 64, True),
    (5, 3, 1, 13, 64, "bf16", "bshd", 16, False),
    (5, 3, 1, 13, 64, "bf16", "bshd", 32, True),
    (2, 5, 5, 9, 128, "f32", "bshd", 96, False),
    (2, 4, 2, 11, 64, "f32", "bhsd", 48, False),
    (1, 40, 8, 3, 128, "bf16", "bshd", 0, False),   # norm alone
    (2, 33, 2, 1300, 64, "bf16", "bshd", 64, False),  # four tokens per CTA
    (3, 2, 2, 901, 128, "f32", "bhsd", 128, True),
    (1, 64, 1, 2500, 128, "bf16", "bhsd", 112, False),
]
IDS = ["B%dH%dKV%dL%dd%d_%s_%s_r%d_%d" % c for c in CASES]


@pytest.mark.parametrize("c", CASES, ids=IDS)
@pytest.mark.parametrize("norm", [(True, True), (False, False), (True, False)],
                         ids=["norm", "bare", "qnorm"])
def test_forward_and_backward(c, norm):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    B, H, Hkv, L, d, dt, layout, rotary, inter = c
    s = make(B, H, Hkv, L, d, dt, layout, rotary, 11, norm, far=100000)
    g = on_gpu(s, dt)
    kw = dict(q_weight=g["qw"], k_weight=g["kw"], positions=g["pos"], inv_freq=g["freq"],
              layout=layout, interleaved=inter, eps=1e-5)
    qo, ko = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], **kw)
    dq, dk, dqw, dkw = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], **kw)
    again = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], **kw)
    torch.cuda.synchronize()
    pos = np.expand_dims(s["pos"], s["axis"])
    for x, w, gy, out, dx, dw, which in (("q", "qw", "gq", qo, dq, dqw, 0),
                                         ("k", "kw", "gk", ko, dk, dkw, 1)):
        a = (f64(s[x], dt), f64(s[w], dt))
        b = (pos, s["freq"], inter, 1e-5)
        check(f64(from_device(out), dt), ref.norm_rope(*a, *b), ref.norm_rope_tol(*a, *b, dt), x)
        wx, ww = ref.norm_rope_bwd(*a, f64(s[gy], dt), *b)
        # additions behind one another: a lane's rows, the CTA's slots, the CTAs
        tx, tw = ref.norm_rope_bwd_tol(*a, f64(s[gy], dt), *b, dt, chain=64 + 400)
        check(f64(from_device(dx), dt), wx, tx, "d" + x)
        assert (dw is None) == (ww is None)
        if dw is not None:
            check(dw.double().cpu().numpy(), ww, tw, "d" + x + " weight")
        for one, two in ((dx, again[which]), (dw, again[2 + which])):
            assert one is None or torch.equal(one, two)


@pytest.mark.parametrize("dt,layout", [("bf16", "bshd"), ("f32", "bhsd")])
def test_in_place_and_one_tensor_alone(dt, layout):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    s = make(2, 6, 2, 50, 128, dt, layout, 128, 5)
    g = on_gpu(s, dt)
    kw = dict(positions=g["pos"], inv_freq=g["freq"], layout=layout)
    qo, ko = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], q_weight=g["qw"], k_weight=g["kw"], **kw)
    q2, k2 = g["q"].clone(), g["k"].clone()
    mha.mha_qk_norm_rope_fwd(q2, k2, q2, k2, q_weight=g["qw"], k_weight=g["kw"], **kw)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    only_q = mha.mha_qk_norm_rope_fwd(g["q"], None, q_weight=g["qw"], **kw)
    only_k = mha.mha_qk_norm_rope_fwd(None, g["k"], k_weight=g["kw"], **kw)
    assert only_q[1] is None and only_k[0] is None
    assert torch.equal(only_q[0], qo) and torch.equal(only_k[1], ko)
    full = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], q_weight=g["qw"],
                                    k_weight=g["kw"], **kw)
    a, b = g["gq"].clone(), g["gk"].clone()
    mha.mha_qk_norm_rope_bwd(g["q"], g["k"], a, b, a, b, q_weight=g["qw"], k_weight=g["kw"], **kw)
    assert torch.equal(a, full[0]) and torch.equal(b, full[1])
    alone = mha.mha_qk_norm_rope_bwd(g["q"], None, g["gq"], None, q_weight=g["qw"], **kw)
    assert torch.equal(alone[0], full[0]) and alone[3] is None
    # the rows are shared out over the warps by how many there are of both tensors, so
    # alone the weight's sum runs in another order: each order is within the bound of
    # any order of these additions
    pos = np.expand_dims(s["pos"], s["axis"])
    args = (f64(s["q"], dt), f64(s["qw"], dt), f64(s["gq"], dt), pos, s["freq"], False, 1e-6)
    want, tol = ref.norm_rope_bwd(*args)[1], ref.norm_rope_bwd_tol(*args, dt, chain=464)[1]
    for w in (alone[2], full[2]):
        check(w.double().cpu().numpy(), want, tol, "weight")


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_rows_of_one_tensor_alone(dt, layout):
    # enough rows that a warp goes through many, across tokens and sequences
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    s = make(7, 9, 5, 801, 64, dt, layout, 64, 12, far=5000)
    g = on_gpu(s, dt)
    kw = dict(positions=g["pos"], inv_freq=g["freq"], layout=layout)
    full = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], q_weight=g["qw"],
                                    k_weight=g["kw"], **kw)
    q = mha.mha_qk_norm_rope_bwd(g["q"], None, g["gq"], None, q_weight=g["qw"], **kw)
    k = mha.mha_qk_norm_rope_bwd(None, g["k"], None, g["gk"], k_weight=g["kw"], **kw)
    assert torch.equal(q[0], full[0]) and torch.equal(k[1], full[1])
    pos = np.expand_dims(s["pos"], s["axis"])
    for x, w, gy, dx, dw in (("q", "qw", "gq", full[0], full[2]), ("k", "kw", "gk", full[1], full[3])):
        args = (f64(s[x], dt), f64(s[w], dt), f64(s[gy], dt), pos, s["freq"], False, 1e-6)
        (wx, ww), (tx, tw) = ref.norm_rope_bwd(*args), ref.norm_rope_bwd_tol(*args, dt, chain=464)
        check(f64(from_device(dx), dt), wx, tx, "d" + x)
        check(dw.double().cpu().numpy(), ww, tw, "d" + x + " weight")


def test_positions():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    # none: 0 .. L - 1; and any 32-bit position, negative ones among them
    s = make(3, 2, 1, 19, 64, "f32", "bshd", 64, 6)
    g = on_gpu(s, "f32")
    a = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], inv_freq=g["freq"], layout="bshd")
    pos = torch.arange(19, dtype=torch.int32, device="cuda").expand(3, 19).contiguous()
    b = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], inv_freq=g["freq"], positions=pos, layout="bshd")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    rng = np.random.default_rng(7)
    p = rng.integers(-2 ** 31, 2 ** 31, (3, 19)).astype(np.int32)
    p[0, :4] = (2 ** 31 - 1, -2 ** 31, 0, -1)
    out, _ = mha.mha_qk_norm_rope_fwd(g["q"], None, inv_freq=g["freq"], layout="bshd",
                                      positions=torch.from_numpy(p).cuda())
    x = s["q"].astype(np.float64)
    args = (x, None, p[:, :, None], s["freq"], False, 1e-6)
    # the angle itself: position times a frequency in turns, held to 2^-53 of it
    turns = np.abs(p[:, :, None, None]) * s["freq"] / (2 * np.pi)
    far = np.zeros_like(x)
    far[..., :32] = far[..., 32:] = 2 * np.pi * turns * 2.0 ** -52
    check(out.double().cpu().numpy(), ref.norm_rope(*args),
          ref.norm_rope_tol(*args, "f32") + far * ref.pair_size(x, 64, False), "far positions")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zero_and_extreme_rows(dt):
    import transformer_head_scaled_mha_gb300 as mha
    s = make(1, 4, 1, 8, 64, dt, "bshd", 32, 8)
    x = f64(s["q"], dt)
    x[0, 0] = 0.0                 # a zero row: 0, and its gradient g w / sqrt(eps)
    x[0, 1] *= 1e-15              # eps outweighs the row
    x[0, 2] *= 1e15               # squares near 1e31
    x[0, 3, :, 5] = 1e4           # one element holds the row
    s["q"] = gen.f64_to_bf16_bits(x) if dt == "bf16" else x.astype(np.float32)
    g = on_gpu(s, dt)
    kw = dict(q_weight=g["qw"], positions=g["pos"], inv_freq=g["freq"], layout="bshd", eps=1e-6)
    out, _ = mha.mha_qk_norm_rope_fwd(g["q"], None, **kw)
    dq, _, dqw, _ = mha.mha_qk_norm_rope_bwd(g["q"], None, g["gq"], None, **kw)
    a = (f64(s["q"], dt), f64(s["qw"], dt))
    b = (s["pos"][:, :, None], s["freq"], False, 1e-6)
    check(f64(from_device(out), dt), ref.norm_rope(*a, *b), ref.norm_rope_tol(*a, *b, dt), "out")
    wx, ww = ref.norm_rope_bwd(*a, f64(s["gq"], dt), *b)
    tx, tw = ref.norm_rope_bwd_tol(*a, f64(s["gq"], dt), *b, dt, chain=464)
    check(f64(from_device(dq), dt), wx, tx + 2.0 ** -140, "dq")
    check(dqw.double().cpu().numpy(), ww, tw, "dq weight")
    assert np.all(f64(from_device(out), dt)[0, 0] == 0)


def test_dimensions_outside_the_rotation_keep_infinities():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    x = torch.randn(1, 4, 2, 64, device="cuda").bfloat16()
    x[0, 1, 0, 40], x[0, 2, 1, 63], x[0, 3, 0, 33] = float("inf"), -float("inf"), float("nan")
    freq = mha.rope_inv_freq(32)
    out, _ = mha.mha_qk_norm_rope_fwd(x, None, inv_freq=freq, layout="bshd")
    assert torch.equal(out[..., 32:].nan_to_num(7.0), x[..., 32:].nan_to_num(7.0))
    assert torch.isfinite(out[..., :32]).all()


def test_weights_without_rows_have_zero_gradients():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64)):
        r = mha.mha_qk_norm_rope_bwd(z(*shape), z(*shape), z(*shape), z(*shape), q_weight=w,
                                     k_weight=w, layout="bshd")
        assert (r[2] == 0).all() and (r[3] == 0).all()
    r = mha.mha_qk_norm_rope_bwd(z(2, 3, 4, 64), z(2, 3, 0, 64), z(2, 3, 4, 64), z(2, 3, 0, 64),
                                 q_weight=w, k_weight=w, layout="bshd")
    assert (r[3] == 0).all()


def test_other_stream_and_captured_graph():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    s = make(4, 8, 2, 700, 64, "bf16", "bshd", 64, 9)
    g = on_gpu(s, "bf16")
    kw = dict(q_weight=g["qw"], k_weight=g["kw"], positions=g["pos"], inv_freq=g["freq"],
              layout="bshd")
    want = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], **kw)
    wantb = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        got = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], stream=st, **kw)
        gotb = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], stream=st, **kw)
        torch.cuda.synchronize()
        for a, b in zip((*got, *gotb), (*want, *wantb)):
            assert torch.equal(a, b)
    outs = [torch.empty_like(t) for t in (g["q"], g["k"])]
    grads = [torch.empty_like(t) for t in wantb]
    ws = torch.empty(mha.mha_qk_norm_rope_bwd_workspace_size(64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mha.mha_qk_norm_rope_fwd(g["q"], g["k"], *outs, **kw)
        mha.mha_qk_norm_rope_bwd(g["q"], g["k"], g["gq"], g["gk"], *grads, workspace=ws, **kw)
    for _ in range(3):
        for t in (*outs, *grads):
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*outs, *grads), (*want, *wantb)):
            assert torch.equal(a, b)
