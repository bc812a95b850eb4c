"""A training step through the operators as they are used together: norm and rotation,
attention that keeps its row statistics, its backward pass from them, and the backward
pass of norm and rotation, against the formulas in 64 bits."""
import numpy as np
import pytest

import paged_ref as ref
from helpers import TOL, from_device
from test_bwd_gpu import BWD_TOL
from test_qk_rope_gpu import check, f64, make, on_gpu, rnd

pytestmark = pytest.mark.gpu


def attention_grads(q, k, v, dout, scale):
    """(out, dq, dk, dv) of causal attention, all [B, H or H_kv, L, d] float64."""
    group = q.shape[1] // k.shape[1]
    kk, vv = (np.repeat(t, group, axis=1) for t in (k, v))
    L = q.shape[2]
    s = scale * (q @ kk.swapaxes(-1, -2))
    s = np.where(np.arange(L)[None, :] <= np.arange(L)[:, None], s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out = w @ vv
    dw = dout @ vv.swapaxes(-1, -2)
    ds = w * (dw - (dout * out).sum(-1, keepdims=True))
    share = lambda t: t.reshape(t.shape[0], k.shape[1], group, L, -1).sum(2)  # noqa: E731
    return out, scale * ds @ kk, share(scale * ds.swapaxes(-1, -2) @ q), \
        share(w.swapaxes(-1, -2) @ dout)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hkv,L,d,layout,rotary,inter", [
    (2, 4, 2, 70, 64, "bhsd", 64, False),
    (1, 6, 2, 200, 64, "bshd", 32, True),
    (2, 4, 1, 150, 128, "bshd", 128, False),
    (3, 2, 2, 33, 128, "bhsd", 128, True),
])
def test_norm_rotation_attention_and_back(B, H, Hkv, L, d, layout, rotary, inter, dt):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    s = make(B, H, Hkv, L, d, dt, layout, rotary, 31, far=3000)
    rng = np.random.default_rng(5)
    g = on_gpu(s, dt)
    v, dout = (rnd(rng, s[x].shape, dt) for x in ("k", "q"))
    up = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda() \
        if dt == "bf16" else torch.from_numpy(a).cuda()  # noqa: E731
    scale = d ** -0.5
    kw = dict(q_weight=g["qw"], k_weight=g["kw"], positions=g["pos"], inv_freq=g["freq"],
              layout=layout, interleaved=inter, eps=1e-6)
    qo, ko = mha.mha_qk_norm_rope_fwd(g["q"], g["k"], **kw)
    att = dict(layout=layout, mask_kind=mha.MHA_MASK_CAUSAL, scale=scale)
    out, lse = mha.mha_fwd_lse(qo, ko, up(v), **att)
    dqo, dko, dv = mha.mha_bwd(qo, ko, up(v), out, up(dout), lse=lse, **att)
    dq, dk, dqw, dkw = mha.mha_qk_norm_rope_bwd(g["q"], g["k"], dqo, dko, dqo, dko, **kw)
    assert mha.mha_debug_status() == mha.MHA_OK

    heads_first = lambda t: t.swapaxes(1, 2) if layout == "bshd" else t  # noqa: E731
    get = lambda t: f64(from_device(t), dt)  # noqa: E731
    pos = np.expand_dims(s["pos"], s["axis"])
    rest = (pos, s["freq"], inter, 1e-6)
    stored = {}
    for x, w, o in (("q", "qw", qo), ("k", "kw", ko)):
        a = (f64(s[x], dt), f64(s[w], dt))
        stored[x] = get(o)
        check(stored[x], ref.norm_rope(*a, *rest), ref.norm_rope_tol(*a, *rest, dt), x)
    # attention at the queries and keys as they were stored (each within its rounding)
    want = attention_grads(heads_first(stored["q"]), heads_first(stored["k"]),
                           heads_first(f64(v, dt)), heads_first(f64(dout, dt)), scale)
    want = [heads_first(t) for t in want]
    assert np.abs(get(out) - want[0]).max() <= TOL[dt]["max"]
    assert np.abs(get(dv) - want[3]).max() <= BWD_TOL[dt]["max"] * np.abs(want[3]).max()
    for x, w, dx, dw, gy in (("q", "qw", dq, dqw, want[1]), ("k", "kw", dk, dkw, want[2])):
        a = (f64(s[x], dt), f64(s[w], dt), gy)
        wx, ww = ref.norm_rope_bwd(*a, *rest)
        tx, tw = ref.norm_rope_bwd_tol(*a, *rest, dt, chain=464)
        # the attention's gradient comes in with errors of up to E an element, rotated back up
        # to sqrt(2) E, and goes through dx = r (w g - n mean(w g n)), dw = sum g n
        E = np.sqrt(2.0) * BWD_TOL[dt]["max"] * np.abs(gy).max()
        r = 1.0 / np.sqrt((a[0] ** 2).mean(-1, keepdims=True) + 1e-6)
        n, aw = np.abs(a[0] * r), np.abs(a[1])
        tx = tx + E * r * (aw + n * (aw * n).mean(-1, keepdims=True))
        tw = tw + E * n.reshape(-1, d).sum(0)
        check(get(dx), wx, tx, "d" + x)
        check(dw.double().cpu().numpy(), ww, tw, "d" + x + " weight")
