"""Launches that overlap: paged attention between the other tensor-core kernels, one after
the other without a pause, on one stream and on several, with grids that leave room on the
SMs for the next launch's CTAs."""
import numpy as np
import pytest

from test_paged_gpu import batch, cache_of, dev
from test_qk_rope_gpu import rnd

pytestmark = pytest.mark.gpu


def calls():
    """(name, function of a stream, its outputs) of small calls of every kernel."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(0)
    res = []

    def paged(name, seqs, H, Hkv, d, max_pages=None):
        b = batch(rng, seqs, 64, max_pages=max_pages)
        kc, vc = (dev(c, "bf16") for c in cache_of(rng, b, Hkv, 64, d, "bf16", "bshd"))
        q = dev(rnd(rng, (b["T"], H, d), "bf16"), "bf16")
        out = torch.zeros_like(q)
        n = max(n for n, _ in seqs)
        ws = torch.empty(mha.mha_paged_workspace_size(len(seqs), b["T"], H, Hkv, d, n, q.dtype),
                         dtype=torch.uint8, device="cuda")
        kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
                  max_q=n, layout="bshd", workspace=ws)
        res.append((name, lambda st: mha.mha_paged_fwd(q, kc, vc, out, stream=st, **kw), out))

    # (short caches: no joining launch behind the attention)
    for d in (64, 128):
        paged("few", [(1, 200), (1, 31)], 8, 2, d)
        paged("few cut", [(1, 3000)], 8, 2, d)
        paged("many", [(40, 200), (9, 31)], 4, 2, d)
        paged("many cut", [(40, 3000)], 4, 2, d)

    def dense(name, B, H, Hkv, Lq, Lk, d, mask):
        q, k, v = (dev(rnd(rng, (B, h, n, d), "bf16"), "bf16")
                   for h, n in ((H, Lq), (Hkv, Lk), (Hkv, Lk)))
        out = torch.zeros_like(q)
        res.append((name, lambda st: mha.mha_fwd_ex(q, k, v, out, mask_kind=mask, stream=st), out))
    dense("short", 2, 4, 4, 64, 64, 64, mha.MHA_MASK_CAUSAL)
    dense("long", 1, 2, 2, 300, 300, 128, mha.MHA_MASK_CAUSAL)
    dense("decode", 2, 8, 2, 1, 300, 64, mha.MHA_MASK_CAUSAL_TAIL)
    x, w = (dev(rnd(rng, s, "bf16"), "bf16") for s in ((100, 512), (512, 512)))
    y = torch.zeros(100, 512, dtype=torch.bfloat16, device="cuda")
    res.append(("linear", lambda st: mha.mha_linear_fwd(x, w, out=y, stream=st), y))
    return res


def test_every_pair_of_kernels_back_to_back():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    all_calls = calls()
    st = torch.cuda.current_stream()
    want = []
    for _, f, out in all_calls:
        f(st)
        torch.cuda.synchronize()
        want.append(out.clone())
    for _, fa, _ in all_calls:
        for _, fb, _ in all_calls:
            for _ in range(6):
                fa(st)
                fb(st)
        torch.cuda.synchronize()
        for (name, _, out), w in zip(all_calls, want):
            assert torch.equal(out, w), name
    assert mha.mha_debug_status() == mha.MHA_OK


def test_kernels_on_streams_of_their_own():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    all_calls = calls()
    streams = [torch.cuda.Stream() for _ in all_calls]
    want = []
    for _, f, out in all_calls:
        f(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(out.clone())
    for _ in range(40):
        for (_, f, _), st in zip(all_calls, streams):
            f(st)
    torch.cuda.synchronize()
    for (name, _, out), w in zip(all_calls, want):
        assert torch.equal(out, w), name
    assert mha.mha_debug_status() == mha.MHA_OK
