"""The give-up path of the bounded waits in the kernels beside the short and long ones,
on the GPU, without any fault (test_give_up_gpu.py): a test hook makes an issuer wait on a
barrier that nothing signals, with a limit of 2 ms.  The kernel returns, the status word
tells MHA_ERR_TIMEOUT, and the next normal call is right."""
import numpy as np
import pytest

import gen
from helpers import check_case, run_gpu, spec
from test_paged_gpu import batch, cache_of, check_paged
from test_qk_rope_gpu import rnd

pytestmark = pytest.mark.gpu

STALL_DECODE, STALL_FEW, STALL_MANY = 8, 16, 32


def stalled(stall, call):
    """``call`` with the hook set: it gives up, and the status says so once."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    assert mha.mha_debug_status() == mha.MHA_OK
    assert mha.mha_debug_set_wait(2_000_000, stall) == mha.MHA_OK
    try:
        call()  # output undefined
        torch.cuda.synchronize()
    finally:
        assert mha.mha_debug_set_wait(0, 0) == mha.MHA_OK
    assert mha.mha_debug_status() == mha.MHA_ERR_TIMEOUT
    assert mha.mha_debug_status() == mha.MHA_OK


def stalled_paged(stall, seqs, H, Hkv, d):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(4)
    b = batch(rng, seqs, 64)
    kc, vc = (torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda()
              for x in cache_of(rng, b, Hkv, 64, d, "bf16", "bshd"))
    q = torch.from_numpy(rnd(rng, (b["T"], H, d), "bf16").view(np.int16)).view(torch.bfloat16).cuda()
    arrays = {k: torch.from_numpy(b[n]).cuda() for k, n in (("q_starts", "starts"),
                                                           ("kv_lengths", "lens"),
                                                           ("block_table", "table"))}
    stalled(stall, lambda: mha.mha_paged_fwd(q, kc, vc, max_q=max(n for n, _ in seqs),
                                             layout="bshd", **arrays))


# parts that end with the tile whose wait runs out (the third), and others: units of 1 to 5
# tiles, more of them than CTAs, and long ones that are cut
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("H,Hkv,n,d", [(2, 2, 1, 64), (4, 1, 1, 128), (4, 2, 8, 64)])
def test_few_query_paged_kernel(tiles, H, Hkv, n, d):
    seqs = [(n, 128 * tiles)] * 320
    stalled_paged(STALL_FEW, seqs, H, Hkv, d)
    stalled_paged(STALL_FEW, [(n, 20000 + 128 * tiles)] * 2, H, Hkv, d)
    check_paged(seqs[:40] + [(n, 3000)], H, Hkv, d, "bf16", 64, "bshd")


@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("H,Hkv,Lq,d", [(2, 2, 1, 64), (4, 1, 1, 128), (4, 1, 4, 64)])
def test_decoding_kernel(tiles, H, Hkv, Lq, d):
    # a pair's last tile is the one whose wait runs out (three tiles), and others
    case = spec(200, H, Lq, 128 * tiles + 1, d, mask=gen.MASK_KEY_PADDING, Hkv=Hkv,
                len_range=(128 * tiles, 128 * tiles))
    q, k, v, lens = gen.make_inputs(case, seed=3)
    stalled(STALL_DECODE, lambda: run_gpu(q, k, v, lens, case))
    check_case(spec(3, H, Lq, 128 * tiles + 1, d, Hkv=Hkv), seed=3)


@pytest.mark.parametrize("seqs,H,Hkv,d", [
    ([(512, 1024)] * 40, 2, 2, 128),              # whole tiles, several parts to a CTA
    ([(300, 1000 + 7 * i) for i in range(60)], 4, 2, 64),   # ragged ones
    ([(40, 700)] * 100 + [(60, 33)] * 100, 4, 2, 128),     # rows for one tile: both share them
    ([(100, 20001)], 2, 1, 64),                   # one unit cut over the CTAs
])
def test_many_query_paged_kernel(seqs, H, Hkv, d):
    stalled_paged(STALL_MANY, seqs, H, Hkv, d)
    check_paged(seqs[:3], H, Hkv, d, "bf16", 64, "bshd")


@pytest.mark.parametrize("H,Hkv,n,d,page", [(16, 16, 8192, 128, 128), (16, 16, 8192, 64, 64)])
def test_a_limit_shorter_than_the_kernel(H, Hkv, n, d, page):
    """A prompt of whole tiles takes longer than the limit (about 220 us against 100): no
    wait is for work that others have in hand as long, so nothing gives up."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    g = torch.Generator(device="cuda").manual_seed(0)
    q, kc, vc = (torch.randn(s, generator=g, device="cuda").bfloat16()
                 for s in ((n, H, d), (n // page, page, Hkv, d), (n // page, page, Hkv, d)))
    i32 = dict(dtype=torch.int32, device="cuda")
    kw = dict(q_starts=torch.tensor([0, n], **i32), kv_lengths=torch.tensor([n], **i32),
              block_table=torch.randperm(n // page, generator=g, device="cuda").int()[None],
              max_q=n, layout="bshd")
    want = mha.mha_paged_fwd(q, kc, vc, **kw)
    torch.cuda.synchronize()
    ws = torch.empty(mha.mha_paged_workspace_size(1, n, H, Hkv, d, n, q.dtype),
                     dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(5)]
    torch.cuda.synchronize()
    assert mha.mha_debug_status() == mha.MHA_OK
    assert mha.mha_debug_set_wait(100_000, 0) == mha.MHA_OK
    try:
        for o in outs:
            mha.mha_paged_fwd(q, kc, vc, o, workspace=ws, **kw)
        torch.cuda.synchronize()
    finally:
        assert mha.mha_debug_set_wait(0, 0) == mha.MHA_OK
    assert mha.mha_debug_status() == mha.MHA_OK
    for o in outs:
        assert torch.equal(o, want)
