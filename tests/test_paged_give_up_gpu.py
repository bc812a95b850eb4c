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

STALL_DECODE, STALL_FEW = 8, 16


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
