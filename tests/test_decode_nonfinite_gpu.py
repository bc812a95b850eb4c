"""Decoding steps against a contiguous cache: a query or key that is NaN, and a score
past the range of fp32, make exactly the rows that see them NaN, in the output and in
the row statistics; the other rows stay what they are without them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DECODE = 5  # the few-query kernel


@pytest.mark.parametrize("H,Hkv,Lq,d", [(2, 2, 1, 64), (2, 1, 1, 128), (4, 1, 1, 64),
                                        (8, 2, 2, 128), (8, 2, 4, 64), (8, 2, 4, 128)])
def test_nan_stays_nan(H, Hkv, Lq, d):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    B, L, kind = 4, 300, mha.MHA_MASK_CAUSAL_TAIL
    assert mha.mha_fwd_path_ex(B, H, Hkv, Lq, L, d, d, kind, mha.MHA_DTYPE_BF16) == DECODE
    g = torch.Generator(device="cuda").manual_seed(H + Lq)
    q, k, v = (torch.randn(B, h, n, d, generator=g, device="cuda").abs().bfloat16()
               for h, n in ((H, Lq), (Hkv, L), (Hkv, L)))
    want, want_lse = mha.mha_fwd_lse(q, k, v, mask_kind=kind)
    rows = torch.zeros(B, H, Lq, dtype=torch.bool, device="cuda")
    group = H // Hkv
    q[0, H - 1, Lq - 1, 7] = float("nan")
    rows[0, H - 1, Lq - 1] = True
    k[1, 0, 5, 3] = float("nan")              # seen by every position
    rows[1, :group] = True
    k[2, Hkv - 1, L - 1, 0] = float("nan")    # seen by the last position alone
    rows[2, H - group:, Lq - 1] = True
    q[3, 0, 0] = 2.0 ** 120                   # products past 2^128
    k[3, 0, 9] = 2.0 ** 15
    rows[3, 0, 0] = True
    out, lse = mha.mha_fwd_lse(q, k, v, mask_kind=kind)
    assert torch.equal(torch.isnan(out), rows[..., None].expand_as(out))
    assert torch.equal(torch.isnan(lse), rows)
    same = ~rows
    same[3, :group] = False  # they see the large key
    assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_lse[same])
    assert np.isfinite(lse[~rows].cpu().numpy()).all()
