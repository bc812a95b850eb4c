"""Norm and rotation of tokens whose rows pass 2^31 elements: offsets from token to token
in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu


def test_tokens_of_more_than_2_to_the_31_elements():
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    L, H, d = 3, 2 ** 24 + 5, 128  # 12.9 GB
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(1, L, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    heads = torch.tensor([0, 1, 2, 2 ** 23, H - 9, H - 2, H - 1], device="cuda")
    small = x[:, :, heads].contiguous()
    kw = dict(inv_freq=mha.rope_inv_freq(d), layout="bshd")
    want, _ = mha.mha_qk_norm_rope_fwd(small, None, **kw)
    back = mha.mha_qk_norm_rope_bwd(None, None, want, None, **kw)[0]
    mha.mha_qk_norm_rope_fwd(x, None, x, None, **kw)
    assert torch.equal(x[:, :, heads], want)
    mha.mha_qk_norm_rope_bwd(None, None, x, None, x, **kw)
    assert torch.equal(x[:, :, heads], back)
    del x
    torch.cuda.empty_cache()
