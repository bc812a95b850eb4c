"""The generation step that the project's overview shows, as it stands there, on the GPU."""
import numpy as np
import pytest

import documented_step

pytestmark = pytest.mark.gpu

LAYERS, H, HKV, D = 2, 4, 2, 64


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pages", [250, 30000], ids=["small_pool", "large_pool"])
@pytest.mark.parametrize("forks", [False, True, None], ids=["same_rows", "forks", "one_call"])
def test_steps_lose_no_page(dt, pages, forks):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    B, dtype = 5, {"f32": torch.float32, "bf16": torch.bfloat16}[dt]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    caches = [torch.zeros(LAYERS, pages, 64, HKV, D, dtype=dtype, device="cuda") for _ in range(2)]

    def fill(tokens):  # a token's number in digits, which both types hold exactly
        rows = np.zeros((len(tokens), HKV, D), np.float32)
        for i in range(3):
            rows[:, :, i] = (tokens // 128 ** i % 128)[:, None]
        k = up(rows).to(dtype)
        return torch.ones(len(tokens), H, D, dtype=dtype, device="cuda"), k, -k

    def read(k):
        digits = k[0, :, :, HKV - 1, :3].float().cpu().numpy().astype(np.int64)
        return digits @ (128 ** np.arange(3))

    pool = documented_step.Pool(mha, up, lambda t: t.cpu().numpy(), caches, read, fill,
                                mha.rope_inv_freq(D), B, 40, pages)
    documented_step.run(pool, 24, 7, forks)
    assert bool(torch.isfinite(pool.space["out"].float()).all())
    assert torch.equal(caches[0][0].float(), -caches[1][0].float())
    assert mha.mha_debug_status() == mha.MHA_OK
