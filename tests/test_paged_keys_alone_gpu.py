"""Appending keys and values without queries: the caches that a call with queries leaves,
whatever is given as the queries' weight."""
import numpy as np
import pytest

from test_paged_gpu import batch, dev
from test_qk_rope_gpu import freqs, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,d", [(2, 64), (8, 64), (9, 64), (3, 128), (24, 128)])
@pytest.mark.parametrize("at", [False, True], ids=["append", "append_at"])
def test_keys_and_values_alone(dt, Hkv, d, at):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(Hkv + d)
    b = batch(rng, [(7, 50), (1, 1), (0, 33), (20, 20), (5, 200)], 16, behind=3, before=2)
    q, k, v = (dev(rnd(rng, (b["T"], h, d), dt), dt) for h in (2 * Hkv, Hkv, Hkv))
    w = dev(rnd(rng, (d,), dt, 0.3, 1.0), dt)
    pos = (dev(rng.integers(0, 300, b["T"]).astype(np.int32)),) if at else ()
    kw = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]),
              inv_freq=dev(freqs(d)), k_weight=w, layout="bshd")
    call = mha.mha_paged_append_at if at else mha.mha_paged_append
    got = []
    for queries, weight in ((q, w), (None, None), (None, w), (None, torch.full_like(w, float("nan")))):
        caches = [torch.full((b["pool"], 16, Hkv, d), 5.0, dtype=k.dtype, device="cuda")
                  for _ in range(2)]
        out = call(queries, k, v, *caches, *pos, q_weight=weight, **kw)
        assert (out is None) == (queries is None)
        got.append(caches)
    torch.cuda.synchronize()
    for caches in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(caches, got[0]))
