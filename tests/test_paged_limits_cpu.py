"""Counts at the edge of the 32-bit numbers that the kernels step through: refused on the
host before anything is enqueued."""
import pytest

from test_paged_cpu import Fake, append, mha, recorded, rope_bwd, rope_fwd  # noqa: F401 (fixtures)

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("H,Hkv", [(MOST, 0), (0, 2 ** 30), (2 ** 30, 2 ** 29 + 2 ** 28)])
def test_rows_of_a_token(mha, H, Hkv):  # noqa: F811
    E_UNS = mha.MHA_ERR_UNSUPPORTED
    assert rope_fwd(mha, B=1, L=1, H=H, Hkv=Hkv) == E_UNS
    assert rope_bwd(mha, B=1, L=1, H=H, Hkv=Hkv) == E_UNS
    if Hkv and H % Hkv == 0:
        assert append(mha, B=1, T=1, H=H, Hkv=Hkv, pages=1) == E_UNS


@pytest.mark.parametrize("B,max_pages", [(2 ** 32 + 2, 1), (2, 2 ** 32 + 4), (2 ** 31, 4)])
def test_tables_past_32_bits(recorded, B, max_pages):  # noqa: F811
    mod, calls = recorded
    q, k = Fake((6, 4, 64)), Fake((6, 2, 64))
    cache = Fake((9, 32, 2, 64)), Fake((9, 32, 2, 64))
    kw = dict(q_starts=Fake((B + 1,), "i32"), kv_lengths=Fake((B,), "i32"),
              block_table=Fake((B, max_pages), "i32"), layout="bshd", stream=3)
    with pytest.raises(ValueError):
        mod.mha_paged_append(q, k, k, *cache, Fake((6, 4, 64)), **kw)
    with pytest.raises(ValueError):
        mod.mha_paged_fwd(q, *cache, Fake((6, 4, 64)), max_q=3, workspace=Fake((64,), "u8"), **kw)
    assert not calls
