"""Counts at the edge of the 32-bit numbers that the kernels step through: refused on the
host before anything is enqueued."""
import pytest

from test_paged_cpu import append, mha, paged, rope_bwd, rope_fwd  # noqa: F401 (mha: fixture)

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("H,Hkv", [(MOST, 0), (0, 2 ** 30), (2 ** 30, 2 ** 29 + 2 ** 28)])
def test_rows_of_a_token(mha, H, Hkv):  # noqa: F811
    E_UNS = mha.MHA_ERR_UNSUPPORTED
    assert rope_fwd(mha, B=1, L=1, H=H, Hkv=Hkv) == E_UNS
    assert rope_bwd(mha, B=1, L=1, H=H, Hkv=Hkv) == E_UNS
    if Hkv and H % Hkv == 0:
        assert append(mha, B=1, T=1, H=H, Hkv=Hkv, pages=1) == E_UNS
