"""What the entry points of include/mha_paged.h hand to their kernels, recorded on the host
(paged_launches_host.cu)."""
import ctypes
import os
import shutil
import subprocess
import types

import pytest

from test_paged_cpu import CSRC, P, ROOT, append, mha  # noqa: F401 (fixture)
from test_paged_tree_cpu import append_at


@pytest.fixture(scope="module")
def launches(mha, tmp_path_factory):  # noqa: F811
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path_factory.mktemp("launches") / "launches.so")
    subprocess.run([nvcc, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-Xlinker",
                    "-Bsymbolic", "--expt-relaxed-constexpr", "-I", CSRC, "-o", out,
                    os.path.join(ROOT, "tests", "paged_launches_host.cu")], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(out)
    for name in ("mha_paged_append", "mha_paged_append_at", "mha_paged_tree_fwd",
                 "mha_paged_workspace_size"):
        entry, known = getattr(lib, name), getattr(mha.lib, name)
        entry.argtypes, entry.restype = known.argtypes, known.restype
    for name in ("rope_q_weight", "rope_k_weight"):
        getattr(lib, name).restype = ctypes.c_void_p
    lib.attention_slots_end.restype = ctypes.c_longlong
    return types.SimpleNamespace(lib=lib)


@pytest.mark.parametrize("call", [append, append_at], ids=["append", "append_at"])
def test_queries_without_heads_have_no_weight(launches, call):
    """With H = 0 the queries' weight is not an argument that is checked, so no kernel may get
    hold of it."""
    assert call(launches) == 0
    assert launches.lib.rope_q_weight() and launches.lib.rope_k_weight()
    if call is append:
        for weight in (None, P[6], P[6] + 2, P[3], P[4]):  # any address, misaligned, another's
            assert append(launches, q=None, qo=None, H=0, qw=weight) == 0
            assert launches.lib.rope_q_weight() is None and launches.lib.rope_k_weight() == P[7]
    else:
        assert append_at(launches, q=None, qo=None, H=0) == 0
        assert launches.lib.rope_q_weight() is None and launches.lib.rope_k_weight() == P[7]


def tree_call(launches, group, max_q, d, dtype, B=16, T=None, Hkv=2, max_pages=512):
    """A call of B trees of max_q tokens; its unit's rows and tokens, its CTAs, and where its
    sums end in a workspace of the size that it asks for."""
    lib, T = launches.lib, B * max_q if T is None else T
    n = lib.mha_paged_workspace_size(B, T, group * Hkv, Hkv, d, max_q, dtype)
    st = lib.mha_paged_tree_fwd(P[0], P[1], P[2], P[3], P[8], P[4], P[5], P[6], B, T, group * Hkv, Hkv, d,
                                max_q, 9000, 16, max_pages, -(-max_q // 32), 1, 0.125, dtype, P[7], n, None)
    assert st == 0
    assert lib.attention_slots_end(d) <= n
    return lib.attention_kernel(), lib.attention_rows(), lib.attention_tokens(), lib.attention_ctas()


@pytest.mark.parametrize("tokens", [33, 64, 150])
def test_units_of_large_fp32_trees(launches, tokens):
    """At d 128 units of 32 rows where that makes for a third fewer, whatever the heads that
    share a key/value head; at d 64 16."""
    def units(group, rows):
        heads = min(group, rows)
        tb = rows // heads
        return -(-tokens // tb) * -(-group // heads), heads * tb, tb
    for group in range(1, 41):
        usual, larger = units(group, 16), units(group, 32)
        want = larger if 3 * larger[0] <= 2 * usual[0] else usual
        kernel, rows, tb, ctas = tree_call(launches, group, tokens, 128, 0)
        assert (kernel, rows, tb) == (1, *want[1:]), group
        assert ctas <= 152
        assert tree_call(launches, group, tokens, 64, 0)[:3] == (1, *usual[1:]), group
        assert launches.lib.attention_merged() == 1
