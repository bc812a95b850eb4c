"""What of the drafted-tree operators runs without a GPU: refusals of the C entry points and
the bindings, the masks of trees, and the kernels' reading of them (compiled for the host)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import tree_ref
from test_paged_cpu import CSRC, P, Fake, mha, recorded  # noqa: F401


def append_at(mha, pos=P[12], q=P[0], k=P[1], qo=P[3], kc=P[4], freq=P[8], starts=P[9], B=2, T=6,  # noqa: F811
              H=4, Hkv=2, d=64, pages=9, page=16, rot=64, dtype=1):
    return mha.lib.mha_paged_append_at(q, k, P[2], qo, kc, P[5], P[6], P[7], freq, pos, starts,
                                       P[10], P[11], B, T, H, Hkv, d, pages, page, 3, rot, 0, 0,
                                       1e-6, dtype, None)


def test_append_at_rejects_before_launch(mha):  # noqa: F811
    for kw in (dict(pos=None), dict(pos=P[12] + 2), dict(pos=P[3]), dict(pos=P[4]), dict(q=None),
               dict(k=None), dict(freq=None), dict(starts=None), dict(page=24), dict(H=3),
               dict(rot=66), dict(dtype=3), dict(qo=P[12])):
        assert append_at(mha, **kw) == mha.MHA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(d=96), dict(page=8), dict(rot=8)):
        assert append_at(mha, **kw) == mha.MHA_ERR_UNSUPPORTED, kw
    for kw in (dict(T=0), dict(B=0), dict(H=0, Hkv=0)):
        assert append_at(mha, pos=None, **kw) == mha.MHA_OK, kw


def tree_fwd(mha, mask=P[8], q=P[0], kc=P[1], out=P[3], starts=P[4], B=2, T=6, H=4, Hkv=2, d=64,  # noqa: F811
             max_q=3, pages=9, page=16, max_pages=3, words=2, layout=0, scale=0.125, dtype=1,
             ws=P[7], ws_n=1 << 31):
    return mha.lib.mha_paged_tree_fwd(q, kc, P[2], out, mask, starts, P[5], P[6], B, T, H, Hkv, d,
                                      max_q, pages, page, max_pages, words, layout, scale, dtype,
                                      ws, ws_n, None)


def test_tree_fwd_rejects_before_launch(mha):  # noqa: F811
    n = mha.mha_paged_workspace_size(2, 6, 4, 2, 64, 3, 1)
    for kw in (dict(mask=None), dict(mask=P[8] + 2), dict(words=0), dict(words=-1), dict(out=P[8]),
               dict(ws=P[8]), dict(q=None), dict(kc=None), dict(out=None), dict(starts=None),
               dict(max_q=0), dict(H=3), dict(Hkv=0), dict(page=48), dict(layout=2),
               dict(scale=float("inf")), dict(dtype=4), dict(ws=None), dict(ws_n=n - 1),
               dict(out=P[0])):
        assert tree_fwd(mha, **kw) == mha.MHA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(page=4), dict(d=80), dict(T=1 << 30), dict(T=1 << 28, words=1 << 30)):
        assert tree_fwd(mha, **kw) == mha.MHA_ERR_UNSUPPORTED, kw
    for kw in (dict(T=0), dict(B=0), dict(H=0, Hkv=0)):
        assert tree_fwd(mha, mask=None, q=None, out=None, ws=None, ws_n=0, **kw) == mha.MHA_OK, kw


def test_bindings(recorded):  # noqa: F811
    mod, calls = recorded
    q, k, v = Fake((6, 4, 64)), Fake((6, 2, 64)), Fake((6, 2, 64))
    kc, vc = Fake((9, 32, 2, 64)), Fake((9, 32, 2, 64))
    batch = dict(q_starts=Fake((3,), "i32"), kv_lengths=Fake((2,), "i32"),
                 block_table=Fake((2, 5), "i32"), layout="bshd", stream=3)
    pos, mask = Fake((6,), "i32"), Fake((6, 2), "i32")
    mod.mha_paged_append_at(q, k, v, kc, vc, pos, Fake((6, 4, 64)), **batch)
    assert calls[-1][0] == "mha_paged_append_at" and calls[-1][1][13:21] == (2, 6, 4, 2, 64, 9, 32, 5)
    tree = dict(out=Fake((6, 4, 64)), max_q=3, workspace=Fake((4096,), "u8"))
    mod.mha_paged_tree_fwd(q, kc, vc, mask, **tree, **batch)
    assert calls[-1][0] == "mha_paged_tree_fwd"
    assert calls[-1][1][8:20] == (2, 6, 4, 2, 64, 3, 9, 32, 5, 2, 1, 0.125)
    for bad in (Fake((5,), "i32"), Fake((6,)), Fake((6, 1), "i32"),
                Fake((6,), "i32", device="cuda:1"), Fake((6,), "i32", contiguous=False)):
        with pytest.raises(ValueError):
            mod.mha_paged_append_at(q, k, v, kc, vc, bad, Fake((6, 4, 64)), **batch)
    for bad in (Fake((5, 2), "i32"), Fake((6, 2)), Fake((6,), "i32"), Fake((6, 0), "i32"),
                Fake((6, 2), "i32", device="cpu"), Fake((6, 2), "i32", contiguous=False)):
        with pytest.raises(ValueError):
            mod.mha_paged_tree_fwd(q, kc, vc, bad, **tree, **batch)


def test_masks_of_trees(mha):  # noqa: F811
    rng = np.random.default_rng(0)
    for n in (0, 1, 31, 32, 33, 70):
        parents = [int(rng.integers(-1, i)) for i in range(n)]
        rows, depth = mha.tree_mask(parents, device="cpu")
        assert rows.shape == (n, max(1, -(-n // 32))) and depth.shape == (n,)
        for i in range(n):
            chain, at = set(), i
            while at >= 0:
                chain.add(at)
                at = parents[at]
            assert {m for m in range(n) if tree_ref.bits(rows[i].tolist()) >> m & 1} == chain
            assert depth[i] == len(chain) - 1
        wide, _ = mha.tree_mask(parents, words=4, device="cpu")
        assert wide.shape == (n, 4) and (wide[:, rows.shape[1]:] == 0).all()
    for bad in ([0], [-1, 1], [-1, -2], [1, -1]):
        with pytest.raises(ValueError):
            mha.tree_mask(bad, device="cpu")
    with pytest.raises(ValueError):
        mha.tree_mask([-1] * 40, words=1, device="cpu")


def test_windows_of_a_row(tmp_path):
    """The 32 positions that a kernel looks at at a time, from any place, against bit by bit."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src, out = tmp_path / "w.cu", str(tmp_path / "w.so")
    src.write_text('''#include "paged.cuh"
extern "C" unsigned window(const unsigned *row, int words, int from) {
  return mha::tree_window(mha::tree_word(row, words, from >> 5),
                          mha::tree_word(row, words, (from >> 5) + 1), from);
}
''')
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-o",
                    out, str(src)], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.window.restype = ctypes.c_uint
    rng = np.random.default_rng(1)
    for words in (1, 2, 5):
        row = rng.integers(0, 2 ** 32, words).astype(np.uint32)
        number = tree_ref.bits(row)
        for start in list(range(-70, 32 * words + 70)) + [-2 ** 31, -2 ** 31 + 5, 2 ** 31 - 40]:
            got = lib.window(row.ctypes.data_as(ctypes.c_void_p), words, start)
            want = sum(1 << e for e in range(32)
                       if start + e < 0 or (start + e < 32 * words and number >> (start + e) & 1))
            assert got == want, (words, start)
    assert os.path.exists(out)
