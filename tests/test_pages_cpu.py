"""What of the page pool's operators runs without a GPU: refusals of the C entry points and
the bindings, and the kernels' integer logic (compiled for the host)."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest

import pages_ref
from test_paged_cpu import CSRC, P, Fake, mha, recorded  # noqa: F401


def reserve(mha, table=P[0], lens=P[1], new=P[2], par=P[3], refs=P[4], table_out=P[5], lens_out=P[6],  # noqa: F811
            refs_out=P[7], moves=P[8], counts=P[9], B_old=3, B=4, pages=20, page=16, max_pages=5,
            ws=P[10], ws_n=1 << 30):
    return mha.lib.mha_paged_reserve(table, lens, new, par, refs, table_out, lens_out, refs_out,
                                     moves, counts, B_old, B, pages, page, max_pages, ws, ws_n, None)


def test_reserve_rejects_before_launch(mha):  # noqa: F811
    n = mha.mha_paged_reserve_workspace_size(4, 20)
    assert n > 0 and n % 256 == 0
    assert mha.mha_paged_reserve_workspace_size(-1, 20) == 0
    assert mha.mha_paged_reserve_workspace_size(4, 2 ** 31 - 1) == 0
    for kw in (dict(B_old=-1), dict(B=-1), dict(pages=-1), dict(max_pages=-1), dict(page=0),
               dict(page=24), dict(table=None), dict(lens=None), dict(new=None), dict(refs=None),
               dict(table_out=None), dict(lens_out=None), dict(refs_out=None), dict(moves=None),
               dict(ws=None), dict(ws_n=n - 1), dict(ws=P[10] + 128), dict(table=P[0] + 2),
               dict(moves=P[8] + 1), dict(counts=P[9] + 3), dict(table_out=P[0]),
               dict(table_out=P[0] + 4), dict(lens_out=P[1]), dict(lens_out=P[2]),
               dict(moves=P[3]), dict(refs_out=P[4] + 4), dict(refs_out=P[5]), dict(counts=P[6]),
               dict(ws=P[0]), dict(par=P[8])):
        assert reserve(mha, **kw) == mha.MHA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(page=8), dict(page=1 << 20, max_pages=1 << 11), dict(pages=2 ** 31 - 1),
               dict(B=2 ** 31 - 1, max_pages=1), dict(B=1 << 16, max_pages=1 << 15),
               dict(B_old=1 << 16, max_pages=1 << 15)):
        assert reserve(mha, **kw) == mha.MHA_ERR_UNSUPPORTED, kw
    assert reserve(mha, B_old=0, B=0, pages=0, counts=None, ws=None, ws_n=512) == mha.MHA_OK


def copy(mha, k=P[0], v=P[1], moves=P[2], n=3, layers=2, Hkv=2, d=64, pages=9, page=16, dtype=1):  # noqa: F811
    return mha.lib.mha_paged_copy(k, v, moves, n, layers, Hkv, d, pages, page, dtype, None)


def test_copy_rejects_before_launch(mha):  # noqa: F811
    for kw in (dict(n=-1), dict(layers=-1), dict(Hkv=-1), dict(d=0), dict(pages=-1), dict(page=24),
               dict(dtype=2), dict(k=None), dict(v=None), dict(moves=None), dict(k=P[0] + 8),
               dict(moves=P[2] + 2), dict(k=P[1]), dict(v=P[2]), dict(v=P[0] + 16)):
        assert copy(mha, **kw) == mha.MHA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(page=8), dict(d=96), dict(n=2 ** 31 - 1), dict(pages=2 ** 31 - 1),
               dict(layers=2 ** 31 - 1, pages=1 << 30), dict(Hkv=2 ** 31 - 1, page=1 << 30),
               dict(layers=2 ** 30, pages=1)):
        assert copy(mha, **kw) == mha.MHA_ERR_UNSUPPORTED, kw
    for kw in (dict(n=0), dict(layers=0), dict(Hkv=0), dict(pages=0)):
        assert copy(mha, k=None, v=None, moves=None, **kw) == mha.MHA_OK, kw


def compact(mha, k=P[0], v=P[1], out=P[2], keep=P[3], counts=P[4], starts=P[5], lens=P[6], src=P[7],  # noqa: F811
            table=P[8], B=3, layers=2, Hkv=2, d=64, pages=9, page=16, max_pages=4, most=7, layout=0,
            dtype=1):
    return mha.lib.mha_paged_compact(k, v, out, keep, counts, starts, lens, src, table, B, layers,
                                     Hkv, d, pages, page, max_pages, most, layout, dtype, None)


def test_compact_rejects_before_launch(mha):  # noqa: F811
    for kw in (dict(B=-1), dict(layers=-1), dict(Hkv=-1), dict(d=-64), dict(pages=-1), dict(page=40),
               dict(max_pages=-1), dict(most=-1), dict(layout=2), dict(dtype=7), dict(k=None),
               dict(v=None), dict(out=None), dict(keep=None), dict(counts=None), dict(lens=None),
               dict(table=None), dict(k=P[0] + 8), dict(starts=P[5] + 2), dict(src=P[7] + 1),
               dict(out=P[6]), dict(out=P[5]), dict(out=P[4]), dict(out=P[3] + 80), dict(out=P[8]),
               dict(v=P[0]), dict(k=P[3]), dict(v=P[7]), dict(k=P[8])):
        assert compact(mha, **kw) == mha.MHA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(page=8), dict(d=32), dict(B=2 ** 31 - 1), dict(layers=2 ** 30, pages=1),
               dict(page=1 << 20, max_pages=1 << 11), dict(B=1 << 30, Hkv=0, layers=0),
               dict(pages=2 ** 31 - 1), dict(most=(1 << 30) + 1), dict(B=2 ** 31 - 1, Hkv=2 ** 31 - 1, layers=2 ** 31 - 1)):
        assert compact(mha, **kw) == mha.MHA_ERR_UNSUPPORTED, kw
    assert compact(mha, B=0, k=None, v=None, out=None, keep=None, counts=None, lens=None,
                   table=None) == mha.MHA_OK


def test_bindings(recorded):  # noqa: F811
    mod, calls = recorded
    i32 = lambda *s, **kw: Fake(s, "i32", **kw)  # noqa: E731
    ins = dict(block_table=i32(3, 5), kv_lengths=i32(3), new_lengths=i32(4), refs=i32(20))
    kw = dict(page_size=32, parents=i32(4), table_out=i32(4, 5), lengths_out=i32(4),
              refs_out=i32(20), moves=i32(4, 2), counts=i32(2), workspace=Fake((4096,), "u8"),
              stream=5)
    got = mod.mha_paged_reserve(*ins.values(), **kw)
    assert got == tuple(kw[x] for x in ("table_out", "lengths_out", "refs_out", "moves", "counts"))
    name, a = calls[-1]
    assert name == "mha_paged_reserve" and a[10:15] == (3, 4, 20, 32, 5) and a[-2:] == (4096, 5)
    for bad in (dict(kv_lengths=i32(4)), dict(block_table=i32(15)), dict(new_lengths=i32(4, 1)),
                dict(refs=i32(4, 5)), dict(refs=Fake((20,), "f32")),
                dict(kv_lengths=i32(3, device="cuda:1")), dict(block_table=i32(3, 5, contiguous=False))):
        with pytest.raises(ValueError):
            mod.mha_paged_reserve(*{**ins, **bad}.values(), **kw)
    for bad in (dict(parents=i32(3)), dict(table_out=i32(3, 5)), dict(lengths_out=i32(3)),
                dict(refs_out=i32(19)), dict(moves=i32(8)), dict(counts=i32(3)),
                dict(workspace=Fake((4096,), "u8", device="cpu")), dict(moves=Fake((4, 2), "f32"))):
        with pytest.raises(ValueError):
            mod.mha_paged_reserve(*ins.values(), **{**kw, **bad})

    for shape, layers in (((9, 32, 2, 64), 1), ((6, 9, 32, 2, 64), 6)):
        kc, vc = Fake(shape), Fake(shape)
        mod.mha_paged_copy(kc, vc, i32(7, 2), stream=1)
        assert calls[-1][1][3:10] == (7, layers, 2, 64, 9, 32, 1)
        lens = i32(3)
        c = dict(keep=i32(3, 8), keep_counts=i32(3), lengths_out=lens, starts=i32(3),
                 kv_lengths=i32(3), block_table=i32(3, 5), layout="bshd", stream=1)
        assert mod.mha_paged_compact(kc, vc, **c) is lens
        assert calls[-1][1][9:19] == (3, layers, 2, 64, 9, 32, 5, 8, 1, 1)
        assert calls[-1][1][7] is None
        mod.mha_paged_compact(kc, vc, **{**c, "src_table": i32(3, 5)})
        assert calls[-1][1][7] is not None
        for bad in (Fake(shape[:-1]), Fake(shape, "f32"), Fake(shape, device="cuda:1"),
                    Fake(shape, contiguous=False)):
            with pytest.raises(ValueError):
                mod.mha_paged_copy(kc, bad, i32(7, 2))
            with pytest.raises(ValueError):
                mod.mha_paged_compact(kc, bad, **c)
        for bad in (i32(7), i32(7, 3), Fake((7, 2), "f32")):
            with pytest.raises(ValueError):
                mod.mha_paged_copy(kc, vc, bad)
        for bad in (dict(keep=i32(24)), dict(keep_counts=i32(2)), dict(starts=i32(2)),
                    dict(kv_lengths=i32(4)), dict(block_table=i32(2, 5)), dict(block_table=i32(15)),
                    dict(src_table=i32(3, 6)), dict(lengths_out=i32(2)), dict(layout="hbsd"),
                    dict(keep=Fake((3, 8), "f32"))):
            with pytest.raises(ValueError):
                mod.mha_paged_compact(kc, vc, **{**c, **bad})
    with pytest.raises(TypeError):
        mod.mha_paged_copy(Fake((9, 32, 2, 64), "f16"), Fake((9, 32, 2, 64), "f16"), i32(7, 2))
    with pytest.raises(ValueError):
        mod.mha_paged_copy(Fake((2 ** 31, 32, 2, 64)), Fake((2 ** 31, 32, 2, 64)), i32(7, 2))


def test_rows_and_lengths_on_the_host(tmp_path):
    """What a row keeps and how far it reaches, as the kernels find it, against the plain form
    of one row at a time."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src, out = tmp_path / "r.cu", str(tmp_path / "r.so")
    src.write_text('''#include <cstring>
#include "pages.cuh"
using namespace mha;
extern "C" void row(const int *table, const int *lens, const int *new_lens, const int *parents,
                    int B_old, int pages, int shift, int width, int i, int got, int *out) {
  ReserveArgs a;
  std::memset(&a, 0, sizeof a);
  a.table = table; a.lens = lens; a.new_lens = new_lens; a.parents = parents;
  a.B_old = B_old; a.num_pages = pages; a.page_shift = shift; a.max_pages = width;
  const ReserveRow r = reserve_row(a, i);
  const int x[9] = {r.parent, r.keep, r.next, r.full, r.had, r.want, r.last,
                    reserve_length(a, r, false, got), reserve_length(a, r, true, got)};
  std::memcpy(out, x, sizeof x);
}
extern "C" int stands(int before, int k, int start, int len) {
  return compact_stands(before, k, start, len);
}
''')
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-o",
                    out, str(src)], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    rng = np.random.default_rng(0)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    for _ in range(400):
        width, page, pool, old = int(rng.integers(1, 6)), 16, 12, 3
        table = rng.integers(-2, pool + 2, (old, width)).astype(np.int32)
        lens = rng.integers(-20, 120, old).astype(np.int32)
        new = rng.integers(-20, 120, 4).astype(np.int32)
        par = rng.integers(-2, 5, 4).astype(np.int32)
        got = int(rng.integers(0, 8))
        res = np.zeros(9, dtype=np.int32)
        for i in range(4):
            lib.row(ptr(table), ptr(lens), ptr(new), ptr(par), old, pool, 4, width, i, got, ptr(res))
            cap = width * page
            p = int(par[i]) if 0 <= par[i] < old else -1
            n = min(max(int(lens[p]), 0), cap) if p >= 0 else 0
            nxt = min(max(int(new[i]), 0), cap)
            keep = min(n, nxt)
            had, want = -(-keep // page), -(-nxt // page)
            last = int(table[p, keep // page]) if keep % page else -1
            last = last if 0 <= last < pool else -1
            short = nxt if got >= want - had else (had + got) * page
            copy_ = nxt if got >= want - had + 1 else \
                (keep // page * page if got == 0 else (had + got - 1) * page)
            assert res.tolist() == [p, keep, nxt, keep // page, had, want, last, short, copy_]
    for _ in range(300):
        keep = np.sort(rng.integers(-1, 30, 6))
        if rng.random() < 0.5:
            rng.shuffle(keep)
        start, ln = int(rng.integers(0, 10)), int(rng.integers(10, 40))
        n = 0
        while n < 6 and lib.stands(int(keep[n - 1]) if n else -1, int(keep[n]), start, ln):
            n += 1
        assert n == pages_ref.stands(keep, 6, start, ln)


def test_the_plain_form_itself():
    """Sequences, forks and a copy, written out."""
    page = 16
    table = np.array([[3, 5, -1], [2, -1, -1]], np.int32)
    lens, refs = np.array([20, 16], np.int32), np.array([0, 0, 1, 1, 0, 1], np.int32)
    # row 0 goes on; rows 1 and 2 fork from it; the old row 1 ends
    t, ln, r, m, c = pages_ref.reserve(table, lens, np.array([21, 20, 40], np.int32),
                                       np.array([0, 0, 0], np.int32), refs, page)
    assert t.tolist() == [[3, 5, -1], [3, 0, -1], [3, 1, 2]]
    assert ln.tolist() == [21, 20, 40] and r.tolist() == [1, 1, 1, 3, 0, 1]
    assert m.tolist() == [[-1, -1], [5, 0], [5, 1]] and c.tolist() == [3, 1]
    # no page is left for the last one's third
    t, ln, r, m, c = pages_ref.reserve(table, lens, np.array([21, 33, 48], np.int32), None,
                                       np.array([9, 9, 1, 1, 0, 1], np.int32), page)
    assert t.tolist() == [[3, 5, -1], [2, 4, -1], [-1, -1, -1]]
    assert ln.tolist() == [21, 32, 0] and c.tolist() == [1, 0]
