"""What of the paged operators runs without a GPU: refusals of the C entry points
and of the bindings, the split of attention work over CTAs and the lookup of
positions (the kernels' own code, compiled for the host), and the plain forms
that the GPU tests compare with."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import paged_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_head_scaled_mha_gb300", "csrc")
FAKE = 0x7F0000000000  # never dereferenced: every call below ends in validation


@pytest.fixture(scope="module")
def mha():
    import __graft_entry__
    __graft_entry__._load_build_module().build()
    import transformer_head_scaled_mha_gb300 as m
    return m


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-o",
                    out, os.path.join(ROOT, "tests", "paged_split_host.cu")], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(out)
    lib.cell.restype = ctypes.c_longlong
    return lib


def i32(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def declared():
    src = open(os.path.join(ROOT, "include", "mha_paged.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(mha_\w+)\s*\(", src)))


def test_header_library_and_binding_agree(mha):
    from transformer_head_scaled_mha_gb300 import paged
    assert declared() == sorted(paged.EXPORTED)
    lib = ctypes.CDLL(mha.LIB_PATH)
    for name in declared():
        assert hasattr(lib, name), name
        assert hasattr(mha, name), name
    src = open(os.path.join(ROOT, "include", "mha_paged.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    for name in declared():  # the binding passes as many arguments as the header declares
        args = re.search(name + r"\s*\(([^)]*)\)", src).group(1)
        assert len(args.split(",")) == len(getattr(mha.lib, name).argtypes), name


P = [FAKE + (i << 32) for i in range(16)]


def rope_fwd(mha, q=P[0], k=P[1], qo=P[2], ko=P[3], qw=P[4], kw=P[5], pos=P[6], freq=P[7], B=2,
             H=4, Hkv=2, L=8, d=64, rot=64, layout=0, style=0, eps=1e-6, dtype=1):
    return mha.lib.mha_qk_norm_rope_fwd(q, k, qo, ko, qw, kw, pos, freq, B, H, Hkv, L, d, rot,
                                        layout, style, eps, dtype, None)


def test_rope_rejects_before_launch(mha):
    E_ARG, E_UNS = mha.MHA_ERR_INVALID_ARGUMENT, mha.MHA_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(H=-1), dict(Hkv=-1), dict(L=-1), dict(d=0), dict(layout=2),
               dict(style=2), dict(dtype=2), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(rot=-16), dict(rot=80), dict(q=None), dict(ko=None),
               dict(freq=None), dict(q=P[0] + 8), dict(pos=P[6] + 2), dict(freq=P[7] + 1),
               dict(qw=P[4] + 4), dict(qo=P[0] + 16), dict(qo=P[1]), dict(ko=P[0]),
               dict(ko=P[2] + 64), dict(qo=P[6]), dict(ko=P[7]), dict(qo=P[4]), dict(qo=P[5])):
        assert rope_fwd(mha, **kw) == E_ARG, kw
    for kw in (dict(d=96), dict(d=256), dict(rot=24), dict(B=1 << 16, L=1 << 15), dict(B=1, L=(1 << 31) - 1000),
               dict(H=1 << 30, Hkv=0, B=1 << 10, L=1 << 20)):
        assert rope_fwd(mha, **kw) == E_UNS, kw
    for kw in (dict(B=0), dict(L=0), dict(H=0, Hkv=0)):
        assert rope_fwd(mha, q=None, k=None, qo=None, ko=None, **kw) == mha.MHA_OK, kw


def rope_bwd(mha, q=P[0], k=P[1], gq=P[2], gk=P[3], dq=P[4], dk=P[5], dqw=P[6], dkw=P[7], qw=P[8],
             kw=P[9], pos=P[10], freq=P[11], B=2, H=4, Hkv=2, L=8, d=64, rot=64, layout=0, style=0,
             eps=1e-6, dtype=1, ws=P[12], ws_n=None):
    ws_n = mha.mha_qk_norm_rope_bwd_workspace_size(d) if ws_n is None else ws_n
    return mha.lib.mha_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dqw, dkw, qw, kw, pos, freq, B, H,
                                        Hkv, L, d, rot, layout, style, eps, dtype, ws, ws_n, None)


def test_rope_bwd_rejects_before_launch(mha):
    E_ARG, E_UNS = mha.MHA_ERR_INVALID_ARGUMENT, mha.MHA_ERR_UNSUPPORTED
    n = mha.mha_qk_norm_rope_bwd_workspace_size(64)
    assert n > 0 and n % 256 == 0 and mha.mha_qk_norm_rope_bwd_workspace_size(96) == 0
    for kw in (dict(B=-1), dict(layout=3), dict(style=-1), dict(dtype=5), dict(eps=-0.5),
               dict(rot=65), dict(q=None), dict(gk=None), dict(dq=None), dict(dqw=None),
               dict(kw=None), dict(ws=None), dict(ws_n=n - 1), dict(ws=P[12] + 128),
               dict(dq=P[2] + 32), dict(dq=P[0]), dict(dk=P[2]), dict(dk=P[4]), dict(ws=P[0]),
               dict(dqw=P[8]), dict(dkw=P[6]), dict(dqw=P[6] + 4), dict(freq=None),
               dict(dq=P[10])):
        assert rope_bwd(mha, **kw) == E_ARG, kw
    for kw in (dict(d=32, rot=32), dict(rot=8), dict(B=1 << 16, L=1 << 15)):
        assert rope_bwd(mha, **kw) == E_UNS, kw
    assert rope_bwd(mha, B=0, dqw=None, dkw=None, qw=None, kw=None) == mha.MHA_OK


def append(mha, q=P[0], k=P[1], v=P[2], qo=P[3], kc=P[4], vc=P[5], qw=P[6], kw=P[7], freq=P[8],
           starts=P[9], lens=P[10], table=P[11], B=2, T=6, H=4, Hkv=2, d=64, pages=9, page=16,
           max_pages=3, rot=64, layout=0, style=0, eps=1e-6, dtype=1):
    return mha.lib.mha_paged_append(q, k, v, qo, kc, vc, qw, kw, freq, starts, lens, table, B, T, H,
                                    Hkv, d, pages, page, max_pages, rot, layout, style, eps, dtype,
                                    None)


def test_append_rejects_before_launch(mha):
    E_ARG, E_UNS = mha.MHA_ERR_INVALID_ARGUMENT, mha.MHA_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(T=-1), dict(H=3), dict(Hkv=-2), dict(Hkv=0), dict(pages=-1),
               dict(max_pages=-1), dict(page=0), dict(page=24), dict(page=-16), dict(layout=2),
               dict(style=7), dict(dtype=9), dict(eps=math.nan), dict(rot=66), dict(q=None),
               dict(k=None), dict(v=None), dict(qo=None), dict(kc=None), dict(freq=None),
               dict(starts=None), dict(lens=None), dict(table=None), dict(starts=P[9] + 2),
               dict(kc=P[4] + 8), dict(kc=P[5]), dict(kc=P[1]), dict(vc=P[2]), dict(qo=P[1]),
               dict(qo=P[0] + 16), dict(qo=P[4]), dict(kc=P[11]), dict(vc=P[10])):
        assert append(mha, **kw) == E_ARG, kw
    for kw in (dict(page=8), dict(d=96), dict(rot=8), dict(pages=(1 << 31) - 1, page=1 << 30),
               dict(B=(1 << 31) - 1, max_pages=(1 << 31) - 1)):
        assert append(mha, **kw) == E_UNS, kw
    for kw in (dict(T=0), dict(B=0), dict(H=0, Hkv=0)):
        assert append(mha, **kw) == mha.MHA_OK, kw


def paged(mha, q=P[0], kc=P[1], vc=P[2], out=P[3], starts=P[4], lens=P[5], table=P[6], B=2, T=6,
          H=4, Hkv=2, d=64, max_q=3, pages=9, page=16, max_pages=3, layout=0, mask=8, scale=0.125,
          dtype=1, ws=P[7], ws_n=1 << 31):
    return mha.lib.mha_paged_fwd(q, kc, vc, out, starts, lens, table, B, T, H, Hkv, d, max_q,
                                 pages, page, max_pages, layout, mask, scale, dtype, ws, ws_n, None)


def test_paged_fwd_rejects_before_launch(mha):
    E_ARG, E_UNS = mha.MHA_ERR_INVALID_ARGUMENT, mha.MHA_ERR_UNSUPPORTED
    n = mha.mha_paged_workspace_size(2, 6, 4, 2, 64, 3, 1)
    assert n > 0
    for kw in (dict(B=-1), dict(T=-1), dict(H=-4), dict(H=3), dict(Hkv=0), dict(Hkv=-1),
               dict(max_q=0), dict(pages=-1), dict(page=48), dict(max_pages=-1), dict(layout=2),
               dict(mask=1), dict(mask=2), dict(mask=10), dict(scale=math.inf), dict(dtype=4),
               dict(q=None), dict(kc=None), dict(vc=None), dict(out=None), dict(starts=None),
               dict(lens=None), dict(table=None), dict(ws=None), dict(ws=P[7] + 16),
               dict(ws_n=n - 1), dict(out=P[0]), dict(out=P[0] + 16), dict(out=P[1]),
               dict(out=P[6]), dict(ws=P[0]), dict(ws=P[2]), dict(out=P[3] + 8),
               dict(lens=P[5] + 1)):
        assert paged(mha, **kw) == E_ARG, kw
    for kw in (dict(page=4), dict(d=80), dict(T=1 << 30), dict(B=1 << 30),
               dict(pages=(1 << 31) - 1, page=1 << 30),
               # positions, rounded up to whole tiles of keys, stay below 2^31
               dict(page=1 << 20, max_pages=1 << 11), dict(page=16, max_pages=(1 << 27) - 63)):
        assert paged(mha, **kw) == E_UNS, kw
    for kw in (dict(T=0), dict(B=0), dict(H=0, Hkv=0), dict(H=0),
               dict(T=0, page=16, max_pages=(1 << 27) - 64)):
        assert paged(mha, q=None, out=None, ws=None, ws_n=0, **kw) == mha.MHA_OK, kw


def test_paged_path_and_workspace_sizes(mha):
    path, size = mha.mha_paged_path, mha.mha_paged_workspace_size
    assert path(0, 4, 8, 8, 64, 1, 16, 1) == 0
    assert path(4, 4, 8, 8, 64, 1, 16, 0) == 1 and path(4, 4, 32, 4, 64, 2, 16, 1) == 2
    assert path(4, 9, 32, 4, 64, 3, 16, 1) == 3 and path(4, 9, 32, 4, 64, 3, 16, 0) == 1
    assert path(4, 4, 8, 3, 64, 1, 16, 1) == -1
    assert path(4, 4, 8, 8, 64, 0, 16, 1) == -1
    assert path(4, 4, 8, 8, 64, 1, 24, 1) == -1
    assert path(4, 4, 8, 8, 64, 1, 8, 1) == -2
    assert path(4, 4, 8, 8, 96, 1, 16, 1) == -2
    assert size(0, 4, 8, 8, 64, 1, 1) == 0 and size(4, 4, 8, 3, 64, 1, 1) == 0
    for dt in (0, 1):
        for max_q in (1, 5, 400):
            for H, Hkv in ((8, 8), (32, 8), (32, 1), (6, 2), (256, 1)):
                n = size(4, 4, H, Hkv, 128, max_q, dt)
                assert 0 < n < 1 << 28 and n % 256 == 0


# ---------------------------------------------------------------------------
# bindings
# ---------------------------------------------------------------------------
class Fake:
    """A CUDA tensor as the bindings see it; nothing is dereferenced."""

    def __init__(self, shape, dtype="bf16", device="cuda:0", contiguous=True, ptr=FAKE):
        import torch
        self.shape = torch.Size(shape)
        self.dtype = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32,
                      "u8": torch.uint8, "f16": torch.float16}[dtype]
        self.device = torch.device(device)
        self.is_cuda = self.device.type == "cuda"
        self._contiguous, self._ptr = contiguous, ptr

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return self._ptr

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def recorded(mha, monkeypatch):
    """The bindings on a library that records each call's arguments."""
    import torch
    from transformer_head_scaled_mha_gb300 import paged as mod
    calls = []

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                calls.append((name, args))
                return 0
            return fn
    real = mod.lib
    monkeypatch.setattr(mod, "lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    yield mod, calls
    for name, args in calls:
        assert len(args) == len(getattr(real, name).argtypes), name


def test_rope_binding(recorded):
    mod, calls = recorded
    q, k = Fake((2, 8, 4, 64)), Fake((2, 8, 2, 64))
    good = dict(q_out=Fake((2, 8, 4, 64)), k_out=Fake((2, 8, 2, 64)), q_weight=Fake((64,)),
                k_weight=Fake((64,)), positions=Fake((2, 8), "i32"), inv_freq=Fake((16,), "f32"),
                layout="bshd", interleaved=True, eps=1e-5, stream=7)
    mod.mha_qk_norm_rope_fwd(q, k, **good)
    name, a = calls[-1]
    assert name == "mha_qk_norm_rope_fwd" and a[8:16] == (2, 4, 2, 8, 64, 32, 1, 1) and a[-1] == 7
    for bad in (dict(q_out=Fake((2, 8, 2, 64))), dict(k_out=Fake((2, 8, 2, 64), "f32")),
                dict(q_weight=Fake((32,))), dict(k_weight=Fake((64,), "f32")),
                dict(positions=Fake((2, 9), "i32")), dict(positions=Fake((2, 8), "f32")),
                dict(inv_freq=Fake((16,), "bf16")), dict(layout="sbhd"),
                dict(q_out=Fake((2, 8, 4, 64), device="cuda:1")),
                dict(inv_freq=Fake((16,), "f32", device="cpu")),
                dict(k_out=Fake((2, 8, 2, 64), contiguous=False))):
        with pytest.raises(ValueError):
            mod.mha_qk_norm_rope_fwd(q, k, **{**good, **bad})
    for bad_k in (Fake((2, 9, 2, 64)), Fake((2, 8, 2, 128)), Fake((2, 8, 2, 64), "f32")):
        with pytest.raises(ValueError):
            mod.mha_qk_norm_rope_fwd(q, bad_k, **good)
    with pytest.raises(TypeError):
        mod.mha_qk_norm_rope_fwd(Fake((2, 8, 4, 64), "f16"), None, stream=0)
    with pytest.raises(ValueError):
        mod.mha_qk_norm_rope_fwd(None, None)
    gq, gk = Fake((2, 8, 4, 64)), Fake((2, 8, 2, 64))
    kw = dict(good, dq=Fake((2, 8, 4, 64)), dk=Fake((2, 8, 2, 64)), dq_weight=Fake((64,), "f32"),
              dk_weight=Fake((64,), "f32"), workspace=Fake((1 << 20,), "u8"))
    kw.pop("q_out"), kw.pop("k_out")
    calls.clear()
    import torch
    import contextlib
    mod._on = lambda stream, device: contextlib.nullcontext()
    mod.mha_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    assert calls[-1][1][12:20] == (2, 4, 2, 8, 64, 32, 1, 1)
    for bad in (dict(dq_weight=Fake((64,))), dict(dq=Fake((2, 8, 4, 64), "f32")),
                dict(q_weight=None), dict(workspace=Fake((1 << 20,), "u8", device="cuda:1"))):
        with pytest.raises(ValueError):
            mod.mha_qk_norm_rope_bwd(q, k, gq, gk, **{**kw, **bad})
    with pytest.raises(ValueError):
        mod.mha_qk_norm_rope_bwd(None, k, gq, gk, **kw)
    assert torch is not None


def test_paged_bindings(recorded):
    mod, calls = recorded
    q, k, v = Fake((6, 4, 64)), Fake((6, 2, 64)), Fake((6, 2, 64))
    kc, vc = Fake((9, 32, 2, 64)), Fake((9, 32, 2, 64))
    batch = dict(q_starts=Fake((3,), "i32"), kv_lengths=Fake((2,), "i32"),
                 block_table=Fake((2, 5), "i32"), layout="bshd", stream=3)
    more = dict(q_out=Fake((6, 4, 64)), q_weight=Fake((64,)), inv_freq=Fake((32,), "f32"))
    mod.mha_paged_append(q, k, v, kc, vc, **more, **batch)
    assert calls[-1][1][12:22] == (2, 6, 4, 2, 64, 9, 32, 5, 64, 1)
    assert mod.mha_paged_append(None, k, v, kc, vc, **batch) is None
    assert calls[-1][1][0] is None and calls[-1][1][14] == 0
    paged_kw = dict(out=Fake((6, 4, 64)), max_q=3, workspace=Fake((4096,), "u8"))
    mod.mha_paged_fwd(q, kc, vc, **paged_kw, **batch)
    assert calls[-1][1][7:18] == (2, 6, 4, 2, 64, 3, 9, 32, 5, 1, 8)
    assert calls[-1][1][-2] == 4096
    for bad in (dict(q_starts=Fake((2,), "i32")), dict(kv_lengths=Fake((3,), "i32")),
                dict(block_table=Fake((10,), "i32")), dict(block_table=Fake((2, 5), "f32")),
                dict(kv_lengths=Fake((2,), "i32", device="cuda:1"))):
        with pytest.raises(ValueError):
            mod.mha_paged_append(q, k, v, kc, vc, **more, **{**batch, **bad})
        with pytest.raises(ValueError):
            mod.mha_paged_fwd(q, kc, vc, **paged_kw, **{**batch, **bad})
    for bad_kc in (Fake((9, 32, 2, 128)), Fake((9, 32, 2, 64), "f32"), Fake((9, 64, 64)),
                   Fake((9, 32, 2, 64), contiguous=False)):
        with pytest.raises(ValueError):
            mod.mha_paged_append(q, k, v, bad_kc, vc, **more, **batch)
        with pytest.raises(ValueError):
            mod.mha_paged_fwd(q, bad_kc, vc, **paged_kw, **batch)
    for bad in (dict(out=Fake((6, 2, 64))), dict(workspace=Fake((4096,), "u8", device="cpu"))):
        with pytest.raises(ValueError):
            mod.mha_paged_fwd(q, kc, vc, **{**paged_kw, **bad}, **batch)


# ---------------------------------------------------------------------------
# the split of attention work
# ---------------------------------------------------------------------------
SIMT, FEW, MANY = range(3)  # the kernels' ways to split


def all_parts(host, starts, lens, H, Hkv, hpu, tb, causal, page_shift, max_pages, grid, which=FEW):
    (s, sp), (ln, lp) = i32(starts), i32(lens)
    out = np.zeros((400000, 11), dtype=np.int32)
    n = host.parts(sp, lp, len(lens), int(s[-1]), H, Hkv, hpu, tb, causal,
                   page_shift, max_pages, grid, which, out.ctypes.data_as(ctypes.c_void_p), len(out))
    assert n >= 0
    return out[:n]


def check_split(host, starts, lens, H, Hkv, hpu, tb, causal, page_shift, max_pages, grid,
                which=FEW):
    """Every key tile of every unit is taken once, in order, by neighbouring CTAs;
    no CTA needs more than its two slots; every row of every sequence has a unit."""
    rows = all_parts(host, starts, lens, H, Hkv, hpu, tb, causal, page_shift, max_pages, grid,
                     which)
    units = {}
    slots = set()
    load = np.zeros(grid, dtype=np.int64)
    for c, b, i0, i1, h0, heads, kv, nt, t0, t1, slot in rows.tolist():
        assert 0 <= t0 <= t1 <= nt and heads >= 1 and h0 // (H // Hkv) == kv
        assert (h0 + heads - 1) // (H // Hkv) == kv
        units.setdefault((b, i0, h0), []).append((c, i1, heads, nt, t0, t1, slot))
        load[c] += (8 if which == MANY else 3) + 2 * (t1 - t0)
        if slot >= 0:
            assert (c, slot) not in slots
            slots.add((c, slot))
    cap = max_pages << page_shift
    want = 0
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        want += n * H
        base, ln = lens[b] - n, min(lens[b], cap)
        for (bb, i0, h0), parts in units.items():
            if bb != b:
                continue
            c, i1, heads, nt = parts[0][:4]
            want -= (i1 - i0) * heads
            end = max(min(base + i1, ln), 0) if causal else ln
            assert nt == -(-end // 128)
            at = 0
            for k, (ck, _, _, _, t0, t1, slot) in enumerate(parts):
                assert ck == c + k and t0 == at and (t1 > t0 or nt == 0)
                at = t1
                assert slot == (-1 if len(parts) == 1 else 1 if k == 0 else 0)
            assert at == nt
    assert want == 0
    return load


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("which", [SIMT, FEW, MANY])
@pytest.mark.parametrize("seed", range(12))
def test_every_tile_is_taken_once(host, seed, which, causal):
    rng = np.random.default_rng(seed)
    for _ in range(12):
        B = int(rng.integers(1, 40))
        most = int(rng.choice([1, 3, 40]))
        n = rng.integers(0, most + 1, B)
        lens = np.maximum(rng.integers(0, int(rng.choice([5, 300, 9000])), B) +
                          n * rng.integers(0, 2, B), 0)
        starts = np.concatenate([[0], np.cumsum(n)])
        Hkv = int(rng.choice([1, 2, 8]))
        group = int(rng.choice([1, 3, 4, 20]))
        hpu = min(group, 16)
        tb = int(rng.integers(1, (256 if which == MANY else 16) // hpu + 1))
        shift = int(rng.choice([4, 6, 9]))
        max_pages = max(1, -(-int(lens.max()) >> shift) - int(rng.integers(0, 2)))
        grid = int(rng.choice([1, 2, 7, 152, 456]))
        check_split(host, starts.tolist(), lens.tolist(), group * Hkv, Hkv, hpu, tb, causal, shift,
                    max_pages, grid, which)


@pytest.mark.parametrize("which", [SIMT, FEW, MANY])
def test_a_unit_over_many_ctas(host, which):
    # one unit as long as the grid and longer, alone and among empty ones
    for tiles in (1, 2, 3, 4, 5, 7, 100, 151, 152, 153, 157, 300, 304, 305, 700, 2000):
        for grid in (2, 152, 304, 608):
            for off in (0, 1, 127):
                ln = tiles * 128 - off
                check_split(host, [0, 1], [ln], 2, 1, 2, 1, 1, 4, -(-ln // 16), grid, which)
                check_split(host, list(range(43)), [0] * 20 + [ln] + [0] * 20 + [ln // 3], 2, 1, 2,
                            1, 1, 4, -(-ln // 16), grid, which)


def test_split_balances_long_and_short_sequences(host):
    # one sequence of 20000 keys among 31 short ones: no CTA does much more than the mean
    lens = [20000] + [200] * 31
    load = check_split(host, list(range(33)), lens, 8, 8, 1, 1, 1, 4, 1250, 152)
    assert load.max() <= 2 * load.sum() / 152
    # a single token over a long cache uses every CTA
    load = check_split(host, [0, 1], [65536], 8, 2, 4, 1, 1, 6, 1024, 152)
    assert (load > 0).all()
    # one short sequence: a CTA per head, nothing split
    load = check_split(host, [0, 1], [300], 8, 8, 1, 1, 1, 4, 20, 152)
    assert (load > 0).sum() == 8


def test_slots_of_sums_are_aligned(host):
    # 16-byte accesses at row and column multiples of 4 floats
    host.slot_floats.restype = ctypes.c_longlong
    for rows in range(1, 257):
        for d in (64, 128):
            n = host.slot_floats(rows, d)
            assert n % 4 == 0 and rows * (d + 2) <= n < rows * (d + 2) + 4


def test_empty_units_are_taken_once(host):
    # no keys at all, and tokens before the first position: zeros to write
    check_split(host, [0, 3, 3, 9], [0, 0, 2], 4, 2, 2, 8, 1, 4, 4, 5)
    check_split(host, [0, 3, 3, 9], [0, 0, 2], 4, 2, 2, 8, 0, 4, 0, 5)
    rows = all_parts(host, [0, 0, 0], [5, 7], 4, 2, 2, 8, 1, 4, 4, 5)
    assert len(rows) == 0


def test_unit_lengths_have_their_closed_form(host):
    rng = np.random.default_rng(5)
    for _ in range(3000):
        n = int(rng.choice([0, 1, 7, 130, 3000]))
        ln = int(rng.integers(0, int(rng.choice([2, 400, 5000])) + 1))
        max_pages = int(rng.choice([0, 3, 400]))
        (a, ap), (l, lp) = i32([0, n]), i32([ln])
        for causal in (0, 1):
            for split in (SIMT, FEW, MANY):
                assert host.unit_sums(ap, lp, n, int(rng.integers(1, 300)), causal, 4, max_pages,
                                      split) == 0


@pytest.mark.parametrize("causal", [0, 1])
def test_chunks_are_split_evenly(host, causal):
    # units of 256 rows: a long prompt from its beginning, and chunks behind caches
    load = check_split(host, [0, 8192], [8192], 16, 16, 1, 256, causal, 7, 64, 152, MANY)
    assert load.max() <= 1.25 * load.sum() / 152
    load = check_split(host, [0, 512, 600, 601], [4096, 3000, 2500], 32, 8, 4, 64, causal, 6, 64, 152,
                       MANY)
    assert load.max() <= 1.4 * load.sum() / 152


def test_lengths_out_of_range_are_clamped(host):
    out = np.zeros(4, dtype=np.int32)
    op = out.ctypes.data_as(ctypes.c_void_p)

    def seq(starts, lens, T, max_pages=4):
        (a, ap), (l, lp) = i32(starts), i32(lens)
        host.seq(ap, lp, T, 4, max_pages, 0, op)
        return out.tolist()
    assert seq([0, 5], [30], 10) == [0, 5, 30, 25]
    assert seq([-7, 5], [30], 10) == [0, 5, 30, 25]     # rows before the buffer
    assert seq([8, 50], [30], 10) == [8, 2, 30, 28]     # rows past it
    assert seq([50, 60], [30], 10) == [10, 0, 30, 30]
    assert seq([6, 2], [30], 10) == [6, 0, 30, 30]      # decreasing
    assert seq([0, 5], [-3], 10) == [0, 5, 0, -5]
    assert seq([0, 5], [2 ** 31 - 1], 10) == [0, 5, 64, 2 ** 31 - 6]
    assert seq([0, 5], [30], 10, max_pages=0) == [0, 5, 0, 25]
    assert seq([-2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1], 10, 2 ** 31 - 1)[:3] == [0, 10, 2 ** 31 - 1]


def test_cells_of_bad_pages_are_absent(host):
    pages, shift, max_pages, heads = 7, 4, 3, 2
    table = np.array([[5, -1, 6], [7, 0, 2 ** 31 - 1], [-2 ** 31, 3, 1]], dtype=np.int32)
    (t, tp) = i32(table)

    def cell(layout, b, pos, head):
        return host.cell(tp, pages, shift, max_pages, layout, b, pos, head, heads)
    for layout in (0, 1):
        for b in range(3):
            for pos in list(range(-3, 60)) + [2 ** 31 - 1, -2 ** 31]:
                for head in range(heads):
                    got = cell(layout, b, pos, head)
                    page = pos // 16
                    ok = 0 <= pos < 48 and 0 <= table[b, page] < pages
                    if not ok:
                        assert got == -1
                        continue
                    idx = (table[b, page], head, pos % 16) if layout == 0 else \
                        (table[b, page], pos % 16, head)
                    shape = (pages, heads, 16) if layout == 0 else (pages, 16, heads)
                    assert got == np.ravel_multi_index(idx, shape)
    # a cache of more than 2^31 rows: 64-bit
    big = np.array([[2 ** 28]], dtype=np.int32)
    (t, tp) = i32(big)
    assert host.cell(tp, 2 ** 29, 7, 1, 0, 0, 3, 1, 2) == ((2 ** 28 * 2 + 1) << 7) + 3


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 64])
def test_plain_gradient_against_differences(rotary, interleaved):
    rng = np.random.default_rng(3)
    x, w, dy = rng.normal(size=(5, 64)), 1 + 0.1 * rng.normal(size=64), rng.normal(size=(5, 64))
    pos = np.array([0, 1, 7, 100, 5000])
    freq = 10000.0 ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))
    f = lambda a, b: (ref.norm_rope(a, b, pos, freq, interleaved, 1e-6) * dy).sum()  # noqa: E731
    dx, dw = ref.norm_rope_bwd(x, w, dy, pos, freq, interleaved, 1e-6)
    h = 1e-6
    for i, j in [(0, 0), (1, 5), (2, 33), (3, 63), (4, 16)]:
        step = np.zeros_like(x)
        step[i, j] = h
        assert (f(x + step, w) - f(x - step, w)) / (2 * h) == pytest.approx(dx[i, j], abs=1e-7)
    for j in (0, 15, 40):
        step = np.zeros_like(w)
        step[j] = h
        assert (f(x, w + step) - f(x, w - step)) / (2 * h) == pytest.approx(dw[j], abs=1e-7)


def test_plain_paged_attention_against_the_oracle(oracle_lib):
    rng = np.random.default_rng(4)
    B, H, Hkv, n, L, d, page = 3, 4, 2, 3, 50, 64, 16
    q = rng.normal(size=(B, n, H, d)).astype(np.float32)
    k, v = (rng.normal(size=(B, L, Hkv, d)).astype(np.float32) for _ in range(2))
    lens = np.array([50, 17, 2], dtype=np.int32)
    want = oracle_lib.mha_fwd(q, k, v, mask_kind=10, key_lengths=lens, scale=0.125, layout="bshd")
    table = rng.permutation(B * 4).reshape(B, 4).astype(np.int32)
    for layout in ("bshd", "bhsd"):
        caches = []
        for t in (k, v):
            c = np.zeros((B * 4, page, Hkv, d))
            for b in range(B):
                for j in range(L):
                    c[table[b, j // page], j % page] = t[b, j]
            caches.append(c if layout == "bshd" else c.transpose(0, 2, 1, 3))
        got, tol = ref.paged_attention(
            q.reshape(B * n, H, d).astype(np.float64), *caches, np.arange(B + 1) * n, lens, table,
            np.zeros((B * n, H, d)), page=page, layout=layout, causal=True, scale=0.125,
            dtype="f32")
        np.testing.assert_allclose(got.reshape(want.shape), want, atol=1e-9)
        assert (tol < 2e-4).all()  # the bound says something
