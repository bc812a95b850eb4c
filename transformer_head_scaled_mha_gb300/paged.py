"""Python binding of the C ABI in include/mha_paged.h (ctypes; argument marshalling only).

The per-head norm and position rotation of queries and keys with its gradients,
the paged key/value cache and the attention over it, for trees of drafted tokens
too, and the page pool under it.  Same library, same errors
and same conventions as ``mha.py``: torch CUDA tensors in, nothing computed here.
Where binding.cpp is built it checks the tensors and makes the calls, those of a
generation step whole where the caller brings the results along; what is refused, and
how, stays the same.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os

from . import _build
from .mha import (MHA_DTYPE_BF16, MHA_DTYPE_F32, MHA_LAYOUT_BHSD, MHA_LAYOUT_BSHD,
                  MHA_MASK_CAUSAL_TAIL, MHA_OK, MhaError, lib)

MHA_ROPE_HALVES, MHA_ROPE_INTERLEAVED = 0, 1
PAGED_PATH_NAMES = {0: "none", 1: "paged_simt", 2: "paged_few_tc", 3: "paged_many_tc"}

_INT_MAX = 0x7fffffff

EXPORTED = ("mha_qk_norm_rope_fwd", "mha_qk_norm_rope_bwd_workspace_size", "mha_qk_norm_rope_bwd",
            "mha_paged_append", "mha_paged_append_at", "mha_paged_workspace_size", "mha_paged_fwd",
            "mha_paged_tree_fwd", "mha_paged_path", "mha_paged_reserve_workspace_size",
            "mha_paged_reserve", "mha_paged_copy", "mha_paged_compact")


def _declare() -> None:
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    numbers = [i32] * 8 + [f32, i32]  # B, H, H_kv, L, d, rotary_dim, layout, style, eps, dtype
    lib.mha_qk_norm_rope_fwd.restype = i32
    lib.mha_qk_norm_rope_fwd.argtypes = [vp] * 8 + numbers + [vp]
    lib.mha_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.mha_qk_norm_rope_bwd_workspace_size.argtypes = [i32]
    lib.mha_qk_norm_rope_bwd.restype = i32
    lib.mha_qk_norm_rope_bwd.argtypes = [vp] * 12 + numbers + [vp, sz, vp]
    lib.mha_paged_append.restype = i32
    lib.mha_paged_append.argtypes = [vp] * 12 + [i32] * 11 + [f32, i32, vp]
    lib.mha_paged_append_at.restype = i32
    lib.mha_paged_append_at.argtypes = [vp] * 13 + [i32] * 11 + [f32, i32, vp]
    lib.mha_paged_workspace_size.restype = sz
    lib.mha_paged_workspace_size.argtypes = [i32] * 7
    lib.mha_paged_fwd.restype = i32
    lib.mha_paged_fwd.argtypes = [vp] * 7 + [i32] * 11 + [f32, i32, vp, sz, vp]
    lib.mha_paged_tree_fwd.restype = i32
    lib.mha_paged_tree_fwd.argtypes = [vp] * 8 + [i32] * 11 + [f32, i32, vp, sz, vp]
    lib.mha_paged_path.restype = i32
    lib.mha_paged_path.argtypes = [i32] * 8
    lib.mha_paged_reserve_workspace_size.restype = sz
    lib.mha_paged_reserve_workspace_size.argtypes = [i32] * 2
    lib.mha_paged_reserve.restype = i32
    lib.mha_paged_reserve.argtypes = [vp] * 10 + [i32] * 5 + [vp, sz, vp]
    lib.mha_paged_copy.restype = i32
    lib.mha_paged_copy.argtypes = [vp] * 3 + [i32] * 7 + [vp]
    lib.mha_paged_compact.restype = i32
    lib.mha_paged_compact.argtypes = [vp] * 9 + [i32] * 10 + [vp]


_declare()


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, device="cuda"):
    """The usual frequencies base^(-2 i / rotary_dim), i < rotary_dim / 2, as the
    float32 tensor ``inv_freq`` that the operators take."""
    import torch
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    return (float(base) ** (-2.0 * i / rotary_dim)).float().to(device)


def tree_mask(parents, words=None, device="cuda"):
    """Rows of mha_paged_tree_fwd's ``tree_mask`` and depths of one tree of drafted tokens.

    ``parents``: for each token the number of its parent, which comes before it, or -1
    (a root).  Returns (int32 [n, words], int32 [n]): every token sees its ancestors and
    itself, and its position is the cached length before the tree plus its depth.
    ``words``: of a row (default: as many as the tree needs)."""
    import torch
    n = len(parents)
    if words is None:
        words = max(1, -(-n // 32))
    if n > 32 * words:
        raise ValueError("a tree of %d tokens needs rows of more than %d words" % (n, words))
    sees, depth = [], []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError("token %d: its parent must be -1 or a token before it, not %d" % (i, p))
        sees.append(1 << i | (sees[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    rows = [[(s >> 32 * w & 0xffffffff) for w in range(words)] for s in sees]
    rows = [[x - (1 << 32) if x >> 31 else x for x in r] for r in rows]
    return (torch.tensor(rows, dtype=torch.int32).reshape(n, words).to(device),
            torch.tensor(depth, dtype=torch.int32).to(device))


_modules = {}


def _torch():
    """torch, imported at the first call that needs it (an import statement in every
    call costs a third of a microsecond each)."""
    torch = _modules.get("torch")
    if torch is None:
        import torch
        _modules["torch"] = torch
        _use_binding()
    return torch


_LIB = lib      # (a test may put another one in lib's place)
_native = None  # binding.cpp's module


def _use_binding() -> None:
    """Takes binding.cpp's checks and calls, where it is built (torch is imported: it links
    to it)."""
    global _native, _at
    if not os.path.exists(_build.BINDING):
        return
    loader = importlib.machinery.ExtensionFileLoader("_mha_binding", _build.BINDING)
    try:
        native = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_mha_binding", loader))
        loader.exec_module(native)
    except ImportError:  # built against another PyTorch
        return
    native.refuse_with(_at_plain)
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        native.stream_with(raw)
    for name in EXPORTED:
        native.bind(name, ctypes.cast(getattr(_LIB, name), ctypes.c_void_p).value)
    _native, _at = native, native.at


def _dtype_of(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return MHA_DTYPE_BF16
    if t.dtype == torch.float32:
        return MHA_DTYPE_F32
    raise TypeError("tensors must be float32 or bfloat16, not %s" % t.dtype)


def _layout_of(layout: str) -> int:
    if layout == "bshd":
        return MHA_LAYOUT_BSHD
    if layout == "bhsd":
        return MHA_LAYOUT_BHSD
    raise ValueError("layout must be 'bhsd' or 'bshd'")


def _device_of(t) -> int:
    """Number of a CUDA tensor's device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _at_plain(name, t, shape, dtype, dev):
    """Address of a tensor or array of the call (None: none): contiguous, of that
    shape, dtype and device.  Every tensor of every call of a generation step passes
    here: plain attribute reads, the device by its number."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d, not %s of shape "
                         "%s on %s" % (name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape),
                                       t.device))
    return t.data_ptr()


_at = _at_plain


def _scratch(t, dev):
    """(address, bytes) of a workspace, or (None, 0)."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    return t.data_ptr(), t.numel() * t.element_size()


def _rotary(inv_freq, dev):
    """(address, rotary_dim) of the frequencies; (None, 0) without."""
    if inv_freq is None:
        return None, 0
    n = inv_freq.numel()
    return _at("inv_freq", inv_freq, (n,), _torch().float32, dev), 2 * n


def _on(stream, device):
    """Context in which this call's own tensors are allocated: its stream, so that
    the memory is not handed to other work while the call's kernels use it."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _torch()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _call(name, dev, stream, args):
    torch = _torch()
    if stream is None:
        handle = _current_stream(dev)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    entry = getattr(_native if _native is not None and lib is _LIB else lib, name)
    if _only_device() or torch.cuda.current_device() == dev:
        st = entry(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = entry(*args, handle)
    if st != MHA_OK:
        raise MhaError(st, name)


def _whole():
    """binding.cpp's module where it may make whole calls, else None: it knows no other
    device than the current one, and no other library than its own."""
    return _native if _native is not None and lib is _LIB and _only_device() else None


def _made(status, name) -> bool:
    """Whether a whole call has been made (None: its arguments are not all as they should
    be, and Python says how, or brings along what is missing)."""
    if status is None:
        return False
    if status != MHA_OK:
        raise MhaError(status, name)
    return True


def _only_device() -> bool:
    """Whether the process has one CUDA device, which then is the current one (asking for
    that takes a quarter of a microsecond)."""
    one = _modules.get("one device")
    if one is None:
        one = _modules["one device"] = _torch().cuda.device_count() == 1
    return one


def _current_stream(dev: int) -> int:
    """Handle of torch's current stream on device ``dev``."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a tenth of the public call's time
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _head_rows(q, k, layout):
    """Dimensions of the row operators: (B, H, H_kv, L, d, q shape, k shape)."""
    if q is None and k is None:
        raise ValueError("q or k must be given")
    ref = q if q is not None else k
    if ref.dim() != 4:
        raise ValueError("q and k must have 4 dimensions")
    if layout == MHA_LAYOUT_BSHD:
        B, L, _, d = ref.shape
        H, Hkv = (0 if t is None else t.shape[2] for t in (q, k))
        return B, H, Hkv, L, d, (B, L, H, d), (B, L, Hkv, d)
    B, _, L, d = ref.shape
    H, Hkv = (0 if t is None else t.shape[1] for t in (q, k))
    return B, H, Hkv, L, d, (B, H, L, d), (B, Hkv, L, d)


def mha_qk_norm_rope_fwd(q, k, q_out=None, k_out=None, *, q_weight=None, k_weight=None,
                         positions=None, inv_freq=None, layout: str = "bhsd",
                         interleaved: bool = False, eps: float = 1e-6, stream=None):
    """Per-head RMS norm (with ``q_weight`` / ``k_weight`` [d]; None: no norm) and
    position rotation (with ``inv_freq`` float32 [rotary_dim / 2]; None: none) of the
    rows of q and k, in one pass.  Returns (q_out, k_out).

    layout "bhsd": q [B,H,L,d], k [B,H_kv,L,d]; "bshd": q [B,L,H,d], k [B,L,H_kv,d];
    either may be None.  ``positions`` int32 [B, L] (None: 0 .. L - 1).  Pairs are
    (i, i + rotary_dim / 2), or (2i, 2i + 1) when ``interleaved``.  ``q_out`` and
    ``k_out`` may be q and k themselves.  Enqueued on ``stream`` (default: torch's
    current stream).
    """
    torch = _torch()
    lay = _layout_of(layout)
    B, H, Hkv, L, d, qs, ks = _head_rows(q, k, lay)
    ref = q if q is not None else k
    dtype, dt, dev = _dtype_of(ref), ref.dtype, _device_of(ref)
    if q_out is None or k_out is None:
        with _on(stream, ref.device):
            q_out = torch.empty_like(q) if q_out is None and q is not None else q_out
            k_out = torch.empty_like(k) if k_out is None and k is not None else k_out
    freq, rotary = _rotary(inv_freq, dev)
    args = (_at("q", q, qs, dt, dev), _at("k", k, ks, dt, dev), _at("q_out", q_out, qs, dt, dev),
            _at("k_out", k_out, ks, dt, dev), _at("q_weight", q_weight, (d,), dt, dev),
            _at("k_weight", k_weight, (d,), dt, dev),
            _at("positions", positions, (B, L), torch.int32, dev), freq, B, H, Hkv, L, d, rotary,
            lay, 1 if interleaved else 0, eps, dtype)
    _call("mha_qk_norm_rope_fwd", dev, stream, args)
    return q_out, k_out


def mha_qk_norm_rope_bwd_workspace_size(d: int) -> int:
    return int(lib.mha_qk_norm_rope_bwd_workspace_size(int(d)))


def mha_qk_norm_rope_bwd(q, k, dq_out, dk_out, dq=None, dk=None, dq_weight=None, dk_weight=None,
                         *, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                         layout: str = "bhsd", interleaved: bool = False, eps: float = 1e-6,
                         workspace=None, stream=None):
    """Gradients through mha_qk_norm_rope_fwd: (dq, dk, dq_weight, dk_weight), the
    last two float32 [d] (None where the weight is None).  q, k: the forward's
    inputs; dq_out, dk_out: the gradients of its results (dk_out None: queries
    alone; dq_out None: keys alone).  ``dq`` and ``dk`` may be dq_out and dk_out
    themselves.  ``workspace``: uint8 CUDA tensor of at least
    mha_qk_norm_rope_bwd_workspace_size(d) bytes (allocated here when None and
    needed)."""
    torch = _torch()
    lay = _layout_of(layout)
    B, H, Hkv, L, d, qs, ks = _head_rows(dq_out, dk_out, lay)
    ref = dq_out if dq_out is not None else dk_out
    dtype, dt, dev = _dtype_of(ref), ref.dtype, _device_of(ref)
    weights = q_weight is not None or k_weight is not None
    if q_weight is None and dq_weight is not None or k_weight is None and dk_weight is not None:
        raise ValueError("dq_weight and dk_weight go with q_weight and k_weight")
    if any(t is None for t in (dq, dk, dq_weight, dk_weight, workspace)):
        with _on(stream, ref.device):
            dq = torch.empty_like(dq_out) if dq is None and dq_out is not None else dq
            dk = torch.empty_like(dk_out) if dk is None and dk_out is not None else dk
            new = lambda: torch.empty(d, dtype=torch.float32, device=ref.device)  # noqa: E731
            dq_weight = new() if dq_weight is None and q_weight is not None else dq_weight
            dk_weight = new() if dk_weight is None and k_weight is not None else dk_weight
            if workspace is None and weights:
                workspace = torch.empty(max(mha_qk_norm_rope_bwd_workspace_size(d), 1),
                                        dtype=torch.uint8, device=ref.device)
    for name, x, w, shape in (("q", q, q_weight, qs), ("k", k, k_weight, ks)):
        if x is None and w is not None and 0 not in shape:
            raise ValueError("%s is needed with %s_weight" % (name, name))
    freq, rotary = _rotary(inv_freq, dev)
    args = (_at("q", q, qs, dt, dev), _at("k", k, ks, dt, dev), _at("dq_out", dq_out, qs, dt, dev),
            _at("dk_out", dk_out, ks, dt, dev), _at("dq", dq, qs, dt, dev),
            _at("dk", dk, ks, dt, dev), _at("dq_weight", dq_weight, (d,), torch.float32, dev),
            _at("dk_weight", dk_weight, (d,), torch.float32, dev),
            _at("q_weight", q_weight, (d,), dt, dev), _at("k_weight", k_weight, (d,), dt, dev),
            _at("positions", positions, (B, L), torch.int32, dev), freq, B, H, Hkv, L, d, rotary,
            lay, 1 if interleaved else 0, eps, dtype, *_scratch(workspace, dev))
    _call("mha_qk_norm_rope_bwd", dev, stream, args)
    return dq, dk, dq_weight, dk_weight


def _cache(k_cache, v_cache, d, Hkv, layout, dt, dev):
    """(k address, v address, num_pages, page_size) of a paged cache."""
    if k_cache.dim() != 4:
        raise ValueError("the caches must have 4 dimensions")
    pages, a, b, _ = shape = k_cache.shape
    page = a if layout == MHA_LAYOUT_BSHD else b
    if (b if layout == MHA_LAYOUT_BSHD else a) != Hkv or shape[3] != d:
        raise ValueError("the caches must have %d heads of %d, not shape %s"
                         % (Hkv, d, tuple(shape)))
    return (_at("k_cache", k_cache, shape, dt, dev), _at("v_cache", v_cache, shape, dt, dev), pages,
            page)


def _batch(q_starts, kv_lengths, block_table, dev):
    """(addresses of the three arrays, B, max_pages) of a ragged batch."""
    i32 = _torch().int32
    if block_table.dim() != 2:
        raise ValueError("block_table must have 2 dimensions")
    B, max_pages = table = block_table.shape
    if B > _INT_MAX or max_pages > _INT_MAX:  # ctypes would keep the low 32 bits
        raise ValueError("block_table has more than 2^31 - 1 rows or columns")
    return (_at("q_starts", q_starts, (B + 1,), i32, dev),
            _at("kv_lengths", kv_lengths, (B,), i32, dev),
            _at("block_table", block_table, table, i32, dev)), B, max_pages


def mha_paged_append(q, k, v, k_cache, v_cache, q_out=None, *, q_starts, kv_lengths, block_table,
                     q_weight=None, k_weight=None, inv_freq=None, layout: str = "bhsd",
                     interleaved: bool = False, eps: float = 1e-6, stream=None):
    """The norm and rotation of mha_qk_norm_rope_fwd for the new tokens of a ragged
    batch at their positions; keys and values go into the pages of the cache.
    Returns q_out (None when q is None).

    q [T,H,d] (or None), k, v [T,H_kv,d]; sequence b's tokens are rows q_starts[b] ..
    q_starts[b+1] - 1 (int32 [B+1]) and the last ones of its kv_lengths[b] (int32 [B])
    positions; position p lies in page block_table[b][p // page_size] (int32
    [B, max_pages]).  Caches: layout "bhsd" [pages,H_kv,page_size,d], "bshd"
    [pages,page_size,H_kv,d].  Rows of no sequence keep what ``q_out`` held (zeros
    when it is allocated here); ``q_out`` may be q itself.
    """
    return _append("mha_paged_append", (), q, k, v, k_cache, v_cache, q_out, q_starts, kv_lengths,
                   block_table, q_weight, k_weight, inv_freq, layout, interleaved, eps, stream)


def mha_paged_append_at(q, k, v, k_cache, v_cache, positions, q_out=None, *, q_starts, kv_lengths,
                        block_table, q_weight=None, k_weight=None, inv_freq=None,
                        layout: str = "bhsd", interleaved: bool = False, eps: float = 1e-6,
                        stream=None):
    """mha_paged_append whose tokens are rotated at ``positions`` (int32 [T]) instead of
    their cells': those of a drafted tree lie behind one another in the cache, each at
    the position of its depth (``tree_mask``)."""
    return _append("mha_paged_append_at", (positions,), q, k, v, k_cache, v_cache, q_out, q_starts,
                   kv_lengths, block_table, q_weight, k_weight, inv_freq, layout, interleaved, eps,
                   stream)


def _append(name, positions, q, k, v, k_cache, v_cache, q_out, q_starts, kv_lengths, block_table,
            q_weight, k_weight, inv_freq, layout, interleaved, eps, stream):
    native = _whole()
    if native is not None and _made(native.append(
            len(positions) == 1, q, k, v, k_cache, v_cache, q_out, positions[0] if positions else None,
            q_starts, kv_lengths, block_table, q_weight, k_weight, inv_freq, layout, interleaved, eps,
            stream), name):
        return q_out
    lay = _layout_of(layout)
    if k.dim() != 3:
        raise ValueError("q, k and v must have 3 dimensions")
    dtype, dt, dev = _dtype_of(k), k.dtype, _device_of(k)
    T, Hkv, d = ks = k.shape
    H = 0 if q is None else q.shape[1]
    if q is None:
        q_out = None
    elif q_out is None:
        with _on(stream, k.device):
            q_out = _torch().zeros_like(q)
        if native is not None:  # (now that it is there)
            return _append(name, positions, q, k, v, k_cache, v_cache, q_out, q_starts, kv_lengths,
                           block_table, q_weight, k_weight, inv_freq, layout, interleaved, eps, stream)
    kc, vc, pages, page = _cache(k_cache, v_cache, d, Hkv, lay, dt, dev)
    arrays, B, max_pages = _batch(q_starts, kv_lengths, block_table, dev)
    freq, rotary = _rotary(inv_freq, dev)
    args = (_at("q", q, (T, H, d), dt, dev), _at("k", k, ks, dt, dev), _at("v", v, ks, dt, dev),
            _at("q_out", q_out, (T, H, d), dt, dev), kc, vc,
            _at("q_weight", q_weight, (d,), dt, dev), _at("k_weight", k_weight, (d,), dt, dev), freq,
            *[_at("positions", t, (T,), _torch().int32, dev) for t in positions],
            *arrays, B, T, H, Hkv, d, pages, page, max_pages, rotary, lay, 1 if interleaved else 0,
            eps, dtype)
    _call(name, dev, stream, args)
    return q_out


def mha_paged_workspace_size(B, T, H, H_kv, d, max_q, dtype) -> int:
    """Bytes of workspace of mha_paged_fwd; ``dtype``: a torch dtype or MHA_DTYPE_*."""
    if not isinstance(dtype, int):
        torch = _torch()
        dtype = {torch.bfloat16: MHA_DTYPE_BF16, torch.float32: MHA_DTYPE_F32}[dtype]
    return int(lib.mha_paged_workspace_size(B, T, H, H_kv, d, max_q, dtype))


def mha_paged_path(B, T, H, H_kv, d, max_q, page_size, dtype) -> int:
    return int(lib.mha_paged_path(B, T, H, H_kv, d, max_q, page_size, dtype))


def mha_paged_fwd(q, k_cache, v_cache, out=None, *, q_starts, kv_lengths, block_table, max_q: int,
                  layout: str = "bhsd", mask_kind: int = MHA_MASK_CAUSAL_TAIL, scale=None,
                  workspace=None, stream=None):
    """Attention of the new tokens of a ragged batch (mha_paged_append) over the
    paged cache.  q [T,H,d]; returns ``out`` like q.  mask_kind: MHA_MASK_CAUSAL_TAIL
    (a token sees the positions up to its own) or MHA_MASK_NONE (all of its
    sequence).  ``max_q``: the most new tokens of a sequence that are expected (it
    chooses the kernel; the result is right whatever it is).  Rows of no sequence
    keep what ``out`` held (zeros when it is allocated here).  ``scale`` defaults to
    1/sqrt(d).  ``workspace``: uint8 CUDA tensor of at least
    mha_paged_workspace_size(B, T, H, H_kv, d, max_q, q.dtype) bytes (allocated here
    when None)."""
    return _attend("mha_paged_fwd", (), q, k_cache, v_cache, out, q_starts, kv_lengths, block_table,
                   max_q, layout, (mask_kind,), scale, workspace, stream)


def mha_paged_tree_fwd(q, k_cache, v_cache, tree_mask, out=None, *, q_starts, kv_lengths,
                       block_table, max_q: int, layout: str = "bhsd", scale=None, workspace=None,
                       stream=None):
    """mha_paged_fwd for new tokens that form a drafted tree in each sequence: a token sees
    every position before its sequence's new tokens, and of those the ones in its row
    of ``tree_mask``, int32 [T, words]: bit m % 32 of word m // 32 for new token m of
    its sequence (the module's ``tree_mask`` makes the rows of a tree).  Everything else,
    the workspace too, as mha_paged_fwd's."""
    return _attend("mha_paged_tree_fwd", (tree_mask,), q, k_cache, v_cache, out, q_starts,
                   kv_lengths, block_table, max_q, layout, (), scale, workspace, stream)


def _attend(name, tree, q, k_cache, v_cache, out, q_starts, kv_lengths, block_table, max_q, layout,
            mask, scale, workspace, stream):
    native = _whole()
    if native is not None and (not tree or tree[0] is not None) and _made(native.attend(
            q, k_cache, v_cache, out, tree[0] if tree else None, q_starts, kv_lengths, block_table,
            max_q, layout, mask[0] if mask else 0, scale, workspace, stream), name):
        return out
    lay = _layout_of(layout)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must have 3 dimensions and the caches 4")
    dtype, dt, dev = _dtype_of(q), q.dtype, _device_of(q)
    T, H, d = qs = q.shape
    Hkv = k_cache.shape[2 if lay == MHA_LAYOUT_BSHD else 1]
    kc, vc, pages, page = _cache(k_cache, v_cache, d, Hkv, lay, dt, dev)
    arrays, B, max_pages = _batch(q_starts, kv_lengths, block_table, dev)
    if out is None or workspace is None:
        torch = _torch()
        with _on(stream, q.device):
            out = torch.zeros_like(q) if out is None else out
            if workspace is None:
                n = mha_paged_workspace_size(B, T, H, Hkv, d, max_q, dtype)
                workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
        if native is not None:  # (now that they are there)
            return _attend(name, tree, q, k_cache, v_cache, out, q_starts, kv_lengths, block_table,
                           max_q, layout, mask, scale, workspace, stream)
    words = ()
    if tree:
        if tree[0].dim() != 2 or not 1 <= tree[0].shape[1] <= _INT_MAX:
            raise ValueError("tree_mask must have 2 dimensions, at least one word to a row")
        words = (tree[0].shape[1],)
        tree = (_at("tree_mask", tree[0], (T, *words), _torch().int32, dev),)
    args = (_at("q", q, qs, dt, dev), kc, vc, _at("out", out, qs, dt, dev), *tree, *arrays, B, T, H,
            Hkv, d, max_q, pages, page, max_pages, *words, lay, *mask,
            d ** -0.5 if scale is None else scale, dtype, *_scratch(workspace, dev))
    _call(name, dev, stream, args)
    return out


def _counted(name, shape):
    """A shape whose counts the C entry points take (ctypes would keep their low 32 bits)."""
    for n in shape:
        if n > _INT_MAX:
            raise ValueError("%s has more than 2^31 - 1 rows or columns" % name)
    return shape


def mha_paged_reserve_workspace_size(B: int, num_pages: int) -> int:
    return int(lib.mha_paged_reserve_workspace_size(int(B), int(num_pages)))


def mha_paged_reserve(block_table, kv_lengths, new_lengths, refs, *, page_size: int, parents=None,
                      table_out=None, lengths_out=None, refs_out=None, moves=None, counts=None,
                      workspace=None, stream=None):
    """The block tables of the next step: row i continues row ``parents[i]`` (int32 [B];
    None: its own number; -1: a new sequence) with ``new_lengths[i]`` positions, sharing
    whole pages with its parent and taking free ones as it needs them.  Sequences grow,
    shrink, fork, end (length 0) and begin.

    block_table int32 [B_old, max_pages], kv_lengths [B_old]: how far those tables reach (the
    ``lengths_out`` they came with: after mha_paged_compact more than the sequences' lengths,
    which go into ``new_lengths`` to give back the pages of rejected tokens before rows fork),
    new_lengths [B], refs [num_pages] (references to each page; 0: free).  Returns (table_out, lengths_out,
    refs_out, moves, counts): the new tables, how far each row's pages go (less than its
    length where the free pages ran out), the new references (``refs_out`` may be refs),
    the page copies that the rows need, [B, 2], for ``mha_paged_copy``, and int32 [2]: pages
    given out and pages still free."""
    native = _whole()
    if native is not None and _made(native.reserve(
            block_table, kv_lengths, new_lengths, parents, refs, table_out, lengths_out, refs_out,
            moves, counts, page_size, workspace, stream), "mha_paged_reserve"):
        return table_out, lengths_out, refs_out, moves, counts
    torch = _torch()
    i32, dev = torch.int32, _device_of(block_table)
    if block_table.dim() != 2 or new_lengths.dim() != 1 or refs.dim() != 1:
        raise ValueError("block_table must have 2 dimensions, new_lengths and refs 1")
    B_old, width = _counted("block_table", block_table.shape)
    (B,), (pages,) = _counted("new_lengths", new_lengths.shape), _counted("refs", refs.shape)
    if (table_out is None or lengths_out is None or refs_out is None or moves is None or
            counts is None or workspace is None):
        with _on(stream, block_table.device):
            new = lambda *n: torch.empty(n, dtype=i32, device=block_table.device)  # noqa: E731
            table_out = new(B, width) if table_out is None else table_out
            lengths_out = new(B) if lengths_out is None else lengths_out
            refs_out = new(pages) if refs_out is None else refs_out
            moves = new(B, 2) if moves is None else moves
            counts = new(2) if counts is None else counts
            if workspace is None:
                workspace = torch.empty(max(mha_paged_reserve_workspace_size(B, pages), 1),
                                        dtype=torch.uint8, device=block_table.device)
    args = (_at("block_table", block_table, (B_old, width), i32, dev),
            _at("kv_lengths", kv_lengths, (B_old,), i32, dev),
            _at("new_lengths", new_lengths, (B,), i32, dev),
            _at("parents", parents, (B,), i32, dev), _at("refs", refs, (pages,), i32, dev),
            _at("table_out", table_out, (B, width), i32, dev),
            _at("lengths_out", lengths_out, (B,), i32, dev),
            _at("refs_out", refs_out, (pages,), i32, dev), _at("moves", moves, (B, 2), i32, dev),
            _at("counts", counts, (2,), i32, dev), B_old, B, pages, page_size, width,
            *_scratch(workspace, dev))
    _call("mha_paged_reserve", dev, stream, args)
    return table_out, lengths_out, refs_out, moves, counts


def _stack(k_cache, v_cache):
    """(layers, shape of one layer's cache, its dtype, device) of caches with or without a
    dimension of layers in front."""
    if k_cache.dim() not in (4, 5):
        raise ValueError("the caches must have 4 dimensions, or 5 with the layers in front")
    shape = _counted("k_cache", k_cache.shape)
    layers = shape[0] if len(shape) == 5 else 1
    return layers, shape[-4:], k_cache.dtype, _device_of(k_cache)


def mha_paged_copy(k_cache, v_cache, moves, *, stream=None):
    """Copies page moves[i][0] to page moves[i][1] (int32 [n, 2]; pairs with a number that
    is no page's are skipped) in both caches, [pages, ...] or [layers, pages, ...] in either
    layout.  What mha_paged_reserve leaves to be copied."""
    native = _whole()
    if native is not None and _made(native.copy(k_cache, v_cache, moves, stream), "mha_paged_copy"):
        return
    layers, (pages, a, b, d), dt, dev = _stack(k_cache, v_cache)
    if moves.dim() != 2:
        raise ValueError("moves must have 2 dimensions")
    n, _ = _counted("moves", moves.shape)
    # (a page's bytes are copied whatever their order: which of its two inner dimensions is
    # the page's and which the heads' does not matter, but a page's is a power of two)
    page, heads = (a, b) if a >= 16 and a & (a - 1) == 0 else (b, a)
    args = (_at("k_cache", k_cache, k_cache.shape, dt, dev),
            _at("v_cache", v_cache, k_cache.shape, dt, dev),
            _at("moves", moves, (n, 2), _torch().int32, dev), n, layers, heads, d, pages, page,
            _dtype_of(k_cache))
    _call("mha_paged_copy", dev, stream, args)


def mha_paged_compact(k_cache, v_cache, keep, keep_counts, lengths_out=None, *, starts=None,
                      kv_lengths, block_table, src_table=None, layout: str = "bhsd", stream=None):
    """Moves the tokens that stay: position starts[b] + keep[b][i] to starts[b] + i for i <
    keep_counts[b], in both caches, [pages, ...] or [layers, pages, ...].  Returns the new
    lengths, starts[b] + keep_counts[b]; the pages behind them are held until
    mha_paged_reserve(block_table, kv_lengths, those lengths, ...) gives them back.

    keep int32 [B, max_keep]: ascending lists, which end before an entry that is not; starts
    int32 [B] (None: 0); kv_lengths [B]: the lengths before; ``block_table`` [B, max_pages]:
    the pages written, ``src_table`` those read (None: the same, in place; else no cell is
    both written and read)."""
    native = _whole()
    if native is not None and _made(native.compact(
            k_cache, v_cache, keep, keep_counts, lengths_out, starts, kv_lengths, block_table,
            src_table, layout, stream), "mha_paged_compact"):
        return lengths_out
    torch = _torch()
    i32, lay = torch.int32, _layout_of(layout)
    layers, (pages, a, b, d), dt, dev = _stack(k_cache, v_cache)
    page, heads = (a, b) if lay == MHA_LAYOUT_BSHD else (b, a)
    if keep.dim() != 2 or block_table.dim() != 2:
        raise ValueError("keep and block_table must have 2 dimensions")
    B, most = _counted("keep", keep.shape)
    _, width = _counted("block_table", block_table.shape)
    if lengths_out is None:
        with _on(stream, k_cache.device):
            lengths_out = torch.empty(B, dtype=i32, device=k_cache.device)
    args = (_at("k_cache", k_cache, k_cache.shape, dt, dev),
            _at("v_cache", v_cache, k_cache.shape, dt, dev),
            _at("lengths_out", lengths_out, (B,), i32, dev), _at("keep", keep, (B, most), i32, dev),
            _at("keep_counts", keep_counts, (B,), i32, dev), _at("starts", starts, (B,), i32, dev),
            _at("kv_lengths", kv_lengths, (B,), i32, dev),
            _at("src_table", src_table, (B, width), i32, dev),
            _at("block_table", block_table, (B, width), i32, dev), B, layers, heads, d, pages, page,
            width, most, lay, _dtype_of(k_cache))
    _call("mha_paged_compact", dev, stream, args)
    return lengths_out
