"""Python binding of the C ABI in include/mha_paged.h (ctypes; argument marshalling only).

The per-head norm and position rotation of queries and keys with its gradients,
the paged key/value cache and the attention over it.  Same library, same errors
and same conventions as ``mha.py``: torch CUDA tensors in, nothing computed here.
"""
from __future__ import annotations

import contextlib
import ctypes

from .mha import (MHA_DTYPE_BF16, MHA_DTYPE_F32, MHA_LAYOUT_BHSD, MHA_LAYOUT_BSHD,
                  MHA_MASK_CAUSAL_TAIL, MHA_OK, MhaError, lib)

MHA_ROPE_HALVES, MHA_ROPE_INTERLEAVED = 0, 1
PAGED_PATH_NAMES = {0: "none", 1: "paged_simt", 2: "paged_few_tc", 3: "paged_many_tc"}

_INT_MAX = 0x7fffffff

EXPORTED = ("mha_qk_norm_rope_fwd", "mha_qk_norm_rope_bwd_workspace_size", "mha_qk_norm_rope_bwd",
            "mha_paged_append", "mha_paged_workspace_size", "mha_paged_fwd", "mha_paged_path")


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
    lib.mha_paged_workspace_size.restype = sz
    lib.mha_paged_workspace_size.argtypes = [i32] * 7
    lib.mha_paged_fwd.restype = i32
    lib.mha_paged_fwd.argtypes = [vp] * 7 + [i32] * 11 + [f32, i32, vp, sz, vp]
    lib.mha_paged_path.restype = i32
    lib.mha_paged_path.argtypes = [i32] * 8


_declare()


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, device="cuda"):
    """The usual frequencies base^(-2 i / rotary_dim), i < rotary_dim / 2, as the
    float32 tensor ``inv_freq`` that the operators take."""
    import torch
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    return (float(base) ** (-2.0 * i / rotary_dim)).float().to(device)


_modules = {}


def _torch():
    """torch, imported at the first call that needs it (an import statement in every
    call costs a third of a microsecond each)."""
    torch = _modules.get("torch")
    if torch is None:
        import torch
        _modules["torch"] = torch
    return torch


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


def _at(name, t, shape, dtype, dev):
    """Address of a tensor or array of the call (None: none): contiguous, of that
    shape, dtype and device.  Every tensor of every call of a generation step passes
    here: plain attribute reads, the device by its number."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d, not %s of shape "
                         "%s on %s" % (name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape),
                                       t.device))
    return t.data_ptr()


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
    if torch.cuda.current_device() == dev:
        st = getattr(lib, name)(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = getattr(lib, name)(*args, handle)
    if st != MHA_OK:
        raise MhaError(st, name)


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
    kc, vc, pages, page = _cache(k_cache, v_cache, d, Hkv, lay, dt, dev)
    arrays, B, max_pages = _batch(q_starts, kv_lengths, block_table, dev)
    freq, rotary = _rotary(inv_freq, dev)
    args = (_at("q", q, (T, H, d), dt, dev), _at("k", k, ks, dt, dev), _at("v", v, ks, dt, dev),
            _at("q_out", q_out, (T, H, d), dt, dev), kc, vc,
            _at("q_weight", q_weight, (d,), dt, dev), _at("k_weight", k_weight, (d,), dt, dev), freq,
            *arrays, B, T, H, Hkv, d, pages, page, max_pages, rotary, lay, 1 if interleaved else 0,
            eps, dtype)
    _call("mha_paged_append", dev, stream, args)
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
    args = (_at("q", q, qs, dt, dev), kc, vc, _at("out", out, qs, dt, dev), *arrays, B, T, H, Hkv, d,
            max_q, pages, page, max_pages, lay, mask_kind, d ** -0.5 if scale is None else scale,
            dtype, *_scratch(workspace, dev))
    _call("mha_paged_fwd", dev, stream, args)
    return out
