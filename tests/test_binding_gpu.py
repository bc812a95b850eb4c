"""Calls that the compiled part of the binding makes from their tensors on (binding.cpp) against
the same ones made in Python: equal results, and for arguments that are not as they should be
the same refusals."""
import numpy as np
import pytest

from test_paged_gpu import batch, cache_of, dev
from test_qk_rope_gpu import freqs, rnd

pytestmark = pytest.mark.gpu

H, HKV, D, PAGE = 4, 2, 64, 16


def entries(layout, q=True, extra=True):
    """name -> (function, arguments by name) of one small batch; all results brought along."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(1)
    b = batch(rng, [(3, 20), (1, 40), (5, 5)], PAGE)
    kc, vc = (dev(x, "bf16") for x in cache_of(rng, b, HKV, PAGE, D, "bf16", layout))
    rows = dev(rnd(rng, (b["T"], H, D), "bf16"), "bf16")
    k, v = (dev(rnd(rng, (b["T"], HKV, D), "bf16"), "bf16") for _ in range(2))
    of = dict(q_starts=dev(b["starts"]), kv_lengths=dev(b["lens"]), block_table=dev(b["table"]))
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    weight = lambda: dev(rnd(rng, (D,), "bf16"), "bf16") if extra else None  # noqa: E731
    append = dict(q=rows if q else None, k=k, v=v, k_cache=kc, v_cache=vc,
                  q_out=torch.zeros_like(rows) if q else None, q_weight=weight(),
                  k_weight=weight(), inv_freq=dev(freqs(D)) if extra else None, layout=layout,
                  interleaved=extra, eps=1e-5, **of)
    ws = torch.empty(mha.mha_paged_workspace_size(3, b["T"], H, HKV, D, 5, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    attend = dict(q=rows, k_cache=kc, v_cache=vc, out=torch.zeros_like(rows), max_q=5, layout=layout,
                  scale=0.2 if extra else None, workspace=ws, **of)
    pool, width = b["pool"], b["table"].shape[1]
    stack = [torch.stack([x, x]) for x in (kc, vc)] if extra else [kc, vc]
    refs = i32(pool).zero_()
    return {
        "append": (mha.mha_paged_append, append),
        "append_at": (mha.mha_paged_append_at, dict(append, positions=i32(b["T"]).abs_())),
        "fwd": (mha.mha_paged_fwd, dict(
            attend, mask_kind=mha.MHA_MASK_NONE if extra else mha.MHA_MASK_CAUSAL_TAIL)),
        "tree_fwd": (mha.mha_paged_tree_fwd, dict(attend, tree_mask=i32(b["T"], 2))),
        "copy": (mha.mha_paged_copy, dict(k_cache=stack[0], v_cache=stack[1], moves=dev(
            np.array([[0, 1], [-1, 2], [3, 9999]], np.int32)))),
        "compact": (mha.mha_paged_compact, dict(
            k_cache=stack[0], v_cache=stack[1], keep=dev(np.array([[0, 2]] * 3, np.int32)),
            keep_counts=dev(np.array([2, 1, 2], np.int32)), lengths_out=i32(3),
            starts=dev(np.array([17, 39, 0], np.int32)) if extra else None,
            kv_lengths=of["kv_lengths"], block_table=of["block_table"],
            src_table=of["block_table"].clone() if extra else None, layout=layout)),
        "reserve": (mha.mha_paged_reserve, dict(
            block_table=of["block_table"], kv_lengths=of["kv_lengths"], new_lengths=i32(4).abs_(),
            refs=refs, page_size=PAGE, parents=i32(4).fill_(1) if extra else None,
            table_out=i32(4, width), lengths_out=i32(4), refs_out=i32(pool), moves=i32(4, 2),
            counts=i32(2), workspace=torch.empty(
                mha.mha_paged_reserve_workspace_size(4, pool), dtype=torch.uint8, device="cuda"))),
    }


NAMES = ["append", "append_at", "fwd", "tree_fwd", "copy", "compact", "reserve"]


@pytest.fixture
def paged():
    import torch
    from transformer_head_scaled_mha_gb300 import paged
    paged._torch()
    if paged._native is None or torch.cuda.device_count() != 1:
        pytest.skip("calls are made in Python here")
    return paged


def called(paged, monkeypatch, native, layout, name, change=None, **kw):
    """What a call did: its refusal, or every tensor it was given, afterwards."""
    import torch
    f, args = entries(layout, **kw)[name]
    if change is not None:
        args[change[0]] = change[1](args[change[0]])
    with monkeypatch.context() as m:
        made = []
        if native:
            real = paged._made
            m.setattr(paged, "_made", lambda st, n: made.append(st) or real(st, n))
        else:
            m.setattr(paged, "_whole", lambda: None)
        try:
            f(**args)
        except Exception as e:  # noqa: BLE001 (both ways are compared)
            return type(e), str(e)
        finally:
            torch.cuda.synchronize()
    return made, [(k, x.contiguous().view(torch.uint8).cpu()) for k, x in sorted(args.items())
                  if isinstance(x, torch.Tensor) and k != "workspace"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("q,extra", [(True, True), (False, True), (True, False)])
def test_the_same_results(paged, monkeypatch, name, layout, q, extra):
    import torch
    made, got = called(paged, monkeypatch, True, layout, name, q=q, extra=extra)
    assert made == [0]  # not by Python
    _, want = called(paged, monkeypatch, False, layout, name, q=q, extra=extra)
    for (k, x), (_, y) in zip(got, want):
        assert torch.equal(x, y), k


@pytest.mark.parametrize("name", ["append", "append_at", "fwd", "tree_fwd"])
@pytest.mark.parametrize("native", [True, False])
def test_results_made_by_the_call(paged, monkeypatch, name, native):
    import torch
    f, args = entries("bshd")[name]
    want = f(**args).clone()
    if not native:
        monkeypatch.setattr(paged, "_whole", lambda: None)
    for key in ("q_out", "out", "workspace"):
        args.pop(key, None)
    got = f(**args)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    with pytest.raises((ValueError, AttributeError)):
        f(**dict(args, kv_lengths=args["kv_lengths"].float()))
    with pytest.raises(ValueError):
        f(**dict(args, layout="sbhd"))


def changes(x):
    """Other values of an argument, none of which a call would take for what it is not."""
    import torch
    if isinstance(x, torch.Tensor):
        other = torch.float32 if x.dtype != torch.float32 else torch.bfloat16
        return [("none", lambda t: None), ("type", lambda t: t.to(other)), ("host", lambda t: t.cpu()),
                ("number", lambda t: 3), ("longer", lambda t: torch.cat([t, t])),
                ("deeper", lambda t: t[None, None]),
                ("apart", lambda t: torch.stack([t, t], -1)[..., 0])]
    if isinstance(x, str):
        return [("unknown", lambda t: "sbhd"), ("none", lambda t: None)]
    if isinstance(x, bool):
        return [("number", lambda t: 0)]
    return [("text", lambda t: "3"), ("large", lambda t: 1 << 40 if isinstance(t, int) else float("nan"))]


@pytest.mark.parametrize("name", NAMES)
def test_the_same_refusals(paged, monkeypatch, name):
    import torch
    args = entries("bshd")[name][1]
    refused = 0
    for key, value in args.items():
        for what, change in changes(value):
            if key == "workspace" and what in ("type", "longer", "deeper", "none"):
                continue  # (any that is large enough will do)
            got, want = (called(paged, monkeypatch, native, "bshd", name,
                                (key, lambda _, v=value: change(v))) for native in (True, False))
            if isinstance(want[0], type):
                assert got == want, (key, what)
                refused += 1
            else:
                assert all(torch.equal(x, y) for (_, x), (_, y) in zip(got[1], want[1])), (key, what)
    assert refused > 15


def test_streams_of_any_kind(paged):
    """The current stream, a stream, its number."""
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    s = torch.cuda.Stream()
    x, y = (torch.arange(3 * 16 * 2 * 64, device="cuda").bfloat16().view(3, 16, 2, 64) for _ in range(2))
    moves = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for stream in (None, s, s.cuda_stream):
        x[2] = 0
        torch.cuda.synchronize()
        mha.mha_paged_copy(x, y, moves, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(x[2], x[0])
    with torch.cuda.stream(s):  # in the order of that stream
        for _ in range(20):
            x[0] += 1
            mha.mha_paged_copy(x, y, moves)
            assert torch.equal(x[2], x[0])
