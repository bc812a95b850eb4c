"""The compiled inner part of the paged operators' binding (binding.cpp): the same checks as
its Python form, and calls that hand over what they are given."""
import ctypes

import pytest

from test_paged_cpu import P, Fake, declared, mha  # noqa: F401


@pytest.fixture(scope="module")
def native(mha):  # noqa: F811
    from transformer_head_scaled_mha_gb300 import paged
    paged._torch()
    if paged._native is None:
        pytest.skip("binding.cpp is not built here")
    return paged


def test_every_entry_point_is_there(native):
    for name in declared():
        assert callable(getattr(native._native, name)), name


def test_checked_addresses(native):
    import torch
    x = torch.zeros(3, 4, 5)
    for t, shape in ((x, (3, 4, 5)), (x, x.shape), (x[1], (4, 5)), (x[:0], (0, 4, 5)),
                     (torch.zeros(()), ()), (x.view(-1), (60,)), (x[:1].transpose(0, 1), (4, 1, 5))):
        want = native._at_plain("x", t, shape, torch.float32, -1)
        assert native._native.at("x", t, shape, torch.float32, -1) == want == t.data_ptr()
    assert native._native.at("x", torch.nn.Parameter(x), x.shape, torch.float32, -1) == x.data_ptr()
    assert native._native.at("x", None, (3,), torch.float32, 0) is None
    for t, shape, dtype, dev in ((x, (3, 4), torch.float32, -1), (x, (3, 4, 6), torch.float32, -1),
                                 (x, (3, 4, 5, 1), torch.float32, -1), (x, x.shape, torch.bfloat16, -1),
                                 (x, x.shape, torch.float32, 0), (x.transpose(0, 1), (4, 3, 5), torch.float32, -1),
                                 (x[:, :2], (3, 2, 5), torch.float32, -1), (x.to("meta"), x.shape, torch.float32, 0)):
        errors = []
        for at in (native._at_plain, native._native.at):
            with pytest.raises(ValueError) as e:
                at("the name", t, shape, dtype, dev)
            errors.append(str(e.value))
        assert errors[0] == errors[1] and errors[0].startswith("the name must be")
    # what is no tensor is asked as Python asks it
    f = Fake((3, 4), "f32")
    assert native._native.at("x", f, (3, 4), torch.float32, 0) == f.data_ptr()
    with pytest.raises(ValueError):
        native._native.at("x", f, (3, 5), torch.float32, 0)
    with pytest.raises(AttributeError):
        native._native.at("x", 7, (3,), torch.float32, 0)
    with pytest.raises(TypeError):
        native._native.at("x", x)


def test_calls_hand_over_their_arguments(native):
    n, lib = native._native, native._LIB
    # (refused, or with nothing to do: no call below reaches CUDA)
    assert n.mha_paged_copy(P[0], P[1], P[2], -1, 2, 2, 64, 9, 16, 1, None) == 1
    assert n.mha_paged_copy(None, None, None, 0, 2, 2, 64, 9, 16, 1, 0) == 0
    assert n.mha_paged_copy(P[0], P[1], P[2], 3, 2, 2, 96, 9, 16, 1, None) == 2
    assert n.mha_paged_path(4, 9, 32, 4, 64, 3, 16, 1) == 3
    assert n.mha_paged_path(4, 4, 8, 3, 64, 1, 16, 1) == -1
    for args in ((8, 64, 32, 8, 128, 8, 1), (8, 64, 32, 8, 128, 8, 0), (0, 0, 1, 1, 64, 1, 1)):
        assert n.mha_paged_workspace_size(*args) == lib.mha_paged_workspace_size(*args)
    assert n.mha_paged_reserve_workspace_size(7, 1000) == lib.mha_paged_reserve_workspace_size(7, 1000)
    # a number after numbers and one that is no whole number
    fwd = [None] * 8 + [0, 4, 2, 8, 64, 64, 0, 0]
    assert n.mha_qk_norm_rope_fwd(*fwd, 1e-6, 1, None) == 0
    assert n.mha_qk_norm_rope_fwd(*fwd, -1.0, 1, None) == 1
    assert n.mha_qk_norm_rope_fwd(*fwd, float("nan"), 1, None) == 1
    # a size past 32 bits
    tree = [P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], 2, 6, 4, 2, 64, 3, 9, 16, 3, 0, 0, 0.125, 1]
    assert n.mha_paged_tree_fwd(*tree, P[8], 1 << 40, None) == 1  # (no words to a row)


def test_calls_refuse_what_does_not_fit(native):
    n = native._native
    good = [None, None, None, 0, 2, 2, 64, 9, 16, 1, None]
    for i, bad in ((3, 1 << 31), (4, -(1 << 31) - 1), (9, 1 << 80)):
        with pytest.raises(OverflowError):
            n.mha_paged_copy(*good[:i], bad, *good[i + 1:])
    for i, bad in ((0, "k"), (3, 1.5), (8, None), (10, object())):
        with pytest.raises(TypeError):
            n.mha_paged_copy(*good[:i], bad, *good[i + 1:])
    for args in (good[:-1], good + [0]):
        with pytest.raises(TypeError):
            n.mha_paged_copy(*args)
    with pytest.raises(KeyError):
        n.bind("mha_fwd", 1)


def test_another_library_in_its_place_is_called(native, monkeypatch):
    """What tests do: the recorded calls go to that library, not past it."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0
    import torch
    monkeypatch.setattr(native, "lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    native.mha_paged_copy(Fake((9, 16, 2, 64)), Fake((9, 16, 2, 64)), Fake((3, 2), "i32"), stream=4)
    assert seen[0][0] == "mha_paged_copy" and seen[0][1][-1] == 4
    assert isinstance(ctypes.cast(native._LIB.mha_paged_copy, ctypes.c_void_p).value, int)
