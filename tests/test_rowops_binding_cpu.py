"""What the binding of the row operators makes of its arguments, without a GPU:
tensors here are on the CPU, with the binding's own check of that taken out
where a function would refuse them, and nothing is launched."""

import copy
import ctypes
import os

import pytest
import torch

import sparse_convolution_hash_amd.binding as B


@pytest.fixture
def cpu_tensors(monkeypatch):
    def need(t, name, dtype=None, dev=None):
        if not isinstance(t, torch.Tensor) or (dtype is not None and t.dtype != dtype):
            raise TypeError(name)
    monkeypatch.setattr(B, "_need", need)


def passed(drop):
    """The descriptor that a call hands to the library."""
    return ctypes.cast(B._drop_arg(drop, torch.device("cpu")), ctypes.POINTER(B._DropArg)).contents


def test_dropout_passes_its_current_values(cpu_tensors):
    a, b = torch.tensor([1, 2]), torch.tensor([3, 4])
    d = B.Dropout(a, 0.5, 7)
    assert (passed(d).rng, passed(d).p, passed(d).layer) == (a.data_ptr(), 0.5, 7)
    d.p, d.layer = 0.25, 9
    assert (passed(d).rng, passed(d).p, passed(d).layer) == (a.data_ptr(), 0.25, 9)
    d.rng = b
    assert d.rng is b and passed(d).rng == b.data_ptr()
    b.set_(torch.tensor([5, 6, 7, 8])[:2])          # another storage under the same tensor
    assert passed(d).rng == b.data_ptr()


def test_dropout_checks_later_values_too(cpu_tensors):
    a = torch.tensor([1, 2])
    d = B.Dropout(a, 0.5, 7)
    for name, bad, error in (("p", 1.5, ValueError), ("p", float("nan"), ValueError), ("layer", -1, ValueError),
                             ("layer", 1 << 32, ValueError), ("rng", torch.tensor([1, 2, 3]), ValueError),
                             ("rng", torch.tensor([1.0, 2.0]), TypeError)):
        with pytest.raises(error):
            setattr(d, name, bad)
    assert (passed(d).rng, passed(d).p, passed(d).layer) == (a.data_ptr(), 0.5, 7)


class Quiet:
    """The library with its size queries, whose other calls do nothing."""

    def __getattr__(self, name):
        return getattr(B._lib, name) if name.endswith("_workspace") else lambda *a: B.SPC_OK


@pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libspc.so not built")
@pytest.mark.parametrize("name", ["group_norm_fwd", "group_norm_bwd", "linear_recurrence_fwd", "linear_recurrence_bwd",
                                  "conv_bwd_filter", "build_kmap", "build_kmap_strided"])
def test_workspaces_are_checked(monkeypatch, name):
    """A workspace is checked as every other tensor is: on the GPU, on the
    call's device, contiguous.  (All tensors are on the CPU here; the others
    pass for GPU tensors.)"""
    B.lib()
    need = B._need

    def others_pass(t, nm, dtype=None, dev=None):
        if nm == "workspace":
            need(t, nm, dtype, dev)
    monkeypatch.setattr(B, "_need", others_pass)
    monkeypatch.setattr(B, "_gate_x", lambda gate, x, names=None: x.shape[1])
    monkeypatch.setattr(B, "lib", Quiet)
    monkeypatch.setattr(B, "_stream", lambda dev: None)
    n, C = 100, 32
    x, i = torch.zeros(n, C), torch.zeros(n, dtype=torch.int32)
    carry = torch.zeros(B.linear_recurrence_workspace(x.dtype, n, C, 1)[1] // 4)
    call = {
        "group_norm_fwd": lambda w: B.group_norm_fwd(x, 4, workspace=w),
        "group_norm_bwd": lambda w: B.group_norm_bwd(x, x, 4, None, None, None, torch.zeros(1, 4, 2), workspace=w),
        "linear_recurrence_fwd": lambda w: B.linear_recurrence_fwd(x, x, workspace=w),
        "linear_recurrence_bwd": lambda w: B.linear_recurrence_bwd(x, x, x, None, carry, workspace=w),
        "conv_bwd_filter": lambda w: B.conv_bwd_filter(x, x, 1, None, None, None, workspace=w),
        "build_kmap": lambda w: B.build_kmap(torch.zeros(n, 4, dtype=torch.int32), 1, (9, 9, 9), 3, workspace=w),
        "build_kmap_strided": lambda w: B.build_kmap(torch.zeros(n, 4, dtype=torch.int32), 1, (9, 9, 9), 3, 2, 1, 1,
                                                     subm=False, count_first=True, workspace=w),
    }[name]
    if name != "build_kmap_strided":         # takes its own workspace, on the CPU here, from its first call to its second
        call(None)
    for bytes_ in (16, 1 << 22):             # too small for any call, large enough for each
        with pytest.raises(TypeError, match="workspace"):
            call(torch.zeros(bytes_, dtype=torch.uint8))


def test_workspace_device_and_layout(monkeypatch):
    # what passes for a GPU tensor: is_cuda, on device 0
    class Fake(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 0)
    w = torch.zeros(64, dtype=torch.uint8).as_subclass(Fake)
    assert B._scratch(w, 64, w) is w and B._scratch(None, 0, w) is None
    assert B._scratch(w, 65, torch.zeros(1).as_subclass(Fake)).numel() == 65
    with pytest.raises(ValueError, match="workspace is on"):
        B._scratch(w, 64, torch.zeros(1))
    with pytest.raises(ValueError, match="contiguous"):
        B._scratch(w[::2], 16, w)
    with pytest.raises(ValueError, match="contiguous"):
        B._scratch(w[:1].expand(64), 64, w)


def test_dropout_copies_are_their_own(cpu_tensors):
    a = torch.tensor([1, 2])
    d = B.Dropout(a, 0.5, 7)
    for c in (copy.copy(d), copy.deepcopy(d)):
        assert (c.p, c.layer) == (0.5, 7) and torch.equal(c.rng, a)
        c.p, c.layer = 0.25, 9
        assert (passed(c).rng, passed(c).p, passed(c).layer) == (c.rng.data_ptr(), 0.25, 9)
        assert (passed(d).rng, passed(d).p, passed(d).layer) == (a.data_ptr(), 0.5, 7)
    assert copy.copy(d).rng is a
