"""What the binding of the row operators makes of its arguments, without a GPU:
tensors here are on the CPU, with the binding's own check of that taken out
where a function would refuse them, and nothing is launched."""

import ctypes

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
