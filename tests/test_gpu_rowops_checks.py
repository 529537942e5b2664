"""The binding's checks of the row operators' tensors."""

import pytest
import torch

import sparse_convolution_hash_amd as spc

pytestmark = pytest.mark.gpu


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_dropout_tensors():
    r = z(2, dtype=torch.int64)
    x = z(4, 16)
    for bad in (lambda: spc.Dropout(z(2), 0.5), lambda: spc.dropout_fwd(x, 0.5), lambda: spc.dropout_fwd(x, None),
                lambda: spc.dropout_fwd(z(4, 16, dtype=torch.float64), spc.Dropout(r, 0.5)),
                lambda: spc.dropout_fwd(x, spc.Dropout(r, 0.5), residual=z(4, 16, dtype=torch.float16)),
                lambda: spc.dropout_bwd(x, spc.Dropout(r, 0.5), din=z(4, 16, dtype=torch.float16))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: spc.Dropout(z(3, dtype=torch.int64), 0.5), lambda: spc.Dropout(r, 1.5),
                lambda: spc.Dropout(r, 0.5, -1), lambda: spc.Dropout(r, 0.5, 1 << 32),
                lambda: spc.dropout_fwd(z(16, 4).t(), spc.Dropout(r, 0.5)),
                lambda: spc.dropout_fwd(x, spc.Dropout(r, 0.5), residual=z(4, 32))):
        with pytest.raises(ValueError):
            bad()


def test_group_norm_tensors():
    x = z(8, 32)
    for bad in (lambda: spc.group_norm_fwd(z(8, 32, dtype=torch.float64), 4),
                lambda: spc.group_norm_fwd(x, 4, torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: spc.group_norm_fwd(x, 4, gamma=z(32, dtype=torch.float16)),
                lambda: spc.group_norm_fwd(x, 4, dropout=0.5)):
        with pytest.raises(TypeError):
            bad()
    st = z(1, 4, 2)
    for bad in (lambda: spc.group_norm_fwd(x, 4, act="gelu"), lambda: spc.group_norm_fwd(z(32, 8).t(), 4),
                lambda: spc.group_norm_fwd(z(32), 4), lambda: spc.group_norm_fwd(x, 4, gamma=z(16)),
                lambda: spc.group_norm_fwd(x, 4, z(1, dtype=torch.int32)),
                lambda: spc.group_norm_fwd(x, 4, out=z(8, 16)),
                lambda: spc.group_norm_bwd(x, x, 4, None, None, None, z(1, 8, 2)),
                lambda: spc.group_norm_bwd(z(4, 32), x, 4, None, None, None, st)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: spc.group_norm_fwd(z(8, 24), 4), lambda: spc.group_norm_fwd(x, 5),
                lambda: spc.group_norm_fwd(x, 4, eps=0.0)):
        with pytest.raises(spc.SpcError):
            bad()


def test_linear_recurrence_tensors():
    x = z(8, 32)
    c = spc.linear_recurrence_fwd(x, x, want_carry=True)[2]
    for bad in (lambda: spc.linear_recurrence_fwd(x, z(8, 32, dtype=torch.float64)),
                lambda: spc.linear_recurrence_fwd(x, x, order=torch.zeros(8, dtype=torch.int64, device="cuda")),
                lambda: spc.linear_recurrence_fwd(x, x, h0=z(1, 32, dtype=torch.float16))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: spc.linear_recurrence_fwd(x, z(8, 32, dtype=torch.float16)),
                lambda: spc.linear_recurrence_fwd(z(32, 8).t(), z(32, 8).t()),
                lambda: spc.linear_recurrence_fwd(x, z(8, 64)[:, :32]),
                lambda: spc.linear_recurrence_fwd(x, x, h0=z(2, 32)),
                lambda: spc.linear_recurrence_fwd(x, x, order=z(7, dtype=torch.int32)),
                lambda: spc.linear_recurrence_bwd(z(8, 16), x, x, None, c),
                lambda: spc.linear_recurrence_bwd(x, x, x, None, c[:-4].clone()),
                lambda: spc.linear_recurrence_bwd(x, x, x, None, c, dgate=x),
                lambda: spc.linear_recurrence_bwd(x, x, x, None, c, dgate=x, dx=z(8, 64)[:, :32]),
                lambda: spc.linear_recurrence_step(x, x, z(7, 32)),
                lambda: spc.linear_recurrence_step(x, x, x, new_state=z(7, 32))):
        with pytest.raises(ValueError):
            bad()
    wide = z(8, 68, dtype=torch.float16)        # rows 136 bytes apart: not 16-byte aligned
    with pytest.raises(spc.SpcError):
        spc.linear_recurrence_fwd(wide[:, :32], wide[:, 32:64])
    shifted = z(8, 72, dtype=torch.float16)     # a slice that starts 8 bytes in
    with pytest.raises(spc.SpcError):
        spc.linear_recurrence_fwd(shifted[:, 4:36], shifted[:, 36:68])
