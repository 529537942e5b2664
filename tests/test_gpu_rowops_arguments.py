"""The row operators' workspaces are checked, and a dropout's later values take effect."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from sparse_convolution_hash_amd import binding as B

pytestmark = pytest.mark.gpu


def test_workspaces_are_checked():
    n, C = 5000, 64
    x = torch.randn(n, C, device="cuda")
    _, stats = spc.group_norm_fwd(x, 8)
    _, _, carry = spc.linear_recurrence_fwd(x, x, want_carry=True)
    need = max(B.group_norm_workspace(n, C, 8, 1), B.linear_recurrence_workspace(x.dtype, n, C, 1)[0])
    coords = torch.stack([torch.zeros(n, dtype=torch.int32), *(torch.arange(n, dtype=torch.int32) // d % 20 for d in (400, 20, 1))], 1).cuda()
    calls = [lambda w: spc.group_norm_fwd(x, 8, workspace=w),
             lambda w: spc.group_norm_bwd(x, x, 8, None, None, None, stats, workspace=w),
             lambda w: spc.linear_recurrence_fwd(x, x, workspace=w),
             lambda w: spc.linear_recurrence_bwd(x, x, x, None, carry, workspace=w),
             lambda w: spc.conv_bwd_filter(x, x, 1, None, None, None, workspace=w),
             lambda w: spc.build_kmap(coords, 1, (20, 20, 20), 3, workspace=w)]
    for call in calls:
        with pytest.raises(TypeError, match="workspace"):
            call(torch.empty(need, dtype=torch.uint8))
        with pytest.raises(ValueError, match="workspace"):
            call(torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
        call(torch.empty(need + (1 << 22), dtype=torch.uint8, device="cuda"))


def test_dropout_values_set_later():
    x = torch.randn(3000, 16, device="cuda")
    a, b = (torch.tensor(v, dtype=torch.int64, device="cuda") for v in ([5, 6], [7, 8]))
    drop = spc.Dropout(a, 0.5, 1)
    fresh = lambda *args: spc.dropout_fwd(x, spc.Dropout(*args))
    assert torch.equal(spc.dropout_fwd(x, drop), fresh(a, 0.5, 1))
    drop.p = 0.1
    assert torch.equal(spc.dropout_fwd(x, drop), fresh(a, 0.1, 1))
    drop.layer = 4
    assert torch.equal(spc.dropout_fwd(x, drop), fresh(a, 0.1, 4))
    drop.rng = b
    want = fresh(b, 0.1, 4)
    del b
    assert torch.equal(spc.dropout_fwd(x, drop), want) and not torch.equal(want, fresh(a, 0.1, 4))
    y, st = spc.group_norm_fwd(x, 2, dropout=drop)
    assert torch.equal(y, spc.group_norm_fwd(x, 2, dropout=spc.Dropout(drop.rng, 0.1, 4))[0])
    with pytest.raises(TypeError):
        drop.rng = torch.zeros(2, dtype=torch.int64)
