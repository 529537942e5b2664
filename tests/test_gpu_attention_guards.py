"""Offsets that fall or leave the arrays, and order entries that name no row:
nothing outside the arrays is written, and nothing from outside reaches a result.
Every array is the middle of a larger one: inputs lie between NaN, outputs between
marks."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from tests.rowops_cases import DTYPES

pytestmark = pytest.mark.gpu

N, SIDE, MARK = 100, 70, 55.0


def between(t, around):
    w = torch.full((t.shape[0] + 2 * SIDE,) + tuple(t.shape[1:]), around, dtype=t.dtype, device="cuda")
    w[SIDE:-SIDE] = t.to("cuda")
    return w, w[SIDE:-SIDE]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("offsets", [[0, 60, 20, 100], [-5, 30, 400, 1000], [90, 10, 95, 3], [-(2 ** 31), 2 ** 31 - 1, 50, 50], [100, 100, 100, 0]])
@pytest.mark.parametrize("entries", [None, [-1, N, 2 ** 31 - 1, -(2 ** 31)]])
def test_guards(entries, offsets, causal, D, dtype):
    g = torch.Generator().manual_seed(9)
    r = lambda h: torch.randn(N, h, D, generator=g).to(dtype)
    ins = [between(r(h), float("nan")) for h in (4, 2, 2, 4)]
    q, k, v, do = (t for _, t in ins)
    ptr = between(torch.tensor(offsets, dtype=torch.int32), -7)[1].clone()     # a call's offsets are aligned to 16 bytes
    order = None
    if entries is not None:
        order = torch.randperm(N, generator=g).int()
        order[::9] = torch.tensor(entries)[torch.arange(0, N, 9) % 4].int()
        order = order.to("cuda")
    outs = [between(torch.full((N, h, D), 1.0, dtype=dtype), MARK) for h in (4, 4, 2, 2)]
    out, dq, dk, dv = (t for _, t in outs)
    _, st = spc.attention_fwd(q, k, v, ptr, order, causal=causal, want_stats=True, out=out)
    assert torch.isfinite(out.float()).all()
    # rows of no sample have no statistics: what they are left with is of no consequence, but has to be numbers here
    st = (torch.nan_to_num(st[0], 0.0, 0.0, 0.0), None if st[1] is None else torch.nan_to_num(st[1], 0.0, 0.0, 0.0))
    spc.attention_bwd(do, q, k, v, out, st, ptr, order, causal=causal, dq=dq, dk=dk, dv=dv)
    for w, _ in outs:
        assert (w[:SIDE] == MARK).all() and (w[-SIDE:] == MARK).all()
    for w, _ in ins:
        assert w[:SIDE].isnan().all() and w[-SIDE:].isnan().all()
