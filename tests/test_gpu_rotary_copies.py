"""Rotary positions: pairs past the axes are copied bit by bit, whatever they hold."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from tests.parity import cuda
from tests.rowops_cases import DTYPES

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,pairs", [(16, (0,)), (16, (1,)), (16, (4,)), (32, (2, 3, 0)), (48, (5, 5, 6)), (128, (10, 0, 20))])
def test_pairs_past_the_axes_are_copied(D, pairs, inverse, dtype):
    g = torch.Generator().manual_seed(D + len(pairs))
    x = torch.randn(200, 3, D, generator=g).to(dtype)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf"), -0.0, 0.0, torch.finfo(dtype).max, torch.finfo(dtype).tiny / 8])
    at = torch.randint(0, 14, x.shape, generator=g)
    x = torch.where(at < 7, odd.to(dtype)[at.clamp(max=6)], x)
    rotated = 2 * sum(pairs)
    x[..., :rotated] = torch.randn(200, 3, rotated, generator=g).to(dtype)
    pos = torch.randint(-1600, 1600, (200, len(pairs)), generator=g, dtype=torch.int32)
    f = torch.rand(sum(pairs), generator=g)
    out = spc.rotary(cuda(x), cuda(pos), cuda(f), pairs, inverse=inverse)
    assert torch.equal(bits(out)[..., rotated:], bits(x)[..., rotated:])
    assert torch.isfinite(out[..., :rotated].float()).all()
    y = cuda(x)
    assert torch.equal(bits(spc.rotary(y, cuda(pos), cuda(f), pairs, inverse=inverse, out=y)), bits(out))
