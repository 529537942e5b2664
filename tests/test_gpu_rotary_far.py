"""Rotary positions as far as int32 reaches."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle.rowops import EPS
from tests.parity import cuda
from tests.rowops_cases import within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("span", [1, 1 << 20, (1 << 31) - 1])
def test_angles_of_far_positions(span):
    """The product of an int32 and an fp32 number, up to 2^33 radians here, is
    reduced exactly: the bound is the fp32 sine's and rotation's alone.  The
    reference takes it in 64 bits of fraction, off by less than 2^33 2^-64."""
    if np.finfo(np.longdouble).nmant < 63:
        pytest.skip("no 64-bit fractions on this host")
    g = torch.Generator().manual_seed(7)
    n = 4000
    pos = torch.randint(span - span // 100, span + 1, (n, 1), generator=g, dtype=torch.int64)
    pos = torch.where(torch.rand(n, 1, generator=g) < 0.5, pos, -pos).int()
    f = torch.rand(16, generator=g) * 3 + 1
    x = torch.randn(n, 1, 32, generator=g)
    out = spc.rotary(cuda(x), cuda(pos), cuda(f), (16,))
    t = pos.numpy().astype(np.longdouble) * f.numpy().astype(np.longdouble)[None]
    c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
    a, b = x.double().numpy()[..., 0::2], x.double().numpy()[..., 1::2]
    ref, env = np.empty((n, 1, 32)), np.empty((n, 1, 32))
    ref[..., 0::2], ref[..., 1::2] = a * c - b * s, a * s + b * c
    env[..., 0::2] = env[..., 1::2] = 6 * EPS * (np.abs(a) + np.abs(b))
    within(out, ref, env, torch.float32, "out")
