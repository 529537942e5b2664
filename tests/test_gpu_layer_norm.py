"""Layer norm, forward and backward, against the fp64 oracle: channels from one
pair of lanes to eight steps of a wave, a residual, rows far from 0, no rows."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from sparse_convolution_hash_amd import binding as B
from tests.parity import cuda
from tests.rowops_cases import DTYPES, half_step, within

pytestmark = pytest.mark.gpu

SIZES = [(1, 16), (7, 48), (130, 16), (1000, 80), (513, 128), (77, 512), (64, 528), (33, 1024), (21, 1040), (9, 2064), (5, 4096),
         (9000, 64)]


def inputs(n, C, dtype, seed, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (r(n, C) * (0.5 + torch.rand(C, generator=g)) + mean * r(C)).to(dtype)
    return x, (r(n, C) * 0.7).to(dtype), 1.0 + 0.3 * r(C), 0.3 * r(C), r(n, C).to(dtype), r(n, C).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C", SIZES)
def test_forward_and_backward(n, C, dtype):
    print(f"layer norm {n} x {C} {dtype}", flush=True)
    x, _, gamma, beta, dy, _ = inputs(n, C, dtype, n + C)
    y, stats, total = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta), 1e-5)
    assert total is None
    ref, mean, rstd, env = A.layer_norm_fwd(x, gamma, beta, 1e-5)
    within(y, ref, env, dtype, "y")
    assert np.allclose(f64(stats)[:, 1], rstd, rtol=1e-5) and np.allclose(f64(stats)[:, 0], mean, rtol=1e-5, atol=1e-5)
    dx, dg, db = spc.layer_norm_bwd(cuda(dy), cuda(x), cuda(gamma), stats)
    rx, rg, rb, ex, eg, eb = A.layer_norm_bwd(dy, x, gamma, 1e-5)
    within(dx, rx, ex, dtype, "dx")
    within(dg, rg, eg, torch.float32, "dgamma")
    within(db, rb, eb, torch.float32, "dbeta")
    again = spc.layer_norm_bwd(cuda(dy), cuda(x), cuda(gamma), stats, dx=cuda(dy))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dg) and torch.equal(again[2], db)
    assert torch.equal(spc.layer_norm_bwd(cuda(dy), cuda(x), cuda(gamma), stats, want_affine=False)[0], dx)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C", [(300, 48), (70, 1024)])
def test_residual(n, C, dtype):
    x, res, gamma, beta, dy, dt = inputs(n, C, dtype, n * C)
    y, stats, total = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta), 1e-5, residual=cuda(res))
    assert torch.equal(total.cpu(), (x.float() + res.float()).to(dtype))
    ref, _, _, env = A.layer_norm_fwd(total, gamma, beta, 1e-5)
    within(y, ref, env, dtype, "y")
    dx, dg, _ = spc.layer_norm_bwd(cuda(dy), total, cuda(gamma), stats, dtotal=cuda(dt))
    rx, rg, _, ex, eg, _ = A.layer_norm_bwd(dy, total, gamma, 1e-5, dtotal=dt)
    within(dx, rx, ex, dtype, "dx")
    within(dg, rg, eg, torch.float32, "dgamma")
    # in place: the sum over x, the result over x, the gradient over dtotal
    a = cuda(x)
    y2, _, t2 = spc.layer_norm_fwd(a, cuda(gamma), cuda(beta), 1e-5, residual=cuda(res), total=a)
    assert t2 is a and torch.equal(a, total) and torch.equal(y2, y)
    b = cuda(dt)
    assert torch.equal(spc.layer_norm_bwd(cuda(dy), total, cuda(gamma), stats, dtotal=b, dx=b)[0], dx)
    c = cuda(x)
    plain = spc.layer_norm_fwd(cuda(x), cuda(gamma))[0]
    assert torch.equal(spc.layer_norm_fwd(c, cuda(gamma), out=c)[0], plain)


@pytest.mark.parametrize("scale", [1.0, 300.0, 10000.0])
def test_rows_far_from_zero(scale):
    # the spread next to the mean is down to 1e-4: the envelope grows with it only by the mean's own rounding
    x, _, gamma, beta, dy, _ = inputs(64, 96, torch.float32, 5, 0.0)
    x = x + scale * torch.arange(1.0, 65.0)[:, None]
    y, stats, _ = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta))
    ref, _, _, env = A.layer_norm_fwd(x, gamma, beta, 1e-5)
    within(y, ref, env, torch.float32, "y")
    assert env.max() < 1e-4 * max(1.0, np.abs(ref).max())
    dx, dg, db = spc.layer_norm_bwd(cuda(dy), cuda(x), cuda(gamma), stats)
    rx, rg, rb, ex, eg, eb = A.layer_norm_bwd(dy, x, gamma, 1e-5)
    within(dx, rx, ex, torch.float32, "dx")
    within(dg, rg, eg, torch.float32, "dgamma")


def test_constant_rows_and_defaults():
    x = torch.full((5, 32), 3.0)
    y, stats, _ = spc.layer_norm_fwd(cuda(x))
    assert not y.any() and np.allclose(f64(stats), [[3.0, 1e-5 ** -0.5]] * 5, rtol=1e-6)
    dx, dg, db = spc.layer_norm_bwd(cuda(torch.ones(5, 32)), cuda(x), None, stats)
    assert not dx.any() and not dg.any() and torch.equal(db.cpu(), torch.full((32,), 5.0))


def test_no_rows():
    x = torch.empty(0, 32, device="cuda")
    y, stats, _ = spc.layer_norm_fwd(x)
    assert y.shape == (0, 32) and stats.shape == (0, 2)
    dx, dg, db = spc.layer_norm_bwd(x, x, None, stats)
    assert dx.shape == (0, 32) and not dg.any() and not db.any()


def test_nan_stays_in_its_row():
    x, _, gamma, beta, dy, _ = inputs(40, 64, torch.bfloat16, 9)
    y0 = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta))[0].clone()
    x[7, 3], x[9, 5] = float("nan"), float("inf")
    y = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta))[0]
    keep = [i for i in range(40) if i not in (7, 9)]
    assert y[7].isnan().all() and y[9].isnan().all() and torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("n,C", [(5000, 64), (70000, 128)])
def test_workspace(n, C):
    x, _, gamma, _, dy, _ = inputs(n, C, torch.bfloat16, 3)
    x, dy, gamma = cuda(x), cuda(dy), cuda(gamma)
    stats = spc.layer_norm_fwd(x, gamma)[1]
    need, runs = B.layer_norm_workspace(n, C), []
    assert need > 0
    for byte in (0, 255, 127):
        buf = torch.full((need + 4096,), byte, dtype=torch.uint8, device="cuda")
        runs.append(spc.layer_norm_bwd(dy, x, gamma, stats, workspace=buf[:need]))
        assert (buf[need:] == byte).all()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_gradient_against_differences():
    x, _, gamma, beta, dy, _ = inputs(3, 16, torch.float32, 8)
    f = lambda x: (A.layer_norm_fwd(x, gamma, beta, 1e-5)[0] * f64(dy)).sum()
    stats = spc.layer_norm_fwd(cuda(x), cuda(gamma), cuda(beta))[1]
    dx = f64(spc.layer_norm_bwd(cuda(dy), cuda(x), cuda(gamma), stats)[0])
    x = f64(x).copy()
    for i in np.ndindex(x.shape):
        s, d = x[i], []
        for e in (1e-5, -1e-5):
            x[i] = s + e
            d.append(f(x))
        x[i] = s
        assert abs((d[0] - d[1]) / 2e-5 - dx[i]) < 1e-5
