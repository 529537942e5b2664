"""GPU group norm (activation, dropout, ragged samples) and its backward
against the fp64 oracle."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, half_step, ptr_of, ragged, within

pytestmark = pytest.mark.gpu

EPS_VAR = 1e-5


def case(seed, n, C, dtype, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, C, generator=g) * (0.5 + torch.rand(C, generator=g)) + offset * torch.randn(C, generator=g))
    dy = torch.randn(n, C, generator=g)
    return x.to(dtype), dy.to(dtype), 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)


def segment_means(v, ptr, G):
    out = np.zeros_like(v)
    for a, b in zip(ptr, ptr[1:]):
        if b > a:
            m = v[a:b].reshape(b - a, G, -1).mean((0, 2))
            out[a:b] = np.repeat(m, v.shape[1] // G)[None]
    return out


def envelopes(x, dy, G, ptr, gamma, beta, name, factor, K):
    """Bounds on the fp32 computation.  xhat: the mean's rounding, and K
    roundings of values of the size of the spread (sums of a run, their
    combination, rstd); everything after it is a handful of roundings."""
    xhat, mean, rstd = R._norm(x, G, ptr, EPS_VAR)
    n, C = x.shape
    rs, mm = np.zeros((n, C)), np.zeros((n, C))
    for s, (a, b) in enumerate(zip(ptr, ptr[1:])):
        rs[a:b], mm[a:b] = np.repeat(rstd[s], C // G)[None], np.repeat(mean[s], C // G)[None]
    e_hat = R.EPS * (rs * np.abs(mm) + K * (1 + np.abs(xhat)))
    ag, z = np.abs(gamma), np.abs(gamma * xhat) + np.abs(beta)
    e_y = factor * (1.1 * ag * e_hat + 16 * R.EPS * z)
    if dy is None:
        return e_y, None, None, None
    d = np.abs(dy * factor)
    # the slope of an activation is at most 1.1 and changes at most 0.5 per unit of z
    dz = 1.1 * d
    e_dz = d * (0.5 * ag * e_hat + 16 * R.EPS * (1 + z))
    w, e_w = ag * dz, ag * e_dz
    mean_of = lambda v: segment_means(v, ptr, G)
    e_m1 = mean_of(e_w) + 64 * R.EPS * mean_of(w)
    m2 = mean_of(w * np.abs(xhat))
    e_m2 = mean_of(e_w * np.abs(xhat) + w * e_hat) + 64 * R.EPS * m2
    e_dx = rs * (e_w + e_m1 + np.abs(xhat) * e_m2 + m2 * e_hat + K * R.EPS * (w + mean_of(w) + np.abs(xhat) * m2))
    e_dgamma = (dz * e_hat + np.abs(xhat) * e_dz).sum(0) + 64 * R.EPS * (dz * np.abs(xhat)).sum(0)
    e_dbeta = e_dz.sum(0) + 64 * R.EPS * dz.sum(0)
    return e_y, e_dx, e_dgamma, e_dbeta


def run(n, C, G, lengths, dtype, name, drop=None, seed=0, K=256, x=None, ptr=None):
    xr, dy, gamma, beta = case(seed, n, C, dtype)
    x = xr if x is None else x
    ptr = ptr_of(lengths) if ptr is None else ptr
    print(f"group norm n={n} C={C} G={G} lengths={str(lengths)[:60]} {dtype} {name} drop={drop}", flush=True)
    if name == "relu":      # next to its corner the slope is whichever side fp32 falls on: no gradient comes in there
        near = np.abs(R._norm(R.f64(x), G, ptr, EPS_VAR)[0] * R.f64(gamma) + R.f64(beta)) < 1e-4
        dy = torch.where(torch.from_numpy(near), torch.zeros_like(dy), dy)
    factor, d = 1.0, None
    if drop:
        factor = R.drop_factor(drop[0], drop[1], drop[2], drop[3], (n, C))
        d = spc.Dropout(torch.tensor(drop[:2], dtype=torch.int64, device="cuda"), drop[3], drop[2])
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    y, stats = spc.group_norm_fwd(cuda(x), G, sp, cuda(gamma), cuda(beta), eps=EPS_VAR, act=name, dropout=d)
    ga, be, xx, dd = R.f64(gamma), R.f64(beta), R.f64(x), R.f64(dy)
    e_y, e_dx, e_g, e_b = envelopes(xx, dd, G, ptr, ga, be, name, factor, K)
    ry, mean, rstd = R.group_norm_fwd(xx, G, ptr, ga, be, EPS_VAR, name, factor)
    rows = slice(ptr[0], ptr[-1])
    within(y[rows], ry[rows], e_y[rows], dtype, "y")
    spread = (rstd ** -2 - EPS_VAR).clip(0) ** 0.5
    within(stats[..., 0], mean, R.EPS * K * spread, torch.float32, "mean")
    within(stats[..., 1], rstd, R.EPS * K * rstd, torch.float32, "rstd")
    dx, dgamma, dbeta = spc.group_norm_bwd(cuda(dy), cuda(x), G, sp, cuda(gamma), cuda(beta), stats, act=name, dropout=d)
    rx, rg, rb = R.group_norm_bwd(dd, xx, G, ptr, ga, be, EPS_VAR, name, factor)
    within(dx[rows], rx[rows], e_dx[rows], dtype, "dx")
    within(dgamma, rg, e_g, torch.float32, "dgamma")
    within(dbeta, rb, e_b, torch.float32, "dbeta")
    return y, stats, dx, dgamma, dbeta


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu"])
@pytest.mark.parametrize("n,C,G,s", [(300, 64, 8, 3), (129, 48, 3, 5), (1000, 80, 10, 1)])
def test_norm_activations(dtype, name, n, C, G, s):
    run(n, C, G, ragged(n, n, s), dtype, name, seed=n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 2049, 5000])
def test_norm_row_counts(dtype, n):
    run(n, 32, 4, [n], dtype, "silu", seed=n)
    run(n, 32, 4, ragged(n, n, 7), dtype, "none", seed=n + 1)


@pytest.mark.parametrize("C,G", [(16, 16), (16, 1), (48, 16), (48, 48), (112, 7), (128, 1), (272, 17), (528, 33), (1040, 5)])
def test_norm_channels_and_groups(C, G):
    # one-channel groups, groups within eight channels, across workgroups, one group
    run(400, C, G, [150, 0, 1, 249], torch.float32, "silu", seed=C)
    run(400, C, G, [400], torch.bfloat16, "none", seed=C + 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_large(dtype):
    run(70001, 64, 16, [40000, 0, 1, 30000], dtype, "silu", seed=3)


def test_norm_many_short_samples():
    run(3000, 32, 8, [1, 0, 2, 3] * 500, torch.float32, "silu", seed=4)
    run(1200, 64, 8, [1] * 1200, torch.float16, "none", seed=5)


def test_norm_dropout_is_the_composition():
    n, C, G = 700, 96, 12
    drop = (12345678901, 77, 9, 0.3)
    y, *_ = run(n, C, G, [200, 500], torch.bfloat16, "silu", drop=drop, seed=6)
    # the kept positions are those of the dropout call on the same tensor
    keep = torch.from_numpy(R.keep_mask(*drop, n * C).reshape(n, C))
    assert (y.cpu()[~keep] == 0).all() and (y.cpu()[keep] != 0).float().mean() > 0.99
    run(333, 16, 1, [333], torch.float32, "none", drop=(1, 2, 3, 1.0), seed=7)


def test_norm_far_from_zero():
    # mean 1000 times the spread: the variance comes from differences
    g = torch.Generator().manual_seed(9)
    x = 1000.0 + torch.randn(3000, 32, generator=g)
    run(3000, 32, 4, [1000, 2000], torch.float32, "none", seed=9, x=x)


def test_norm_first_row_is_an_outlier():
    # the row that differences are taken from lies far from all others: its
    # square enters the sum once per row, so K grows by up to the 128 rows of a run
    g = torch.Generator().manual_seed(10)
    x = torch.randn(1000, 32, generator=g)
    x[0] = 1e4
    run(1000, 32, 4, [1000], torch.float32, "none", seed=10, x=x, K=256 * 128)


def test_norm_constant_sample():
    x = torch.full((500, 32), 3.25)
    y, stats, dx, _, _ = run(500, 32, 4, [500], torch.float32, "none", seed=11, x=x)
    assert (stats[..., 0] == 3.25).all()


def test_norm_rows_outside_every_sample():
    n, C = 600, 32
    x, dy, gamma, beta = case(12, n, C, torch.float32)
    ptr = [100, 250, 500]
    run(n, C, 4, "100..250..500", torch.float32, "silu", seed=12, ptr=ptr)
    sp, out = cuda(torch.tensor(ptr, dtype=torch.int32)), torch.full((n, C), 7.0, device="cuda")
    x = x.clone()
    x[:100], x[500:] = float("nan"), float("inf")
    y, stats = spc.group_norm_fwd(cuda(x), 4, sp, act="silu", out=out)
    assert (y[:100] == 7).all() and (y[500:] == 7).all() and torch.isfinite(y).all()
    dx, dg, db = spc.group_norm_bwd(cuda(dy), cuda(x), 4, sp, None, None, stats, act="silu",
                                    dx=torch.full((n, C), 7.0, device="cuda"))
    assert (dx[:100] == 7).all() and (dx[500:] == 7).all()
    assert torch.isfinite(dx).all() and torch.isfinite(dg).all() and torch.isfinite(db).all()


def test_norm_nan_stays_in_its_group():
    n, C, G = 500, 64, 4
    x, dy, gamma, beta = case(13, n, C, torch.bfloat16)
    ptr = [0, 200, 500]
    x[130, 17] = float("nan")
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    y, stats = spc.group_norm_fwd(cuda(x), G, sp, cuda(gamma), cuda(beta), act="silu")
    bad = torch.isnan(y).cpu()
    assert bad[:200, 16:32].all() and not bad[200:].any() and not bad[:, :16].any() and not bad[:, 32:].any()
    dx, _, _ = spc.group_norm_bwd(cuda(dy), cuda(x), G, sp, cuda(gamma), cuda(beta), stats, act="silu")
    bad = torch.isnan(dx).cpu()
    assert bad[:200, 16:32].all() and not bad[200:].any() and not bad[:, :16].any() and not bad[:, 32:].any()


def test_norm_no_rows_no_affine_in_place():
    sp = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, stats = spc.group_norm_fwd(torch.empty((0, 32), device="cuda"), 4, sp)
    assert y.shape == (0, 32) and (stats[..., 0] == 0).all()
    assert torch.allclose(stats[..., 1], torch.tensor(1e-5 ** -0.5, device="cuda"))
    dx, dg, db = spc.group_norm_bwd(y, y, 4, sp, None, None, stats)
    assert (dg == 0).all() and (db == 0).all()
    x, dy, *_ = case(14, 900, 48, torch.float16)
    xc = cuda(x)
    y, stats = spc.group_norm_fwd(xc, 6, act="silu")
    one, zero = torch.ones(48, device="cuda"), torch.zeros(48, device="cuda")
    assert torch.equal(y, spc.group_norm_fwd(xc, 6, cuda(torch.tensor([0, 900], dtype=torch.int32)), one, zero, act="silu")[0])
    buf = xc.clone()
    assert torch.equal(spc.group_norm_fwd(buf, 6, act="silu", out=buf)[0], y)
    dx, dg, db = spc.group_norm_bwd(cuda(dy), xc, 6, None, None, None, stats, act="silu")
    buf = cuda(dy)
    dx2, no1, no2 = spc.group_norm_bwd(buf, xc, 6, None, None, None, stats, act="silu", want_affine=False, dx=buf)
    assert torch.equal(dx, dx2) and no1 is None and no2 is None


def test_norm_repeats_bit_for_bit():
    x, dy, gamma, beta = (cuda(t) for t in case(15, 40000, 96, torch.bfloat16))
    sp = cuda(torch.tensor([0, 15000, 40000], dtype=torch.int32))

    def once():
        y, st = spc.group_norm_fwd(x, 12, sp, gamma, beta, act="silu")
        return (y, st) + spc.group_norm_bwd(dy, x, 12, sp, gamma, beta, st, act="silu")
    a, b = once(), once()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_norm_gradient_by_differences():
    # the directional derivative of sum(y * w) against the returned gradients
    n, C, G = 200, 16, 4
    x, w, gamma, beta = (cuda(t) for t in case(16, n, C, torch.float32))
    sp = cuda(torch.tensor([0, 80, 200], dtype=torch.int32))
    y, stats = spc.group_norm_fwd(x, G, sp, gamma, beta, act="silu")
    dx, dg, db = spc.group_norm_bwd(w, x, G, sp, gamma, beta, stats, act="silu")
    g = torch.Generator().manual_seed(17)
    ux, ug, ub = cuda(torch.randn(n, C, generator=g)), cuda(torch.randn(C, generator=g)), cuda(torch.randn(C, generator=g))
    h = 2.0 ** -7

    def loss(t):
        y, _ = spc.group_norm_fwd(x + t * ux, G, sp, gamma + t * ug, beta + t * ub, act="silu")
        return (y.double() * w.double()).sum().item()
    diff = (loss(h) - loss(-h)) / (2 * h)
    want = sum((a.double() * b.double()).sum().item() for a, b in ((dx, ux), (dg, ug), (db, ub)))
    # third derivative along a unit-variance direction, times h^2 / 6; and 3200 roundings of y over 2 h
    assert abs(diff - want) < 3200 * (h * h) + 3200 * 2.0 ** -22 / h
