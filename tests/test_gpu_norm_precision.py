"""GPU group norm statistics on whole numbers: every difference, square and sum
of a run is exact in fp32, so what is left are the roundings of the runs' stored
means and spreads and of the results, a few units whatever the sizes."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, ptr_of, ragged

pytestmark = pytest.mark.gpu

EPS_VAR = 1e-5


def runs_of(ptr, step):
    """(sample, rows) of the pieces that multiples of step cut the samples into."""
    for s, (a, b) in enumerate(zip(ptr, ptr[1:])):
        while a < b:
            e = min(b, (a // step + 1) * step)
            yield s, slice(a, e)
            a = e


def check_stats(x, ptr, G, stats, step, what):
    """stats against 64 bits.  Per run and channel two numbers are stored in
    fp32: the spread (one rounding) and the mean (one, of half a unit of the
    mean); the rest is in double.  A mean that is off by e moves the variance by
    rows (2 |mean - group mean| e + e^2) / count."""
    x = R.f64(x)
    S, C = len(ptr) - 1, x.shape[1]
    cg, u = C // G, R.EPS
    _, mean, rstd = R._norm(x, G, ptr, EPS_VAR)
    e_var, e_mean = np.zeros((S, G)), np.zeros((S, G))
    for s, rows in runs_of(ptr, step):
        v = x[rows]
        m, count = v.mean(0), (ptr[s + 1] - ptr[s]) * cg
        spread, e = ((v - m) ** 2).sum(0), u * np.abs(m)
        far = np.abs(m - np.repeat(mean[s], cg))
        e_var[s] += (u * spread + len(v) * (2 * far * e + e * e)).reshape(G, cg).sum(1) / count
        e_mean[s] += (len(v) * e).reshape(G, cg).sum(1) / count
    # the last roundings, and the double arithmetic (far below a unit)
    b_mean = e_mean + u * np.abs(mean) + 1e-12
    b_rstd = rstd * (0.5 * e_var * rstd ** 2 * (1 + 1e-6) + u + 1e-9)
    g = stats.double().cpu().numpy()
    for got, want, bound, name in ((g[..., 0], mean, b_mean, "mean"), (g[..., 1], rstd, b_rstd, "rstd")):
        worst = (np.abs(got - want) / bound).max()
        assert worst <= 1, f"{what}: {name} off by {worst:.3g} times its bound"


def whole(seed, n, C, top):
    return torch.randint(-top, top + 1, (n, C), generator=torch.Generator().manual_seed(seed)).float()


@pytest.mark.parametrize("C,G,tile", [(16, 1, 512), (16, 2, 512), (64, 8, 128), (48, 3, 168)])
def test_norm_first_rows_of_runs_are_outliers(C, G, tile):
    # first rows 700 from all others: at a sample's start and at the start of a
    # later tile, in runs of lengths that are no powers of two
    ptr = [0, 1733, 5000, 9000]
    x = whole(C, 9000, C, 2)
    for r in (0, 1536, 1733, 4608, 5000, 8704):
        x[r] = 700.0 if r % 2 else -700.0
    print(f"outliers C={C} G={G}", flush=True)
    _, stats = spc.group_norm_fwd(cuda(x), G, cuda(torch.tensor(ptr, dtype=torch.int32)), eps=EPS_VAR)
    check_stats(x, ptr, G, stats, tile, "outliers")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C,G,S,tile", [(500, 32, 4, 3, 500), (1000, 16, 2, 1, 1000), (20011, 48, 3, 37, 168), (30000, 64, 8, 4, 128)])
def test_norm_whole_numbers(dtype, n, C, G, S, tile):
    ptr = ptr_of(ragged(n, n, S))
    x, dy = whole(n, n, C, 8).to(dtype), whole(n + 1, n, C, 8).to(dtype)
    print(f"whole numbers n={n} C={C} {dtype}", flush=True)
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    _, stats = spc.group_norm_fwd(cuda(x), G, sp, eps=EPS_VAR)
    check_stats(x, ptr, G, stats, tile, "whole numbers")
    _, _, db = spc.group_norm_bwd(cuda(dy), cuda(x), G, sp, None, None, stats)
    assert torch.equal(db.cpu().double(), dy.double().sum(0))      # below 2^24: exact
