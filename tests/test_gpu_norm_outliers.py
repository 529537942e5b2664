"""GPU group norm of samples whose first rows lie far from all others, which are
nearly or wholly constant: the variance keeps fp32's precision."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda

pytestmark = pytest.mark.gpu

EPS_VAR, U = 1e-5, R.EPS


def rstd_bound(x, ptr, G, lanes, tile):
    """(rstd, bound).  A thread sums differences from k, the median of a run's
    first, middle and last row, over its m rows of the run, in fp32: s1 is off by
    (1 + m) U sum |d|, s2 by (3 + m) U sum d^2, and around the run's mean that is
    e2 + 2 |k - mean| e1 of the spread.  Everything above is double but the stored
    pair of a run, its spread and mean (tile: rows of a run; in one launch nothing
    is stored)."""
    x = R.f64(x)
    C = x.shape[1]
    S, cg = len(ptr) - 1, C // G
    _, mean, rstd = R._norm(x, G, ptr, EPS_VAR)
    e_var = np.zeros((S, G))
    for s, (a, b) in enumerate(zip(ptr, ptr[1:])):
        start = a
        while start < b:
            end = min(b, (start // tile + 1) * tile) if tile else b
            v = x[start:end]
            m = v.mean(0)
            e, k = np.zeros(C), np.median(v[[0, len(v) // 2, -1]], axis=0)
            for lane in range(min(lanes, len(v))):
                w = v[lane::lanes]
                d = np.abs(w - k)
                e += (3 + len(w)) * U * (d * d).sum(0) + 2 * np.abs(k - m) * (1 + len(w)) * U * d.sum(0)
            if tile:
                off = U * np.abs(m)
                e += U * ((v - m) ** 2).sum(0) + len(v) * (2 * np.abs(m - np.repeat(mean[s], cg)) * off + off * off)
            e_var[s] += e.reshape(G, cg).sum(1) / ((b - a) * cg)
            start = end
    return rstd, rstd * (0.5 * e_var * rstd ** 2 * (1 + 1e-3) + U + 1e-8)


# lanes: rows that a workgroup of 512 (one launch) or 256 threads takes side by side
@pytest.mark.parametrize("n,C,G,ptr,lanes,tile", [
    (1000, 32, 4, [0, 1000], 512, 0),
    (2000, 16, 2, [0, 700, 2000], 512, 0),
    (9000, 16, 1, [0, 1733, 9000], 128, 512),
    (9000, 64, 8, [0, 4000, 9000], 32, 128),
    (9000, 48, 3, [0, 4000, 9000], 42, 168),
])
@pytest.mark.parametrize("noise", [0.0, 1e-3])
def test_norm_first_row_far_from_the_others(n, C, G, ptr, lanes, tile, noise):
    g = torch.Generator().manual_seed(n + C)
    x = torch.randn(1, C, generator=g) + noise * torch.randn(n, C, generator=g)
    for a in ptr[:-1]:
        x[a] = 1e4 * (1 + torch.rand(C, generator=g))
    print(f"outlier rows n={n} C={C} noise={noise}", flush=True)
    _, stats = spc.group_norm_fwd(cuda(x), G, cuda(torch.tensor(ptr, dtype=torch.int32)), eps=EPS_VAR)
    rstd, bound = rstd_bound(x, ptr, G, lanes, tile)
    worst = (np.abs(R.f64(stats[..., 1]) - rstd) / bound).max()
    assert worst <= 1, f"rstd off by {worst:.3g} times its bound, {(bound / rstd).max() / U:.1f} units of 2^-24"
