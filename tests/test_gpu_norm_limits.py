"""GPU group norm with more (sample, group) pairs than one launch has workgroups
for: a launch holds fewer than 2^32 threads."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import within
from tests.test_gpu_norm import EPS_VAR, case, envelopes

pytestmark = pytest.mark.gpu


# 2^23 and some groups of workgroups of 512 threads; the second in the channels
# and rows that one launch would take
@pytest.mark.parametrize("n,C,G,S", [(5000, 32, 32, (1 << 18) + 3), (1000, 16, 2, (1 << 22) + 3)])
def test_norm_more_groups_than_a_launch(n, C, G, S):
    print(f"group norm n={n} C={C} G={G} S={S}", flush=True)
    # nearly all samples are empty; rows lie in the first, the last and some between
    at = [0, 1, 77, S // 2, S // 2 + 1, S - 2, S - 1]
    cut = [0] + sorted(int(v) for v in np.random.default_rng(S).integers(1, n, size=len(at) - 1)) + [n]
    ptr = np.zeros(S + 1, np.int64)
    for s, m in zip(at, np.diff(cut)):
        ptr[s + 1] = m
    ptr = cuda(torch.from_numpy(np.cumsum(ptr).astype(np.int32)))
    x, dy, gamma, beta = case(n, n, C, torch.float32)
    args = (G, ptr, cuda(gamma), cuda(beta))
    y, stats = spc.group_norm_fwd(cuda(x), *args, eps=EPS_VAR, act="silu")
    dx, dg, db = spc.group_norm_bwd(cuda(dy), cuda(x), *args, stats, act="silu")
    empty = torch.ones(S, dtype=torch.bool, device="cuda")
    empty[at] = False
    assert (stats[empty][..., 0] == 0).all()
    within(stats[empty][..., 1].cpu().unique(), np.array([EPS_VAR ** -0.5]), R.EPS * EPS_VAR ** -0.5, torch.float32, "rstd")

    xx, dd, ga, be = (R.f64(t) for t in (x, dy, gamma, beta))
    K = 256
    e_y, e_dx, e_g, e_b = envelopes(xx, dd, G, cut, ga, be, "silu", 1.0, K)
    ry, mean, rstd = R.group_norm_fwd(xx, G, cut, ga, be, EPS_VAR, "silu")
    rx, rg, rb = R.group_norm_bwd(dd, xx, G, cut, ga, be, EPS_VAR, "silu")
    within(y, ry, e_y, torch.float32, "y")
    within(stats[at][..., 0], mean, R.EPS * K * (rstd ** -2 - EPS_VAR).clip(0) ** 0.5, torch.float32, "mean")
    within(stats[at][..., 1], rstd, R.EPS * K * rstd, torch.float32, "rstd")
    within(dx, rx, e_dx, torch.float32, "dx")
    within(dg, rg, e_g, torch.float32, "dgamma")
    within(db, rb, e_b, torch.float32, "dbeta")
