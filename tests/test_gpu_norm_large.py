"""GPU group norm beyond the sizes that one launch takes, in the shapes that the
smaller tests cover below them."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, ragged, within
from tests.test_gpu_norm import EPS_VAR, case, envelopes, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu"])
@pytest.mark.parametrize("C,G", [(64, 8), (48, 3), (80, 10)])
def test_norm_large_activations_and_dropout(dtype, name, C, G):
    run(9001, C, G, ragged(C, 9001, 5), dtype, name, drop=(77 + C, 1 << 33, 5, 0.2), seed=C)


@pytest.mark.parametrize("C,G", [(16, 16), (16, 1), (48, 16), (48, 48), (112, 7), (128, 1), (272, 17), (272, 16), (528, 33)])
def test_norm_large_channels_and_groups(C, G):
    run(5000, C, G, [2500, 0, 1, 2499], torch.float32, "silu", seed=C)
    run(5000, C, G, [5000], torch.bfloat16, "none", seed=C + 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_large_many_samples(dtype):
    # more samples than a wave has lanes, several in a tile and several tiles to one, empty ones among them
    run(12000, 32, 4, [1, 0, 2, 3, 114] * 100, dtype, "silu", seed=4)
    run(20000, 64, 4, ragged(6, 20000, 90), dtype, "none", seed=5)


@pytest.mark.parametrize("n", [511, 512, 513, 1023, 1025, 4095, 4096, 4097])
def test_norm_around_the_one_launch_limits(n):
    run(n, 32, 2, [n], torch.float32, "silu", seed=n)
    run(n, 32, 1, ragged(n, n, 4), torch.bfloat16, "silu", drop=(5, n, 1, 0.1), seed=n)


def test_norm_large_nan_stays_in_its_group():
    n, C, G = 9000, 64, 4
    ptr = [0, 3000, 5200, 9000]
    x, dy, gamma, beta = case(13, n, C, torch.bfloat16)
    x[3000, 17], x[4000, 20] = float("nan"), float("inf")      # a run's first row, and a later one
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    y, stats = spc.group_norm_fwd(cuda(x), G, sp, cuda(gamma), cuda(beta), act="silu")
    dx, _, _ = spc.group_norm_bwd(cuda(dy), cuda(x), G, sp, cuda(gamma), cuda(beta), stats, act="silu")
    for t in (y, dx):
        bad = torch.isnan(t).cpu()
        assert bad[3000:5200, 16:32].all() and bad.sum() == 2200 * 16


def test_norm_large_rows_outside_and_in_place():
    n, C, G = 9000, 48, 3
    ptr = [700, 4000, 4000, 8001]
    x, dy, gamma, beta = case(14, n, C, torch.float16)
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    ga, be = cuda(gamma), cuda(beta)
    clean, stats = spc.group_norm_fwd(cuda(x), G, sp, ga, be, act="relu")
    dclean = spc.group_norm_bwd(cuda(dy), cuda(x), G, sp, ga, be, stats, act="relu")
    x[:700], x[8001:], dy[:700], dy[8001:] = float("nan"), float("inf"), float("inf"), float("nan")
    buf = cuda(x)
    y, st = spc.group_norm_fwd(buf, G, sp, ga, be, act="relu", out=buf)
    assert torch.equal(st, stats) and torch.equal(y[700:8001], clean[700:8001])
    assert torch.isnan(y[:700]).all() and torch.isinf(y[8001:]).all()      # not written
    buf = cuda(dy)
    dx, dg, db = spc.group_norm_bwd(buf, cuda(x), G, sp, ga, be, stats, act="relu", dx=buf)
    assert torch.equal(dx[700:8001], dclean[0][700:8001]) and torch.equal(dg, dclean[1]) and torch.equal(db, dclean[2])
    assert torch.isinf(dx[:700]).all() and torch.isnan(dx[8001:]).all()


def test_norm_past_32_bits():
    # 2^31 elements and more: addresses and slots are 64 bits wide
    C, G, tail = 64, 8, 2000
    n = (1 << 31) // C + 3000
    print(f"group norm n={n} C={C}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn((n, C), generator=g, device="cuda", dtype=torch.bfloat16)
    x[:n - tail] += 1
    ptr = cuda(torch.tensor([0, n - tail, n], dtype=torch.int32))
    y, stats = spc.group_norm_fwd(x, G, ptr, act="silu")
    dx, dg, db = spc.group_norm_bwd(x, x, G, ptr, None, None, stats, act="silu")
    # the long sample's statistics in pieces
    s1, s2 = torch.zeros(G, dtype=torch.float64, device="cuda"), torch.zeros(G, dtype=torch.float64, device="cuda")
    for a in range(0, n - tail, 1 << 22):
        v = x[a:min(a + (1 << 22), n - tail)].double().view(-1, G, C // G) - 1
        s1 += v.sum((0, 2))
        s2 += (v * v).sum((0, 2))
    m = s1 / ((n - tail) * (C // G))
    var = s2 / ((n - tail) * (C // G)) - m * m
    within(stats[0, :, 0], (1 + m).cpu().numpy(), R.EPS * 16, torch.float32, "mean")
    within(stats[0, :, 1], ((var + EPS_VAR) ** -0.5).cpu().numpy(), R.EPS * 16, torch.float32, "rstd")
    # the last sample, whose elements lie past 2^31, against the oracle
    xt = x[n - tail:].cpu()
    one, zero = np.ones(C), np.zeros(C)
    e_y, e_dx, _, _ = envelopes(R.f64(xt), R.f64(xt), G, [0, tail], one, zero, "silu", 1.0, 256)
    within(y[n - tail:], R.group_norm_fwd(xt, G, [0, tail], one, zero, EPS_VAR, "silu")[0], e_y, torch.bfloat16, "y")
    within(dx[n - tail:], R.group_norm_bwd(xt, xt, G, [0, tail], one, zero, EPS_VAR, "silu")[0], e_dx, torch.bfloat16, "dx")
    # and the first rows of the long one, from its statistics
    z = (x[:1000].double() - (1 + m).repeat_interleave(C // G)) * ((var + EPS_VAR) ** -0.5).repeat_interleave(C // G)
    within(y[:1000], (z * torch.sigmoid(z)).cpu().numpy(), 64 * R.EPS * (1 + np.abs(z.cpu().numpy())), torch.bfloat16, "y")
    assert torch.isfinite(dg).all() and torch.isfinite(db).all()
