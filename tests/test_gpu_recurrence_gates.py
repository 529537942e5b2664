"""GPU recurrence at gates that are nearly open or closed: the small one of
sigmoid(g) and sigmoid(-g) keeps its relative precision, and the gradients and
states that it scales keep theirs."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES

pytestmark = pytest.mark.gpu

U = R.EPS
# The small gate is e / (1 + e), e = exp(-|g|): the exp and reciprocal instructions
# are off by a unit in the last place each (2 U), and three roundings come on top
# (e's correction, the sum, the product); the rest of the correction is below U.
GATE = 8 * U
# For 16-bit gates exp2's argument log2(e) |g| keeps its rounding (|g| U in e) and
# its constant's (0.23 |g| U): far below the gate's own.
GATE_16 = 1.25 * U


def near(got, want, rel, what):
    worst = ((got.double().cpu() - want).abs() / (want.abs() * rel)).max().item()
    assert worst <= 1, f"{what}: off by {worst:.3g} times its bound"


def gates(n, C, dtype, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    v = (lo + (hi - lo) * torch.rand(n, C, generator=g)).to(dtype)
    return v * (2 * torch.randint(0, 2, (n, C), generator=g) - 1).to(dtype)


@pytest.mark.parametrize("lo,hi", [(0, 4), (4, 12), (12, 40), (40, 80)])
@pytest.mark.parametrize("n", [60, 3000])      # one tile, and several
def test_gates_keep_relative_precision(n, lo, hi):
    # every row a sample: nothing but the gate, its complement and products of them
    C = 16
    gate = gates(n, C, torch.float32, lo, hi, n + hi)
    g = torch.Generator().manual_seed(hi)
    x, dout, h0 = (0.5 + torch.rand(n, C, generator=g) for _ in range(3))
    zero = torch.zeros(n, C)
    sp = cuda(torch.arange(n + 1, dtype=torch.int32))
    a, na = torch.sigmoid(gate.double()), torch.sigmoid(-gate.double())
    print(f"gates n={n} {lo}..{hi}", flush=True)
    # a from h0 alone, 1 - a from x alone
    out, last, carry = spc.linear_recurrence_fwd(cuda(gate), cuda(zero), sp, cuda(h0), want_carry=True)
    near(out, a * h0.double(), GATE + 2 * U, "a h0")
    assert torch.equal(out, last)
    dg, dx, dh0 = spc.linear_recurrence_bwd(cuda(dout), cuda(gate), cuda(zero), sp, carry, cuda(h0), want_dh0=True)
    near(dx, na * dout.double(), GATE + 2 * U, "dx")
    near(dh0, a * dout.double(), GATE + 2 * U, "dh0")
    near(dg, a * na * h0.double() * dout.double(), GATE + U + 4 * U, "dgate")
    out, _, _ = spc.linear_recurrence_fwd(cuda(gate), cuda(x), sp)
    near(out, na * x.double(), GATE + 2 * U, "(1 - a) x")
    step = spc.linear_recurrence_step(cuda(gate), cuda(x), torch.zeros(n, C, device="cuda"))
    near(step, na * x.double(), GATE + 2 * U, "step")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [20, 2000])      # one tile, and several
def test_products_of_closed_gates(dtype, k):
    # samples of three rows with x = 0: the state, fp32 in every type, is a product of three gates
    C = 16
    gate = -gates(3 * k, C, dtype, 12, 25, k).abs()
    sp = cuda(torch.arange(k + 1, dtype=torch.int32) * 3)
    print(f"products k={k} {dtype}", flush=True)
    _, last, _ = spc.linear_recurrence_fwd(cuda(gate), cuda(torch.zeros_like(gate)), sp, torch.ones(k, C, device="cuda"))
    rel = 3 * (GATE + U) + (0 if dtype == torch.float32 else GATE_16 * gate.double().abs().view(k, 3, C).sum(1))
    near(last, torch.sigmoid(gate.double()).view(k, 3, C).prod(1), rel, "h_last")


@pytest.mark.parametrize("dtype", DTYPES)
def test_gates_at_infinity_and_nan(dtype):
    n, C = 40, 16
    gate = torch.zeros(n, C)
    gate[:, 0], gate[:, 1], gate[:, 2], gate[:, 3] = float("inf"), float("-inf"), 60000.0, -60000.0
    gate[7, 4] = float("nan")
    g = torch.Generator().manual_seed(3)
    x, dout, h0 = (torch.randn(*s, generator=g) for s in ((n, C), (n, C), (n, C)))
    x, dout = x.to(dtype), dout.to(dtype)
    sp = cuda(torch.arange(n + 1, dtype=torch.int32))
    gate = gate.to(dtype)
    out, last, carry = spc.linear_recurrence_fwd(cuda(gate), cuda(x), sp, cuda(h0), want_carry=True)
    dg, dx, dh0 = (t.cpu() for t in spc.linear_recurrence_bwd(cuda(dout), cuda(gate), cuda(x), sp, carry, cuda(h0), want_dh0=True))
    last = last.cpu()
    for c, opened in ((0, True), (1, False), (2, True), (3, False)):
        assert torch.equal(last[:, c], h0[:, c] if opened else x[:, c].float())
        assert torch.equal(dx[:, c], torch.zeros_like(dx[:, c]) if opened else dout[:, c])
        assert torch.equal(dh0[:, c], dout[:, c].float() if opened else torch.zeros(n)) and (dg[:, c] == 0).all()
    for t in (out.cpu(), last, dg, dx, dh0):
        bad = torch.isnan(t)
        assert bad[7, 4] and bad.sum() == 1
