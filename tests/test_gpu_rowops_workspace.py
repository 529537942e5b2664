"""The row operators take nothing from what a workspace or an output held before
the call, and write no further than the workspace's stated size."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from sparse_convolution_hash_amd import binding as B
from tests.parity import cuda
from tests.rowops_cases import ptr_of, ragged

pytestmark = pytest.mark.gpu

GUARD = 4096


def poisoned(need, byte):
    """A workspace of exactly need bytes within a larger buffer of one value."""
    buf = torch.full((need + GUARD,), byte, dtype=torch.uint8, device="cuda")
    return buf, buf[:need]


def same(runs):
    for a, b in zip(runs, runs[1:]):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("n,C,G,S", [(300, 48, 3, 4), (9000, 64, 8, 5), (9000, 16, 1, 1), (60000, 128, 16, 3)])
def test_norm_workspace(n, C, G, S):
    print(f"norm workspace n={n} C={C}", flush=True)
    g = torch.Generator().manual_seed(n)
    x, dy = (cuda(torch.randn(n, C, generator=g).bfloat16()) for _ in range(2))
    gamma, beta = (cuda(torch.randn(C, generator=g)) for _ in range(2))
    sp = cuda(torch.tensor(ptr_of(ragged(n, n, S)), dtype=torch.int32))
    need = B.group_norm_workspace(n, C, G, S)
    runs = []
    for byte in (0, 255, 127):
        buf, ws = poisoned(max(need, 16), byte)
        out = torch.full_like(x, float("nan"))
        y, st = spc.group_norm_fwd(x, G, sp, gamma, beta, act="silu", out=out, workspace=ws)
        runs.append((y, st) + spc.group_norm_bwd(dy, x, G, sp, gamma, beta, st, act="silu", workspace=ws))
        assert (buf[max(need, 16):] == byte).all()
    same(runs)


@pytest.mark.parametrize("n,C,S", [(100, 64, 3), (1500, 48, 4), (40000, 64, 5), (300000, 64, 2)])
def test_recurrence_workspace(n, C, S):
    print(f"recurrence workspace n={n} C={C}", flush=True)
    g = torch.Generator().manual_seed(n)
    gate, x, dh = (cuda((torch.randn(n, C, generator=g) + 1).half()) for _ in range(3))
    h0, dl = (cuda(torch.randn(S, C, generator=g)) for _ in range(2))
    sp = cuda(torch.tensor(ptr_of(ragged(n, n, S)), dtype=torch.int32))
    need, _ = B.linear_recurrence_workspace(x.dtype, n, C, S)
    runs = []
    for byte in (0, 255, 127):
        buf, ws = poisoned(need, byte)
        out = torch.full_like(x, float("nan"))
        h, last, carry = spc.linear_recurrence_fwd(gate, x, sp, h0, want_carry=True, out=out, workspace=ws)
        runs.append((h, last) + spc.linear_recurrence_bwd(dh, gate, x, sp, carry, h0, dh_last=dl, want_dh0=True, workspace=ws))
        assert (buf[need:] == byte).all()
    same(runs)
