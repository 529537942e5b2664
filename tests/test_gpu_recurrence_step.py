"""GPU single step of the recurrence on rows of a wider tensor."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, within
from tests.test_gpu_recurrence import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C,gap", [(2, 16, 0), (7, 64, 16), (33, 48, 80), (600, 272, 8), (5, 4096, 16)])
def test_step_of_wide_rows(dtype, n, C, gap):
    # gate and x as the halves of one product's rows, with a gap of NaN behind them
    if dtype == torch.float32:
        gap = gap // 2      # rows stay a multiple of 16 bytes
    gate, x, _, h0, _ = case(n + C, n, C, n, dtype)
    both = torch.full((n, 2 * C + gap), float("nan"), dtype=dtype, device="cuda")
    both[:, :C], both[:, C:2 * C] = cuda(gate), cuda(x)
    print(f"step n={n} C={C} gap={gap} {dtype}", flush=True)
    state, new = cuda(h0), torch.full((n, C), float("nan"), device="cuda")
    out = spc.linear_recurrence_step(both[:, :C], both[:, C:2 * C], state, new_state=new)
    ro, rl, _, eo, el = R.recurrence_fwd(gate, x, list(range(n + 1)), h0)
    within(new, rl, el, torch.float32, "state")
    within(out, ro, eo, dtype, "out")
    assert torch.equal(state, cuda(h0))
    dense = torch.empty_like(new)
    assert torch.equal(out, spc.linear_recurrence_step(cuda(gate), cuda(x), state, new_state=dense)) and torch.equal(new, dense)
    buf = torch.full((n, C), 7.0, dtype=dtype, device="cuda")
    assert spc.linear_recurrence_step(both[:, :C], both[:, C:2 * C], state, out=buf) is buf
    assert torch.equal(buf, out) and torch.equal(state, new)
