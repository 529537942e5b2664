"""Heads of every width between 32 and 128 in workgroups of four waves and, with
few queries or few keys, in split walks."""

import pytest
import torch

from tests.attn_cases import Case, check
from tests.rowops_cases import DTYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [48, 80, 96, 112])
def test_widths(D, causal, dtype):
    print(f"attention width {D} causal={causal} {dtype}", flush=True)
    check(Case([130] * 40, None, 8, 8, D, dtype, seed=61, causal=causal, ordered=causal))
    check(Case([3], [1500], 2, 1, D, dtype, seed=62, causal=causal))
    check(Case([1300], [5], 2, 2, D, dtype, seed=63, causal=causal, ordered=True))
