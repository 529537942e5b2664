"""Few rows against many keys (pooling, single queries) take their probabilities
as two numbers of a 16-bit type: what is left of their rounding is the square of
half a step, and the result is as near as its own rounding."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import Case, split_of
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [16, 48, 64, 96, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk,H,Hk", [([1, 1, 2], [400, 700, 3], 2, 2), ([1], [3000], 4, 1), ([7] * 5, [900, 0, 1500, 1, 640], 2, 1)])
def test_probabilities_in_two_numbers(lq, lk, H, Hk, causal, D, dtype):
    c = Case(lq, lk, H, Hk, D, dtype, seed=71, causal=causal, gain=2.0)
    h = half_step(dtype)
    ref = A.attention(c.q, c.k, c.v, c.q_ptr, c.kv_ptr, c.scale, causal, step=h * h, floor=2.0 ** -30 if dtype == torch.float16 else 2.0 ** -126,
                      split=split_of(dtype, D, c.scale) if dtype == torch.bfloat16 else (0.0, 0.0))
    q, k, v, _ = c.on_gpu()
    within(f64(spc.attention_fwd(q, k, v, **c.kw())[0]), ref["out"], ref["e_out"], dtype, "out")
