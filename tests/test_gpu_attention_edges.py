"""Heads of up to 32 elements of a 16-bit type take ds as two numbers of the
type for dq, wherever a row's tiles lie: at a causal mask's edge, at the end of
a sample, in between."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import FLOOR, Case
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [16, 32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,H", [([20], 1), ([64, 33], 2), ([150, 7], 1), ([300] * 30, 8)])
def test_dq_of_even_rows(lens, H, causal, D, dtype):
    """Queries of 0 make every probability one over a count, which the forward
    takes as exact powers of two: the roundings left are those of ds (the square
    of half a step h as two numbers, h alone would not fit) and of out, in two
    numbers as well."""
    c = Case(lens, None, H, H, D, dtype, seed=51, causal=causal)
    c.q.zero_()
    h = half_step(dtype)
    ref = A.attention(c.q, c.k, c.v, c.q_ptr, c.kv_ptr, c.scale, causal, dout=c.dout, step=h * h, floor=FLOOR[dtype])
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    dq = spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())[0]
    within(f64(dq), ref["dq"], ref["e_dq"], dtype, "dq")
