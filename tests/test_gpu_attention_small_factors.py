"""scale q far below 1 in half precision against keys of some 10^4: no factor of
a score loses bits among the type's smallest numbers."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import Case
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.mark.parametrize("size,scale", [(1e-3, 0.25), (1e-4, 0.25), (1.0, 1e-5), (30.0, 3e-7)])
@pytest.mark.parametrize("D", [16, 32])
def test_small_factors_against_large_keys(D, size, scale):
    """The scores are off by roundings of fp32 alone (no term of the type's)."""
    c = Case([70, 33], [40, 5], 2, 2, D, F16, seed=43, scale=scale)
    c.q = (c.q.float() * size).to(F16)
    c.k = (c.k.float() * 5000).to(F16)
    q, k, v, _ = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    ref = A.attention(c.q, c.k, c.v, c.q_ptr, c.kv_ptr, scale, step=half_step(F16), floor=2.0 ** -30)
    st = f64(stats[0])
    lse = (st[..., 0] + np.log2(st[..., 1])) * np.log(2.0)
    assert (np.abs(lse - ref["lse"]) <= ref["e_lse"] + 4e-7 * (1 + np.abs(ref["lse"]))).all()
    within(f64(out), ref["out"], ref["e_out"], F16, "out")
