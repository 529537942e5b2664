"""Values, and so outputs, near half precision's smallest numbers: dout . out
keeps the precision of dout . v, from which it is subtracted."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import Case
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.mark.parametrize("lq,lk", [([400], None), ([3], [3000])])
@pytest.mark.parametrize("D", [16, 32])
@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** -10, 1.0])
def test_gradients_of_small_values(size, D, lq, lk):
    """dq is linear in v.  Queries of 0 make every probability one over a count,
    exact in the forward, and keys of one sign let an error of dout . out through.
    out is kept in two numbers of the type, the second one times 2^11: off by the
    square of half a step, and by 2^-25 2^-11 at least."""
    c = Case(lq, lk, 1, 1, D, F16, seed=44)
    c.q.zero_()
    c.k.copy_((16 + 5 * c.k.float()).to(F16))
    c.v.copy_((c.v.float() * size).to(F16))
    ref = A.attention(c.q, c.k, c.v.double() / size, c.q_ptr, c.kv_ptr, c.scale, dout=c.dout, step=half_step(F16) ** 2,
                      floor=2.0 ** -36 / size)
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    dq = spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())[0]
    within(f64(dq), ref["dq"] * size, ref["e_dq"] * size, F16, "dq")
