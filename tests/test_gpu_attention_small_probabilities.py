"""Probabilities far below 1 in half precision, whose smallest normal number is
2^-14: the forward's (relative to the row's largest) and the backward's."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import Case
from tests.parity import cuda
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.mark.parametrize("D", [16, 48, 64])
@pytest.mark.parametrize("lq", [5, 64, 300])
def test_dv_of_small_probabilities(lq, D):
    """One key outweighs the others, whose probabilities are 2^-15 to 2^-20: p is
    off by half a step of the type, not of its smallest numbers."""
    c = Case([lq], [300], 2, 1, D, F16, seed=42, gain=0.3, scale=1.0)
    c.q[:, :, 0], c.k[:, :, 0], c.k[0] = 4.0, -3.0, 0.0
    s = 2.0 ** 12
    c.dout = (c.dout * s).to(F16)
    ref = A.attention(c.q, c.k, c.v, c.q_ptr, c.kv_ptr, c.scale, dout=c.dout.double() / s, step=half_step(F16), floor=2.0 ** -40)
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    dv = spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())[2]
    r, e = ref["dv"] * s, ref["e_dv"] * s
    fits = np.abs(r) + e < 65000           # the one key's gradient passes 65,504 here and there
    assert fits[1:].all()
    within(f64(dv)[fits], r[fits], e[fits], F16, "dv")


@pytest.mark.parametrize("D", [16, 48, 64, 128])
@pytest.mark.parametrize("lq,H", [(3, 1), (8400, 8)])
def test_one_key_above_many(lq, H, D):
    """One key has the largest score and no value, the result is that of keys with
    probabilities of some 2^-20, all alike: their roundings do not cancel."""
    n = 2000
    q, k, v = torch.zeros(lq, H, D), torch.zeros(n, H, D), torch.full((n, H, D), 500.0)
    q[:, :, 0], k[:, :, 0] = 1.0, -13.6
    k[0], v[0] = 0.0, 0.0
    q, k, v = q.to(F16), k.to(F16), v.to(F16)
    out, _ = spc.attention_fwd(cuda(q), cuda(k), cuda(v), scale=1.0)
    ref = A.attention(q[:1, :1], k[:, :1], v[:, :1], [0, 1], [0, n], 1.0, step=half_step(F16), floor=2.0 ** -30)
    within(f64(out), np.broadcast_to(ref["out"], out.shape), ref["e_out"], F16, "out")
