"""A query with an infinity reaches its own results only: its scores may all be
minus infinity for some tiles, or for the whole walk, while those of the queries
next to it grow from one tile to the next by more than an exponent holds."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle.rowops import f64
from tests.attn_cases import Case
from tests.rowops_cases import DTYPES, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("what", ["until_130", "throughout"])
@pytest.mark.parametrize("n,lq,H,D", [(1, 70, 2, 16), (1, 70, 2, 48), (1, 70, 2, 64), (1, 70, 2, 128), (16, 256, 8, 16), (16, 256, 8, 128)])
def test_rows_next_to_infinity(n, lq, H, D, what, causal, dtype):
    print(f"infinite query {n} x {lq} x {H} x {D} {what} causal={causal} {dtype}", flush=True)
    c = Case([lq] * n, [lq + 430] * n, H, H, D, dtype, seed=31, causal=causal, scale=1.0)
    c.q[:, :, 0], c.k[:, :, 0], c.k[:, :, 1] = 16.0, -16.0, 1.0
    for a, b in zip(c.kv_ptr, c.kv_ptr[1:]):
        c.k[a + 130:b, :, 0] = 16.0
    ref = c.ref()
    bad = np.array([a + 5 for a in c.q_ptr[:-1]] + [a + lq - 3 for a in c.q_ptr[:-1]])
    if what == "until_130":
        c.q[bad, :, 0] = float("inf")      # minus infinity against the first 130 keys, infinity against the others
    else:
        c.q[bad, :, 1] = float("-inf")     # minus infinity against every key
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    dq = spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())[0]
    rows = np.ones(c.n, bool)
    rows[bad] = False
    assert not torch.isfinite(out[torch.from_numpy(bad)].float()).any()
    within(f64(out)[rows], ref["out"][rows], ref["e_out"][rows], dtype, "out")
    within(f64(dq)[rows], ref["dq"][rows], ref["e_dq"][rows], dtype, "dq")
