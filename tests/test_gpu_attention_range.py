"""Half precision has 40 binades: ds of long rows and of small or large
gradients leaves them at its own size.  Results keep the precision that the
formulas give them.

Gradients are linear in dout: for dout = s u the bounds are s times those of u,
a bound that no rounding at a size of its own (2^-25 whatever s is) fits in."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import FLOOR, Case, split_of
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu

F16 = torch.float16
SIZES = [([1024], None, 2, 2), ([1000, 1, 70], None, 4, 2), ([3], [3000], 2, 1), ([3000], [7], 1, 1)]
WIDE = ([300] * 26, None, 8, 8)          # workgroups of four waves
CASES = [z + (D,) for z in SIZES for D in (16, 32, 128)] + [WIDE + (D,) for D in (32, 128)]


def scaled(c, s):
    """dout as stored and the bounds that belong to it."""
    c.dout = (c.dout * s).to(F16)
    ref = A.attention(c.q, c.k, c.v, c.q_ptr, c.kv_ptr, c.scale, c.causal, dout=c.dout.double() / s, step=half_step(F16),
                      floor=FLOOR[F16], split=split_of(F16, c.D, c.scale))
    for name in ("dq", "dk", "dv"):
        ref[name], ref["e_" + name] = ref[name] * s, ref["e_" + name] * s
    return ref


def grads(c):
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    return dict(zip(("dq", "dk", "dv"), spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("s", [2.0 ** -17, 2.0 ** 13])
@pytest.mark.parametrize("lq,lk,H,Hk,D", CASES)
def test_gradients_of_any_size(lq, lk, H, Hk, D, s, causal):
    """Queries 64 times as large as they could be against keys 64 times as
    small (and the other way round) put dk (dq) where its own rounding hides nothing,
    or where it does not pass the type's largest number though ds does."""
    print(f"range {lq} {lk} {H}/{Hk} x {D} s={s} causal={causal}", flush=True)
    small = s < 1
    for name, gain in (("dq", 1 / 64), ("dk", 64.0)):
        c = Case(lq, lk, H, Hk, D, F16, seed=41, causal=causal, gain=4.0)
        gain = gain if small else 1 / gain
        c.q.copy_((c.q.float() * gain).to(F16))
        c.k.copy_((c.k.float() / gain).to(F16))
        if not small:
            c.v.copy_((c.v.float() * 16).to(F16))
        ref, got = scaled(c, s), grads(c)
        for t in (name, "dv"):
            r, e = ref[t], ref["e_" + t]
            fits = ref["rows" if t == "dq" else "keys"][:, None, None] & (np.abs(r) + e < 65000)
            assert t == "dv" or fits.mean() > 0.5
            within(f64(got[t])[fits], r[fits], e[fits], F16, t)
