"""Shared inputs and checks of the attention tests."""

import math

import numpy as np
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.parity import cuda
from tests.rowops_cases import half_step, ptr_of, within

#: What p and ds are off by at least: a rounding to fp16 by half its smallest number, 2^-25; and the
#: fp32 exponential, like bf16's conversion, gives 0 for results below the smallest normal number,
#: 2^-126, so that p, which is that result or less (divided by a sum of at least 1), is off by up to that.
FLOOR = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


#: Heads of up to 32 elements of a 16-bit type: scale log2(e) q is kept as hi + lo, two numbers of the
#: type.  hi is off by up to half a step h of the product (2^-9 for bf16, 2^-11 for fp16) and lo, which is
#: that remainder, by h of itself: h^2 of the product.  fp16's lo is off by 2^-25 at least (half its
#: smallest number), and its heads are not split where scale log2(e) is above 1.
def split_of(dtype, D, scale=0.0):
    if dtype == torch.float32 or D > 32 or dtype == torch.float16 and scale * math.log2(math.e) > 1:
        return 0.0, 0.0
    return half_step(dtype) ** 2, 2.0 ** -25 if dtype == torch.float16 else 0.0


class Case:
    def __init__(self, lq, lk, H, Hk, D, dtype, seed=0, causal=False, ordered=False, gain=1.0, scale=None, outside=0):
        """lk None: the rows attend to themselves.  outside: rows of no sample, before and after."""
        g = torch.Generator().manual_seed(seed * 1000003 + H * 131 + D)
        r = lambda *s: torch.randn(*s, generator=g)
        self.causal, self.H, self.Hk, self.D, self.dtype = causal, H, Hk, D, dtype
        self.scale = D ** -0.5 if scale is None else scale
        self.own = lk is None
        self.q_ptr = [outside + v for v in ptr_of(lq)]
        self.kv_ptr = self.q_ptr if self.own else [outside + v for v in ptr_of(lk)]
        n, m = self.q_ptr[-1] + outside, self.kv_ptr[-1] + outside
        if self.own:
            x = (r(n, H + 2 * Hk, D)).to(dtype)
            x[:, :H] = (x[:, :H].float() * gain).to(dtype)
            self.q, self.k, self.v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        else:
            self.q, self.k, self.v = (r(n, H, D) * gain).to(dtype), r(m, Hk, D).to(dtype), r(m, Hk, D).to(dtype)
        self.dout = r(n, H, D).to(dtype)
        self.order = self.kv_order = None
        if ordered:
            perm = lambda k: torch.randperm(k, generator=g).int()
            self.order = perm(n)
            self.kv_order = self.order if self.own else perm(m)
        self.n, self.m = n, m

    def ref(self, bwd=True):
        np_ = lambda t: None if t is None else t.numpy()
        return A.attention(self.q, self.k, self.v, self.q_ptr, self.kv_ptr, self.scale, self.causal, np_(self.order),
                           np_(self.kv_order), dout=self.dout if bwd else None,
                           step=half_step(self.dtype) if self.dtype != torch.float32 else 0.0, floor=FLOOR[self.dtype],
                           split=split_of(self.dtype, self.D, self.scale))

    def kw(self):
        i32 = lambda v: cuda(torch.tensor(v, dtype=torch.int32))
        kw = dict(seg_ptr=i32(self.q_ptr), causal=self.causal, scale=self.scale)
        if self.order is not None:
            kw["order"] = cuda(self.order)
        if not self.own:
            kw["kv_ptr"] = i32(self.kv_ptr)
            if self.kv_order is not None:
                kw["kv_order"] = cuda(self.kv_order)
        return kw

    def on_gpu(self):
        if self.own:
            x = cuda(torch.cat([self.q, self.k, self.v], dim=1))
            return x[:, :self.H], x[:, self.H:self.H + self.Hk], x[:, self.H + self.Hk:], cuda(self.dout)
        kv = cuda(torch.cat([self.k, self.v], dim=1))
        return cuda(self.q), kv[:, :self.Hk], kv[:, self.Hk:], cuda(self.dout)


def check(c, bwd=True, q=None):
    """Runs the case and holds every output to the oracle; returns the outputs."""
    ref = c.ref(bwd)
    q, k, v, dout = c.on_gpu()
    kw = c.kw()
    mark = 77.0
    fill = lambda t: torch.full(t.shape, mark, dtype=t.dtype, device="cuda")
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, out=fill(q), **kw)
    rows, keys = ref["rows"], ref["keys"]
    within(f64(out)[rows], ref["out"][rows], ref["e_out"][rows], c.dtype, "out")
    assert (out[~torch.from_numpy(rows)] == mark).all()
    st = f64(stats[0])[:, rows]
    with np.errstate(divide="ignore"):
        lse = (st[..., 0] + np.log2(st[..., 1])) * np.log(2.0)
    lse[st[..., 1] == 0] = -np.inf
    want, env = ref["lse"][:, rows], ref["e_lse"][:, rows]
    assert np.array_equal(np.isneginf(lse), np.isneginf(want))
    some = np.isfinite(want)
    lse, want, env = lse[some], want[some], env[some]
    assert (np.abs(lse - want) <= env + 4e-7 * (1 + np.abs(want))).all()
    if not bwd:
        return out, stats[0]
    got = spc.attention_bwd(dout, q, k, v, out, stats, dq=fill(q), dk=fill(k), dv=fill(v), **kw)
    for t, name, there in zip(got, ("dq", "dk", "dv"), (rows, keys, keys)):
        within(f64(t)[there], ref[name][there], ref["e_" + name][there], c.dtype, name)
        assert (t[~torch.from_numpy(there)] == mark).all()
    return (out, stats[0]) + got
