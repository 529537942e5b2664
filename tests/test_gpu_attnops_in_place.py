"""Layouts that share memory where the contract allows it give what separate
tensors give; those that overlap otherwise are refused by the binding's calls."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from tests.parity import cuda
from tests.rowops_cases import DTYPES

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype):
    return cuda(torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C", [(1, 16), (700, 80), (65, 1040), (3000, 512)])
def test_layer_norm(n, C, dtype):
    x, res, dy, dt = (randn(n, C, seed=s, dtype=dtype) for s in range(4))
    y, stats, total = spc.layer_norm_fwd(x, residual=res)
    for place in ("y over residual", "y over x", "total over x, y over residual", "total over residual, y over x"):
        a, b = x.clone(), res.clone()
        out = b if "y over residual" in place else a
        tot = a if "total over x" in place else b if "total over residual" in place else None
        y2, s2, t2 = spc.layer_norm_fwd(a, residual=b, out=out, total=tot)
        assert torch.equal(y2, y) and torch.equal(t2, total) and torch.equal(s2, stats), place
    dx = spc.layer_norm_bwd(dy, total, None, stats, dtotal=dt)[0]
    for over in ("dout", "dtotal"):
        a, b = dy.clone(), dt.clone()
        assert torch.equal(spc.layer_norm_bwd(a, total, None, stats, dtotal=b, dx=a if over == "dout" else b)[0], dx)
    wide = torch.empty((n + 1) * C, dtype=dtype, device="cuda")
    for bad in (lambda: spc.layer_norm_bwd(dy, total, None, stats, dx=total),
                lambda: spc.layer_norm_fwd(x, residual=res, out=wide[:n * C].view(n, C), total=wide[C:].view(n, C)) if n > 1 else
                spc.layer_norm_fwd(x, residual=res, out=x, total=x)):
        with pytest.raises(spc.SpcError):
            bad()


@pytest.mark.parametrize("dtype", DTYPES)
def test_columns_of_one_tensor(dtype):
    n, H, Hk, D = 300, 4, 2, 32
    qkv, do = randn(n, H + 2 * Hk, D, seed=5, dtype=dtype), randn(n, H, D, seed=6, dtype=dtype)
    q, k, v = (t.contiguous() for t in (qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]))
    out, st = spc.attention_fwd(q, k, v, want_stats=True)
    grads = spc.attention_bwd(do, q, k, v, out, st)
    # everything in one tensor: q, k, v, out, dout, dq, dk, dv
    w = torch.zeros(n, 4 * H + 4 * Hk, D, dtype=dtype, device="cuda")
    w[:, :H + 2 * Hk], w[:, 2 * H + 2 * Hk:3 * H + 2 * Hk] = qkv, do
    c = lambda a, m: w[:, a:a + m]
    base = H + 2 * Hk
    o2, s2 = spc.attention_fwd(c(0, H), c(H, Hk), c(H + Hk, Hk), want_stats=True, out=c(base, H))
    g2 = spc.attention_bwd(c(base + H, H), c(0, H), c(H, Hk), c(H + Hk, Hk), o2, s2, dq=c(base + 2 * H, H), dk=c(base + 3 * H, Hk),
                           dv=c(base + 3 * H + Hk, Hk))
    assert torch.equal(o2, out) and all(torch.equal(a, b) for a, b in zip(g2, grads))
    with pytest.raises(spc.SpcError):
        spc.attention_fwd(c(0, H), c(H, Hk), c(H + Hk, Hk), out=c(base - 1, H))
    with pytest.raises(spc.SpcError):
        spc.attention_bwd(c(base + H, H), c(0, H), c(H, Hk), c(H + Hk, Hk), o2, s2, dk=c(base + 3 * H, Hk), dv=c(base + 3 * H + 1, Hk))
    f, pos = torch.rand(16, device="cuda"), torch.arange(n, device="cuda", dtype=torch.int32)[:, None]
    r = spc.rotary(q, pos, f, (16,))
    assert torch.equal(spc.rotary(c(0, H), pos, f, (16,), out=c(base, H)), r)
    assert torch.equal(spc.rotary(c(0, H), pos, f, (16,), out=c(0, H)), r)
    with pytest.raises(spc.SpcError):
        spc.rotary(c(0, H), pos, f, (16,), out=c(1, H))
