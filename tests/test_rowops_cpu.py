"""The row operators' refusals without a GPU: host checks return before any
launch (so fake, never-dereferenced pointers are safe here)."""

import ctypes
import os

import pytest
import torch

import sparse_convolution_hash_amd as spc
import sparse_convolution_hash_amd.binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libspc.so not built")

P = ctypes.c_void_p(0x100000)           # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 40


def drop(p=0.5, rng=0x100000, layer=0):
    return ctypes.byref(B._DropArg(rng, layer, p))


def test_dropout_refusals():
    f = lambda dt=2, x=P, n=100, res=None, d=drop(), out=P: B.lib().spc_dropout_fwd(dt, x, n, res, d, out, None)
    assert f(n=0) == f(n=0, x=None, out=None) == B.SPC_OK
    assert f(dt=3) == f(n=-1) == f(x=None) == f(out=None) == f(x=ODD) == f(out=ODD) == f(res=ODD) == B.SPC_ERR_ARG
    assert f(d=None) == f(d=drop(-0.1)) == f(d=drop(1.1)) == f(d=drop(float("nan"))) == B.SPC_ERR_ARG
    assert "outside [0, 1]" in B.lib().spc_last_error().decode()
    assert f(d=drop(rng=None)) == f(d=drop(rng=0x100008)) == B.SPC_ERR_ARG
    b = lambda dt=2, x=P, n=100, d=drop(), out=P: B.lib().spc_dropout_bwd(dt, x, n, d, out, None)
    assert b(n=0) == B.SPC_OK
    assert b(dt=-1) == b(n=-1) == b(x=None) == b(out=ODD) == b(d=None) == B.SPC_ERR_ARG


def test_group_norm_refusals():
    L = B.lib()

    def fwd(dt=2, x=P, n=100, C=64, G=8, sp=P, S=2, gamma=P, beta=P, eps=1e-5, act=2, d=None, y=P, stats=P, ws=P, wsb=BIG):
        return L.spc_group_norm_fwd(dt, x, n, C, G, sp, S, gamma, beta, eps, act, d, y, stats, ws, wsb, None)

    def bwd(dt=2, dy=P, x=P, n=100, C=64, G=8, sp=P, S=2, gamma=P, beta=P, stats=P, act=2, d=None, dx=P, dg=P, db=P, ws=P,
            wsb=BIG):
        return L.spc_group_norm_bwd(dt, dy, x, n, C, G, sp, S, gamma, beta, stats, act, d, dx, dg, db, ws, wsb, None)

    for f in (fwd, bwd):
        assert f(C=24) == f(C=0) == f(C=-16) == f(C=65536 * 64, G=1) == B.SPC_ERR_UNSUPPORTED
        assert f(G=0) == f(G=7) == f(G=-8) == f(n=-1) == f(n=1 << 31) == f(S=0) == f(S=1 << 31) == B.SPC_ERR_ARG
        assert f(dt=9) == f(act=3) == f(act=-1) == f(sp=None) == f(sp=ODD) == f(ws=None) == f(ws=ODD) == B.SPC_ERR_ARG
        assert f(x=None) == f(x=ODD) == f(stats=None) == f(stats=ODD) == f(gamma=ODD) == f(beta=ODD) == B.SPC_ERR_ARG
        assert f(d=drop(2.0)) == f(d=drop(rng=None)) == B.SPC_ERR_ARG
        assert f(wsb=64) == B.SPC_ERR_WORKSPACE
    for e in (0.0, -1.0, float("nan")):
        assert fwd(eps=e) == B.SPC_ERR_ARG
    assert fwd(y=None) == fwd(y=ODD) == B.SPC_ERR_ARG
    assert bwd(dy=None) == bwd(dx=None) == bwd(dg=ODD) == bwd(db=ODD) == bwd(dx=ODD) == B.SPC_ERR_ARG
    b = ctypes.c_size_t()
    assert L.spc_group_norm_workspace(100, 64, 8, 2, None) == B.SPC_ERR_ARG
    assert L.spc_group_norm_workspace(100, 64, 8, 2, ctypes.byref(b)) == B.SPC_OK and b.value > 0
    assert fwd(wsb=b.value - 1) == B.SPC_ERR_WORKSPACE


def test_linear_recurrence_refusals():
    L = B.lib()

    def fwd(dt=2, g=P, x=P, ld=64, n=100, C=64, sp=P, S=2, order=None, h0=None, out=P, last=None, carry=None, ws=P, wsb=BIG):
        return L.spc_linear_recurrence_fwd(dt, g, x, ld, n, C, sp, S, order, 0, h0, out, last, carry, ws, wsb, None)

    def bwd(dt=2, dh=P, g=P, x=P, ld=64, n=100, C=64, sp=P, S=2, order=None, h0=None, carry=P, dl=None, dg=P, dx=P, ldg=64,
            dh0=None, ws=P, wsb=BIG):
        return L.spc_linear_recurrence_bwd(dt, dh, g, x, ld, n, C, sp, S, order, 0, h0, carry, dl, dg, dx, ldg, dh0, ws,
                                           wsb, None)

    for f in (fwd, bwd):
        assert f(C=24) == f(C=0) == B.SPC_ERR_UNSUPPORTED
        assert f(dt=5) == f(n=-1) == f(n=1 << 31) == f(S=0) == f(sp=None) == f(sp=ODD) == f(order=ODD) == B.SPC_ERR_ARG
        assert f(ld=63) == f(ld=68) == f(ld=0) == f(ld=1 << 31) == B.SPC_ERR_ARG       # 68 bf16 are 136 bytes
        assert f(g=None) == f(x=None) == f(g=ODD) == f(x=ODD) == f(h0=ODD) == f(ws=None) == f(ws=ODD) == B.SPC_ERR_ARG
        assert f(wsb=0) == B.SPC_ERR_WORKSPACE
    assert fwd(out=None) == fwd(out=ODD) == fwd(last=ODD) == fwd(carry=ODD) == B.SPC_ERR_ARG
    assert bwd(dh=None) == bwd(carry=None) == bwd(dg=None) == bwd(dx=ODD) == bwd(ldg=60) == bwd(dl=ODD) == B.SPC_ERR_ARG
    assert bwd(dh0=ODD) == bwd(ldg=1 << 31) == B.SPC_ERR_ARG
    step = lambda dt=2, g=P, x=P, ld=64, n=3, C=64, s=P, ns=P, out=P: L.spc_linear_recurrence_step(
        dt, g, x, ld, n, C, s, ns, out, None)
    assert step(n=0) == B.SPC_OK
    assert step(C=8) == B.SPC_ERR_UNSUPPORTED
    assert step(dt=4) == step(n=-1) == step(ld=32) == step(g=None) == step(s=None) == step(ns=ODD) == step(out=ODD) == B.SPC_ERR_ARG
    w, c = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.spc_linear_recurrence_workspace(2, 100, 64, 2, ctypes.byref(w), None) == B.SPC_ERR_ARG
    assert L.spc_linear_recurrence_workspace(2, 100, 64, 2, ctypes.byref(w), ctypes.byref(c)) == B.SPC_OK and w.value > 0
    assert fwd(wsb=w.value - 1) == B.SPC_ERR_WORKSPACE


def test_binding_refuses_cpu_tensors():
    x, r = torch.zeros(4, 16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        spc.Dropout(r, 0.5)
    with pytest.raises(TypeError):
        spc.dropout_fwd(x, None)
    with pytest.raises(TypeError):
        spc.group_norm_fwd(x, 4)
    with pytest.raises(TypeError):
        spc.linear_recurrence_fwd(x, x)
    with pytest.raises(TypeError):
        spc.linear_recurrence_step(x, x, x)
