"""The attention-block operators' refusals and limits without a GPU: host checks
return before any launch (so fake, never-dereferenced pointers are safe here)."""

import ctypes
import os

import pytest
import torch

import sparse_convolution_hash_amd as spc
import sparse_convolution_hash_amd.binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libspc.so not built")

P = ctypes.c_void_p(0x100000)           # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 60
END = (1 << 31) - 4096


def test_layer_norm_refusals():
    L = B.lib()

    def fwd(dt=2, x=P, r=None, n=100, C=64, g=P, b=P, eps=1e-5, y=P, t=None, s=P):
        return L.spc_layer_norm_fwd(dt, x, r, n, C, g, b, eps, y, t, s, None)

    def bwd(dt=2, dy=P, x=P, n=100000, C=64, g=P, s=P, dt_=None, dx=P, dg=P, db=P, ws=P, wsb=BIG):
        return L.spc_layer_norm_bwd(dt, dy, x, n, C, g, s, dt_, dx, dg, db, ws, wsb, None)

    for f in (fwd, bwd):
        assert f(C=24) == f(C=0) == f(C=-16) == f(C=4112) == B.SPC_ERR_UNSUPPORTED
        assert f(dt=3) == f(n=-1) == f(n=END) == f(x=None) == f(x=ODD) == f(g=ODD) == f(s=None) == f(s=ODD) == B.SPC_ERR_ARG
    assert fwd(n=0) == fwd(n=0, x=None, y=None, s=None) == B.SPC_OK
    assert fwd(y=None) == fwd(y=ODD) == fwd(b=ODD) == fwd(eps=0.0) == fwd(eps=float("nan")) == B.SPC_ERR_ARG
    assert fwd(r=P) == fwd(t=P) == fwd(r=ODD, t=P) == fwd(r=P, t=ODD) == B.SPC_ERR_ARG     # both or neither
    assert fwd(r=ctypes.c_void_p(0x200000), t=P) == B.SPC_ERR_ARG                          # total over y
    assert bwd(n=0, dg=None, db=None, dy=None, x=None, dx=None, s=None) == B.SPC_OK
    assert bwd(dy=None) == bwd(dx=None) == bwd(dx=ODD) == bwd(dt_=ODD) == bwd(dg=ODD) == bwd(db=ODD) == B.SPC_ERR_ARG
    assert bwd(ws=None) == bwd(ws=ODD) == B.SPC_ERR_ARG
    b = ctypes.c_size_t()
    assert L.spc_layer_norm_workspace(100000, 64, None) == B.SPC_ERR_ARG
    assert L.spc_layer_norm_workspace(100000, 64, ctypes.byref(b)) == B.SPC_OK and b.value > 0
    assert bwd(wsb=b.value - 1) == B.SPC_ERR_WORKSPACE
    # a launch holds fewer than 2^32 threads: 2^26 groups of 4 rows of 64 lanes are 2^34
    ws = lambda n, C: L.spc_layer_norm_workspace(n, C, ctypes.byref(b))
    assert ws((1 << 26) - 4, 512) == ws(END - 1, 16) == ws(1, 4096) == B.SPC_OK
    assert ws(1 << 26, 512) == B.SPC_ERR_UNSUPPORTED


def test_rotary_refusals():
    L = B.lib()

    def f(dt=2, x=P, ldx=128, n=100, H=2, D=64, pos=P, ldp=4, pairs=(8, 8, 8), freq=P, out=P, ldo=128, axes=None):
        a = (ctypes.c_int32 * max(len(pairs), 1))(*pairs)
        return L.spc_rotary(dt, x, ldx, n, H, D, pos, ldp, len(pairs) if axes is None else axes, a, freq, 0, out, ldo, None)

    assert f(n=0) == f(n=0, x=None, pos=None, freq=None, out=None) == B.SPC_OK
    assert f(D=24) == f(D=0) == f(D=4112, ldx=1 << 20, ldo=1 << 20) == B.SPC_ERR_UNSUPPORTED
    assert f(H=1 << 20, D=1024, ldx=1 << 30, ldo=1 << 30) == B.SPC_ERR_UNSUPPORTED
    assert f(dt=4) == f(n=-1) == f(n=END) == f(H=0) == f(ldx=120) == f(ldo=132) == f(ldx=1 << 31) == B.SPC_ERR_ARG
    assert f(axes=0) == f(pairs=(1,) * 9, ldp=9) == f(ldp=2) == f(pairs=(8, -1, 8)) == f(pairs=(16, 16, 1)) == B.SPC_ERR_ARG
    assert f(x=None) == f(out=None) == f(pos=None) == f(freq=None) == f(x=ODD) == f(out=ODD) == B.SPC_ERR_ARG
    assert f(pos=ctypes.c_void_p(0x100002)) == f(freq=ctypes.c_void_p(0x100001)) == B.SPC_ERR_ARG
    assert L.spc_rotary(2, P, 128, 100, 2, 64, P, 4, 3, None, P, 0, P, 128, None) == B.SPC_ERR_ARG


def attn(n_q=1000, n_kv=1000, S=1, H=4, Hk=2, D=32, causal=0, scale=0.5, qp=None, kp=None, qo=None, ko=None):
    return B._AttnArg(n_q, n_kv, S, H, Hk, D, causal, scale, qp, kp, qo, ko)


def test_attention_refusals():
    L, R = B.lib(), ctypes.byref

    def fwd(dt=2, a=None, q=P, ldq=128, k=P, ldk=64, v=P, ldv=64, out=P, ldo=128, st=P, rest=P, ws=P, wsb=BIG, **kw):
        return L.spc_attention_fwd(dt, R(attn(**kw) if a is None else a), q, ldq, k, ldk, v, ldv, out, ldo, st, rest, ws, wsb,
                                   None)

    def bwd(dt=2, a=None, do=P, lddo=128, q=P, ldq=128, k=P, ldk=64, v=P, ldv=64, out=P, ldo=128, st=P, rest=P, dq=P, lddq=128, dk=P,
            lddk=64, dv=P, lddv=64, ws=P, wsb=BIG, **kw):
        return L.spc_attention_bwd(dt, R(attn(**kw) if a is None else a), do, lddo, q, ldq, k, ldk, v, ldv, out, ldo, st, rest,
                                   dq, lddq, dk, lddk, dv, lddv, ws, wsb, None)

    for f in (fwd, bwd):
        assert f(D=24) == f(D=144, ldq=1 << 10, ldk=1 << 10) == f(D=0) == B.SPC_ERR_UNSUPPORTED
        assert f(n_q=1 << 30) == f(n_kv=1 << 30, ) == f(H=1 << 20, Hk=1 << 20) == B.SPC_ERR_UNSUPPORTED
        assert f(dt=3) == f(n_q=-1) == f(n_kv=-1) == f(n_q=END) == f(S=0) == f(S=END) == B.SPC_ERR_ARG
        assert f(H=0) == f(Hk=0) == f(H=3) == f(H=-4) == B.SPC_ERR_ARG
        for s in (0.0, -1.0, float("inf"), float("nan")):
            assert f(scale=s) == B.SPC_ERR_ARG
        assert f(S=2) == f(S=2, qp=0x100000) == f(S=2, kp=0x100000) == B.SPC_ERR_ARG
        assert f(qp=0x100008) == f(kp=0x100008) == f(qo=0x100008) == f(ko=0x100008) == B.SPC_ERR_ARG
        for name in ("q", "k", "v", "out"):
            assert f(**{name: None}) == f(**{name: ODD}) == B.SPC_ERR_ARG, name
        for name in ("ldq", "ldk", "ldv", "ldo"):
            assert f(**{name: 60}) == f(**{name: 132}) == f(**{name: 1 << 31}) == B.SPC_ERR_ARG, name
        assert f(st=ODD) == f(rest=ODD) == f(ws=ODD) == B.SPC_ERR_ARG
    for name in ("do", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == bwd(**{name: ODD}) == B.SPC_ERR_ARG, name
    for name in ("lddo", "lddq", "lddk", "lddv"):
        assert bwd(**{name: 60}) == bwd(**{name: 132}) == B.SPC_ERR_ARG, name
    assert bwd(st=None) == bwd(ws=None) == B.SPC_ERR_ARG
    assert fwd(n_q=0) == fwd(n_q=0, q=None, out=None, st=None) == B.SPC_OK
    f_, b_ = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.spc_attention_workspace(2, R(attn()), None, R(b_)) == B.SPC_ERR_ARG
    assert L.spc_attention_workspace(2, None, R(f_), R(b_)) == B.SPC_ERR_ARG
    one = dict(n_q=4, n_kv=100000)                                     # few queries: split over the keys
    assert L.spc_attention_workspace(2, R(attn(**one)), R(f_), R(b_)) == B.SPC_OK and f_.value > 0 and b_.value > 0
    assert fwd(wsb=f_.value - 1, **one) == bwd(wsb=b_.value - 1, **one) == B.SPC_ERR_WORKSPACE
    assert fwd(ws=None, **one) == B.SPC_ERR_ARG


def test_attention_limits():
    f_, b_ = ctypes.c_size_t(), ctypes.c_size_t()
    f = lambda **kw: B.lib().spc_attention_workspace(2, ctypes.byref(attn(**dict(dict(H=1, Hk=1), **kw))), ctypes.byref(f_),
                                                     ctypes.byref(b_))
    few = (1 << 31) - (1 << 14)
    assert f(n_q=few) == f(n_kv=few) == f(S=(1 << 26) - 512, n_q=0, n_kv=0) == B.SPC_OK
    assert f(n_q=END - 1) == f(n_kv=END - 1) == B.SPC_ERR_UNSUPPORTED  # 2^24 groups of 128 rows, 256 threads each
    assert f(S=1 << 26, n_q=0, n_kv=0) == B.SPC_ERR_UNSUPPORTED        # a wave for each: 2^32 threads
    assert f(S=1 << 24, n_q=END - 1) == B.SPC_ERR_UNSUPPORTED
    assert f(n_q=1 << 20, H=1 << 11, Hk=1 << 11, D=16) == B.SPC_ERR_UNSUPPORTED   # rows x heads
    # the partial results stay small: few rows times few splits
    for n_q, n_kv in ((1, 1 << 28), (1 << 27, 1), (64, 1 << 20), (4096, 1 << 20), (20000, 20000)):
        assert f(n_q=n_q, n_kv=n_kv, H=8, Hk=4, D=128) == B.SPC_OK
        assert max(f_.value, b_.value) <= (1 << 30) + 4 * n_q * 8 + 256


def test_binding_refuses_cpu_tensors():
    x, h = torch.zeros(4, 16), torch.zeros(4, 1, 16)
    for f in (lambda: spc.layer_norm_fwd(x), lambda: spc.layer_norm_bwd(x, x, None, x),
              lambda: spc.rotary(h, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(8), (8,)),
              lambda: spc.attention_fwd(h, h, h), lambda: spc.attention_bwd(h, h, h, h, h, (x, None))):
        with pytest.raises(TypeError):
            f()


def test_calls_go_to_their_tensors_device(monkeypatch):
    """A call on tensors of another device than the current one makes that
    device current for the launch, and only then."""
    log = []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            log.append(("in", self.dev.index))

        def __exit__(self, *a):
            log.append(("out", self.dev.index))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "_stream", lambda dev: ("stream", dev.index))
    f = lambda *a: log.append(a) or 0
    assert B._call(torch.device("cuda", 0), f, 1, 2) == 0 and log == [(1, 2, ("stream", 0))]
    log.clear()
    assert B._call(torch.device("cuda", 1), f, 3) == 0
    assert log == [("in", 1), (3, ("stream", 1)), ("out", 1)]
