"""Outputs that overlap an input or one another, where the contract does not
allow it, are refused before any launch.  Every call here is refused, so the
made-up pointers are never dereferenced; layouts that are allowed run in the GPU
tests (slices of one product, results over their inputs)."""

import ctypes
import os

import pytest

import sparse_convolution_hash_amd.binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libspc.so not built")

BIG = 1 << 60
AT = 1 << 40


def ptr(i, off=0):
    """Buffers far apart, and places in them."""
    return ctypes.c_void_p(AT + (i << 32) + off)


def refused(status):
    return status == B.SPC_ERR_ARG and b"overlap" in B.lib().spc_last_error()


N, C = 100, 64                                   # bf16: rows of 128 bytes, 12,800 in all


def test_layer_norm():
    L = B.lib()

    def fwd(x=ptr(0), r=None, y=ptr(2), t=None):
        return L.spc_layer_norm_fwd(2, x, r, N, C, None, None, 1e-5, y, t, ptr(9), None)

    def bwd(dy=ptr(0), x=ptr(1), dt=None, dx=ptr(3)):
        return L.spc_layer_norm_bwd(2, dy, x, N, C, None, ptr(9), dt, dx, None, None, None, 0, None)

    for off in (128, 12784, -12784, -128):       # rows shifted against each other: rows of one are written before they are read
        base = ptr(0, 1 << 20)
        moved = ptr(0, (1 << 20) + off)
        assert refused(fwd(x=base, y=moved))
        assert refused(fwd(x=base, r=ptr(1), y=ptr(2), t=moved))
        assert refused(fwd(x=ptr(1), r=base, y=ptr(2), t=moved))
        assert refused(fwd(x=ptr(1), r=base, y=moved, t=ptr(3)))
        assert refused(fwd(x=ptr(1), r=ptr(2), y=base, t=moved))
        assert refused(bwd(dy=base, dx=moved))
        assert refused(bwd(x=base, dx=moved))
        assert refused(bwd(dt=base, dx=moved))
    assert refused(fwd(r=ptr(1), y=ptr(2), t=ptr(2)))
    assert refused(bwd(dx=ptr(1)))               # dx over x


def test_rotary():
    pairs = (ctypes.c_int32 * 1)(16)

    def f(x, ldx, out, ldo, n=N, H=2, D=32):
        return B.lib().spc_rotary(2, x, ldx, n, H, D, ptr(7), 1, 1, pairs, ptr(8), 0, out, ldo, None)

    a = ptr(0, 1 << 20)
    for off in (128, 16, -16, 12784, -12784):
        assert refused(f(a, 64, ptr(0, (1 << 20) + off), 64))
    assert refused(f(a, 128, a, 64)) and refused(f(a, 64, a, 128))       # in place needs the same stride
    assert refused(f(a, 192, ptr(0, (1 << 20) + 64), 192))               # columns 0-63 and 32-95 of one tensor
    assert refused(f(a, 128, ptr(0, (1 << 20) + 16384 + 64), 192))       # other strides, a row meets one far down


def attn(n_q=N, n_kv=N, H=4, Hk=2, D=32):
    return B._AttnArg(n_q, n_kv, 1, H, Hk, D, 0, 0.5, None, None, None, None)


def test_attention():
    L, R = B.lib(), ctypes.byref
    lq, lk = 128, 64

    def fwd(q=ptr(0), ldq=lq, k=ptr(1), ldk=lk, v=ptr(2), ldv=lk, out=ptr(3), ldo=lq, rest=None, **kw):
        return L.spc_attention_fwd(2, R(attn(**kw)), q, ldq, k, ldk, v, ldv, out, ldo, None, rest, ptr(9), BIG, None)

    def bwd(do=ptr(0), lddo=lq, q=ptr(1), ldq=lq, k=ptr(2), ldk=lk, v=ptr(3), ldv=lk, out=ptr(4), ldo=lq, rest=None, dq=ptr(5), lddq=lq,
            dk=ptr(6), lddk=lk, dv=ptr(7), lddv=lk, **kw):
        return L.spc_attention_bwd(2, R(attn(**kw)), do, lddo, q, ldq, k, ldk, v, ldv, out, ldo, ptr(8), rest, dq, lddq, dk, lddk, dv,
                                   lddv, ptr(9), BIG, None)

    base = 1 << 20
    b = ptr(0, base)
    for off in (0, 256, 64, -64, 25600 - 16, 16 - 25600):
        m = ptr(0, base + off)
        assert refused(fwd(q=b, out=m))
        for name in ("do", "q", "out"):
            assert refused(bwd(**{name: b}, dq=m)), name
        assert off < -12800 or refused(bwd(do=ptr(10), dq=b, dk=m))
    for off in (0, 128, 64, -64, 12800 - 16):
        m = ptr(0, base + off)
        for name in ("k", "v"):
            assert refused(fwd(q=ptr(10), **{name: b}, out=m)), name
            for d in ("dq", "dk", "dv"):
                assert refused(bwd(do=ptr(10), **{name: b}, **{d: m})), (name, d)
        assert refused(bwd(do=ptr(10), dk=b, dv=m))
    # slices of one product of 256 columns (q 128, k 64, v 64): out or a gradient beside them, a column too far
    s = dict(q=b, ldq=256, k=ptr(0, base + 256), ldk=256, v=ptr(0, base + 384), ldv=256)
    assert refused(fwd(**s, out=ptr(0, base + 240), ldo=256)) and refused(fwd(**s, out=ptr(0, base + 512), ldo=256))
    g = ptr(10, base)
    assert refused(bwd(do=ptr(11), dq=g, lddq=256, dk=ptr(10, base + 240), lddk=256))
    assert refused(bwd(do=ptr(11), dk=g, lddk=128, dv=ptr(10, base + 112), lddv=128))
    # rest, dense, under out and over the gradients
    assert refused(fwd(rest=ptr(3, 25584))) and refused(bwd(do=ptr(11), rest=ptr(5, 25584)))
    # more rows than 32 bits of bytes
    big = dict(n_q=1 << 26, n_kv=1 << 26)
    assert refused(fwd(q=ptr(100), k=ptr(200), v=ptr(300), out=ptr(100, ((1 << 26) - 1) * 256), **big))
