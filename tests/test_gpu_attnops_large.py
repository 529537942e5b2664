"""The attention block's operators on arrays of more than 2^31 elements, dense and
by their strides.  The arrays repeat one block, which is held to the oracle, so
that every row of the whole has to be the block's, bit by bit."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from tests.attn_cases import FLOOR, split_of
from tests.parity import cuda
from tests.rowops_cases import half_step, within

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GIB = 1 << 30


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 64 * GIB:
        pytest.skip("needs 64 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def tiled(t, copies):
    return t.repeat(copies, *[1] * (t.dim() - 1))


def same(got, block, copies):
    """Every copy of the block in got, as bits (a NaN would not equal itself)."""
    g, b = got.view(copies, *block.shape).view(torch.int16), block.view(torch.int16)
    for c in range(copies):
        assert torch.equal(g[c], b), c


@pytest.mark.parametrize("C,rows,copies", [(4096, 1031, 512), (16, 1 << 20, 129)])
def test_layer_norm(C, rows, copies):
    n = rows * copies
    assert n * C > 1 << 31
    print(f"layer norm {n} x {C}", flush=True)
    g = torch.Generator().manual_seed(1)
    r = lambda: cuda(torch.randn(rows, C, generator=g).to(BF16))
    x, res, dy = r(), r(), r()
    gamma, beta = cuda(1 + 0.1 * torch.randn(C, generator=g)), cuda(torch.randn(C, generator=g))
    y, stats, total = spc.layer_norm_fwd(x, gamma, beta, residual=res)
    dx, dg, db = spc.layer_norm_bwd(dy, total, gamma, stats, dtotal=res)
    few = slice(0, 500)
    ref, _, _, env = A.layer_norm_fwd(total[few], gamma, beta, 1e-5)
    within(y[few], ref, env, BF16, "y")
    Y, S, T = spc.layer_norm_fwd(tiled(x, copies), gamma, beta, residual=tiled(res, copies))
    same(T, total, copies)
    same(Y, y, copies)
    assert torch.equal(S.view(copies, rows, 2), stats.expand(copies, rows, 2))
    del Y
    DX, DG, DB = spc.layer_norm_bwd(tiled(dy, copies), T, gamma, S, dtotal=tiled(res, copies))
    same(DX, dx, copies)
    h = (total.double() - stats[:, :1].double()) * stats[:, 1:].double()
    # 16 rows are summed in fp32 and rounded once more: 20 roundings of 2^-24 of the sizes that are added
    for got, terms in ((DG, dy.double() * h), (DB, dy.double())):
        assert ((got.double() - copies * terms.sum(0)).abs() <= copies * 24 * 2.0 ** -24 * terms.abs().sum(0)).all()


def test_rotary():
    rows, copies, H, D = 1024, 257, 256, 32
    assert rows * copies * H * D > 1 << 31
    g = torch.Generator().manual_seed(2)
    x = cuda(torch.randn(rows, H, D, generator=g).to(BF16))
    pos = cuda(torch.randint(-2000, 2000, (rows, 3), generator=g, dtype=torch.int32))
    f, pairs = cuda(torch.rand(14, generator=g)), (5, 5, 4)
    out = spc.rotary(x, pos, f, pairs)
    ref, env = A.rotary(x[:50].cpu(), pos[:50].cpu(), f.cpu(), pairs)
    within(out[:50], ref, env, BF16, "out")
    big = tiled(x, copies)
    spc.rotary(big, tiled(pos, copies), f, pairs, out=big)
    same(big, out, copies)


def far_rows(t, stride, buffer):
    """t's rows `stride` elements apart in the buffer."""
    v = buffer.as_strided((t.shape[0], t.shape[1], t.shape[2]), (stride, t.shape[2], 1))
    v.copy_(t)
    return v


def test_rows_far_apart():
    """21 rows 2^27 - 16 elements apart: 5 GB from the first to the last."""
    n, H, D, stride = 21, 2, 32, (1 << 27) - 16
    g = torch.Generator().manual_seed(3)
    r = lambda h: cuda(torch.randn(n, h, D, generator=g).to(BF16))
    q, k, v, do = r(H), r(H), r(H), r(H)
    out, st = spc.attention_fwd(q, k, v, causal=True, want_stats=True)
    grads = spc.attention_bwd(do, q, k, v, out, st, causal=True)
    buf = torch.zeros(stride * n, dtype=BF16, device="cuda")
    col = H * D                                    # eight tensors side by side in rows of one buffer
    place = lambda i, t: far_rows(t, stride, buf[i * col:])
    Q, K, V, DO = place(0, q), place(1, k), place(2, v), place(3, do)
    O, DQ, DK, DV = (place(i, torch.zeros_like(q)) for i in (4, 5, 6, 7))
    _, st2 = spc.attention_fwd(Q, K, V, causal=True, want_stats=True, out=O)
    spc.attention_bwd(DO, Q, K, V, O, st2, causal=True, dq=DQ, dk=DK, dv=DV)
    for a, b in zip((O, DQ, DK, DV), (out,) + grads):
        assert torch.equal(a, b)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    f = torch.rand(16, device="cuda")
    ref = spc.rotary(q, pos, f, (16,))
    assert torch.equal(spc.rotary(Q, pos, f, (16,), out=O), ref)
    assert not buf.as_strided((n, stride - 8 * col), (stride, 1), 8 * col)[:, :4096].any()


def test_attention():
    w, samples, copies, H, Hk, D = 64, 257, 256, 4, 4, 128
    rows = w * samples
    n = rows * copies
    assert n * H * D > 1 << 31 and n * Hk * D > 1 << 31
    print(f"attention {n} x {H} x {D}", flush=True)
    g = torch.Generator().manual_seed(4)
    r = lambda h: cuda(torch.randn(rows, h, D, generator=g).to(BF16))
    q, k, v, do = r(H), r(Hk), r(Hk), r(H)
    ptr = lambda m: cuda(torch.arange(0, m + 1, w, dtype=torch.int32))
    # along an order, the same within every copy
    order = cuda(torch.cat([w * i + torch.randperm(w, generator=g) for i in range(samples)]).int())
    out, st = spc.attention_fwd(q, k, v, ptr(rows), order, want_stats=True)
    grads = spc.attention_bwd(do, q, k, v, out, st, ptr(rows), order)
    few = 3 * w
    ref = A.attention(q[:few].cpu(), k[:few].cpu(), v[:few].cpu(), [0, w, 2 * w, few], [0, w, 2 * w, few], D ** -0.5,
                      q_order=order[:few].cpu().numpy(), kv_order=order[:few].cpu().numpy(), dout=do[:few].cpu(), step=half_step(BF16),
                      floor=FLOOR[BF16], split=split_of(BF16, D))
    for t, name in zip((out,) + grads, ("out", "dq", "dk", "dv")):
        within(f64(t[:few]), ref[name], ref["e_" + name], BF16, name)
    at = torch.arange(copies, dtype=torch.int32, device="cuda")[:, None] * rows
    O = (order[None] + at).view(-1)
    Q, K, V, DO = (tiled(t, copies) for t in (q, k, v, do))
    OUT, ST = spc.attention_fwd(Q, K, V, ptr(n), O, want_stats=True)
    same(OUT, out, copies)
    same(ST[1], st[1], copies)
    DQ, DK, DV = spc.attention_bwd(DO, Q, K, V, OUT, ST, ptr(n), O)
    for a, b in zip((DQ, DK, DV), grads):
        same(a, b, copies)
