"""GPU gated linear recurrence, its backward and its single step against the
fp64 oracle, within the envelope of its own fp32 roundings."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, ptr_of, ragged, within

pytestmark = pytest.mark.gpu


def case(seed, n, C, S, dtype, gate_mean=2.0):
    g = torch.Generator().manual_seed(seed)
    gate = (torch.randn(n, C, generator=g) + gate_mean + torch.randn(C, generator=g)).to(dtype)
    x, dh = (torch.randn(n, C, generator=g).to(dtype) for _ in range(2))
    return gate, x, dh, torch.randn(S, C, generator=g), torch.randn(S, C, generator=g)


def shuffled(seed, ptr, n):
    r = np.random.default_rng(seed)
    o = np.arange(n, dtype=np.int32)
    for a, b in zip(ptr, ptr[1:]):
        o[a:b] = a + r.permutation(b - a)
    return torch.from_numpy(o)


def run(seed, n, C, lengths, dtype, ordered=False, reverse=False, state=True, wide=False, gate_mean=2.0, ptr=None,
        order=None):
    ptr = ptr_of(lengths) if ptr is None else ptr
    S = len(ptr) - 1
    print(f"recurrence n={n} C={C} S={S} {str(lengths)[:50]} {dtype} ordered={ordered} reverse={reverse} state={state} "
          f"wide={wide}", flush=True)
    gate, x, dh, h0, dl = case(seed, n, C, S, dtype, gate_mean)
    if ordered and order is None:
        order = shuffled(seed, ptr, n)
    h0, dl = (h0, dl) if state else (None, None)
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    if wide:      # gate and x as the two halves of one product's rows, with a gap behind them
        both = torch.full((n, 2 * C + 16), float("nan"), dtype=dtype, device="cuda")
        both[:, :C], both[:, C:2 * C] = cuda(gate), cuda(x)
        gd, xd = both[:, :C], both[:, C:2 * C]
        grads = torch.full((n, 2 * C + 32), 7.0, dtype=dtype, device="cuda")
        dgd, dxd = grads[:, :C], grads[:, C:2 * C]
    else:
        gd, xd, dgd, dxd = cuda(gate), cuda(x), None, None
    on = None if order is None else order.numpy()
    kw = dict(h0=None if h0 is None else cuda(h0), order=None if order is None else cuda(order), reverse=reverse)
    out, last, carry = spc.linear_recurrence_fwd(gd, xd, sp, want_carry=True, **kw)
    dg, dx, dh0 = spc.linear_recurrence_bwd(cuda(dh), gd, xd, sp, carry, dh_last=None if dl is None else cuda(dl),
                                            want_dh0=True, dgate=dgd, dx=dxd, **kw)
    ro, rl, _, eo, el = R.recurrence_fwd(gate, x, ptr, h0, on, reverse)
    rg, rx, r0, eg, ex, e0 = R.recurrence_bwd(dh, gate, x, ptr, h0, dl, on, reverse)
    rows = np.zeros(n, bool)
    for s in range(S):
        rows[R._rows(ptr, s, on, reverse, n)] = True
    t = torch.from_numpy(rows)
    within(out.cpu()[t], ro[rows], eo[rows], dtype, "out")
    within(last, rl, el, torch.float32, "h_last")
    within(dg.cpu()[t], rg[rows], eg[rows], dtype, "dgate")
    within(dx.cpu()[t], rx[rows], ex[rows], dtype, "dx")
    within(dh0, r0, e0, torch.float32, "dh0")
    if wide:
        assert (grads[:, 2 * C:] == 7).all()
    # without a carry the forward is the same, bit for bit, and so is a second run
    out2, last2, none = spc.linear_recurrence_fwd(gd, xd, sp, **kw)
    assert none is None and torch.equal(out.cpu()[t], out2.cpu()[t]) and torch.equal(last, last2)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1025])
def test_recurrence_lengths(dtype, n):
    run(n, n, 16, [n], dtype)
    run(n + 1, n, 64, ragged(n, n, 5), dtype, reverse=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ordered", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("C", [16, 32, 48, 64, 80, 112, 272])
def test_recurrence_channels_orders_directions(dtype, ordered, reverse, C):
    run(C, 700, C, ragged(C, 700, 6), dtype, ordered=ordered, reverse=reverse, state=C % 32 == 16, wide=C % 64 == 16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_recurrence_long_memory(dtype, reverse):
    # gates around 6: a memory of hundreds of rows, across many tiles
    run(31, 9001, 32, [9001], dtype, reverse=reverse, gate_mean=6.0)
    run(32, 9001, 16, [4500, 0, 1, 4500], dtype, reverse=reverse, ordered=True, gate_mean=6.0)


@pytest.mark.parametrize("reverse", [False, True])
def test_recurrence_many_tiles(reverse):
    run(33, 70001, 16, [33333, 36668], torch.float32, reverse=reverse, wide=True)


def test_recurrence_many_short_samples():
    run(34, 3000, 32, [0, 1, 2, 0, 3] * 500, torch.float32)
    run(35, 3000, 32, [0, 1, 2, 0, 3] * 500, torch.bfloat16, reverse=True, ordered=True)
    run(36, 40, 16, [0] * 300 + [40] + [0] * 300, torch.float32, reverse=True)


def test_recurrence_gates_at_their_ends():
    # sigmoid of +-100 and of infinities: h keeps its value, or takes x
    n, C = 300, 16
    x = torch.randn(n, C, generator=torch.Generator().manual_seed(37))
    gate = torch.zeros(n, C)
    gate[:, 0], gate[:, 1], gate[:, 2], gate[:, 3] = 100, -100, float("inf"), float("-inf")
    h0 = torch.full((1, C), 1.5)
    out, last, _ = spc.linear_recurrence_fwd(cuda(gate), cuda(x), None, cuda(h0))
    out = out.cpu()
    assert (out[:, 0] == 1.5).all() and (out[:, 2] == 1.5).all()
    assert torch.equal(out[:, 1], x[:, 1]) and torch.equal(out[:, 3], x[:, 3])
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("reverse", [False, True])
def test_recurrence_nan_stays_in_its_sample_and_channel(reverse):
    n, C = 2000, 32
    gate, x, dh, h0, dl = case(38, n, C, 3, torch.float32)
    ptr = [0, 900, 1200, 2000]
    x[1000, 5], gate[1100, 6], dh[1000, 7], h0[1, 8], dl[1, 9] = float("nan"), float("nan"), float("inf"), float("inf"), float("nan")
    sp = cuda(torch.tensor(ptr, dtype=torch.int32))
    kw = dict(h0=cuda(h0), reverse=reverse)
    out, last, carry = spc.linear_recurrence_fwd(cuda(gate), cuda(x), sp, want_carry=True, **kw)
    dg, dx, dh0 = spc.linear_recurrence_bwd(cuda(dh), cuda(gate), cuda(x), sp, carry, dh_last=cuda(dl), want_dh0=True, **kw)
    for t in (out, dg, dx):
        t = t.cpu()
        ok = torch.isfinite(t)
        assert ok[:900].all() and ok[1200:].all() and ok[:, :5].all() and ok[:, 10:].all()
    for t in (last, dh0):
        ok = torch.isfinite(t).cpu()
        assert ok[0].all() and ok[2].all() and ok[:, :5].all() and ok[:, 10:].all()
    assert torch.isnan(out[1000, 5]) and torch.isnan(out[1100, 6])


def test_recurrence_rows_outside_every_sample_and_bad_order():
    n, C = 600, 16
    run(39, n, C, "100..250..500", torch.float32, ptr=[100, 250, 500])
    order = torch.arange(n, dtype=torch.int32)
    order[::7] = -1
    order[3::50] = n + 5
    run(40, n, C, "order with holes", torch.float32, ptr=[0, 250, 600], order=order, ordered=True)
    run(41, n, C, "order with holes", torch.float32, ptr=[0, 250, 600], order=order, ordered=True, reverse=True)
    gate, x, *_ = case(42, n, C, 1, torch.float32)
    out = torch.full((n, C), 7.0, device="cuda")
    spc.linear_recurrence_fwd(cuda(gate), cuda(x), cuda(torch.tensor([100, 500], dtype=torch.int32)), out=out)
    assert (out[:100] == 7).all() and (out[500:] == 7).all()


def test_recurrence_no_rows():
    e = torch.empty((0, 16), device="cuda")
    sp = torch.zeros(4, dtype=torch.int32, device="cuda")
    h0, dl = torch.randn(3, 16, device="cuda"), torch.randn(3, 16, device="cuda")
    out, last, carry = spc.linear_recurrence_fwd(e, e, sp, h0, want_carry=True)
    assert out.shape == (0, 16) and torch.equal(last, h0)
    dg, dx, dh0 = spc.linear_recurrence_bwd(e, e, e, sp, carry, h0, dh_last=dl, want_dh0=True)
    assert torch.equal(dh0, dl)
    assert (spc.linear_recurrence_fwd(e, e, sp)[1] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,C", [(1, 16), (3, 48), (130, 64), (1, 4096)])
def test_recurrence_step_is_one_row(dtype, n, C):
    gate, x, _, h0, _ = case(n + C, n, C, n, dtype)
    state = cuda(h0)
    new = torch.empty_like(state)
    out = spc.linear_recurrence_step(cuda(gate), cuda(x), state, new_state=new)
    assert torch.equal(state, cuda(h0))
    ro, rl, _, eo, el = R.recurrence_fwd(gate, x, list(range(n + 1)), h0)
    within(new, rl, el, torch.float32, "state")
    within(out, ro, eo, dtype, "out")
    out2 = spc.linear_recurrence_step(cuda(gate), cuda(x), state)
    assert torch.equal(state, new) and torch.equal(out, out2)


def test_recurrence_steps_continue_a_sequence():
    # a forward over 20 rows, then 5 single steps, is the forward over 25
    gate, x, _, h0, _ = case(43, 25, 32, 1, torch.float32)
    g, v = cuda(gate), cuda(x)
    _, state, _ = spc.linear_recurrence_fwd(g[:20].contiguous(), v[:20].contiguous(), None, cuda(h0))
    ro, _, _, eo, _ = R.recurrence_fwd(gate, x, [0, 25], h0)
    for t in range(20, 25):
        both = torch.cat([g[t:t + 1], v[t:t + 1]], 1)
        out = spc.linear_recurrence_step(both[:, :32], both[:, 32:], state)
        within(out[0], ro[t], 2 * eo[t], torch.float32, f"step {t}")


def test_recurrence_gradient_by_differences():
    n, C = 300, 16
    gate, x, w, h0, wl = (cuda(t) for t in case(44, n, C, 2, torch.float32, 0.0))
    sp = cuda(torch.tensor([0, 120, 300], dtype=torch.int32))
    out, last, carry = spc.linear_recurrence_fwd(gate, x, sp, h0, want_carry=True)
    dg, dx, dh0 = spc.linear_recurrence_bwd(w, gate, x, sp, carry, h0, dh_last=wl, want_dh0=True)
    g = torch.Generator().manual_seed(45)
    ug, ux, u0 = (cuda(torch.randn(*t.shape, generator=g)) for t in (gate, x, h0))
    h = 2.0 ** -7

    def loss(t):
        o, l, _ = spc.linear_recurrence_fwd(gate + t * ug, x + t * ux, sp, h0 + t * u0)
        return ((o.double() * w.double()).sum() + (l.double() * wl.double()).sum()).item()
    diff = (loss(h) - loss(-h)) / (2 * h)
    want = sum((a.double() * b.double()).sum().item() for a, b in ((dg, ug), (dx, ux), (dh0, u0)))
    assert abs(diff - want) < 4800 * (h * h) + 4800 * 2.0 ** -22 / h


def test_recurrence_past_32_bits():
    # 2^31 elements and more: addresses are 64 bits wide
    C = 512
    n = (1 << 31) // C + 1000
    g = torch.Generator(device="cuda").manual_seed(46)
    gate = torch.zeros((n, C), dtype=torch.bfloat16, device="cuda")      # a = 1/2: 64 rows back is 2^-64
    x = torch.randn((n, C), generator=g, device="cuda", dtype=torch.bfloat16)
    for reverse in (False, True):
        out, last, carry = spc.linear_recurrence_fwd(gate, x, None, reverse=reverse, want_carry=True)
        dg, dx, _ = spc.linear_recurrence_bwd(x, gate, x, None, carry, reverse=reverse)
        m = 400
        for a in (n - m, 0):
            xs, gs = x[a:a + m].cpu(), gate[a:a + m].cpu()
            ro, _, _, eo, _ = R.recurrence_fwd(gs, xs, [0, m], None, None, reverse)
            rg, rx, _, eg, ex, _ = R.recurrence_bwd(xs, gs, xs, [0, m], reverse=reverse)
            mid = slice(100, m - 100)      # the cut ends weigh 2^-100 here
            within(out[a:a + m][mid], ro[mid], eo[mid] + 1e-25, torch.bfloat16, "out")
            within(dg[a:a + m][mid], rg[mid], eg[mid] + 1e-25, torch.bfloat16, "dgate")
            within(dx[a:a + m][mid], rx[mid], ex[mid] + 1e-25, torch.bfloat16, "dx")
        del out, dg, dx, carry
