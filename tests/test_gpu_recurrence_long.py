"""GPU recurrence over long sequences with a long memory: strips of every length
and more tiles than one round of their join takes, against a scan in fp64 by
doubling, within the envelope of the fp32 roundings."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.rowops_cases import half_step, tiny

pytestmark = pytest.mark.gpu


def scan64(a, b):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... (fp64, on the device)."""
    step = 1
    while step < b.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def close(got, ref, env, dtype, what):
    bound = env + half_step(dtype) * (ref.abs() + env) + tiny(dtype)
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("C,dtype,reverse", [(64, torch.float32, False), (64, torch.bfloat16, True), (144, torch.float16, True),
                                             (256, torch.bfloat16, False)])
def test_recurrence_long_sequences(C, dtype, reverse):
    n, K = 300001, 8 * R.EPS
    lengths = [150001, 0, 1, 149999]
    print(f"long recurrence n={n} C={C} {dtype} reverse={reverse}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(C)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    # memories of some thousand rows and values around 1: a lost state shows at once
    gate, x, dh = (rand(n, C) + 8.0).to(dtype), (rand(n, C) + 1.0).to(dtype), (rand(n, C) + 1.0).to(dtype)
    h0, dl = rand(4, C), rand(4, C)
    ptr = [0] + torch.tensor(lengths).cumsum(0).tolist()
    sp = torch.tensor(ptr, dtype=torch.int32, device="cuda")
    out, last, carry = spc.linear_recurrence_fwd(gate, x, sp, h0, reverse=reverse, want_carry=True)
    dg, dx, dh0 = spc.linear_recurrence_bwd(dh, gate, x, sp, carry, h0, dh_last=dl, reverse=reverse, want_dh0=True)

    turn = (lambda t: t.flip(0)) if reverse else (lambda t: t)
    G, X, D = (turn(t.double()) for t in (gate, x, dh))
    a, na = torch.sigmoid(G), torch.sigmoid(-G)
    full = [s for s in range(4) if lengths[s]]
    first = [n - ptr[s + 1] if reverse else ptr[s] for s in full]      # in the order of the walk
    end = [f + lengths[s] - 1 for f, s in zip(first, full)]
    chain = a.clone()
    chain[first] = 0
    b = na * X
    b[first] += a[first] * h0[full].double()
    h = scan64(chain, b)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[full].double()
    he = scan64(chain, K * (before.abs() + X.abs()))
    close(turn(out), h, he, dtype, "out")
    close(last[full], h[end], he[end], torch.float32, "h_last")
    assert torch.equal(last[1], h0[1])

    D = D.clone()
    D[end] += dl[full].double()
    back = torch.cat([a[1:], a[:1]])
    back[end] = 0
    big = scan64(back.flip(0), D.flip(0)).flip(0)
    c = K * (big.abs() + D.abs()) + K * (back * torch.cat([big[1:], big[:1]])).abs()
    be = scan64(back.flip(0), c.flip(0)).flip(0)
    he0 = torch.cat([he[:1], he[:-1]])
    he0[first] = 0
    close(turn(dx), na * big, na * (be + K * big.abs()), dtype, "dx")
    close(turn(dg), a * na * (before - X) * big,
          a * na * ((before - X).abs() * be + big.abs() * (he0 + K * (before.abs() + X.abs()))), dtype, "dgate")
    close(dh0[full], (a * big)[first], (a * be + K * (a * big).abs())[first], torch.float32, "dh0")
    assert torch.equal(dh0[1], dl[1])


@pytest.mark.parametrize("n", [120, 200, 300])
def test_recurrence_few_rows_of_very_many_channels(n):
    # enough elements for long strips, but hardly a tile of rows
    C, K = 180224, 8 * R.EPS
    print(f"wide recurrence n={n} C={C}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    gate, x, dh = (torch.randn(n, C, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, last, carry = spc.linear_recurrence_fwd(gate, x, want_carry=True)
    dg, dx, _ = spc.linear_recurrence_bwd(dh, gate, x, None, carry)
    a, na, X = torch.sigmoid(gate.double()), torch.sigmoid(-gate.double()), x.double()
    h, e = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    before = []
    for t in range(n):
        before.append((h, e))
        e = a[t] * e + K * (h.abs() + X[t].abs())
        h = a[t] * h + na[t] * X[t]
        close(out[t], h, e, torch.bfloat16, f"out {t}")
    close(last[0], h, e, torch.float32, "h_last")
    d, e = torch.zeros_like(h), torch.zeros_like(h)
    for t in range(n - 1, -1, -1):
        hp, he = before[t]
        d = d + dh[t].double()
        e = e + K * (d.abs() + dh[t].double().abs())
        close(dx[t], na[t] * d, na[t] * (e + K * d.abs()), torch.bfloat16, f"dx {t}")
        close(dg[t], a[t] * na[t] * (hp - X[t]) * d,
              a[t] * na[t] * ((hp - X[t]).abs() * e + d.abs() * (he + K * (hp.abs() + X[t].abs()))), torch.bfloat16, f"dgate {t}")
        d, e = a[t] * d, a[t] * e + K * (a[t] * d).abs()
