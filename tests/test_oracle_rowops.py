"""Pins of the row operators' oracle: the generator's published test vectors,
torch's group norm and autograd in fp64, and differences of the recurrence."""

import numpy as np
import pytest
import torch

from oracle import rowops as R


def test_philox_known_answers():
    # the known-answer vectors published with the generator
    for ctr, key, want in [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]:
        assert tuple(int(v) for v in R.philox4x32(ctr, key)) == want


def test_keep_mask_layout_and_rate():
    m = R.keep_mask(7, 5, 3, 0.25, 80)
    w = R.philox4x32((6, 0, 3, 0), (7, 0))
    half = [h for v in w for h in (int(v) & 0xFFFF, int(v) >> 16)]
    assert (m[8:16] == (np.array(half) >= 16384)).all()        # the second group takes counter offset + 1
    assert (m[8:] == R.keep_mask(7, 6, 3, 0.25, 72)).all()
    big = R.keep_mask(1, (1 << 32) - 1, 0, 0.1, 1 << 20)       # the counter's carry into its high word
    # 2^20 draws: the kept share is within 5 standard deviations of 1 - 6554 / 65536
    q = 6554 / 65536
    assert abs(big.mean() - (1 - q)) < 5 * (q * (1 - q) / (1 << 20)) ** 0.5
    assert not R.keep_mask(1, 0, 0, 1.0, 64).any() and R.keep_mask(1, 0, 0, 0.0, 64).all()


@pytest.mark.parametrize("name", ["none", "relu", "silu"])
def test_group_norm_is_torchs(name):
    g = torch.Generator().manual_seed(1)
    ptr, C, G = [0, 5, 5, 6, 20], 16, 4
    x = torch.randn(20, C, generator=g, dtype=torch.float64).requires_grad_()
    gamma = torch.randn(C, generator=g, dtype=torch.float64).requires_grad_()
    beta = torch.randn(C, generator=g, dtype=torch.float64).requires_grad_()
    dy = torch.randn(20, C, generator=g, dtype=torch.float64)
    f = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu}[name]
    y = torch.cat([f(torch.nn.functional.group_norm(x[a:b].t()[None], G, gamma, beta, 1e-3))[0].t()
                   for a, b in zip(ptr, ptr[1:]) if b - a > 1 or (b - a == 1 and C // G > 1)])
    y.backward(dy)
    ours = R.group_norm_fwd(x, G, ptr, gamma, beta, 1e-3, name)[0]
    assert np.allclose(ours, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dgamma, dbeta = R.group_norm_bwd(dy, x, G, ptr, gamma, beta, 1e-3, name)
    for got, want in ((dx, x.grad), (dgamma, gamma.grad), (dbeta, beta.grad)):
        assert np.allclose(got, want.numpy(), rtol=1e-10, atol=1e-11)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("ordered", [False, True])
def test_recurrence_gradient_by_differences(reverse, ordered):
    r = np.random.default_rng(3)
    ptr, C, n = [0, 0, 7, 8, 12], 3, 12
    gate, x, w = r.normal(size=(n, C)), r.normal(size=(n, C)), r.normal(size=(n, C))
    h0, wl = r.normal(size=(4, C)), r.normal(size=(4, C))
    order = np.concatenate([a + r.permutation(b - a) for a, b in zip(ptr, ptr[1:])]) if ordered else None

    def loss(gate, x, h0):
        out, last = R.recurrence_fwd(gate, x, ptr, h0, order, reverse)[:2]
        return (out * w).sum() + (last * wl).sum()

    dg, dx, dh0 = R.recurrence_bwd(w, gate, x, ptr, h0, wl, order, reverse)[:3]
    d = 1e-5
    for k, grad in ((0, dg), (1, dx), (2, dh0)):
        args = [gate, x, h0]
        for i in np.ndindex(grad.shape):
            e = np.zeros(grad.shape)
            e[i] = d
            up, dn = list(args), list(args)
            up[k], dn[k] = args[k] + e, args[k] - e
            # third derivatives are below 10 here: the difference quotient is good to 10 d^2 + 1e-15 / d
            assert abs((loss(*up) - loss(*dn)) / (2 * d) - grad[i]) < 1e-8


def test_recurrence_by_hand():
    z = np.zeros((3, 1))                                     # a = 1/2
    out, last, before, env, _ = R.recurrence_fwd(z, np.array([[8.0], [0.0], [4.0]]), [0, 3], np.array([[2.0]]))
    assert out[:, 0].tolist() == [5.0, 2.5, 3.25] and last[0, 0] == 3.25 and before[:, 0].tolist() == [2.0, 5.0, 2.5]
    out = R.recurrence_fwd(z, np.array([[8.0], [0.0], [4.0]]), [0, 3], None, [2, 9, 0])[0]
    assert out[:, 0].tolist() == [5.0, 0.0, 2.0]             # entry 9 names no row: the state passes
    assert (env > 0).all()
