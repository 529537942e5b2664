"""Pins of the attention-block oracle: torch's own layer norm and attention in
float64 with their autograd, complex rotations, and differences."""

import numpy as np
import pytest
import torch

from oracle import attnops as A

D64 = torch.float64


def test_layer_norm_equals_torch():
    g = torch.Generator().manual_seed(1)
    x, gamma, beta, dy = (torch.randn(*s, generator=g, dtype=D64) for s in ((7, 48), (48,), (48,), (7, 48)))
    x.requires_grad_(), gamma.requires_grad_(), beta.requires_grad_()
    y = torch.nn.functional.layer_norm(x, (48,), gamma, beta, 1e-5)
    y.backward(dy)
    assert np.allclose(A.layer_norm_fwd(x, gamma, beta, 1e-5)[0], y.detach().numpy(), rtol=0, atol=1e-12)
    dx, dg, db = A.layer_norm_bwd(dy, x, gamma, 1e-5)[:3]
    for a, b in ((dx, x.grad), (dg, gamma.grad), (db, beta.grad)):
        assert np.allclose(a, b.numpy(), rtol=0, atol=1e-12)


def test_rotary_is_a_rotation():
    r = np.random.default_rng(2)
    x, pos, freq = r.normal(size=(5, 2, 16)), r.integers(0, 50, size=(5, 3)), r.normal(size=7)
    out, _ = A.rotary(x, pos, freq, (2, 2, 3))
    z = (x[..., 0::2] + 1j * x[..., 1::2])
    axis = [0, 0, 1, 1, 2, 2, 2]
    turn = np.concatenate([np.exp(1j * pos[:, axis] * freq), np.ones((5, 1))], axis=1)
    w = z * turn[:, None, :]
    assert np.allclose(out[..., 0::2], w.real) and np.allclose(out[..., 1::2], w.imag)
    assert np.array_equal(out[..., 14:], x[..., 14:])
    assert np.allclose(A.rotary(out, pos, freq, (2, 2, 3), True)[0], x)
    # the scores of two rows depend on the difference of their positions alone
    q, k = r.normal(size=(1, 1, 16)), r.normal(size=(1, 1, 16))
    f = lambda a, b: (A.rotary(q, np.array([a]), freq, (2, 2, 3))[0] * A.rotary(k, np.array([b]), freq, (2, 2, 3))[0]).sum()
    assert np.isclose(f([3, 9, 4], [1, 2, 8]), f([13, 29, 34], [11, 22, 38]))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_equals_torch(causal):
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(*s, generator=g, dtype=D64) for s in ((11, 4, 16), (11, 2, 16), (11, 2, 16), (11, 4, 16)))
    for t in (q, k, v):
        t.requires_grad_()
    ptr, order = [0, 4, 4, 5, 11], np.random.default_rng(4).permutation(11)
    order = np.concatenate([order[order < 5], order[order >= 5]])
    out = torch.zeros(11, 4, 16, dtype=D64)
    for s in range(4):
        rows = torch.from_numpy(order[ptr[s]:ptr[s + 1]].copy())
        if len(rows):
            a = [t[rows].transpose(0, 1) for t in (q, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1))]
            o = torch.nn.functional.scaled_dot_product_attention(*a, is_causal=causal, scale=0.3)
            out = out.index_copy(0, rows, o.transpose(0, 1))
    out.backward(do)
    r = A.attention(q, k, v, ptr, ptr, 0.3, causal, order, order, dout=do)
    for name, t in (("out", out), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert np.allclose(r[name], t.detach().numpy(), rtol=0, atol=1e-12), name


def test_attention_against_differences_and_empty_rows():
    # more queries than keys: the first rows of a causal sample see nothing
    r = np.random.default_rng(5)
    q, k, v, g = r.normal(size=(5, 2, 16)), r.normal(size=(3, 1, 16)), r.normal(size=(3, 1, 16)), r.normal(size=(5, 2, 16))
    f = lambda q, k, v: (A.attention(q, k, v, [0, 5], [0, 3], 0.4, True)["out"] * g).sum()
    a = A.attention(q, k, v, [0, 5], [0, 3], 0.4, True, dout=g)
    assert not a["out"][:2].any() and np.isneginf(a["lse"][:, :2]).all() and a["out"][2:].all()
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        d = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            save = t[i]
            t[i] = save + 1e-5
            up = f(q, k, v)
            t[i] = save - 1e-5
            d[i] = (up - f(q, k, v)) / 2e-5
            t[i] = save
        assert np.abs(d - a[name]).max() < 1e-8, name


def test_attention_oracle_catches_mistakes():
    # an oracle whose mask were off by one, or whose heads were shared the other way, differs
    r = np.random.default_rng(6)
    q, k = r.normal(size=(6, 4, 16)), r.normal(size=(6, 2, 16))
    a = A.attention(q, k, k, [0, 6], [0, 6], 1.0, True)["out"]
    assert not np.allclose(a, A.attention(q, k, k, [0, 6], [0, 6], 1.0, False)["out"])
    assert not np.allclose(a, A.attention(q, k[:, ::-1], k[:, ::-1], [0, 6], [0, 6], 1.0, True)["out"])
    assert np.allclose(a[0], np.repeat(k[0], 2, axis=0))       # the first row sees itself
