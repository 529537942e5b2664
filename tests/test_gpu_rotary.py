"""Rotary positions of several axes against the fp64 oracle."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from tests.parity import cuda
from tests.rowops_cases import DTYPES, within

pytestmark = pytest.mark.gpu


def freqs(pairs, base=10000.0):
    return torch.tensor([base ** (-j / max(m, 1)) for m in pairs for j in range(m)], dtype=torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,H,D,pairs,span", [
    (1, 1, 16, (8,), 10), (7, 8, 64, (32,), 1 << 20), (100, 3, 16, (2, 3, 3), 1600), (333, 2, 48, (8, 8, 7), 1600),
    (50, 1, 128, (10, 0, 20, 5), 300), (20, 4, 32, (0,), 9), (3000, 8, 32, (5, 5, 6), 128), (3, 1, 4096, (1000, 1048), 50),
    (5000, 1, 16, (4, 4), 77)])
def test_rotation(n, H, D, pairs, span, dtype):
    print(f"rotary {n} x {H} x {D} {pairs} {dtype}", flush=True)
    g = torch.Generator().manual_seed(n + D)
    x = torch.randn(n, H, D, generator=g).to(dtype)
    pos = torch.randint(-span, span, (n, len(pairs) + 1), generator=g, dtype=torch.int32)
    f = freqs(pairs)
    for inverse in (False, True):
        out = spc.rotary(cuda(x), cuda(pos)[:, 1:], cuda(f), pairs, inverse=inverse)
        ref, env = A.rotary(x, pos[:, 1:], f, pairs, inverse)
        within(out, ref, env, dtype, "out")
    y = cuda(x)
    assert spc.rotary(y, cuda(pos)[:, 1:], cuda(f), pairs, inverse=True, out=y) is y and torch.equal(y, out)


def test_far_positions():
    # int32's ends: the angle is some 10^9 radians, its error that of a product in double
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 1], [0]], dtype=torch.int32)
    x = torch.randn(4, 2, 32, generator=torch.Generator().manual_seed(1))
    f = torch.rand(16, generator=torch.Generator().manual_seed(2)) + 0.5
    ref, env = A.rotary(x, pos, f, (16,))
    # 3 roundings of the angle in double: 2^31 * 1.5 * 3 * 2^-53 < 1.1e-6 radians (numpy's cos of the same product has one of them)
    a = np.abs(x.double().numpy())
    env = env + 1.5e-6 * (a + a.reshape(4, 2, 16, 2)[..., ::-1].reshape(a.shape))
    within(spc.rotary(cuda(x), cuda(pos), cuda(f), (16,)), ref, env, torch.float32, "far")


def test_slices_of_one_product():
    g = torch.Generator().manual_seed(3)
    qkv = cuda(torch.randn(60, 3 * 64, generator=g).bfloat16())
    pos = cuda(torch.randint(0, 50, (60, 4), generator=g, dtype=torch.int32))
    f, pairs = cuda(freqs((2, 3, 3))), (2, 3, 3)
    qk = qkv[:, :128].view(60, 8, 16)
    ref = spc.rotary(qk.contiguous(), pos[:, 1:], f, pairs)
    save = qkv.clone()
    spc.rotary(qk, pos[:, 1:], f, pairs, out=qk)
    assert torch.equal(qkv[:, :128].reshape(60, 8, 16), ref) and torch.equal(qkv[:, 128:], save[:, 128:])
    with pytest.raises(ValueError):
        spc.rotary(qkv[:, :64].view(60, 4, 16).transpose(0, 1), pos[:4, 1:], f, pairs)
    with pytest.raises(ValueError):
        spc.rotary(qk, pos, f, pairs)
    with pytest.raises(ValueError):
        spc.rotary(qk, pos[:, 1:], f[:5], pairs)
    with pytest.raises(TypeError):
        spc.rotary(qk, pos[:, 1:].float(), f, pairs)


def test_no_rows_and_nan():
    f, pairs = cuda(freqs((8,))), (8,)
    assert spc.rotary(torch.empty(0, 2, 16, device="cuda"), torch.empty(0, 1, dtype=torch.int32, device="cuda"), f, pairs).shape == (0, 2, 16)
    x = torch.randn(9, 2, 16, generator=torch.Generator().manual_seed(4))
    pos = cuda(torch.arange(9, dtype=torch.int32)[:, None])
    a = spc.rotary(cuda(x), pos, f, pairs)
    x[4, 1, 6] = float("nan")
    b = spc.rotary(cuda(x), pos, f, pairs)
    assert b[4, 1, 6:8].isnan().all()
    b[4, 1, 6:8] = a[4, 1, 6:8]
    assert torch.equal(a, b)
