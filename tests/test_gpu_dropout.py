"""GPU dropout against the oracle's mask and fp64 values."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.parity import cuda
from tests.rowops_cases import DTYPES, within

pytestmark = pytest.mark.gpu


def rng_state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def check(x, res, dy, seed, offset, layer, p, dtype):
    drop = spc.Dropout(rng_state(seed, offset), p, layer)
    f = R.drop_factor(seed, offset, layer, p, tuple(x.shape))
    y = spc.dropout_fwd(cuda(x), drop, None if res is None else cuda(res))
    a, b = R.f64(x) * f, 0.0 if res is None else R.f64(res)
    # fp32: the scale's rounding, the product's, the sum's
    within(y, a + b, 4 * R.EPS * (np.abs(a) + np.abs(b)), dtype, "y")
    d = spc.dropout_bwd(cuda(dy), drop)
    within(d, R.f64(dy) * f, 4 * R.EPS * np.abs(R.f64(dy) * f), dtype, "din")
    # dropped elements are the residual (or 0) exactly
    dead = torch.from_numpy(f == 0)
    assert torch.equal(d.cpu()[dead], torch.zeros_like(dy)[dead])
    assert torch.equal(y.cpu()[dead], (torch.zeros_like(x) if res is None else res)[dead])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("numel", [1, 7, 8, 9, 2047, 2048, 2049, 100003])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_sizes(dtype, numel, residual):
    print(f"dropout {numel} {dtype} residual={residual}", flush=True)
    g = torch.Generator().manual_seed(numel)
    x, res, dy = (torch.randn(numel, generator=g).to(dtype) for _ in range(3))
    check(x, res if residual else None, dy, 1234567890123 + numel, 17, 2, 0.3, dtype)


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.999, 1.0])
def test_dropout_probabilities(p):
    g = torch.Generator().manual_seed(5)
    x, res, dy = (torch.randn(300, 48, generator=g) for _ in range(3))
    check(x, res, dy, 99, (1 << 32) - 100, 0, p, torch.float32)   # the counter's carry too


def test_dropout_negative_words_and_layers():
    # seed and offset are 64 bits, whatever their sign in int64; layers differ
    g = torch.Generator().manual_seed(6)
    x, dy = torch.randn(4096, generator=g), torch.randn(4096, generator=g)
    check(x, None, dy, -3, -5, 0xFFFFFFFF, 0.4, torch.float32)
    r = rng_state(3, 0)
    a, b = (spc.dropout_fwd(cuda(x), spc.Dropout(r, 0.5, k)) for k in (0, 1))
    assert not torch.equal(a, b)


def test_dropout_of_infinities_and_nans():
    x = torch.full((512,), float("nan"))
    x[::2] = float("inf")
    drop = spc.Dropout(rng_state(1, 1), 0.5)
    y = spc.dropout_fwd(cuda(x), drop).cpu()
    keep = torch.from_numpy(R.keep_mask(1, 1, 0, 0.5, 512))
    assert (y[~keep] == 0).all()
    assert torch.isnan(y[keep & torch.isnan(x)]).all() and torch.isinf(y[keep & torch.isinf(x)]).all()


def test_dropout_in_place_and_empty():
    g = torch.Generator().manual_seed(8)
    x, res = cuda(torch.randn(1001, 16, generator=g)), cuda(torch.randn(1001, 16, generator=g))
    drop = spc.Dropout(rng_state(4, 4), 0.25)
    want = spc.dropout_fwd(x, drop, res)
    assert torch.equal(spc.dropout_fwd(x.clone(), drop, res), want)
    buf = res.clone()
    assert spc.dropout_fwd(x, drop, buf, out=buf) is buf and torch.equal(buf, want)
    buf = x.clone()
    assert torch.equal(spc.dropout_fwd(buf, drop, res, out=buf), want)
    buf = x.clone()
    assert torch.equal(spc.dropout_bwd(buf, drop, din=buf), spc.dropout_bwd(x, drop))
    assert spc.dropout_fwd(x[:0], drop).shape == (0, 16)


def test_dropout_past_32_bits():
    # elements beyond 2^32: the counter and the addresses are 64 bits wide
    n = (1 << 32) + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = spc.dropout_fwd(x, spc.Dropout(rng_state(11, 0), 0.5), out=x)
    lo = (n - 5000) // 8 * 8
    keep = R.keep_mask(11, lo // 8, 0, 0.5, n - lo)
    assert torch.equal(y[lo:].float().cpu(), torch.from_numpy(keep * 2.0).float())
