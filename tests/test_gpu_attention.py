"""Attention, forward and backward, against the fp64 oracle: lengths around the
tiles, shared heads, causal masks with rows that see nothing, orders, keys of
another tensor, splits."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from tests.attn_cases import Case, check
from tests.rowops_cases import DTYPES, ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
def test_head_dims(D, dtype):
    print(f"attention head_dim {D} {dtype}", flush=True)
    check(Case([70, 0, 1, 33, 130], None, 2, 2, D, dtype, seed=1))
    check(Case([40, 3, 65], None, 4, 2, D, dtype, seed=2, causal=True, ordered=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [63, 1, 64], [65, 127], [128, 129], [0, 0, 5, 0], [0]])
def test_lengths(lens, dtype):
    print(f"attention lengths {lens} {dtype}", flush=True)
    for causal in (False, True):
        check(Case(lens, None, 1, 1, 32, dtype, seed=3, causal=causal))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 2), (8, 8), (12, 3)])
def test_shared_heads(H, Hk, dtype):
    print(f"attention heads {H}/{Hk} {dtype}", flush=True)
    check(Case([50, 7, 90], None, H, Hk, 16, dtype, seed=4, causal=True, ordered=True))
    check(Case([5, 40], [77, 20], H, Hk, 16, dtype, seed=5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lq,lk", [([5, 1, 9], [3, 1, 40]), ([40, 33], [7, 0]), ([0, 4], [9, 2]), ([1, 1, 1], [100, 0, 35]),
                                   ([130], [1]), ([3], [200])])
def test_queries_and_keys_of_their_own(lq, lk, dtype):
    # with causal, the first lq - lk queries of a sample see no key
    print(f"attention {lq} {lk} {dtype}", flush=True)
    for causal in (False, True):
        for ordered in (False, True):
            check(Case(lq, lk, 2, 1, 32, dtype, seed=6, causal=causal, ordered=ordered))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lq,lk,H,D", [([1, 1], [3000, 1700], 2, 16), ([1], [5000], 4, 64), ([2500], [3], 1, 32),
                                       ([20, 3], [4000, 900], 1, 128), ([1900], None, 1, 16)])
def test_splits(lq, lk, H, D, dtype):
    # few rows on one side: the other is split and joined
    print(f"attention splits {lq} {lk} {dtype}", flush=True)
    check(Case(lq, lk, H, 1, D, dtype, seed=7))
    check(Case(lq, lk, H, 1, D, dtype, seed=8, causal=True, ordered=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 64, 128])
def test_wide_workgroups(D, dtype):
    # enough rows for workgroups of four waves, in even and ragged samples
    H = 16 if D == 16 else 8
    print(f"attention wide {D} {dtype}", flush=True)
    check(Case([257] * 35, None, H, H, D, dtype, seed=9))
    check(Case(ragged(1, 9000, 20), None, H, H // 2, D, dtype, seed=10, causal=True, ordered=True))


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_small_samples(dtype):
    check(Case(ragged(2, 1500, 300), None, 2, 2, 16, dtype, seed=11))
    check(Case([36] * 100, None, 2, 1, 32, dtype, seed=12, causal=True))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_outside_the_samples(dtype):
    for kw in (dict(lk=None), dict(lk=[0, 30, 5])):
        for ordered in (False, True):
            check(Case([20, 0, 45], kw["lk"], 2, 2, 32, dtype, seed=13, ordered=ordered, outside=9))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gain", [0.0, 12.0, 60.0])
def test_flat_and_peaked(gain, dtype):
    # scores up to some hundred: maxima that grow along the walk, rows that see one key in effect
    check(Case([150, 40], None, 2, 2, 32, dtype, seed=14, gain=gain))
    check(Case([150, 40], None, 2, 2, 32, dtype, seed=15, gain=gain, causal=True))


def test_orders_without_rows():
    # positions whose entry is outside [0, n) have no row: keys that are not there, queries that are not written
    c = Case([70, 40], None, 2, 2, 32, torch.float32, seed=16, ordered=True)
    for causal in (False, True):
        c.causal = causal
        order = c.order.clone()
        order[::7] = torch.tensor([-1, 2 ** 31 - 1, c.n, -2 ** 31])[torch.arange(0, c.n, 7) % 4].int()
        c.order = c.kv_order = order
        check(c)


def test_one_sample_without_offsets():
    c = Case([90], [130], 2, 2, 32, torch.bfloat16, seed=17)
    q, k, v, dout = c.on_gpu()
    a, sa = spc.attention_fwd(q, k, v, want_stats=True)
    b, sb = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    assert torch.equal(a, b) and all(torch.equal(u, w) for u, w in zip(sa, sb))
    for x, y in zip(spc.attention_bwd(dout, q, k, v, a, sa), spc.attention_bwd(dout, q, k, v, b, sb, **c.kw())):
        assert torch.equal(x, y)
    assert spc.attention_fwd(q, k, v)[1] is None


def test_offsets_that_fall_or_leave_the_arrays():
    # no defined values, and no access outside (rows past the arrays hold the mark)
    q = torch.randn(100, 2, 32, device="cuda")
    for p in ([0, 60, 20, 100], [-5, 30, 400, 1000], [90, 10, 95, 3]):
        ptr = torch.tensor(p, dtype=torch.int32, device="cuda")
        out, stats = spc.attention_fwd(q, q, q, ptr, want_stats=True)
        spc.attention_bwd(q, q, q, q, out, stats, ptr)
    torch.cuda.synchronize()


def test_no_rows():
    e = torch.empty(0, 2, 32, device="cuda")
    q = torch.randn(9, 2, 32, device="cuda")
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    n = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    out, stats = spc.attention_fwd(q, e, e, n, kv_ptr=z, want_stats=True)
    assert not out.any() and not stats[0][..., 1].any()
    dq, dk, dv = spc.attention_bwd(q, q, e, e, out, stats, n, kv_ptr=z)
    assert not dq.any() and dk.shape == (0, 2, 32)
    out, stats = spc.attention_fwd(e, q, q, z, kv_ptr=n, want_stats=True)
    assert out.shape == (0, 2, 32)
    dq, dk, dv = spc.attention_bwd(e, e, q, q, out, stats, z, kv_ptr=n)
    assert not dk.any() and not dv.any()
