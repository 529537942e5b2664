"""Attention with infinite and NaN rows (in hidden places they reach nothing),
strides, poisoned workspaces, repeated calls, differences, refusals."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import attnops as A
from oracle.rowops import f64
from sparse_convolution_hash_amd import binding as B
from tests.attn_cases import FLOOR, Case, check
from tests.parity import cuda
from tests.rowops_cases import DTYPES, half_step, within

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]


def run(c):
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    return (out,) + spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("lens", [[40, 100, 37], [600] * 16])
def test_other_samples_stay_clean(lens, bad, dtype):
    H = 1 if len(lens) == 3 else 8
    for causal in (False, True):
        c = Case(lens, None, H, H, 32, dtype, seed=20, causal=causal, ordered=True)
        good = run(c)
        mid = torch.from_numpy(c.order.numpy()[c.q_ptr[1]:c.q_ptr[2]].copy()).long()
        c.q[mid[3]] = bad
        c.k[mid[5]] = bad
        c.v[mid[7]] = bad
        c.dout[mid[9]] = bad
        rest = torch.ones(c.n, dtype=torch.bool)
        rest[mid] = False
        for a, b, name in zip(good, run(c), ("out", "dq", "dk", "dv")):
            assert torch.equal(a[rest], b[rest]), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("n,at,H,D", [(90, 41, 2, 16), (90, 70, 1, 48), (300, 200, 1, 64), (2100, 1500, 8, 32), (2100, 1500, 8, 128)])
def test_hidden_values_reach_nothing(n, at, H, D, bad, dtype):
    """Row `at` of a causal sample: its key and value reach the queries from
    `at` on, its query and gradient the keys up to `at`, and nothing else."""
    print(f"hidden {n} {at} {D} {bad} {dtype}", flush=True)
    c = Case([n], None, H, H, D, dtype, seed=21, causal=True)
    out, dq, dk, dv = run(c)
    keep = {t: getattr(c, t).clone() for t in ("q", "k", "v", "dout")}

    def only(name):
        for t, u in keep.items():
            getattr(c, t).copy_(u)
        getattr(c, name)[at, :, 1] = bad
        return run(c)

    o2, q2, k2, v2 = only("v")
    assert torch.equal(o2[:at], out[:at]) and torch.equal(q2[:at], dq[:at])
    # visible: the value itself in its column, in every row that sees it
    assert not torch.isfinite(o2[at:, :, 1].float()).any() and torch.equal(o2[at:, :, 2:], out[at:, :, 2:])
    if bad != bad or abs(bad) == float("inf"):
        w = o2[at, :, 1].float()
        assert (w.isnan() if bad != bad else w == bad).all()
    o2, q2, k2, v2 = only("k")
    assert torch.equal(o2[:at], out[:at]) and torch.equal(q2[:at], dq[:at])
    o2, q2, k2, v2 = only("q")
    assert torch.equal(o2[:at], out[:at]) and torch.equal(o2[at + 1:], out[at + 1:])
    assert torch.equal(k2[at + 1:], dk[at + 1:]) and torch.equal(v2[at + 1:], dv[at + 1:])
    o2, q2, k2, v2 = only("dout")
    assert torch.equal(k2[at + 1:], dk[at + 1:]) and torch.equal(v2[at + 1:], dv[at + 1:])
    assert torch.equal(q2[:at], dq[:at]) and torch.equal(q2[at + 1:], dq[at + 1:])
    assert not torch.isfinite(v2[:at + 1, :, 1].float()).any() and torch.equal(v2[:, :, 2:], dv[:, :, 2:])


def test_lowest_values_as_a_mask():
    # keys set to the type's lowest value take no part where others are seen
    for dtype in DTYPES:
        c = Case([70], None, 1, 1, 16, dtype, seed=22)
        c.q[:, :, 0] = 1.0
        c.k[10:30] = 0.0
        c.k[10:30, :, 0] = torch.finfo(dtype).min
        out = run(c)[0]
        d = Case([70], [50], 1, 1, 16, dtype, seed=22)
        rest = torch.cat([torch.arange(10), torch.arange(30, 70)])
        d.q, d.k, d.v = c.q.clone(), c.k[rest].clone(), c.v[rest].clone()
        r = d.ref(False)
        e = c.ref(False)
        assert (np.abs(f64(out) - r["out"]) <= r["e_out"] + torch.finfo(dtype).eps * (1e-30 + np.abs(r["out"]) + r["e_out"])).all()
        assert np.allclose(e["out"], r["out"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lq,lk,H", [([70, 1], [300, 400], 1), ([600] * 16, None, 8), ([2], [3000], 2)])
def test_first_keys_hidden(lq, lk, H, dtype):
    """The first tiles of a walk hold no key that is there, and the scores after
    them are far below 0: what a walk has summed up so far is nothing, not a
    maximum of 0."""
    for causal in (False, True):
        c = Case(lq, lk, H, H, 16, dtype, seed=26, causal=causal, ordered=True, scale=1.0)
        c.q[:, :, 0], c.k[:, :, 0] = 16.0, -16.0
        order = (c.order if lk is None else c.kv_order).clone()
        for a, b in zip(c.kv_ptr, c.kv_ptr[1:]):
            order[a:min(b, a + 200)] = -1
        c.kv_order = order
        if lk is None:
            c.order = order
        check(c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("n,lq,H", [(1, 64, 1), (16, 256, 8)])
def test_rows_without_keys_next_to_growing_scores(n, lq, H, D, dtype):
    """Rows that see no key walk the tiles together with rows whose scores grow
    from one tile to the next by more than an exponent holds."""
    c = Case([lq] * n, [lq + 246] * n, H, H, D, dtype, seed=29, causal=True, ordered=True, scale=1.0)
    c.q[:, :, 0], c.k[:, :, 0] = 16.0, -16.0
    for a, b in zip(c.kv_ptr, c.kv_ptr[1:]):
        c.k[c.kv_order[a + 256:b].long(), :, 0] = 16.0
        c.kv_order[a:a + 252] = -1         # rows 0 to 5 see none of the others, row 6 sees key 252
    check(c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_rows_next_to_nan(D, causal, dtype):
    """A query of NaN is NaN; those next to it, whose scores grow along the keys, are not touched."""
    c = Case([70], [500], 2, 2, D, dtype, seed=30, causal=causal, scale=1.0)
    c.q[:, :, 0], c.k[:, :, 0], c.k[130:, :, 0] = 16.0, -16.0, 16.0
    ref = c.ref(False)
    q, k, v, _ = c.on_gpu()
    q = q.clone()
    q[5] = float("nan")
    out, _ = spc.attention_fwd(q, k, v, **c.kw())
    rows = np.arange(70) != 5
    assert out[5].isnan().all()
    within(f64(out)[rows], ref["out"][rows], ref["e_out"][rows], dtype, "out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,H", [(300, 1), (3000, 1), (9000, 8)])
def test_scores_of_minus_infinity(n, H, dtype):
    """Keys whose scores are minus infinity count for nothing, in the first
    tiles of a walk and in whole parts of a split one; rows with no other score
    are NaN."""
    D = 32 if dtype == torch.float32 else 48       # narrow 16-bit heads give NaN
    q = torch.ones(3, H, D, dtype=dtype)
    g = torch.Generator().manual_seed(27)
    k, v = (torch.randn(n, H, D, generator=g).to(dtype) for _ in range(2))
    k[:n - 50, :, 0] = float("-inf")
    out, stats = spc.attention_fwd(cuda(q), cuda(k), cuda(v), scale=0.25, want_stats=True)
    r = A.attention(q, k[n - 50:], v[n - 50:], [0, 3], [0, 50], 0.25, step=half_step(dtype) if dtype != torch.float32 else 0.0,
                    floor=FLOOR[dtype])
    within(f64(out), r["out"], r["e_out"], dtype, "out")
    assert stats[0].isfinite().all()
    out, stats = spc.attention_fwd(cuda(q), cuda(k[:n - 50]), cuda(v[:n - 50]), scale=0.25, want_stats=True)
    assert out.isnan().all() and stats[0][..., 1].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1e-3, 0.9, 3.0])
def test_scales(scale, dtype):
    # above c = scale log2(e) = 1, 60,000 c is no number of fp16
    c = Case([70, 9], None, 2, 1, 16, dtype, seed=28, scale=scale)
    check(c)
    if dtype == torch.float16 and scale > 1:
        c.q[3], c.k[3] = 60000.0, 0.0
        check(c, bwd=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides(dtype):
    """Rows of wider tensors for every argument, gradients into one tensor."""
    c = Case([30, 50], None, 4, 2, 32, dtype, seed=23, causal=True)
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), want_stats=True, **c.kw())
    grads = spc.attention_bwd(dout, q.contiguous(), k.contiguous(), v.contiguous(), out, stats, **c.kw())
    wide = torch.full((c.n, 13, 32), 5.0, dtype=dtype, device="cuda")
    o2, s2 = spc.attention_fwd(q, k, v, want_stats=True, out=wide[:, 1:5], **c.kw())
    assert torch.equal(o2, out) and all(a is b is None or torch.equal(a, b) for a, b in zip(s2, stats)) and (wide[:, 0] == 5).all() and (wide[:, 5:] == 5).all()
    g = torch.full((c.n, 9, 32), 7.0, dtype=dtype, device="cuda")
    d = torch.empty((c.n, 6, 32), dtype=dtype, device="cuda")
    d[:, 2:] = dout
    got = spc.attention_bwd(d[:, 2:], q, k, v, wide[:, 1:5], s2, dq=g[:, :4], dk=g[:, 4:6], dv=g[:, 6:8], **c.kw())
    assert all(torch.equal(a, b) for a, b in zip(got, grads)) and (g[:, 8] == 7).all()


@pytest.mark.parametrize("lq,lk,H,Hk", [([4], [3000], 2, 1), ([3000], [4], 2, 1), ([500, 900], None, 1, 1), ([600] * 16, None, 8, 8)])
def test_workspace_and_repeats(lq, lk, H, Hk):
    c = Case(lq, lk, H, Hk, 32, torch.bfloat16, seed=24)
    q, k, v, dout = c.on_gpu()
    kw, runs = c.kw(), []
    need = B.attention_workspace(torch.bfloat16, c.n, c.m, len(lq), H, Hk, 32)
    for byte in (0, 255, 127):
        bufs = [torch.full((n + 4096,), byte, dtype=torch.uint8, device="cuda") for n in need]
        out, stats = spc.attention_fwd(q, k, v, want_stats=True, workspace=bufs[0][:max(need[0], 1)], **kw)
        runs.append((out,) + stats + spc.attention_bwd(dout, q, k, v, out, stats, workspace=bufs[1][:need[1]], **kw))
        for b, n in zip(bufs, need):
            assert (b[n:] == byte).all()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_gradients_against_differences():
    c = Case([6, 3], [4, 5], 2, 1, 16, torch.float32, seed=25, causal=True)
    q, k, v, dout = c.on_gpu()
    out, stats = spc.attention_fwd(q, k, v, want_stats=True, **c.kw())
    got = spc.attention_bwd(dout, q, k, v, out, stats, **c.kw())
    base = [f64(t).copy() for t in (c.q, c.k, c.v)]
    f = lambda: (A.attention(*base, c.q_ptr, c.kv_ptr, c.scale, True)["out"] * f64(c.dout)).sum()
    r = np.random.default_rng(1)
    for t, g in zip(base, got):
        for _ in range(25):
            i = tuple(r.integers(0, s) for s in t.shape)
            s, d = t[i], []
            for e in (1e-5, -1e-5):
                t[i] = s + e
                d.append(f())
            t[i] = s
            assert abs((d[0] - d[1]) / 2e-5 - f64(g)[i]) < 2e-5


def test_refusals_of_the_binding():
    q = torch.zeros(8, 4, 32, device="cuda")
    k = torch.zeros(9, 2, 32, device="cuda")
    ptr = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    o8, o9 = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (8, 9))
    bad = [
        lambda: spc.attention_fwd(q, k, k, ptr),                                   # 8 queries, 9 keys, one layout
        lambda: spc.attention_fwd(q, k, k, order=o8),
        lambda: spc.attention_fwd(q, k, k, ptr, kv_order=o9),
        lambda: spc.attention_fwd(q, k, k, ptr, kv_ptr=torch.tensor([0, 1, 9], dtype=torch.int32, device="cuda")),
        lambda: spc.attention_fwd(q, k, k, kv_order=o8),
        lambda: spc.attention_fwd(q, k, k[:, :1]),
        lambda: spc.attention_fwd(q, k[:, :, :16], k),
        lambda: spc.attention_fwd(q.transpose(0, 1), k, k),
        lambda: spc.attention_fwd(q[:, ::2], k, k),
        lambda: spc.attention_fwd(q[:, :, 0], k, k),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        spc.attention_fwd(q, k.half(), k)
    with pytest.raises(TypeError):
        spc.attention_fwd(q, k, k, ptr.long())
    with pytest.raises(TypeError):
        spc.attention_bwd(q, q, k, k, q, spc.attention_fwd(q, k, k)[1])             # a forward without stats
    for kw in (dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(spc.SpcError):
            spc.attention_fwd(q, k, k, **kw)
    with pytest.raises(spc.SpcError):
        spc.attention_fwd(q[:, :3], k, k)                                          # 3 heads over 2
    with pytest.raises(spc.SpcError):
        spc.attention_fwd(q[:, :, :24], k[:, :, :24], k[:, :, :24]) if False else spc.attention_fwd(
            torch.zeros(8, 4, 24, device="cuda"), torch.zeros(9, 2, 24, device="cuda"), torch.zeros(9, 2, 24, device="cuda"))
