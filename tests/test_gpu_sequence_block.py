"""The sequence block of examples/sequence_block.py (convolutions, group norm,
dropout, recurrence, residual) against the composition of the oracles, captured
as a graph, and on a stream of its own."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from examples import sequence_block as SB
from oracle import conv as OC
from oracle import kmap as OK
from oracle import rowops as R
from tests.parity import assert_close, cuda

pytestmark = pytest.mark.gpu

N, BATCH, SIDE, C, G, P = 700, 3, 16, 32, 4, 0.2


def setup(dtype, n=N):
    coords = SB.voxels(n, BATCH, SIDE, 5)
    block = SB.SequenceBlock(C, G, P, dtype, seed=3)
    km, ptr, curve = block.maps(coords, BATCH, (SIDE,) * 3)
    g = torch.Generator().manual_seed(6)
    x, dout = (torch.randn(coords.shape[0], C, generator=g).to(dtype) for _ in range(2))
    return coords, block, km, ptr, curve, x, dout


def test_block_against_the_oracles():
    coords, block, km, ptr, curve, x, dout = setup(torch.float32)
    print(f"sequence block n={coords.shape[0]}", flush=True)
    out, last, saved = block.forward(cuda(x), km, ptr, curve)
    dx, grads = block.backward(cuda(dout), saved, km, ptr, curve)

    n, q = coords.shape[0], [i * N for i in range(BATCH + 1)]
    w = {k: v.cpu() for k, v in block.params.items()}
    nbr = OK.subm_kmap(coords, (SIDE,) * 3, 3)
    ident = np.arange(n, dtype=np.int32)[None]
    order = curve.cpu().numpy()
    assert all((np.sort(order[a:b]) == np.arange(a, b)).all() for a, b in zip(q, q[1:]))
    f0, f1 = (R.drop_factor(4, 0, k, P, (n, C)) for k in (0, 1))
    c = torch.from_numpy(np.asarray(OC.conv_fwd(x, w["w"], None, nbr)))
    y, _, _ = R.group_norm_fwd(c, G, q, w["gamma"], w["beta"], 1e-5, "silu", f0)
    gv = np.asarray(OC.conv_fwd(torch.from_numpy(y), w["w1"], w["b1"], ident))
    h, rl, _, _, _ = R.recurrence_fwd(gv[:, :C], gv[:, C:], q, None, order)
    assert_close(out.cpu(), h * f1 + R.f64(x), 1e-4, "out")
    assert_close(last.cpu(), rl, 1e-4, "last")
    dg, dv, _, _, _, _ = R.recurrence_bwd(R.f64(dout) * f1, gv[:, :C], gv[:, C:], q, None, None, order)
    dgv = np.concatenate([dg, dv], 1)
    t = torch.from_numpy
    assert_close(grads["w1"].cpu(), OC.conv_bwd_filter(t(y), t(dgv), ident), 1e-4, "dw1")
    assert_close(grads["b1"].cpu(), dgv.sum(0), 1e-4, "db1")
    dy = np.asarray(OC.conv_bwd_input(t(dgv), w["w1"], ident, n))
    dc, dgamma, dbeta = R.group_norm_bwd(dy, c, G, q, w["gamma"], w["beta"], 1e-5, "silu", f0)
    assert_close(grads["gamma"].cpu(), dgamma, 1e-4, "dgamma")
    assert_close(grads["beta"].cpu(), dbeta, 1e-4, "dbeta")
    assert_close(grads["w"].cpu(), OC.conv_bwd_filter(x, t(dc), nbr), 1e-4, "dw")
    assert_close(dx.cpu(), np.asarray(OC.conv_bwd_input(t(dc), w["w"], nbr, n)) + R.f64(dout), 1e-4, "dx")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [40, 700])
def test_block_captured(dtype, n):
    """Forward and backward of the block as one graph: every replay equals the
    eager calls with the same dropout words, which move between replays, with
    eager work in between."""
    coords, block, km, ptr, curve, x, dout = setup(dtype, n)
    x, dout = cuda(x), cuda(dout)

    def step():
        out, last, saved = block.forward(x, km, ptr, curve)
        dx, grads = block.backward(dout, saved, km, ptr, curve)
        return [out, last, dx] + [grads[k] for k in sorted(grads)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    print(f"capture n={coords.shape[0]} {dtype}", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(4):
        block.rng[1] = 1000 * rep
        for o in outs:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        eager = step()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, eager)):
            assert torch.equal(a, b), f"replay {rep}: output {k} differs from the eager step"


def test_block_on_two_streams_at_once():
    """Two blocks' steps side by side on streams of their own give what each gives alone."""
    sets = [setup(torch.bfloat16, n) for n in (500, 900)]

    def step(coords, block, km, ptr, curve, x, dout):
        out, last, saved = block.forward(x, km, ptr, curve)
        dx, grads = block.backward(dout, saved, km, ptr, curve)
        return [out, last, dx, grads["w"], grads["gamma"], grads["b1"]]

    sets = [s[:5] + (cuda(s[5]), cuda(s[6])) for s in sets]
    alone = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for rep in range(3):
        both = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                both.append(step(*s))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(u, v) for u, v in zip(a, b)), f"repetition {rep}"


def test_block_trains():
    coords, block, km, ptr, curve, x, _ = setup(torch.bfloat16)
    target = torch.randn(x.shape, generator=torch.Generator().manual_seed(8))
    losses = [block.train_step(cuda(x), cuda(target), km, ptr, curve, 10.0).item() for _ in range(30)]
    assert losses[-1] < losses[0] and np.isfinite(losses).all()
    # the state after the rows goes on one row at a time
    _, state, _ = block.forward(cuda(x), km, ptr, curve)
    before = state.clone()
    row = torch.zeros(BATCH, 2 * C, dtype=torch.bfloat16, device="cuda")
    out = spc.linear_recurrence_step(row[:, :C], row[:, C:], state)
    assert torch.equal(state, before * 0.5) and out.dtype == torch.bfloat16
