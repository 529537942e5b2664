"""The attention block of examples/attention_block.py (layer norms, convolutions,
rotary positions, windowed attention, residual) against the composition of the
oracles, captured as a graph, and on streams of its own."""

import numpy as np
import pytest
import torch

import sparse_convolution_hash_amd as spc
from examples import attention_block as AB
from oracle import attnops as A
from oracle import conv as OC
from oracle import kmap as OK
from oracle.rowops import f64
from tests.parity import assert_close, cuda

pytestmark = pytest.mark.gpu

N, BATCH, SIDE, C, H, HK, W = 500, 2, 16, 64, 4, 2, 96


def setup(dtype, n=N, window=W):
    coords = AB.voxels(n, BATCH, SIDE, 5)
    block = AB.AttentionBlock(C, H, HK, dtype, seed=3)
    maps = block.maps(coords, BATCH, (SIDE,) * 3, window)
    g = torch.Generator().manual_seed(6)
    x, dout = (torch.randn(coords.shape[0], C, generator=g).to(dtype) for _ in range(2))
    return coords, block, maps, x, dout


def test_block_against_the_oracles():
    coords, block, maps, x, dout = setup(torch.float32)
    print(f"attention block n={coords.shape[0]}", flush=True)
    out, saved = block.forward(cuda(x), maps)
    dx, grads = block.backward(cuda(dout), saved, maps)

    n, D = coords.shape[0], C // H
    w = {k: v.cpu() for k, v in block.params.items()}
    nbr, ident = OK.subm_kmap(coords, (SIDE,) * 3, 3), np.arange(n, dtype=np.int32)[None]
    ptr, order = maps[2].cpu().tolist(), maps[3].cpu().numpy()
    assert ptr[-1] == n and max(np.diff(ptr)) == W
    t = torch.from_numpy
    freq, pos = block.freq.cpu(), coords[:, 1:]
    y, _, _, _ = A.layer_norm_fwd(x, w["g1"], w["b1"], 1e-5)
    qkv = np.asarray(OC.conv_fwd(t(y), w["wqkv"], None, ident)).reshape(n, H + 2 * HK, D)
    qk, _ = A.rotary(qkv[:, :H + HK], pos, freq, block.pairs)
    q, k, v = qk[:, :H], qk[:, H:], qkv[:, H + HK:]
    a = A.attention(q, k, v, ptr, ptr, D ** -0.5, False, order, order)
    o = a["out"].reshape(n, C)
    tot = f64(x) + np.asarray(OC.conv_fwd(t(o), w["wo"], None, ident))
    z, _, _, _ = A.layer_norm_fwd(tot, w["g2"], w["b2"], 1e-5)
    assert_close(out.cpu(), tot + np.asarray(OC.conv_fwd(t(z), w["w3"], None, nbr)), 1e-4, "out")

    assert_close(grads["w3"].cpu(), OC.conv_bwd_filter(t(z), dout, nbr), 1e-4, "dw3")
    dz = np.asarray(OC.conv_bwd_input(dout, w["w3"], nbr, n))
    dt, dg, db, _, _, _ = A.layer_norm_bwd(dz, tot, w["g2"], 1e-5, dtotal=dout)
    assert_close(grads["g2"].cpu(), dg, 1e-4, "dg2")
    assert_close(grads["b2"].cpu(), db, 1e-4, "db2")
    assert_close(grads["wo"].cpu(), OC.conv_bwd_filter(t(o), t(dt), ident), 1e-4, "dwo")
    do = np.asarray(OC.conv_bwd_input(t(dt), w["wo"], ident, n)).reshape(n, H, D)
    a = A.attention(q, k, v, ptr, ptr, D ** -0.5, False, order, order, dout=do)
    dqk, _ = A.rotary(np.concatenate([a["dq"], a["dk"]], 1), pos, freq, block.pairs, True)
    dqkv = np.concatenate([dqk, a["dv"]], 1).reshape(n, -1)
    assert_close(grads["wqkv"].cpu(), OC.conv_bwd_filter(t(y), t(dqkv), ident), 1e-4, "dwqkv")
    dy = np.asarray(OC.conv_bwd_input(t(dqkv), w["wqkv"], ident, n))
    rx, dg, db, _, _, _ = A.layer_norm_bwd(dy, x, w["g1"], 1e-5, dtotal=t(dt))
    assert_close(grads["g1"].cpu(), dg, 1e-4, "dg1")
    assert_close(grads["b1"].cpu(), db, 1e-4, "db1")
    assert_close(dx.cpu(), rx, 1e-4, "dx")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,window", [(40, 32), (500, 96), (2000, 4096)])
def test_block_captured(dtype, n, window):
    """Forward and backward of the block as one graph, with windows small and as
    long as a sample (split and joined): every replay equals the eager calls on
    the same inputs, which move between replays."""
    coords, block, maps, x, dout = setup(dtype, n, window)
    x, dout = cuda(x), cuda(dout)

    def step():
        out, saved = block.forward(x, maps)
        dx, grads = block.backward(dout, saved, maps)
        return [out, dx] + [grads[k] for k in sorted(grads)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    print(f"capture n={coords.shape[0]} {window} {dtype}", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(rep)))
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
    sets = [setup(torch.bfloat16, n, w) for n, w in ((500, 4096), (900, 128))]

    def step(coords, block, maps, x, dout):
        out, saved = block.forward(x, maps)
        dx, grads = block.backward(dout, saved, maps)
        return [out, dx] + [grads[k] for k in sorted(grads)]

    sets = [s[:3] + (cuda(s[3]), cuda(s[4])) for s in sets]
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


def test_block_runs_and_pools():
    coords, block, maps, x, _ = setup(torch.bfloat16)
    target = torch.randn(x.shape, generator=torch.Generator().manual_seed(8))
    for _ in range(3):
        assert np.isfinite(block.train_step(cuda(x), cuda(target), maps, 1.0).item())
    rows = block.forward(cuda(x), maps)[0].view(-1, H, C // H)
    ptr = cuda(torch.tensor([0, N, 2 * N], dtype=torch.int32))
    ones = cuda(torch.tensor([0, 1, 2], dtype=torch.int32))
    q = torch.randn(BATCH, H, C // H, generator=torch.Generator().manual_seed(9)).bfloat16()
    pooled, _ = spc.attention_fwd(cuda(q), rows, rows, ones, kv_ptr=ptr)
    ref = A.attention(q, rows.cpu(), rows.cpu(), [0, 1, 2], [0, N, 2 * N], (C // H) ** -0.5)["out"]
    assert_close(pooled.cpu(), ref, 1e-2, "pooled")
