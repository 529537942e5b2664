"""A block of windowed attention on voxels: every sample's rows are walked along
a space-filling curve and attend to the rows of their window, with the voxels'
(z, y, x) as rotary positions, between a layer norm and a residual join.

    y             = layer_norm(x)
    [q, k, v]     = conv1(y)                      one product for all three
    q, k          = rotated by (z, y, x)
    o             = attention within windows of the curve
    t, z          = x + conv1(o), layer_norm of it     one call
    out           = t + conv3(z)                  submanifold, 3 x 3 x 3

    python -m examples.attention_block [--sites N] [--channels C] [--window W] [--steps K]

trains it for a few steps on random voxels towards a random target, eagerly and
as one captured graph, then pools every sample by one query per head.
"""

import argparse

import numpy as np
import torch

import sparse_convolution_hash_amd as spc

from .sequence_block import morton_order, voxels


class AttentionBlock:
    """Parameters, and the forward and backward calls of the block above.  Key
    and value heads may be fewer than query heads."""

    def __init__(self, channels: int, heads: int, kv_heads: int, dtype: torch.dtype, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        C = channels
        self.C, self.H, self.Hk, self.D, self.dtype = C, heads, kv_heads, C // heads, dtype
        kv = kv_heads * self.D
        r = lambda *s, std: torch.randn(*s, generator=g) * std
        self.params = {
            "g1": torch.ones(C), "b1": torch.zeros(C), "wqkv": r(1, C, C + 2 * kv, std=C ** -0.5),
            "wo": r(1, C, C, std=C ** -0.5), "g2": torch.ones(C), "b2": torch.zeros(C),
            "w3": r(27, C, C, std=(27 * C) ** -0.5),
        }
        self.params = {k: v.to(device) for k, v in self.params.items()}
        # the head's pairs, shared out over the three axes
        P = self.D // 2
        self.pairs = [P * (a + 1) // 3 - P * a // 3 for a in range(3)]
        self.freq = torch.tensor([100.0 ** (-j / m) for m in self.pairs for j in range(m)], dtype=torch.float32).to(device)

    def maps(self, coords: np.ndarray, batch: int, shape, window: int):
        """What a set of voxels needs once: its coordinates on the GPU, kernel
        map, windows of the curve as row offsets, and the curve."""
        dev = self.freq.device
        c = torch.from_numpy(coords).to(dev)
        ptr = np.searchsorted(coords[:, 0], np.arange(batch + 1))
        cuts = np.concatenate([np.arange(a, b, window) for a, b in zip(ptr[:-1], ptr[1:])] + [[ptr[-1]]])
        return (c, spc.build_kmap(c, batch, shape, 3, orders=True), torch.from_numpy(cuts.astype(np.int32)).to(dev),
                torch.from_numpy(morton_order(coords)).to(dev))

    def heads_of(self, qkv):
        n, H, Hk, D = qkv.shape[0], self.H, self.Hk, self.D
        h = qkv.view(n, H + 2 * Hk, D)
        return h[:, :H + Hk], h[:, :H], h[:, H:H + Hk], h[:, H + Hk:]

    def forward(self, x, maps):
        P, dt = self.params, self.dtype
        coords, km, windows, curve = maps
        y, s1, _ = spc.layer_norm_fwd(x, P["g1"], P["b1"])
        qkv = spc.subm_conv_fwd(y, P["wqkv"].to(dt), None, None, None)
        qk, q, k, v = self.heads_of(qkv)
        spc.rotary(qk, coords[:, 1:], self.freq, self.pairs, out=qk)
        o, st = spc.attention_fwd(q, k, v, windows, curve, want_stats=True)
        a = spc.subm_conv_fwd(o.view(-1, self.C), P["wo"].to(dt), None, None, None)
        z, s2, t = spc.layer_norm_fwd(a, P["g2"], P["b2"], residual=x)
        out = spc.conv_fwd_fused(z, P["w3"].to(dt), None, km["nbr"], z.shape[0], km["order"], residual=t)
        return out, (x, y, s1, qkv, o, st, z, s2, t)

    def backward(self, dout, saved, maps):
        """Gradients of x and of every parameter."""
        x, y, s1, qkv, o, st, z, s2, t = saved
        P, dt, n = self.params, self.dtype, x.shape[0]
        coords, km, windows, curve = maps
        dw3, _ = spc.conv_bwd_filter(z, dout, 27, km["pair_ptr"], km["pair_in"], km["pair_out"])
        dz = spc.conv_bwd_input(dout, P["w3"].to(dt), km["nbr"], True, n, km["order"])
        dt_, dg2, db2 = spc.layer_norm_bwd(dz, t, P["g2"], s2, dtotal=dout)
        dwo, _ = spc.conv_bwd_filter(o.view(n, -1), dt_, 1, None, None, None)
        do = spc.conv_bwd_input(dt_, P["wo"].to(dt), None, True, n).view_as(o)
        dqkv = torch.empty_like(qkv)
        (_, q, k, v), (dqk, dq, dk, dv) = self.heads_of(qkv), self.heads_of(dqkv)
        spc.attention_bwd(do, q, k, v, o, st, windows, curve, dq=dq, dk=dk, dv=dv)
        spc.rotary(dqk, coords[:, 1:], self.freq, self.pairs, inverse=True, out=dqk)
        dwqkv, _ = spc.conv_bwd_filter(y, dqkv, 1, None, None, None)
        dy = spc.conv_bwd_input(dqkv, P["wqkv"].to(dt), None, True, n)
        dx, dg1, db1 = spc.layer_norm_bwd(dy, x, P["g1"], s1, dtotal=dt_)
        return dx, {"g1": dg1, "b1": db1, "wqkv": dwqkv, "wo": dwo, "g2": dg2, "b2": db2, "w3": dw3}

    def train_step(self, x, target, maps, lr: float):
        """One step of gradient descent on mean (out - target)^2; returns the
        loss.  Nothing leaves the device, so the step can be captured."""
        out, saved = self.forward(x, maps)
        d = out.float() - target
        _, grads = self.backward((d * (2.0 / d.numel())).to(self.dtype), saved, maps)
        for k, v in self.params.items():
            v.sub_(grads[k], alpha=lr)
        return (d * d).mean()


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--sites", type=int, default=20000)
    a.add_argument("--channels", type=int, default=64)
    a.add_argument("--window", type=int, default=1024)
    a.add_argument("--steps", type=int, default=10)
    a = a.parse_args()
    side, batch, dt = 64, 2, torch.bfloat16
    coords = voxels(a.sites, batch, side, 0)
    block = AttentionBlock(a.channels, a.channels // 16, a.channels // 32, dt)
    maps = block.maps(coords, batch, (side,) * 3, a.window)
    g = torch.Generator().manual_seed(1)
    n = coords.shape[0]
    x = torch.randn(n, a.channels, generator=g).to("cuda", dt)
    target = torch.randn(n, a.channels, generator=g).to("cuda")
    step = lambda: block.train_step(x, target, maps, 10.0)

    def timed(f):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        for _ in range(a.steps):
            loss = f()
        e[1].record()
        torch.cuda.synchronize()
        return loss, e[0].elapsed_time(e[1]) / a.steps

    print(f"{n} voxels x {a.channels}, first loss {step().item():.5f}")
    side_stream = torch.cuda.Stream()
    side_stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side_stream):
        step()
    torch.cuda.current_stream().wait_stream(side_stream)
    loss, ms = timed(step)
    print(f"eager: {ms:.3f} ms a step, loss {loss.item():.5f}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    _, ms = timed(graph.replay)
    print(f"graph: {ms:.3f} ms a step, loss {loss.item():.5f}")

    # one query per head and sample pools all its rows
    out, _ = block.forward(x, maps)
    ptr = torch.from_numpy(np.searchsorted(coords[:, 0], np.arange(batch + 1)).astype(np.int32)).to("cuda")
    ones = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    query = torch.randn(batch, block.H, block.D, generator=g).to("cuda", dt)
    rows = out.view(n, block.H, block.D)
    pooled, _ = spc.attention_fwd(query, rows, rows, ones, kv_ptr=ptr)
    print("pooled:", pooled.float().norm().item())


if __name__ == "__main__":
    main()
