"""A residual sequence block on voxels: every sample's rows are walked along a
space-filling curve by a gated recurrence, between a submanifold convolution
and a residual join.

    c      = conv3(x)                                  submanifold, 3 x 3 x 3
    y      = dropout(silu(group_norm(c)))              one call
    [g, v] = conv1(y)                                  one product for gate and value
    h_t    = sigmoid(g_t) h_{t-1} + sigmoid(-g_t) v_t  along the curve
    out    = x + dropout(h)

    python -m examples.sequence_block [--sites N] [--channels C] [--steps K]

trains it for a few steps on random voxels towards a random target, eagerly and
as one captured graph, then feeds single rows to its recurrence.
"""

import argparse

import numpy as np
import torch

import sparse_convolution_hash_amd as spc


def morton_order(coords: np.ndarray) -> np.ndarray:
    """Rows of each sample along the Morton curve (coords int32 [N, 4], rows
    grouped by sample): the row numbers in the order of the walk."""
    z, y, x = (coords[:, i].astype(np.uint64) for i in (1, 2, 3))
    code = np.zeros(coords.shape[0], dtype=np.uint64)
    for b in range(16):
        one, b = np.uint64(1), np.uint64(b)
        for k, v in enumerate((x, y, z)):
            code |= ((v >> b) & one) << (np.uint64(3) * b + np.uint64(k))
    return np.lexsort((code, coords[:, 0])).astype(np.int32)


class SequenceBlock:
    """Parameters, and the forward and backward calls of the block above."""

    def __init__(self, channels: int, groups: int, p: float, dtype: torch.dtype, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        C = channels
        self.C, self.groups, self.p, self.dtype = C, groups, p, dtype
        self.params = {
            "w": torch.randn(27, C, C, generator=g) / (27 * C) ** 0.5,
            "gamma": torch.ones(C), "beta": torch.zeros(C),
            "w1": torch.randn(1, C, 2 * C, generator=g) / C ** 0.5,
            "b1": torch.cat([torch.full((C,), 1.0), torch.zeros(C)]),      # gates start half open
        }
        self.params = {k: v.to(device) for k, v in self.params.items()}
        self.rng = torch.tensor([seed + 1, 0], dtype=torch.int64, device=device)   # {seed, offset}

    def maps(self, coords: np.ndarray, batch: int, shape):
        """What a set of voxels needs once: its kernel map, sample offsets and curve."""
        dev = self.rng.device
        km = spc.build_kmap(torch.from_numpy(coords).to(dev), batch, shape, 3, orders=True)
        ptr = np.searchsorted(coords[:, 0], np.arange(batch + 1)).astype(np.int32)
        return km, torch.from_numpy(ptr).to(dev), torch.from_numpy(morton_order(coords)).to(dev)

    def forward(self, x, km, ptr, curve, h0=None):
        P, C = self.params, self.C
        c = spc.subm_conv_fwd(x, P["w"].to(self.dtype), None, km["nbr"], km["order"])
        y, stats = spc.group_norm_fwd(c, self.groups, ptr, P["gamma"], P["beta"], act="silu",
                                      dropout=spc.Dropout(self.rng, self.p, 0))
        gv = spc.subm_conv_fwd(y, P["w1"].to(self.dtype), P["b1"], None, None)
        h, last, carry = spc.linear_recurrence_fwd(gv[:, :C], gv[:, C:], ptr, h0, order=curve, want_carry=True)
        out = spc.dropout_fwd(h, spc.Dropout(self.rng, self.p, 1), residual=x)
        return out, last, (x, c, stats, y, gv, carry, h0)

    def backward(self, dout, saved, km, ptr, curve):
        """Gradients of x and of every parameter."""
        x, c, stats, y, gv, carry, h0 = saved
        P, C, n = self.params, self.C, x.shape[0]
        dh = spc.dropout_bwd(dout, spc.Dropout(self.rng, self.p, 1))
        dgv = torch.empty_like(gv)
        spc.linear_recurrence_bwd(dh, gv[:, :C], gv[:, C:], ptr, carry, h0, order=curve, dgate=dgv[:, :C], dx=dgv[:, C:])
        dw1, db1 = spc.conv_bwd_filter(y, dgv, 1, None, None, None, want_dbias=True)
        dy = spc.conv_bwd_input(dgv, P["w1"].to(self.dtype), None, True, n)
        dc, dgamma, dbeta = spc.group_norm_bwd(dy, c, self.groups, ptr, P["gamma"], P["beta"], stats, act="silu",
                                               dropout=spc.Dropout(self.rng, self.p, 0))
        dw, _ = spc.conv_bwd_filter(x, dc, 27, km["pair_ptr"], km["pair_in"], km["pair_out"])
        dx = spc.conv_bwd_input(dc, P["w"].to(self.dtype), km["nbr"], True, n, km["order"])
        return dx + dout, {"w": dw, "gamma": dgamma, "beta": dbeta, "w1": dw1, "b1": db1}

    def train_step(self, x, target, km, ptr, curve, lr: float):
        """One step of gradient descent on mean (out - target)^2; returns the
        loss.  Everything stays on the device, the dropout's offset included,
        so the step can be captured and every replay draws new masks."""
        out, _, saved = self.forward(x, km, ptr, curve)
        d = out.float() - target
        _, grads = self.backward((d * (2.0 / d.numel())).to(self.dtype), saved, km, ptr, curve)
        for k, v in self.params.items():
            v.sub_(grads[k], alpha=lr)
        self.rng[1] += (x.numel() + 7) // 8
        return (d * d).mean()


def voxels(sites: int, batch: int, side: int, seed: int) -> np.ndarray:
    """sites random cells of side^3 for each sample, rows grouped by sample."""
    r = np.random.default_rng(seed)
    rows = []
    for b in range(batch):
        lin = r.choice(side ** 3, size=sites, replace=False)
        rows.append(np.stack([np.full(sites, b), *np.unravel_index(lin, (side,) * 3)], axis=1))
    return np.ascontiguousarray(np.concatenate(rows), dtype=np.int32)


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--sites", type=int, default=20000)
    a.add_argument("--channels", type=int, default=64)
    a.add_argument("--steps", type=int, default=10)
    a = a.parse_args()
    side, batch, dt = 64, 2, torch.bfloat16
    coords = voxels(a.sites, batch, side, 0)
    block = SequenceBlock(a.channels, a.channels // 8, 0.1, dt)
    km, ptr, curve = block.maps(coords, batch, (side,) * 3)
    g = torch.Generator().manual_seed(1)
    n = coords.shape[0]
    x = torch.randn(n, a.channels, generator=g).to("cuda", dt)
    target = torch.randn(n, a.channels, generator=g).to("cuda")
    step = lambda: block.train_step(x, target, km, ptr, curve, 10.0)

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

    # the last states go on one row at a time
    _, state, _ = block.forward(x, km, ptr, curve)
    row = torch.randn(batch, 2 * a.channels, generator=g).to("cuda", dt)
    for _ in range(3):
        h = spc.linear_recurrence_step(row[:, :a.channels], row[:, a.channels:], state)
    print("after three more rows:", h.float().norm().item())


if __name__ == "__main__":
    main()
