"""Shared inputs and bounds of the row operators' tests."""

import numpy as np
import torch

from oracle import rowops as R

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def half_step(dtype):
    """A rounding to dtype is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Below the smallest normal number a rounding is off by half of this."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def within(got, ref, env, dtype, what):
    """|got - ref| <= env + the rounding of ref (+ env) to dtype."""
    g, ref = R.f64(got), np.asarray(ref)
    bound = env + half_step(dtype) * (np.abs(ref) + env) + tiny(dtype)
    err = np.abs(g - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(v[0] for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {g[i]!r} ref {ref[i]!r} "
                             f"bound {np.broadcast_to(bound, g.shape)[i]:.3g}")


def ptr_of(lengths):
    return [0] + np.cumsum(lengths).tolist()


def ragged(seed, n, s):
    """s lengths that sum to n, zeros and ones among them."""
    r = np.random.default_rng(seed)
    cut = np.sort(r.integers(0, n + 1, size=s - 1)) if s > 1 else np.zeros(0, int)
    if s > 3 and n > 1:
        cut[1] = cut[0]
        cut[2:] = np.maximum(cut[2:], cut[0])
        cut[2] = min(cut[1] + 1, n)
        cut = np.sort(cut)
    return np.diff(np.concatenate([[0], cut, [n]])).tolist()
