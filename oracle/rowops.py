"""Row operators in fp64 on the CPU: group norm with activation, the dropout
generator and mask, and the gated linear recurrence, each with its backward
from the formulas.  Test infrastructure only.

Every function also returns (or offers) an error envelope: a bound on what an
fp32 computation of the same formula may be off by, from counting its
roundings (``EPS`` is half a unit in the last place of fp32).
"""

import numpy as np

EPS = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


# ---------------------------------------------------------------- dropout

def philox4x32(counter, key):
    """Philox4x32-10 of 32-bit word arrays: counter (4), key (2) -> 4 words."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & lo, (p0 >> sh) ^ c[3] ^ np.uint64(k[1]), p0 & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def keep_mask(seed, offset, layer, p, numel):
    """Whether each of numel elements stays."""
    ctr = (np.arange((numel + 7) // 8, dtype=np.uint64) + np.uint64(offset % (1 << 64)))
    w = philox4x32((ctr & np.uint64(0xFFFFFFFF), ctr >> np.uint64(32), np.full_like(ctr, layer), np.zeros_like(ctr)),
                   (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    half = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=-1)
    return half.reshape(-1)[:numel] >= threshold(p)


def drop_factor(seed, offset, layer, p, shape):
    """0 for dropped elements, the scale for kept ones."""
    thr = threshold(p)
    scale = 65536.0 / (65536 - thr) if thr < 65536 else 0.0
    return keep_mask(seed, offset, layer, p, int(np.prod(shape))).reshape(shape) * scale


# -------------------------------------------------------------- group norm

def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0) * 1.0
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def _norm(x, groups, ptr, eps):
    n, C = x.shape
    S, cg = len(ptr) - 1, C // groups
    xhat, rstd, mean = np.zeros_like(x), np.zeros((S, groups)), np.zeros((S, groups))
    for s in range(S):
        v = x[ptr[s]:ptr[s + 1]].reshape(-1, groups, cg)
        if v.shape[0] == 0:
            rstd[s] = eps ** -0.5
            continue
        mean[s] = v.mean((0, 2))
        rstd[s] = (v.var((0, 2)) + eps) ** -0.5
        xhat[ptr[s]:ptr[s + 1]] = ((v - mean[s][None, :, None]) * rstd[s][None, :, None]).reshape(-1, C)
    return xhat, mean, rstd


def group_norm_fwd(x, groups, ptr, gamma, beta, eps, name, factor=1.0):
    """(y, mean [S, G], rstd [S, G])."""
    xhat, mean, rstd = _norm(f64(x), groups, ptr, eps)
    return act(xhat * f64(gamma) + f64(beta), name) * factor, mean, rstd


def group_norm_bwd(dy, x, groups, ptr, gamma, beta, eps, name, factor=1.0):
    """(dx, dgamma, dbeta)."""
    x, gamma, beta = f64(x), f64(gamma), f64(beta)
    n, C = x.shape
    cg = C // groups
    xhat, _, rstd = _norm(x, groups, ptr, eps)
    dz = f64(dy) * factor * act_slope(xhat * gamma + beta, name)
    inside = np.zeros((n, 1))
    inside[ptr[0]:ptr[-1]] = 1.0
    dz = dz * inside
    w, dx = dz * gamma, np.zeros_like(x)
    for s in range(len(ptr) - 1):
        a, b = ptr[s], ptr[s + 1]
        if a == b:
            continue
        v, h = w[a:b].reshape(-1, groups, cg), xhat[a:b].reshape(-1, groups, cg)
        d = v - v.mean((0, 2))[None, :, None] - h * (v * h).mean((0, 2))[None, :, None]
        dx[a:b] = (d * rstd[s][None, :, None]).reshape(-1, C)
    return dx, (dz * xhat).sum(0), dz.sum(0)


# -------------------------------------------------- gated linear recurrence

def _rows(ptr, s, order, reverse, n):
    q = range(ptr[s], ptr[s + 1])
    q = list(q)[::-1] if reverse else list(q)
    rows = q if order is None else [int(order[i]) for i in q]
    return [r for r in rows if 0 <= r < n]


def recurrence_fwd(gate, x, ptr, h0=None, order=None, reverse=False, roundings=8):
    """(out, h_last, before, envelope of out, envelope of h_last): before is
    the state ahead of each row, the envelope what `roundings` fp32 roundings of
    |h| + |x| per step add up to through the same recurrence."""
    g, x = f64(gate), f64(x)
    n, C = x.shape
    a, na = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    S = len(ptr) - 1
    h_last = np.zeros((S, C)) if h0 is None else f64(h0).copy()
    e_last = np.zeros((S, C))
    out, before, env = np.zeros((n, C)), np.zeros((n, C)), np.zeros((n, C))
    for s in range(S):
        h, e = h_last[s].copy(), np.zeros(C)
        for r in _rows(ptr, s, order, reverse, n):
            before[r] = h
            e = a[r] * e + roundings * EPS * (np.abs(h) + np.abs(x[r]))
            h = a[r] * h + na[r] * x[r]
            out[r], env[r] = h, e
        h_last[s], e_last[s] = h, e
    return out, h_last, before, env, e_last


def recurrence_bwd(dh, gate, x, ptr, h0=None, dh_last=None, order=None, reverse=False, roundings=8):
    """(dgate, dx, dh0) and an envelope of each."""
    g, x, dh = f64(gate), f64(x), f64(dh)
    n, C = x.shape
    a, na = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    _, _, before, henv, _ = recurrence_fwd(gate, x, ptr, h0, order, reverse, roundings)
    S = len(ptr) - 1
    dh0 = np.zeros((S, C)) if dh_last is None else f64(dh_last).copy()
    e0 = np.zeros((S, C))
    dg, dx, eg, ex = (np.zeros((n, C)) for _ in range(4))
    for s in range(S):
        d, e = dh0[s].copy(), np.zeros(C)
        prev_env = None
        rows = _rows(ptr, s, order, reverse, n)
        for i in range(len(rows) - 1, -1, -1):
            r = rows[i]
            d = d + dh[r]
            e = e + roundings * EPS * (np.abs(d) + np.abs(dh[r]))
            hp = henv[rows[i - 1]] if i else 0.0
            dx[r], ex[r] = na[r] * d, na[r] * (e + roundings * EPS * np.abs(d))
            dg[r] = a[r] * na[r] * (before[r] - x[r]) * d
            m = np.abs(before[r]) + np.abs(x[r])
            eg[r] = a[r] * na[r] * (np.abs(before[r] - x[r]) * e + np.abs(d) * (hp + roundings * EPS * m))
            d, e = a[r] * d, a[r] * e + roundings * EPS * np.abs(a[r] * d)
        dh0[s], e0[s] = d, e
    return dg, dx, dh0, eg, ex, e0
