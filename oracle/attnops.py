"""Attention-block operators in fp64 on the CPU: layer norm, rotary positions and
attention over ragged samples, each with its backward from the formulas.  Test
infrastructure only.

Next to each result stands a bound on what an fp32 computation of the same
formula, with the stated roundings to the storage type, may be off by, from
counting roundings (``EPS`` is half a unit in the last place of fp32; a sum of
n terms in any order is off by at most n EPS times the sum of their sizes).
"""

import numpy as np

from .rowops import EPS, f64

# ---------------------------------------------------------------- layer norm


def _norm(x, eps):
    mean = x.mean(1, keepdims=True)
    d = x - mean
    rstd = ((d * d).mean(1, keepdims=True) + eps) ** -0.5
    return d, d * rstd, rstd, mean


def _sums(C):
    """Roundings on the way of one term into a row's sum: 8 channels of a lane
    and step in a tree, its steps, the lanes, the division."""
    return 3 + -(-C // 512) + 6 + 2


def layer_norm_fwd(x, gamma, beta, eps):
    """(y, mean [N], rstd [N], envelope of y).  Differences are taken from a
    rounded mean, whose own error is taken out by their mean."""
    x, gamma, beta = f64(x), f64(gamma), f64(beta)
    d, h, rstd, mean = _norm(x, eps)
    n = _sums(x.shape[1])
    off = n * EPS * np.abs(x).mean(1, keepdims=True)                   # of the first mean
    size = np.abs(d).mean(1, keepdims=True) + off
    ed = 3 * EPS * (np.abs(d) + off) + (n + 2) * EPS * size            # of a difference, its mean taken out
    rel = (n + 8) * EPS + (n + 8) * EPS * off * off * rstd * rstd      # of rstd: half that of the variance, which loses md^2
    env = np.abs(gamma) * (rstd * ed + rel * np.abs(h)) + 4 * EPS * (np.abs(gamma * h) + np.abs(beta))
    return h * gamma + beta, mean[:, 0], rstd[:, 0], env


def layer_norm_bwd(dy, x, gamma, eps, dtotal=None):
    """(dx, dgamma, dbeta) and an envelope of each."""
    dy, x, gamma = f64(dy), f64(x), f64(gamma)
    d, h, rstd, mean = _norm(x, eps)
    w = dy * gamma
    m1, m2 = w.mean(1, keepdims=True), (w * h).mean(1, keepdims=True)
    dx = rstd * (w - m1 - h * m2)
    n = _sums(x.shape[1]) + 4
    off = 2 * EPS * np.abs(mean)                                       # of the mean as saved
    size = np.abs(d).mean(1, keepdims=True) + off
    eh = rstd * (3 * EPS * (np.abs(d) + off) + n * EPS * size) + n * EPS * np.abs(h)
    ew = np.abs(w).mean(1, keepdims=True)
    em2 = (n * EPS) * rstd * ((np.abs(w) * (np.abs(d) + off)).mean(1, keepdims=True) + size * ew) + n * EPS * np.abs(m2)
    env = rstd * (n * EPS * ew + 6 * EPS * (np.abs(w) + np.abs(m1) + np.abs(h * m2)) + eh * np.abs(m2) + np.abs(h) * em2)
    env = env + n * EPS * np.abs(dx)
    if dtotal is not None:
        dx = dx + f64(dtotal)
        env = env + EPS * np.abs(dx)
    eg = (np.abs(dy) * (eh + 20 * EPS * np.abs(h))).sum(0)             # 16 rows in fp32, then double, rounded once between
    return dx, (dy * h).sum(0), dy.sum(0), env, eg, 20 * EPS * np.abs(dy).sum(0)


# -------------------------------------------------------------------- rotary

def rotary(x, pos, freq, pairs, inverse=False):
    """(out, envelope): sines and cosines are off by up to 4 EPS each."""
    x, pos, freq = f64(x), f64(pos), f64(freq)
    out = x.copy()
    env = np.zeros_like(x)
    j = 0
    for a, m in enumerate(pairs):
        for _ in range(m):
            t = pos[:, a] * freq[j] * (-1.0 if inverse else 1.0)
            c, s = np.cos(t)[:, None], np.sin(t)[:, None]
            p, q = x[:, :, 2 * j], x[:, :, 2 * j + 1]
            out[:, :, 2 * j], out[:, :, 2 * j + 1] = p * c - q * s, p * s + q * c
            env[:, :, 2 * j] = env[:, :, 2 * j + 1] = 6 * EPS * (np.abs(p) + np.abs(q))
            j += 1
    return out, env


# ----------------------------------------------------------------- attention

def _rows(ptr, s, order, n):
    q = np.arange(ptr[s], ptr[s + 1])
    return q if order is None else np.asarray(order)[q]


def _samples(nq, nk, q_ptr, kv_ptr, q_order, kv_order, causal):
    """Of each sample: rows of the queries and keys that are there, and which
    pairs see each other.  A position without a row keeps its place."""
    for s in range(len(q_ptr) - 1):
        rq, rk = _rows(q_ptr, s, q_order, nq), _rows(kv_ptr, s, kv_order, nk)
        see = np.ones((len(rq), len(rk)), bool)
        if causal:
            see = np.arange(len(rk))[None, :] <= np.arange(len(rq))[:, None] + len(rk) - len(rq)
        okq, okk = (rq >= 0) & (rq < nq), (rk >= 0) & (rk < nk)
        yield rq[okq], rk[okk], see[okq][:, okk]


def attention(q, k, v, q_ptr, kv_ptr, scale, causal=False, q_order=None, kv_order=None, dout=None, step=0.0, floor=0.0,
              split=(0.0, 0.0)):
    """dict of out, (m + log l) and, with dout, dq, dk, dv, each with its
    envelope under "e_" + name, and "rows"/"keys": which rows are in a sample.
    step: the relative rounding of p and ds (0: none); floor: what p and ds are
    off by at least (their type's smallest numbers).  split: how far the factor
    scale log2(e) times an element of q or k, kept as two numbers of the type,
    may be off, relative and absolute."""
    q, k, v = f64(q), f64(k), f64(v)
    nq, H, D = q.shape
    nk, Hk, _ = k.shape
    r = {"out": np.zeros_like(q), "lse": np.full((H, nq), -np.inf), "e_out": np.zeros_like(q), "dq": np.zeros_like(q),
         "dk": np.zeros_like(k), "dv": np.zeros_like(v), "e_dq": np.zeros_like(q), "e_dk": np.zeros_like(k),
         "e_dv": np.zeros_like(v), "e_lse": np.zeros((H, nq)), "rows": np.zeros(nq, bool), "keys": np.zeros(nk, bool)}
    g = None if dout is None else f64(dout)
    for rq, rk, see in _samples(nq, nk, q_ptr, kv_ptr, q_order, kv_order, causal):
        r["rows"][rq] = True
        r["keys"][rk] = True
        if not len(rq) or not len(rk):
            continue
        L = len(rk)
        for h in range(H):
            kh = h // (H // Hk)
            Q, K, V = q[rq, h], k[rk, kh], v[rk, kh]
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(see, Q @ K.T * scale, -np.inf)
            es = (D + 6) * EPS * scale * (np.abs(Q) @ np.abs(K).T)
            es = es + split[0] * scale * (np.abs(Q) @ np.abs(K).T) + split[1] * (np.abs(Q).sum(1)[:, None] + np.abs(K).sum(1)[None, :])
            es = np.where(see, es, 0.0)
            top = s.max(1, keepdims=True)
            top = np.where(np.isneginf(top), 0.0, top)
            e = np.where(see, np.exp(s - top), 0.0)
            l = e.sum(1, keepdims=True)
            some = l[:, 0] > 0
            p = e / np.where(l > 0, l, 1.0)
            # the exponent's argument carries roundings of its size, the maximum's cancel
            size = np.abs(np.where(see, s, 0.0)) + np.abs(top)
            rel = np.where(see, es + 4 * EPS * (1.0 + size), 0.0)
            mean_rel = (p * rel).sum(1, keepdims=True) + (L + 4) * EPS
            erel = rel + mean_rel + 4 * EPS                            # of a normalised p
            fl = floor * see
            o = p @ V
            aV = np.abs(V)
            eo = (p * (erel + step)) @ aV + (fl @ aV) + (L + 6) * EPS * (p @ aV)
            r["out"][rq, h], r["e_out"][rq, h] = o, eo
            lse = np.where(some, top[:, 0] + np.log(np.where(some, l[:, 0], 1.0)), -np.inf)
            r["lse"][h, rq] = lse
            r["e_lse"][h, rq] = mean_rel[:, 0] + 4 * EPS * (1 + np.abs(top[:, 0]) + np.abs(np.log(np.where(some, l[:, 0], 1.0))))
            if g is None:
                continue
            G = g[rq, h]
            dp = np.where(see, G @ V.T, 0.0)
            delta = (G * o).sum(1, keepdims=True)
            ds = p * (dp - delta)
            eout = eo + step * step * (np.abs(o) + eo) + floor         # out in two numbers of the type
            edelta = (np.abs(G) * eout).sum(1, keepdims=True) + (D + 4) * EPS * (np.abs(G) * np.abs(o)).sum(1, keepdims=True)
            edp = (D + 4) * EPS * (np.abs(G) @ aV.T)
            # p from the saved m and l: the errors of both, and of their sum's rounding
            ep = p * (erel + 4 * EPS * (1.0 + size) + 2 * EPS * np.abs(np.where(some, lse, 0.0))[:, None]) + fl
            eds = ep * np.abs(dp - delta) + p * (edp + edelta) + 3 * EPS * np.abs(ds)
            eds = eds + step * (np.abs(ds) + eds) + fl
            aG = np.abs(G)
            r["dv"][rk, kh] += p.T @ G
            r["e_dv"][rk, kh] += (ep + step * p + fl).T @ aG + (len(rq) * H // Hk + 8) * EPS * (p.T @ aG)
            r["dq"][rq, h] = ds @ K * scale
            r["e_dq"][rq, h] = scale * (eds @ np.abs(K) + (L + 8) * EPS * (np.abs(ds) @ np.abs(K)))
            r["dk"][rk, kh] += ds.T @ Q * scale
            r["e_dk"][rk, kh] += scale * (eds.T @ np.abs(Q) + (len(rq) * H // Hk + 8) * EPS * (np.abs(ds).T @ np.abs(Q)))
    return r
