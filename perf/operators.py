"""Cases of the sequence-block operators next to the sparse convolutions: group
norm with activation, counter-based dropout and the gated linear recurrence,
all on channels-last features [rows, channels] with ragged samples.

``run`` computes a case with elementary torch operations, or, where ``own`` is
true, with the library's own calls; ``exact`` gives the same outputs from the
definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5


# ------------------------------------------------------------------- cases

def listed():
    """The measured cases; row counts and channels are the library's own
    workloads' (2,000 sites x 16; 2 x 60k LiDAR sites x 64; 266,426 shell
    sites x 128 or 96) and generic ragged batches."""
    return [
        # a small scene, one sample: the call's latency
        _norm("norm_fwd_2k_f32", "f32", 2000, 16, 4, 1, "even", "silu", 0.0, False),
        # inference on the two LiDAR samples
        _norm("norm_fwd_lidar_f16", "f16", 120000, 64, 16, 2, "even", "relu", 0.0, False),
        # the training step of a residual block's first half on the shell sets, dropout fused
        _norm("norm_train_shells_bf16", "bf16", 266426, 128, 32, 4, "even", "silu", 0.1, True),
        # a ragged batch with empty and one-row samples, groups of 16 channels, full precision
        _norm("norm_train_ragged_f32", "f32", 20011, 48, 3, 37, "ragged", "none", 0.0, True),
        # dropout of a small scene's features
        _drop("drop_fwd_2k_f32", "f32", 2000, 16, False, 0.5, False),
        # dropout of the odd-sized output of a strided layer
        _drop("drop_fwd_odd_f16", "f16", 33333, 80, False, 0.25, False),
        # the residual join of a block in training on the shell sets
        _drop("drop_train_shells_bf16", "bf16", 266426, 128, True, 0.1, True),
        # one new token for each of seven running sequences
        _step("scan_step_7_bf16", "bf16", 7, 64),
        # inference over the serialised LiDAR samples
        _scan("scan_fwd_lidar_f16", "f16", 120000, 64, 2, "even", False, False, False, False),
        # one very long sequence
        _scan("scan_fwd_long_bf16", "bf16", 1000003, 64, 1, "even", False, False, True, False),
        # training over the shell sets along a space-filling order, backwards
        _scan("scan_train_shells_bf16", "bf16", 266426, 128, 4, "even", True, True, True, True),
        # many short sequences with empty and one-row ones, full precision
        _scan("scan_train_ragged_f32", "f32", 30011, 48, 301, "ragged", False, False, True, True),
    ]


def _norm(name, dtype, rows, channels, groups, samples, spread, act, p, train):
    c = dict(op="norm", dtype=dtype, rows=rows, channels=channels, groups=groups, samples=samples, spread=spread,
             act=act, p=p, train=train)
    return dict(c, name=name) if name else c


def _drop(name, dtype, rows, channels, residual, p, train):
    c = dict(op="drop", dtype=dtype, rows=rows, channels=channels, residual=residual, p=p, train=train)
    return dict(c, name=name) if name else c


def _scan(name, dtype, rows, channels, samples, spread, ordered, reverse, state, train):
    c = dict(op="scan", dtype=dtype, rows=rows, channels=channels, samples=samples, spread=spread, ordered=ordered,
             reverse=reverse, state=state, train=train)
    return dict(c, name=name) if name else c


def _step(name, dtype, rows, channels):
    c = dict(op="step", dtype=dtype, rows=rows, channels=channels)
    return dict(c, name=name) if name else c


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "norm", "drop", "scan", "scan", "step"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    channels = 16 * log_int(1, 16)
    cap = 266426 * 128 * 2 // (channels * _SIZE[dtype])      # no larger than the largest listed case
    if op == "step":
        return _step(None, dtype, log_int(1, 4096), channels)
    rows = log_int(1, max(1, min(cap, 500000)))
    train = rng.random() < 0.6
    if op == "drop":
        return _drop(None, dtype, rows, channels, rng.random() < 0.5, rng.choice((0.05, 0.1, 0.25, 0.5)), train)
    samples = log_int(1, 64 if op == "norm" else 512)
    spread = rng.choice(("even", "ragged"))
    if op == "norm":
        groups = rng.choice([g for g in (1, 2, 3, 4, 8, 16, 32, channels // 16) if channels % g == 0])
        # the derivative of relu jumps at 0, so its gradient has no value to compare there
        act = rng.choice(("none", "silu") if train else ("none", "silu", "relu"))
        return _norm(None, dtype, rows, channels, groups, samples, spread, act, rng.choice((0.0, 0.1)), train)
    return _scan(None, dtype, rows, channels, samples, spread, rng.random() < 0.5, rng.random() < 0.5,
                 rng.random() < 0.7, train)


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    n, s = case["rows"], case["samples"]
    if case["spread"] == "even":
        return [n * (i + 1) // s - n * i // s for i in range(s)]
    r = np.random.default_rng(seed)
    w = r.exponential(size=s) ** 2
    if s > 3:
        w[r.permutation(s)[:max(1, s // 8)]] = 0.0       # empty samples
    cut = np.floor(np.cumsum(w) / w.sum() * n + 0.5).astype(np.int64)
    cut[-1] = n
    return np.diff(np.concatenate([[0], cut])).tolist()


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _DT[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    n, c = case["rows"], case["channels"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std

    st = {"case": case}
    if case["op"] in ("norm", "scan"):
        st["lengths"] = _lengths(case, seed)
        st["ptr"] = torch.tensor([0] + np.cumsum(st["lengths"]).tolist(), dtype=torch.int32).to(dev)
    if case["op"] in ("norm", "drop"):
        st["rng"] = torch.tensor([(seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), seed % 1000 + (1 << 33)],
                                 dtype=torch.int64).to(dev)
    if case["op"] == "norm":
        # a convolution's output: every channel has a mean and a spread of its own
        st["x"] = (normal(n, c) * (0.5 + torch.rand(c, generator=g, device=dev)) + normal(c)).to(dt)
        st["gamma"], st["beta"] = 1.0 + normal(c, std=0.2), normal(c, std=0.2)
        if case["train"]:
            st["dy"] = normal(n, c).to(dt)
    elif case["op"] == "drop":
        st["x"] = normal(n, c).to(dt)
        if case["residual"]:
            st["residual"] = normal(n, c).to(dt)
        if case["train"]:
            st["dy"] = normal(n, c).to(dt)
    elif case["op"] == "scan":
        # gates from nearly closed to a memory of some thousand rows
        gx = torch.empty(n, 2 * c, dtype=dt, device=dev)
        gx[:, :c] = (normal(n, c) + 2.0 + 2.0 * normal(c)).to(dt)
        gx[:, c:] = normal(n, c).to(dt)
        st["gate"], st["x"] = gx[:, :c], gx[:, c:]          # one projection gives both
        if case["ordered"]:
            st["order"] = torch.empty(n, dtype=torch.int32, device=dev)
            a = 0
            for m in st["lengths"]:                         # each sample's rows along its own curve
                st["order"][a:a + m] = a + torch.randperm(m, generator=g, device=dev)
                a += m
        if case["state"]:
            st["h0"] = normal(case["samples"], c)
        if case["train"]:
            st["dh"] = normal(n, c).to(dt)
            if case["state"]:
                st["dh_last"] = normal(case["samples"], c)
    else:
        st["gate"], st["x"] = (normal(n, c) + 2.0).to(dt), normal(n, c).to(dt)
        st["state"], st["next"] = normal(n, c), torch.empty(n, c, device=dev)
    return st


# -------------------------------------------------------------- plain forms

_M32 = 0xFFFFFFFF


def _mul_hi_lo(a, m):
    """High and low words of the product of 32-bit a (in int64) and constant m."""
    p0, p1 = (a & 0xFFFF) * m, (a >> 16) * m
    t = p0 + ((p1 & 0xFFFF) << 16)
    return (p1 >> 16) + (t >> 32), t & _M32


def _keep(rng, numel, p, layer=0):
    """Truth values [numel]: element i stays iff its 16 bits of Philox4x32-10
    (key = seed, counter = offset + i // 8 and the layer) reach 65536 p."""
    seed, off = rng[0], rng[1]
    ctr = off + torch.arange((numel + 7) // 8, device=rng.device, dtype=torch.int64)
    c0, c1 = ctr & _M32, (ctr >> 32) & _M32
    c2, c3 = torch.full_like(c0, layer), torch.zeros_like(c0)
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    half = torch.stack([w for c in (c0, c1, c2, c3) for w in (c & 0xFFFF, c >> 16)], dim=1)
    return half.reshape(-1)[:numel] >= round(p * 65536)


def _scale(p):
    return 65536.0 / (65536 - round(p * 65536))


def _norm_plain(st):
    case, x = st["case"], st["x"].float()
    n, c, gr = case["rows"], case["channels"], case["groups"]
    cg, gamma, beta = c // gr, st["gamma"], st["beta"]
    xhat = torch.empty_like(x)
    stats, a = [], 0
    for m in st["lengths"]:
        if m:
            v = x[a:a + m].view(m, gr, cg)
            cnt = float(m * cg)
            mean = v.sum((0, 2), dtype=torch.float64) / cnt
            d = v - mean.float().view(1, gr, 1)
            var = (d * d).sum((0, 2), dtype=torch.float64) / cnt
            r = torch.rsqrt(var + _EPS).float().view(1, gr, 1)
            xhat[a:a + m] = (d * r).view(m, c)
            stats.append((a, m, r))
        a += m
    z = xhat * gamma + beta
    sig = torch.sigmoid(z) if case["act"] == "silu" else None
    y = z * sig if sig is not None else z.clamp(min=0) if case["act"] == "relu" else z
    keep = _keep(st["rng"], n * c, case["p"]).view(n, c) if case["p"] > 0 else None
    if keep is not None:
        y = torch.where(keep, y * _scale(case["p"]), 0.0)
    y = y.to(st["x"].dtype)
    if not case["train"]:
        return y
    dz = st["dy"].float()
    if keep is not None:
        dz = torch.where(keep, dz * _scale(case["p"]), 0.0)
    if sig is not None:
        dz = dz * sig * (1.0 + z * (1.0 - sig))
    dbeta, dgamma = dz.sum(0, dtype=torch.float64).float(), (dz * xhat).sum(0, dtype=torch.float64).float()
    gz, dx = dz * gamma, torch.empty_like(x)
    for a, m, r in stats:
        gv, hv = gz[a:a + m].view(m, gr, cg), xhat[a:a + m].view(m, gr, cg)
        cnt = float(m * cg)
        m1 = (gv.sum((0, 2), dtype=torch.float64) / cnt).float().view(1, gr, 1)
        m2 = ((gv * hv).sum((0, 2), dtype=torch.float64) / cnt).float().view(1, gr, 1)
        dx[a:a + m] = ((gv - m1 - hv * m2) * r).view(m, c)
    return y, dx.to(st["x"].dtype), dgamma, dbeta


def _drop_plain(st):
    case, x = st["case"], st["x"].float()
    keep, s = _keep(st["rng"], x.numel(), case["p"]).view(x.shape), _scale(case["p"])
    y = torch.where(keep, x * s, 0.0)
    if case["residual"]:
        y = y + st["residual"].float()
    y = y.to(st["x"].dtype)
    if not case["train"]:
        return y
    return y, torch.where(keep, st["dy"].float() * s, 0.0).to(st["x"].dtype)


def _doubling(a, b, longest):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... by windows of doubling length."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _scan_plain(st):
    case, dt, dev = st["case"], st["x"].dtype, st["x"].device
    n, c, s = case["rows"], case["channels"], case["samples"]
    lengths = torch.tensor(st["lengths"], device=dev)
    ptr = st["ptr"].long()
    longest, full = max(st["lengths"]), lengths > 0
    first, last = ptr[:-1][full], ptr[1:][full] - 1
    if case["reverse"]:
        first, last = n - 1 - last, n - 1 - first
    row = st["order"].long() if case["ordered"] else torch.arange(n, device=dev)
    row = row.flip(0) if case["reverse"] else row
    g, x = st["gate"].float()[row], st["x"].float()[row]
    h0 = st["h0"] if case["state"] else torch.zeros(s, c, device=dev)
    a, na = torch.sigmoid(g), torch.sigmoid(-g)
    b, a_in = na * x, a.clone()
    b[first] += a[first] * h0[full]
    a_in[first] = 0.0
    h = _doubling(a_in, b, longest)
    out = torch.empty(n, c, dtype=dt, device=dev)
    out[row] = h.to(dt)
    h_last = h0.clone()
    h_last[full] = h[last]
    if not case["train"]:
        return out, h_last
    d = st["dh"].float()[row]
    dlast = st["dh_last"] if case["state"] else torch.zeros(s, c, device=dev)
    d[last] += dlast[full]
    a_next = torch.cat([a[1:], torch.zeros(1, c, device=dev)])
    a_next[last] = 0.0
    big = _doubling(a_next.flip(0), d.flip(0), longest).flip(0)
    prev = torch.cat([torch.zeros(1, c, device=dev), h[:-1]])
    prev[first] = h0[full]
    dx, dg = torch.empty(n, c, dtype=dt, device=dev), torch.empty(n, c, dtype=dt, device=dev)
    dx[row] = (na * big).to(dt)
    dg[row] = (a * na * (prev - x) * big).to(dt)
    dh0 = dlast.clone()
    dh0[full] = a[first] * big[first]
    return out, h_last, dg, dx, dh0


def _step_plain(st):
    g, x = st["gate"].float(), st["x"].float()
    h = torch.sigmoid(g) * st["state"] + torch.sigmoid(-g) * x
    return h.to(st["x"].dtype), h


# ---------------------------------------------------------------- own calls

def _run_own(st):
    import sparse_convolution_hash_amd as spc

    case = st["case"]
    if case["op"] == "norm":
        drop = spc.Dropout(st["rng"], case["p"]) if case["p"] > 0 else None
        args = (case["groups"], st["ptr"], st["gamma"], st["beta"])
        y, stats = spc.group_norm_fwd(st["x"], *args, eps=_EPS, act=case["act"], dropout=drop)
        if not case["train"]:
            return y
        return (y,) + spc.group_norm_bwd(st["dy"], st["x"], *args, stats, act=case["act"], dropout=drop)
    if case["op"] == "drop":
        drop = spc.Dropout(st["rng"], case["p"])
        y = spc.dropout_fwd(st["x"], drop, residual=st.get("residual"))
        return (y, spc.dropout_bwd(st["dy"], drop)) if case["train"] else y
    if case["op"] == "scan":
        kw = dict(h0=st.get("h0"), order=st.get("order"), reverse=case["reverse"])
        out, h_last, carry = spc.linear_recurrence_fwd(st["gate"], st["x"], st["ptr"], want_carry=case["train"], **kw)
        if not case["train"]:
            return out, h_last
        return (out, h_last) + spc.linear_recurrence_bwd(st["dh"], st["gate"], st["x"], st["ptr"], carry,
                                                         dh_last=st.get("dh_last"), want_dh0=True, **kw)
    return spc.linear_recurrence_step(st["gate"], st["x"], st["state"], new_state=st["next"]), st["next"]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "drop": _drop_plain, "scan": _scan_plain, "step": _step_plain}[
        state["case"]["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    n, c, e = case["rows"], case["channels"], _SIZE[case["dtype"]]
    cells = n * c
    if case["op"] == "norm":
        per = 4 if case["train"] else 2          # x in, y out; in training dy in and dx out too
        return {"bytes": cells * e * per + 8 * c + (16 * c if case["train"] else 0) + 4 * (case["samples"] + 1),
                "flops": cells * (40 if case["train"] else 14)}
    if case["op"] == "drop":
        per = 2 + (1 if case["residual"] else 0) + (2 if case["train"] else 0)
        return {"bytes": cells * e * per + 16, "flops": cells * (2 if case["train"] else 1)}
    if case["op"] == "scan":
        per = 3 + (3 if case["train"] else 0)    # gate, x in, h out; in training dh in, two gradients out
        ends = 4 * c * case["samples"] * ((2 if case["state"] else 1) + (2 if case["train"] else 0)
                                          + (1 if case["train"] and case["state"] else 0))
        order = 4 * n if case["ordered"] else 0
        return {"bytes": cells * e * per + ends + order + 4 * (case["samples"] + 1),
                "flops": cells * (28 if case["train"] else 10)}
    return {"bytes": cells * (3 * e + 8), "flops": cells * 10}


# ------------------------------------------------------------- definitions

def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _philox_keep(rng, numel, p):
    seed, off = (int(v) & 0xFFFFFFFFFFFFFFFF for v in rng.cpu().tolist())
    u64, lo = np.uint64, np.uint64(0xFFFFFFFF)
    blocks = np.arange((numel + 7) // 8, dtype=np.uint64) + u64(off)
    x = [blocks & lo, blocks >> u64(32), np.zeros_like(blocks), np.zeros_like(blocks)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        a, b = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)     # below 2^64
        x = [(b >> u64(32)) ^ x[1] ^ u64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), b & lo,
             (a >> u64(32)) ^ x[3] ^ u64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF), a & lo]
    words = np.stack(x, axis=1).astype(np.uint32)
    half = np.ascontiguousarray(words).view(np.uint16).reshape(-1)   # little endian: low half first
    return half[:numel] >= int(round(p * 65536))


def _exact_norm(case, st):
    x, gamma, beta = _np(st["x"]), _np(st["gamma"]), _np(st["beta"])
    n, c, gr = case["rows"], case["channels"], case["groups"]
    cg = c // gr
    factor = np.ones((n, c))
    if case["p"] > 0:
        factor = _philox_keep(st["rng"], n * c, case["p"]).reshape(n, c) * _scale(case["p"])
    y, dx = np.zeros((n, c)), np.zeros((n, c))
    dgamma, dbeta, a = np.zeros(c), np.zeros(c), 0
    dy = _np(st["dy"]) if case["train"] else None
    for m in st["lengths"]:
        rows = slice(a, a + m)
        a += m
        for k in range(gr if m else 0):
            ch = slice(k * cg, (k + 1) * cg)
            v = x[rows, ch]
            r = 1.0 / math.sqrt(v.var() + _EPS)
            hat = (v - v.mean()) * r
            z = hat * gamma[ch] + beta[ch]
            s = 1.0 / (1.0 + np.exp(-z))
            val = {"none": z, "relu": np.maximum(z, 0.0), "silu": z * s}[case["act"]]
            y[rows, ch] = val * factor[rows, ch]
            if dy is None:
                continue
            slope = {"none": np.ones_like(z), "relu": (z > 0) * 1.0, "silu": s + z * s * (1.0 - s)}[case["act"]]
            dz = dy[rows, ch] * factor[rows, ch] * slope
            dbeta[ch] += dz.sum(0)
            dgamma[ch] += (dz * hat).sum(0)
            w = dz * gamma[ch]
            dx[rows, ch] = r * (w - w.mean() - hat * (w * hat).mean())
    return y if dy is None else (y, dx, dgamma, dbeta)


def _exact_drop(case, st):
    x = _np(st["x"])
    f = _philox_keep(st["rng"], x.size, case["p"]).reshape(x.shape) * _scale(case["p"])
    y = x * f + (_np(st["residual"]) if case["residual"] else 0.0)
    return (y, _np(st["dy"]) * f) if case["train"] else y


def _exact_scan(case, st):
    n, c, s = case["rows"], case["channels"], case["samples"]
    g, x = _np(st["gate"]), _np(st["x"])
    a, na = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    order = st["order"].cpu().numpy() if case["ordered"] else np.arange(n)
    out, dg, dx = np.zeros((n, c)), np.zeros((n, c)), np.zeros((n, c))
    h_last = _np(st["h0"]) if case["state"] else np.zeros((s, c))
    dh0 = _np(st["dh_last"]) if case["train"] and case["state"] else np.zeros((s, c))
    dh = _np(st["dh"]) if case["train"] else None
    start = 0
    for k, m in enumerate(st["lengths"]):
        rows = order[start:start + m].tolist()
        start += m
        if case["reverse"]:
            rows.reverse()
        before = np.zeros((m, c)) if dh is not None else None
        h = h_last[k].copy()
        for t, r in enumerate(rows):
            if before is not None:
                before[t] = h
            h = a[r] * h + na[r] * x[r]
            out[r] = h
        h_last[k] = h
        if dh is None:
            continue
        d = dh0[k].copy()
        for t in range(m - 1, -1, -1):
            r = rows[t]
            d = d + dh[r]
            dx[r] = na[r] * d
            dg[r] = a[r] * na[r] * (before[t] - x[r]) * d
            d = a[r] * d
        dh0[k] = d
    return (out, h_last) if dh is None else (out, h_last, dg, dx, dh0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        res = _exact_norm(case, st)
    elif case["op"] == "drop":
        res = _exact_drop(case, st)
    elif case["op"] == "scan":
        res = _exact_scan(case, st)
    else:
        g, x, h = _np(st["gate"]), _np(st["x"]), _np(st["state"])
        a = 1.0 / (1.0 + np.exp(-g))
        new = a * h + x / (1.0 + np.exp(g))
        res = (new, new)
    if isinstance(res, tuple):
        return tuple(torch.from_numpy(r) for r in res)
    return torch.from_numpy(res)
