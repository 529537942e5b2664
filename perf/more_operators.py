"""Cases of the attention-block operators next to the sparse convolutions: layer
norm, rotary positions of several axes and attention over ragged samples, on
channels-last features [rows, channels] of voxels.

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
    sites x 128) and generic ragged batches."""
    return [
        # a small scene: the call's latency
        _norm("ln_fwd_2k_f32", "f32", 2000, 16, False, False),
        # the odd-sized output of a strided layer
        _norm("ln_train_odd_f16", "f16", 33333, 80, False, True),
        # the join before a block's second half, in training on the shell sets
        _norm("ln_train_shells_bf16", "bf16", 266426, 128, True, True),
        # wide rows
        _norm("ln_train_wide_f32", "f32", 4099, 1024, False, True),
        # one new row for each of seven running sequences, one axis, far along
        _rotary("rotary_step_7_bf16", "bf16", 7, 8, 64, 1, 1 << 20, False),
        # queries and keys of the LiDAR samples by (z, y, x)
        _rotary("rotary_lidar_f16", "f16", 120000, 8, 16, 3, 1600, False),
        # their gradients on the shell sets
        _rotary("rotary_inverse_shells_bf16", "bf16", 266426, 8, 32, 3, 128, True),
        # a small scene in windows of 125 rows along the curve: the call's latency
        _attn("attn_fwd_2k_f32", "f32", 2000, 0, 1, 1, 16, 1, "windows", 125, True, False, False),
        # one query for each sample pools all its rows
        _attn("attn_pool_shells_bf16", "bf16", 4, 266426, 8, 8, 16, 4, "even", 0, False, False, False),
        # one long sequence, each row after those before it, four query heads to a pair of keys and values
        _attn("attn_fwd_long_bf16", "bf16", 16411, 0, 8, 2, 128, 1, "even", 0, False, True, False),
        # training in windows of 1,024 rows along a curve on the shell sets
        _attn("attn_train_shells_bf16", "bf16", 266426, 0, 4, 4, 32, 4, "windows", 1024, True, False, True),
        # a ragged batch with empty and one-row samples, full precision, shared keys
        _attn("attn_train_ragged_f32", "f32", 5003, 0, 6, 2, 48, 23, "ragged", 0, False, True, True),
    ]


def _norm(name, dtype, rows, channels, residual, train):
    c = dict(op="norm", dtype=dtype, rows=rows, channels=channels, residual=residual, train=train)
    return dict(c, name=name) if name else c


def _rotary(name, dtype, rows, heads, dim, axes, span, inverse):
    c = dict(op="rotary", dtype=dtype, rows=rows, heads=heads, dim=dim, axes=axes, span=span, inverse=inverse)
    return dict(c, name=name) if name else c


def _attn(name, dtype, rows, kv_rows, heads, kv_heads, dim, samples, spread, window, ordered, causal, train):
    """kv_rows 0: the rows attend to themselves."""
    c = dict(op="attn", dtype=dtype, rows=rows, kv_rows=kv_rows, heads=heads, kv_heads=kv_heads, dim=dim, samples=samples,
             spread=spread, window=window, ordered=ordered, causal=causal, train=train)
    return dict(c, name=name) if name else c


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "rotary", "attn", "attn", "attn"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    cells = 266426 * 128 * 2 // _SIZE[dtype]                 # no larger than the largest listed case
    if op == "norm":
        channels = 16 * log_int(1, 64)
        return _norm(None, dtype, log_int(1, min(266426, cells // channels)), channels, rng.random() < 0.5,
                     rng.random() < 0.6)
    dim = 16 * rng.choice((1, 2, 3, 4, 4, 5, 6, 8))
    if op == "rotary":
        heads = log_int(1, 16)
        return _rotary(None, dtype, log_int(1, min(266426, cells // (heads * dim))), heads, dim, rng.choice((1, 2, 3, 4)),
                       rng.choice((32, 1600, 1 << 20)), rng.random() < 0.5)
    kv_heads = rng.choice((1, 2, 3, 4))
    heads = kv_heads * rng.choice((1, 1, 2, 4))
    train = rng.random() < 0.5
    kind = rng.choice(("windows", "even", "ragged", "cross"))
    ordered = rng.random() < 0.5
    if kind == "windows":
        window = log_int(16, 2048)
        rows = log_int(1, max(1, min(266426, cells // (heads * dim), (1 << 30) // (heads * window))))
        return _trained(_attn(None, dtype, rows, 0, heads, kv_heads, dim, log_int(1, 8), "windows", window, ordered, False,
                              train))
    causal = rng.random() < 0.5
    samples = log_int(1, 32)
    spread = "ragged" if kind == "ragged" else rng.choice(("even", "ragged"))
    rows, kv_rows = log_int(1, 12000), 0
    if kind == "cross":                                      # a few rows each way against many
        rows, kv_rows = log_int(1, 64), log_int(1, 100000)
        if rng.random() < 0.3:
            rows, kv_rows = kv_rows, rows
    while True:
        c = _attn(None, dtype, rows, kv_rows, heads, kv_heads, dim, samples, spread, 0, ordered, causal, train)
        lq, lk = _lengths(c, 0)
        if samples * heads * max(lq) * max(lk) <= 1 << 30:   # the plain form's scores, padded
            return _trained(c)
        rows, kv_rows = -(-rows // 2), -(-kv_rows // 2)


def _trained(case):
    """The case, trained only where some sample has four keys: gradients of a
    query that sees one key are 0, and a case of only these says nothing."""
    return dict(case, train=case["train"] and any(a and b >= 4 for a, b in zip(*_lengths(case, 0))))


# ------------------------------------------------------------------ inputs

def _spread(n, s, spread, seed):
    if spread == "even":
        return np.array([n * (i + 1) // s - n * i // s for i in range(s)])
    r = np.random.default_rng(seed)
    w = r.exponential(size=s) ** 2
    if s > 3:
        w[r.permutation(s)[:max(1, s // 8)]] = 0.0           # empty samples
    cut = np.floor(np.cumsum(w) / w.sum() * n + 0.5).astype(np.int64)
    cut[-1] = n
    return np.diff(np.concatenate([[0], cut]))


def _lengths(case, seed):
    """Rows of queries and of keys of each sample (or window); the seed only
    permutes them, so that every seed has the same work."""
    n, s = case["rows"], case["samples"]
    if case["spread"] == "windows":
        w = case["window"]
        each = [m for m in _spread(n, s, "even", 0) for m in [w] * (m // w) + ([m % w] if m % w else [])]
        lq = np.array(each)
        return lq.tolist(), lq.tolist()
    lq = _spread(n, s, case["spread"], 1)
    lk = _spread(case["kv_rows"], s, case["spread"], 2) if case["kv_rows"] else lq
    p = np.random.default_rng(seed).permutation(s)
    return lq[p].tolist(), lk[p].tolist()


def _pairs(dim, axes):
    """Rotated pairs of each axis: as even as they come, the first ones fewer."""
    return [dim // 2 * (a + 1) // axes - dim // 2 * a // axes for a in range(axes)]


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _DT[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    n = case["rows"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std

    def order(lengths):
        at = np.cumsum([0] + lengths)
        ids = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).to(dev)
        key = ids.double() + torch.rand(int(at[-1]), generator=g, device=dev, dtype=torch.float64) * 0.999
        return torch.argsort(key).int()                      # each sample's rows along its own curve

    def ptr(lengths):
        return torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32).to(dev)

    st = {"case": case}
    if case["op"] == "norm":
        c = case["channels"]
        # a block's features: every channel has a mean and a spread of its own
        st["x"] = (normal(n, c) * (0.5 + torch.rand(c, generator=g, device=dev)) + normal(c)).to(dt)
        st["gamma"], st["beta"] = 1.0 + normal(c, std=0.2), normal(c, std=0.2)
        if case["residual"]:
            st["residual"] = normal(n, c).to(dt)
        if case["train"]:
            st["dy"] = normal(n, c).to(dt)
            if case["residual"]:
                st["dtotal"] = normal(n, c).to(dt)
    elif case["op"] == "rotary":
        st["x"] = normal(n, case["heads"], case["dim"]).to(dt)
        cells = torch.randint(0, case["span"], (n, case["axes"] + 1), generator=g, device=dev, dtype=torch.int32)
        st["pos"], st["pairs"] = cells[:, 1:], _pairs(case["dim"], case["axes"])   # the first column is the sample
        st["axis"] = torch.tensor([a for a, p in enumerate(st["pairs"]) for _ in range(p)], device=dev)
        st["freq"] = torch.tensor([10000.0 ** (-j / p) for p in st["pairs"] for j in range(p)], dtype=torch.float32).to(dev)
    else:
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        st["lq"], st["lk"] = _lengths(case, seed)
        st["ptr"] = ptr(st["lq"])
        gain = 0.5 + 2.0 * torch.rand(h, 1, generator=g, device=dev)             # from flat to peaked heads
        if case["kv_rows"]:
            q, kv = normal(n, h, d), normal(case["kv_rows"], 2 * hk, d).to(dt)
            st["q"], st["k"], st["v"] = (q * gain).to(dt), kv[:, :hk], kv[:, hk:]
            st["kv_ptr"] = ptr(st["lk"])
        else:
            x = normal(n, h + 2 * hk, d)                     # one projection gives all three
            x[:, :h] *= gain
            x = x.to(dt)
            st["q"], st["k"], st["v"] = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        if case["ordered"]:
            st["order"] = order(st["lq"])
            if case["kv_rows"]:
                st["kv_order"] = order(st["lk"])
        if case["train"]:
            st["dout"] = normal(n, h, d).to(dt)
    return st


# -------------------------------------------------------------- plain forms

def _norm_plain(st):
    case, dt = st["case"], st["x"].dtype
    total = (st["x"].float() + st["residual"].float()).to(dt) if case["residual"] else st["x"]
    u = total.float()
    d = u - u.mean(1, keepdim=True)
    r = torch.rsqrt((d * d).mean(1, keepdim=True) + _EPS)
    hat = d * r
    y = (hat * st["gamma"] + st["beta"]).to(dt)
    res = (total, y) if case["residual"] else (y,)
    if not case["train"]:
        return res
    dy = st["dy"].float()
    w = dy * st["gamma"]
    dx = r * (w - w.mean(1, keepdim=True) - hat * (w * hat).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + st["dtotal"].float()
    sums = (dy * hat).sum(0, dtype=torch.float64).float(), dy.sum(0, dtype=torch.float64).float()
    return res + (dx.to(dt),) + sums


def _rotary_plain(st):
    x = st["x"].float()
    n, h, d = x.shape
    t = st["pos"].double()[:, st["axis"]] * st["freq"].double()
    c, s = torch.cos(t).float().unsqueeze(1), torch.sin(t).float().unsqueeze(1)
    if st["case"]["inverse"]:
        s = -s
    pair = x.view(n, h, d // 2, 2)
    a, b = pair[..., 0], pair[..., 1]
    return torch.stack([a * c - b * s, a * s + b * c], dim=-1).view(n, h, d).to(st["x"].dtype)


def _slots(lengths, order, dev):
    """Rows of each sample, padded to the longest: [S, L], and which are there."""
    m = torch.tensor(lengths, device=dev).unsqueeze(1)
    at = torch.cumsum(m, 0) - m
    i = torch.arange(max(lengths), device=dev).unsqueeze(0)
    rows = torch.where(i < m, at + i, 0)
    return (rows if order is None else order.long()[rows]), i < m


def _attn_plain(st):
    case, dev, dt = st["case"], st["q"].device, st["q"].dtype
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    scale = 1.0 / math.sqrt(d)
    qr, qv = _slots(st["lq"], st.get("order"), dev)
    kr, kv = _slots(st["lk"], st.get("kv_order"), dev) if case["kv_rows"] else (qr, qv)
    s, lq, lk = qr.shape[0], qr.shape[1], kr.shape[1]

    def queries(t):                                          # [S, kv heads, shared heads x Lq, D]
        t = t[qr].float() * qv[..., None, None]
        return t.view(s, lq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(s, hk, -1, d)

    def keys(t):
        return (t[kr].float() * kv[..., None, None]).permute(0, 2, 1, 3).contiguous()

    def back(t, like, rows, there, shared):
        t = t.view(s, hk, shared, -1, d).permute(0, 3, 1, 2, 4).reshape(s, t.shape[2] // shared, -1, d)
        out = torch.empty(like.shape, dtype=dt, device=dev)
        out[rows[there]] = t[there].to(dt)
        return out

    q, k, v = queries(st["q"]), keys(st["k"]), keys(st["v"])
    see = (qv[:, :, None] & kv[:, None, :])
    if case["causal"]:
        ends = torch.tensor(st["lk"], device=dev) - torch.tensor(st["lq"], device=dev)
        i, j = torch.arange(lq, device=dev), torch.arange(lk, device=dev)
        see = see & (j[None, None, :] <= i[None, :, None] + ends[:, None, None])
    see = see[:, None, None].expand(s, 1, h // hk, lq, lk).reshape(s, 1, -1, lk)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(scale).masked_fill_(~see, -math.inf)
    top = p.amax(3, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(3, keepdim=True)
    p = p.div_(torch.where(total == 0.0, 1.0, total))
    o = torch.matmul(p, v)
    out = back(o, st["q"], qr, qv, h // hk)
    if not case["train"]:
        return out
    do = queries(st["dout"])
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(3, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)
    return out, back(dq, st["q"], qr, qv, h // hk), back(dk, st["k"], kr, kv, 1), back(dv, st["v"], kr, kv, 1)


# ---------------------------------------------------------------- own calls

def _run_own(st):
    import sparse_convolution_hash_amd as spc

    case = st["case"]
    if case["op"] == "norm":
        y, stats, total = spc.layer_norm_fwd(st["x"], st["gamma"], st["beta"], _EPS, residual=st.get("residual"))
        res = (total, y) if case["residual"] else (y,)
        if not case["train"]:
            return res
        return res + spc.layer_norm_bwd(st["dy"], total if case["residual"] else st["x"], st["gamma"], stats,
                                        dtotal=st.get("dtotal"))
    if case["op"] == "rotary":
        return spc.rotary(st["x"], st["pos"], st["freq"], st["pairs"], inverse=case["inverse"])
    kw = dict(order=st.get("order"), kv_ptr=st.get("kv_ptr"), kv_order=st.get("kv_order"), causal=case["causal"])
    out, stats = spc.attention_fwd(st["q"], st["k"], st["v"], st["ptr"], want_stats=case["train"], **kw)
    if not case["train"]:
        return out
    return (out,) + spc.attention_bwd(st["dout"], st["q"], st["k"], st["v"], out, stats, st["ptr"], **kw)


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "rotary": _rotary_plain, "attn": _attn_plain}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work

def _scores(case):
    """(query, key) pairs of one head."""
    lq, lk = (np.array(v, dtype=np.int64) for v in _lengths(case, 0))
    if not case["causal"]:
        return int((lq * lk).sum())
    return int(sum(np.clip(np.arange(a) + 1 + b - a, 0, b).sum() for a, b in zip(lq, lk)))


def work(case):
    n, e = case["rows"], _SIZE[case["dtype"]]
    if case["op"] == "norm":
        c = case["channels"]
        per = 2 + (2 if case["train"] else 0) + (2 if case["residual"] else 0) + (1 if case["train"] and case["residual"] else 0)
        return {"bytes": n * c * e * per + 8 * c + (8 * c if case["train"] else 0),
                "flops": n * c * ((22 if case["train"] else 8) + (1 if case["residual"] else 0))}
    if case["op"] == "rotary":
        cells = n * case["heads"] * case["dim"]
        return {"bytes": 2 * cells * e + 4 * n * case["axes"] + 2 * case["dim"], "flops": 3 * cells}
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    m = case["kv_rows"] or n
    rows = e * d * (2 * n * h + 2 * m * hk)                  # q, k, v in, out out
    if case["train"]:
        rows += e * d * (2 * n * h + 2 * m * hk)             # dout in, three gradients out
    if case["ordered"]:
        rows += 4 * (n + case["kv_rows"])
    return {"bytes": rows + 4 * (case["samples"] + 1), "flops": _scores(case) * h * d * (14 if case["train"] else 4)}


# ------------------------------------------------------------- definitions

def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _exact_norm(case, st):
    x = _np(st["x"])
    if case["residual"]:
        x = x + _np(st["residual"])
        total = x
        x = _np(torch.from_numpy(x).to(st["x"].dtype))       # what is normed is the sum as stored
    gamma, beta = _np(st["gamma"]), _np(st["beta"])
    r = 1.0 / np.sqrt(x.var(axis=1, keepdims=True) + _EPS)
    hat = (x - x.mean(axis=1, keepdims=True)) * r
    y = hat * gamma + beta
    res = (total, y) if case["residual"] else (y,)
    if not case["train"]:
        return res
    dy = _np(st["dy"])
    w = dy * gamma
    dx = r * (w - w.mean(axis=1, keepdims=True) - hat * (w * hat).mean(axis=1, keepdims=True))
    if case["residual"]:
        dx = dx + _np(st["dtotal"])
    return res + (dx, (dy * hat).sum(0), dy.sum(0))


def _exact_rotary(case, st):
    x, pos, freq = _np(st["x"]), _np(st["pos"]), _np(st["freq"])
    z = x[..., 0::2] + 1j * x[..., 1::2]
    j = 0
    for a, pairs in enumerate(st["pairs"]):
        for _ in range(pairs):
            t = pos[:, a] * freq[j]
            z[:, :, j] *= np.exp((-1j if case["inverse"] else 1j) * t)[:, None]
            j += 1
    out = np.empty_like(x)
    out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return (out,)


def _exact_attn(case, st):
    """Sample by sample and head by head on the GPU."""
    h, hk, scale = case["heads"], case["kv_heads"], case["dim"] ** -0.5
    f = lambda t: t.double()
    q, k, v = f(st["q"]), f(st["k"]), f(st["v"])
    out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = f(st["dout"]) if case["train"] else None
    qo = st["order"].long() if case["ordered"] else torch.arange(q.shape[0], device=q.device)
    if case["kv_rows"]:
        ko = st["kv_order"].long() if case["ordered"] else torch.arange(k.shape[0], device=q.device)
    else:
        ko = qo
    a = b = 0
    for lq, lk in zip(st["lq"], st["lk"]):
        rq, rk = qo[a:a + lq], ko[b:b + lk]
        a, b = a + lq, b + lk
        if lq == 0 or lk == 0:
            continue
        for i in range(hk):
            heads = slice(i * (h // hk), (i + 1) * (h // hk))
            qs, ks, vs = q[rq, heads].transpose(0, 1), k[rk, i], v[rk, i]          # [shared, lq, D], [lk, D]
            s = (qs.reshape(-1, qs.shape[2]) @ ks.T).view(-1, lq, lk) * scale
            if case["causal"]:
                hidden = torch.ones(lq, lk, dtype=torch.bool, device=q.device).triu(1 + lk - lq)
                s = s.masked_fill(hidden, -math.inf)
                del hidden
            p = torch.nan_to_num(torch.softmax(s, dim=2), nan=0.0)                  # a row that sees nothing: 0
            del s
            o = (p.view(-1, lk) @ vs).view(-1, lq, vs.shape[1])
            out[rq, heads] = o.transpose(0, 1)
            if do is None:
                continue
            g = do[rq, heads].transpose(0, 1)
            flat = g.reshape(-1, g.shape[2])
            ds = (flat @ vs.T).view(-1, lq, lk) - (g * o).sum(2, keepdim=True)
            ds = (ds * p * scale).view(-1, lk)
            dq[rq, heads] = (ds @ ks).view(-1, lq, ks.shape[1]).transpose(0, 1)
            dk[rk, i] = ds.T @ qs.reshape(-1, qs.shape[2])
            dv[rk, i] = p.view(-1, lk).T @ flat
    res = (out, dq, dk, dv) if case["train"] else (out,)
    return tuple(t.cpu().numpy() for t in res)


def exact(case, seed):
    st = prepare(case, seed)
    res = {"norm": _exact_norm, "rotary": _exact_rotary, "attn": _exact_attn}[case["op"]](case, st)
    res = tuple(torch.from_numpy(np.ascontiguousarray(r)) for r in res)
    single = case["op"] == "rotary" or (case["op"] == "attn" and not case["train"])
    return res[0] if single else res
