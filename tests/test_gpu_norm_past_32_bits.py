"""GPU group norm's backward past 2^31 elements: sums over all rows and the means
of a sample of 33 million rows against fp64 sums of pieces."""

import pytest
import torch

import sparse_convolution_hash_amd as spc
from oracle import rowops as R
from tests.rowops_cases import within

pytestmark = pytest.mark.gpu

EPS_VAR = 1e-5


def test_norm_backward_past_32_bits():
    C, G, tail, head, U = 64, 8, 2000, 1000, R.EPS
    n = (1 << 31) // C + 3000
    print(f"group norm backward n={n} C={C}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(31)
    rand = lambda *s, **k: torch.randn(*s, generator=g, device="cuda", **k)
    x = rand(n, C, dtype=torch.bfloat16)
    x[:n - tail] += 1
    # no gradient cancels another: a tile that is missing, or counted twice, shows in every sum
    dy = rand(n, C, dtype=torch.bfloat16).abs_().add_(0.5)
    gamma, beta = 1 + 0.2 * rand(C), 0.2 * rand(C)
    ptr = torch.tensor([0, n - tail, n], dtype=torch.int32, device="cuda")
    _, stats = spc.group_norm_fwd(x, G, ptr, gamma, beta, eps=EPS_VAR, act="silu")
    dx, dgamma, dbeta = spc.group_norm_bwd(dy, x, G, ptr, gamma, beta, stats, act="silu")

    def pieces():
        for s, (a, b) in enumerate(((0, n - tail), (n - tail, n))):
            for i in range(a, b, 1 << 21):
                yield s, slice(i, min(i + (1 << 21), b))

    wide = lambda v: v.repeat_interleave(C // G)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    count = torch.tensor([n - tail, tail], dtype=torch.float64, device="cuda")[:, None] * (C // G)
    s1, s2 = zeros(2, G), zeros(2, G)
    for s, r in pieces():
        v = x[r].double().view(-1, G, C // G) - 1
        s1[s] += v.sum((0, 2))
        s2[s] += (v * v).sum((0, 2))
    mean = 1 + s1 / count
    rstd = (s2 / count - (s1 / count) ** 2 + EPS_VAR) ** -0.5

    # dz, xhat and the bounds of their fp32 forms: 16 roundings of the slope and the product on
    # top of what xhat's own (the mean's rounding, 16 of the statistics and the product) moves z by
    def parts(s, r):
        hat = (x[r].double() - wide(mean[s])) * wide(rstd[s])
        z = hat * gamma.double() + beta.double()
        sig = torch.sigmoid(z)
        d = dy[r].double()
        dz = d * sig * (1 + z * (1 - sig))
        e_hat = U * (wide(rstd[s] * mean[s].abs()) + 16 * (1 + hat.abs()))
        e_dz = d * (0.5 * gamma.double().abs() * e_hat + 16 * U * (1 + z.abs()))
        return hat, dz, e_hat, e_dz

    g64 = gamma.double()
    sums, env, m1, m2, e1, e2 = zeros(2, C), zeros(2, C), zeros(2, G), zeros(2, G), zeros(2, G), zeros(2, G)
    fold = lambda v: v.view(G, C // G).sum(1)
    for s, r in pieces():
        hat, dz, e_hat, e_dz = parts(s, r)
        b, h = dz.sum(0), (dz * hat).sum(0)
        # a thread's up to 16 additions, and the stored fp32 sums
        e_b = (e_dz + 20 * U * dz.abs()).sum(0)
        e_h = (dz.abs() * e_hat + hat.abs() * e_dz + 24 * U * (dz * hat).abs()).sum(0)
        sums += torch.stack([b, h])
        env += torch.stack([e_b, e_h])
        m1[s] += fold(g64 * b)
        m2[s] += fold(g64 * h)
        e1[s] += fold(g64.abs() * e_b)
        e2[s] += fold(g64.abs() * e_h)
    num = lambda t: t.cpu().numpy()
    within(dbeta, num(sums[0]), num(env[0]), torch.float32, "dbeta")
    within(dgamma, num(sums[1]), num(env[1]), torch.float32, "dgamma")
    # one tile more or less, 512 rows of 33 million, is beyond these bounds
    assert (env < sums.abs() * 512 / n).all()

    m1, m2, e1, e2 = (v / count for v in (m1, m2, e1, e2))
    for s, r in ((0, slice(0, head)), (0, slice(n - tail - head, n - tail)), (1, slice(n - head, n))):
        hat, dz, e_hat, e_dz = parts(s, r)
        w = g64 * dz
        rs, a1, a2 = wide(rstd[s]), wide(m1[s]), wide(m2[s])
        e = rs * (g64.abs() * e_dz + wide(e1[s]) + hat.abs() * wide(e2[s]) + a2.abs() * e_hat
                  + 24 * U * (w.abs() + a1.abs() + (hat * a2).abs()))
        within(dx[r], num(rs * (w - a1 - hat * a2)), num(e), torch.bfloat16, f"dx of sample {s}")
