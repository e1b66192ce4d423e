"""64-bit reference of linear attention's gate gradient as a sum over pairs, nothing subtracted:
    dg_t = sum_{j < t <= i} w_ij (q_i . k_j)(do_i . v_j) + (the state h0 as step -1, dhT as step n),
with the sum of its terms' absolute values, and with what the suffix sum
    dg_t = dg_end + sum_{t <= s < end} (q_s . dq_s - v_s . dv_s)
over the steps between two resets adds up in absolute values."""
from __future__ import annotations

import torch

RESET = -87.33655   # a factor below fp32's normal numbers


def gate_gradient(q, k, v, g, h0, do, dhT):
    """One head's: q, k [n, dk], v, do [n, dv], g [n], h0 and dhT [dv, dk] or None.  Returns
    (dg, sum of |terms|, sum over the run between resets of |steps|) in fp64."""
    n = q.shape[0]
    q, k, v, do, g = (t.double() for t in (q, k, v, do, g))
    S0 = torch.zeros(v.shape[1], q.shape[1], dtype=torch.float64, device=q.device) if h0 is None else h0.double()
    D1 = torch.zeros_like(S0) if dhT is None else dhT.double()
    c = g.clamp_min(-1000.0).cumsum(0)
    low = torch.ones(n, n, device=q.device).tril() > 0
    w = torch.where(low, c[:, None] - c[None, :], -torch.inf).exp()
    up, left, all_ = c.exp(), (c[-1] - c).exp(), c[-1].exp()
    out = []
    for x, y, z, e, s, d in ((q, k, v, do, S0, D1), (q.abs(), k.abs(), v.abs(), do.abs(), S0.abs(), D1.abs())):
        # pairs (i, j): rows 0 .. n (n: dhT), columns 0 .. n (0: h0, j + 1 else); gate t straddles j < t <= i
        E = torch.zeros(n + 1, n + 1, dtype=torch.float64, device=q.device)
        E[:n, 1:] = w * (x @ y.T) * (e @ z.T)
        E[:n, 0] = up * ((x @ s.T) * e).sum(-1)
        E[n, 1:] = left * ((y @ d.T) * z).sum(-1)
        E[n, 0] = all_ * (s * d).sum()
        before = E.cumsum(1)[:, :n]                       # [i, t]: columns up to t (steps before t)
        out.append(before.flip(0).cumsum(0).flip(0).diagonal()[:n].clone())   # sum over i >= t
    val, mag = out
    if h0 is None:
        val[0] = mag[0] = 0.0
    cut = g < RESET
    # the absolute values that the sum over a run of steps passes through: |a_s| + |b_s|, and its ends
    x, y, z, e, s, d = (t.abs() for t in (q, k, v, do, S0, D1))
    dp = (e @ z.T) * w
    steps = (x * (dp @ y + up[:, None] * (e @ s))).sum(-1) + \
            (z * ((((x @ y.T) * w).T @ e) + left[:, None] * (y @ d.T))).sum(-1)
    run = torch.zeros(n, dtype=torch.float64, device=q.device)
    edges = [0] + [t for t in range(1, n) if bool(cut[t])] + [n]
    for a, b in zip(edges, edges[1:]):
        run[a:b] = steps[a:b].sum() + mag[a] + (0.0 if b == n and d.abs().sum() == 0 else mag[b - 1])
    val[cut] = 0.0
    return val, mag, run
