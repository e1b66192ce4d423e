"""64-bit reference of the gated linear recurrence, step by step from its definition, with
elementwise bounds on what fp32 rounding may do to a kernel's result."""
from __future__ import annotations

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24   # half a step of bf16 and of fp32, relative

# Roundings of fp32 that a step may add to what it passes on, in half steps of the sum of the
# terms' absolute values: the decay's exponential 2 (one unit of its instruction) and its
# argument's rounding |g| e^-|g| * 1.5 < 1, the series or difference of the coupled weight 4
# and its product 1, the step's own multiply-add 1; and once in a run of 16 steps the run's
# decay, whose argument is a sum of 16 gates: 16 |G| e^-|G| < 6, its exponential 2; joining it
# to the runs before it in its tile 2, the tile's map to the state 2, the state to the run 1.
# Together 22.
STEP = 24


def reference(x, g, h0=None, lens=None, coupled=False, do=None, dhT=None):
    """Returns ({name: value}, {name: bound of the fp32 error}); gradients where ``do`` is given.
    A row behind its length: everything zero there, not read."""
    B, H, T, d = x.shape
    f64, dev = torch.float64, x.device
    n = torch.full((B,), T, device=dev) if lens is None else lens.long().clamp(0, T)
    live = (torch.arange(T, device=dev) < n[:, None])[:, None, :, None]
    X = torch.where(live, x.double(), 0.0)
    G = torch.where(live, g.double(), 0.0)
    a, w = G.exp(), (-G.expm1() if coupled else torch.ones_like(G))
    h = torch.zeros(B, H, d, dtype=f64, device=dev) if h0 is None else h0.double()
    m, e = h.abs(), torch.zeros_like(h)
    hs, ms, es = [h], [m], [e]
    for t in range(T):
        on = live[:, :, t]
        b = w[:, :, t] * X[:, :, t]
        h = torch.where(on, a[:, :, t] * h + b, h)
        m = torch.where(on, a[:, :, t] * m + b.abs(), m)
        e = torch.where(on, a[:, :, t] * e + STEP * U32 * m, e)
        hs.append(h), ms.append(m), es.append(e)
    hs, ms, es = (torch.stack(z, 2) for z in (hs, ms, es))
    val = {"o": hs[:, :, 1:] * live, "hT": h}
    err = {"o": es[:, :, 1:] * live, "hT": e}
    if do is None:
        return val, err
    Y = torch.where(live, do.double(), 0.0)
    r = torch.zeros_like(h) if dhT is None else dhT.double()
    m, e = r.abs(), torch.zeros_like(r)
    D, DM, DE, R, RM, RE = ([None] * T for _ in range(6))
    for t in range(T - 1, -1, -1):
        on, y, f = live[:, :, t], Y[:, :, t], a[:, :, t]
        D[t], DM[t], DE[t] = y + r, y.abs() + m, e + U32 * (y.abs() + m)
        R[t], RM[t], RE[t] = f * D[t], f * DM[t], f * DE[t] + STEP * U32 * f * DM[t]
        r, m, e = torch.where(on, R[t], r), torch.where(on, RM[t], m), torch.where(on, RE[t], e)
    zero = torch.zeros(B, H, 0, d, dtype=f64, device=dev)
    D, DM, DE, R, RM, RE = (torch.stack(z, 2) if T else zero for z in (D, DM, DE, R, RM, RE))
    before, bm, be = hs[:, :, :-1], ms[:, :, :-1], es[:, :, :-1]
    if coupled:
        before, bm = before - X, bm + X.abs()
        be = be + U32 * bm
    val["dx"], err["dx"] = w * D * live, (w.abs() * (DE + 6 * U32 * DM)) * live
    val["dg"] = R * before * live
    err["dg"] = (RE * bm + RM * be + 4 * U32 * RM * bm) * live
    val["dh0"], err["dh0"] = r, e
    return val, err


def check(got, val, err, label=""):
    """Every element within its bound: the fp32 one and, of a bf16 result, its own rounding."""
    bad = []
    for n, v in val.items():
        x = got[n]
        assert x.shape == v.shape, (label, n, x.shape, v.shape)
        lim = err[n] + 1e-30
        if x.dtype == torch.bfloat16:
            lim = lim * (1 + U16) + U16 * v.abs()
        assert torch.isfinite(x).all(), (label, n)
        if not v.numel():
            continue
        over = float(((x.double() - v).abs() / lim).max())
        print(f"{label} {n}: worst element at {over:.3f} of its bound", flush=True)
        if not over <= 1:
            bad.append((n, over))
    assert not bad, (label, bad)
