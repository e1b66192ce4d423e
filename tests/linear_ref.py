"""64-bit reference of linear attention with a decay per head, from its definition (the
matrix of all pairs of steps), with elementwise bounds on what rounding may do to a
kernel's result."""
from __future__ import annotations

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24   # half a step of bf16 and of fp32, relative


def log_decay(g, b, h, n, dev):
    """Running log-decay of n steps of one head; below -1000 a gate is a reset."""
    if g is None:
        return torch.zeros(n, dtype=torch.float64, device=dev)
    s = (g[h].expand(n) if g.dim() == 1 else g[b, h, :n]).double().clamp_min(-1000.0)
    return s.cumsum(0)


def reference(q, k, v, g, h0, lens=None, do=None, dhT=None):
    """Returns ({name: value}, {name: sum of the absolute values of the terms}) in fp64;
    gradients where ``do`` is given."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    dims = {"o": (T, dv), "hT": (dv, dk)}
    if do is not None:
        dims.update(dq=(T, dk), dk=(T, dk), dv=(T, dv), dh0=(dv, dk))
        if g is not None and g.dim() == 3:
            dims["dg"] = (T,)
    val = {n: torch.zeros((B, H) + d, dtype=torch.float64, device=dev) for n, d in dims.items()}
    mag = {n: torch.zeros_like(t) for n, t in val.items()}
    zero = torch.zeros(dv, dk, dtype=torch.float64, device=dev)
    for b in range(B):
        n = T if lens is None else max(0, min(T, int(lens[b])))
        for h in range(H):
            s0 = zero if h0 is None else h0[b, h].double()
            d1 = zero if dhT is None else dhT[b, h].double()
            if n == 0:
                val["hT"][b, h] = s0
                if do is not None:
                    val["dh0"][b, h] = d1
                continue
            c = log_decay(g, b, h, n, dev)
            w = torch.where(torch.ones(n, n, device=dev).tril() > 0, c[:, None] - c[None, :], -torch.inf).exp()
            up, left, end = c.exp()[:, None], (c[-1] - c).exp()[:, None], c[-1].exp()
            f = [t[b, h, :n].double() for t in (q, k, v)] + ([] if do is None else [do[b, h, :n].double()])
            for out, (x, y, z, *e), S0, D1 in ((val, f, s0, d1), (mag, [t.abs() for t in f], s0.abs(), d1.abs())):
                p = (x @ y.T) * w
                out["o"][b, h, :n] = p @ z + up * (x @ S0.T)
                out["hT"][b, h] = hT = (left * z).T @ y + end * S0
                if do is None:
                    continue
                e = e[0]
                dp = (e @ z.T) * w
                dq = dp @ y + up * (e @ S0)
                dkk = dp.T @ x + left * (z @ D1)
                out["dq"][b, h, :n], out["dk"][b, h, :n] = dq, dkk
                out["dv"][b, h, :n] = p.T @ e + left * (y @ D1.T)
                out["dh0"][b, h] = (up * e).T @ x + end * D1
                if "dg" in val:
                    sign = -1.0 if out is val else 1.0
                    t = (x * dq).sum(-1) + sign * (y * dkk).sum(-1)
                    t[-1] += (hT * D1).sum()
                    out["dg"][b, h, :n] = t.flip(0).cumsum(0).flip(0)
                    if h0 is None:
                        val["dg"][b, h, 0] = 0   # the first gate decays nothing: exactly zero
    return val, mag


def bounds(val, mag, dtype, roundings=400):
    """Elementwise bound of each result.  fp32 parts: at most ``roundings`` fp32 roundings of
    partial sums on the way of a term (products of up to 128, chunks of 64, a few dozen chunk
    updates, exponentials good to some 2^-21).  bf16 I/O adds half a bf16 step of the result
    and, for the operands rounded to bf16 (pairs of a chunk, state of earlier chunks), half a
    step of every term."""
    out = {}
    for n, r in val.items():
        b = roundings * U32 * mag[n]
        if dtype == torch.bfloat16 and n in ("o", "dq", "dk", "dv"):
            b = b + U16 * r.abs() + U16 * (1 + U16) * mag[n]
        out[n] = b + 1e-30
    return out


def check(got, val, mag, dtype, label=""):
    """Every result within its bound, and as a whole (2-norm) within what independent
    roundings leave: three of bf16 for bf16 results (0.43 half steps each, root mean square),
    under 200 half steps of fp32 for the others."""
    lim = bounds(val, mag, dtype)
    bad = []
    for n, r in val.items():
        x = got[n].double()
        assert x.shape == r.shape, (label, n)
        assert torch.isfinite(x).all(), (label, n)
        if not r.numel():
            continue
        over = ((x - r).abs() / lim[n]).max()
        norm = float(r.norm())
        rel = float((x - r).norm()) / norm if norm else float((x - r).norm())
        far = 3 ** 0.5 * 0.5 * U16 if got[n].dtype == torch.bfloat16 else 200 * U32
        print(f"{label} {n}: rel {rel:.2e}, worst element at {float(over):.3f} of its bound", flush=True)
        if not (over <= 1 and rel <= far):
            bad.append((n, rel, float(over)))
    assert not bad, (label, bad)
