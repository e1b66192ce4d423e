"""64-bit reference of the norms and rotations of queries and keys, row by row from their
definition, with elementwise bounds on what fp32 rounding may do to a kernel's result."""
from __future__ import annotations

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24   # half a step of bf16 and of fp32, relative


def turn(y, rot, angle, amplitude, interleaved, both=False):
    """Rows y rotated by angle [B,1,T,rot/2]; both: the sum of the absolute values of a result's terms."""
    c, s = angle.cos() * amplitude, angle.sin() * amplitude
    out = y.clone()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = y[..., i], y[..., j]
    if both:
        out[..., i] = out[..., j] = abs(amplitude) * (u + v)
    else:
        out[..., i], out[..., j] = u * c - v * s, v * c + u * s
    return out


def reference(x, w=None, norm=None, eps=0.0, freqs=None, pos=None, interleaved=False, amplitude=1.0, lens=None, dy=None):
    """Returns ({name: value}, {name: bound of the fp32 error}) of y and, where ``dy`` is given, dx and dw."""
    B, H, T, d = x.shape
    dev = x.device
    n = torch.full((B,), T, device=dev) if lens is None else lens.long()
    live = (torch.arange(T, device=dev) < n[:, None])[:, None, :, None]
    X = torch.where(live, x.double(), 0.0)
    rot = 0 if freqs is None else 2 * freqs.shape[0]
    p = torch.arange(T, device=dev).expand(B, T).double()
    if pos is not None:
        p = pos.double() if pos.dim() == 2 else p + pos.double()[:, None]
    angle = None if freqs is None else (p[..., None] * freqs)[:, None]
    share = {None: 0.0, "l2": 1.0, "rms": 1.0 / d}[norm]
    W = 1.0 if w is None else w.double()
    r = 1.0 if norm is None else ((X * X).sum(-1, keepdim=True) * share + eps).rsqrt()
    unit = X * r
    f = (lambda y, a: y) if rot == 0 else (lambda y, a: turn(y, rot, a * angle, amplitude, interleaved))
    m = (lambda y: y) if rot == 0 else (lambda y: turn(y, rot, angle, amplitude, interleaved, both=True))
    # r: 8 + 4 additions of squares, halved by the root, its instruction 2, share and eps 1; two
    # products; a rotation's cosine and sine 3 each (series 1, reduction 1, amplitude 1), two
    # products and a sum: 20 at most
    val, err = {"y": f(unit * W, 1.0) * live}, {"y": 24 * U32 * m((unit * W).abs()) * live}
    if dy is None:
        return val, err
    Y = torch.where(live, dy.double(), 0.0)
    u, um = f(Y, -1.0), m(Y.abs())
    e, em = u * W, um * (1.0 if w is None else w.double().abs())
    # the sum of a row's products: 8 + 4 additions of terms 20 off at most; what follows doubles it
    s, sm = (unit * e).sum(-1, keepdim=True), (unit.abs() * em).sum(-1, keepdim=True)
    val["dx"] = (r * (e - share * unit * s) if norm else u) * live
    err["dx"] = (80 * U32 * r * (em + share * unit.abs() * sm) if norm else 24 * U32 * um) * live
    if w is not None:
        # a thread's rows, 64 at most in these tests, then some 40 additions across threads
        val["dw"], err["dw"] = (unit * u).sum((0, 1, 2)), 150 * U32 * (unit.abs() * um).sum((0, 1, 2))
    return val, err


def check(got, val, err, label=""):
    """Every element within its bound: the fp32 one and, of a bf16 result, its own rounding."""
    bad = []
    for n, v in val.items():
        x = got[n]
        assert x.shape == v.shape, (label, n, x.shape, v.shape)
        assert torch.isfinite(x).all(), (label, n)
        lim = err[n] + 1e-30
        if x.dtype == torch.bfloat16:
            lim = lim * (1 + U16) + U16 * v.abs()
        if not v.numel():
            continue
        over = float(((x.double() - v).abs() / lim).max())
        print(f"{label} {n}: worst element at {over:.3f} of its bound", flush=True)
        if not over <= 1:
            bad.append((n, over))
    assert not bad, (label, bad)
