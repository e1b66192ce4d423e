"""Cases that measure the gated linear recurrence and the pass that brings queries and
keys to the operators: norms for each head and rotary positions.

scan         h_t = e^{g_t} h_{t-1} + w_t x_t for every channel, o_t = h_t, w_t = 1 or (coupled)
             1 - e^{g_t}, over whole sequences with ragged lengths (``gated_scan_fwd``)
scan_train   the same and its gradients (``gated_scan_fwd`` with saved states, ``gated_scan_bwd``)
scan_step    tokens of every sequence, the state updated in place (``gated_scan_recurrent_fwd``)
norm         queries and keys of a fused projection, normalised for each head (l2: by the length
             of the row; rms: by its root mean square, with weights), then rotated by position
             where the case has positions, laid out head by head (``qk_norm_fwd``)
norm_train   the same and its gradients (``qk_norm_fwd``, ``qk_norm_bwd``)
rotary       the rotation alone (``rotary_fwd``)
rotary_train the same and its gradients (``rotary_fwd``, ``rotary_bwd``)

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits
(angles in 64); with ``own`` true it calls the framework.  ``exact`` evaluates the
definitions in 64 bits.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the smallest sequence: one head of width 16, where only the call's latency counts
        {"name": "scan_one", "op": "scan", "B": 1, "H": 1, "T": 64, "d": 16, "dtype": "fp32", "coupled": False,
         "ragged": False, "h0": False},
        # one long document on one sequence: few channels, so the work has to be split over the steps
        {"name": "scan_long", "op": "scan", "B": 1, "H": 16, "T": 32768, "d": 128, "dtype": "bf16", "coupled": True,
         "ragged": False, "h0": True},
        # training at the widths and batch of the repository's headline workload
        {"name": "scan_train_batch", "op": "scan_train", "B": 8, "H": 16, "T": 4096, "d": 128, "dtype": "bf16",
         "coupled": True, "ragged": False, "h0": False},
        # full-precision training of odd widths and a padded batch that goes on from a state
        {"name": "scan_train_odd", "op": "scan_train", "B": 3, "H": 5, "T": 777, "d": 67, "dtype": "fp32",
         "coupled": False, "ragged": True, "h0": True},
        # serving: one token for each of 64 sequences
        {"name": "scan_step_batch", "op": "scan_step", "B": 64, "H": 16, "T": 1, "d": 128, "dtype": "bf16",
         "coupled": True},
        # serving: a few accepted tokens of one sequence, full precision
        {"name": "scan_step_few", "op": "scan_step", "B": 1, "H": 32, "T": 5, "d": 128, "dtype": "fp32",
         "coupled": False},
        # prompts of a padded batch on their way to the delta rule: unit queries and keys, no positions
        {"name": "norm_prompt_ragged", "op": "norm", "B": 8, "Hq": 16, "Hk": 16, "T": 4096, "d": 128, "rot": 0,
         "dtype": "bf16", "norm": "l2", "interleaved": False, "scaling": "none", "pos": "none", "ragged": True},
        # long-context training on the way to linear attention: rms with weights, halves rotated
        {"name": "norm_train_long", "op": "norm_train", "B": 1, "Hq": 32, "Hk": 32, "T": 32768, "d": 128, "rot": 128,
         "dtype": "bf16", "norm": "rms", "interleaved": False, "scaling": "linear", "pos": "none", "ragged": False},
        # serving: one token for each of 64 sequences, each at its own far position, fewer key heads
        {"name": "norm_step_batch", "op": "norm", "B": 64, "Hq": 16, "Hk": 4, "T": 1, "d": 128, "rot": 128,
         "dtype": "bf16", "norm": "rms", "interleaved": True, "scaling": "yarn", "pos": "start", "ragged": False},
        # a long prompt rotated with positions scaled beyond the trained length
        {"name": "rotary_prompt_long", "op": "rotary", "B": 1, "Hq": 32, "Hk": 32, "T": 32768, "d": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "scaling": "yarn", "pos": "none", "ragged": False},
        # full-precision training of odd, packed sequences, half of the head rotated in pairs of neighbours
        {"name": "rotary_train_part", "op": "rotary_train", "B": 3, "Hq": 5, "Hk": 5, "T": 777, "d": 64, "rot": 32,
         "dtype": "fp32", "interleaved": True, "scaling": "none", "pos": "each", "ragged": False},
        # serving: one token of one sequence
        {"name": "rotary_step_one", "op": "rotary", "B": 1, "Hq": 32, "Hk": 32, "T": 1, "d": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "scaling": "ntk", "pos": "start", "ragged": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan_train", "scan_step", "norm", "norm_train", "rotary", "rotary_train"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op.startswith("scan"):
        c["coupled"] = rng.random() < 0.5
        c["T"] = rng.choice([1, 1, 1, 2, 5]) if op == "scan_step" else _spread(rng, 1, 65536)
        n = _spread(rng, 1, max(1, min(262144, 67108864 // c["T"])))   # channels of all sequences
        c["d"] = min(n, rng.choice([16, 64, 67, 100, 128, 200, 1024, 2048]))
        n = max(1, n // c["d"])
        c["H"] = min(n, rng.choice([1, 1, 3, 8, 16]))
        c["B"] = max(1, n // c["H"])
        if op != "scan_step":
            c["ragged"] = rng.random() < 0.5
            c["h0"] = rng.random() < 0.5
        return c
    c["d"] = rng.choice([16, 32, 64, 128, 128])
    c["T"] = _spread(rng, 1, 32768)
    n = _spread(rng, 1, max(1, min(2048, 134217728 // (c["T"] * c["d"]))))   # heads of all sequences
    c["Hq"] = min(n, rng.choice([1, 3, 4, 8, 16, 32]))
    c["Hk"] = rng.choice([c["Hq"], c["Hq"], max(1, c["Hq"] // 4)])
    c["B"] = max(1, n // c["Hq"])
    c["interleaved"] = rng.random() < 0.5
    c["rot"] = 8 * rng.randint(1, c["d"] // 8) if rng.random() < 0.5 else c["d"]
    if op.startswith("norm"):
        c["norm"] = rng.choice(["l2", "rms"])
        if rng.random() < 0.3:
            c["rot"] = 0
    c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
    c["pos"] = rng.choice(["none", "start", "each"])
    c["ragged"] = rng.random() < 0.4
    return c


# ------------------------------------------------------------------ inputs


def _frequencies(rot, scaling):
    """Angle a position of each pair, fp64 [rot / 2], for contexts 8 times the trained 4096
    positions, and the factor of the rotated part."""
    base, factor, trained = 10000.0, 8.0, 4096
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":   # whole turns in the trained length: 32 and more stay, 1 and fewer are stretched
        keep = ((trained * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return f, 1.0


def prepare(case, seed):
    """Inputs on the GPU.  Log-gates -softplus(N(0,1)) / 16; queries and keys are slices of one
    projection's output [B, T, heads, d], two times normal; weights about 1."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    B, T, d, io = case["B"], case["T"], case["d"], IO[case["dtype"]]

    def normal(*dims):
        return torch.randn(dims, generator=gen, device="cuda")

    def uniform(*dims):
        return torch.rand(dims, generator=gen, device="cuda")

    s = {"case": case, "lens": None}
    if case.get("ragged"):
        lens = (uniform(B) * (T + 1)).to(torch.int32).clamp_max(T)
        lens[0] = T
        s["lens"] = lens
    if case["op"].startswith("scan"):
        H = case["H"]
        s["g"] = -torch.log1p(torch.exp(normal(B, H, T, d))) / 16
        s["x"] = normal(B, H, T, d).to(io)
        if case["op"] == "scan_step":
            s["state"] = normal(B, H, d)
            return s
        s["h0"] = normal(B, H, d) if case["h0"] else None
        if case["op"] == "scan_train":
            s["do"], s["dhT"] = normal(B, H, T, d).to(io), normal(B, H, d)
        return s
    Hq, Hk = case["Hq"], case["Hk"]
    both = (2 * normal(B, T, Hq + Hk, d)).to(io)
    s["q"], s["k"] = both[:, :, :Hq].transpose(1, 2), both[:, :, Hq:].transpose(1, 2)
    f, s["amplitude"] = _frequencies(case["rot"], case["scaling"]) if case["rot"] else (None, 1.0)
    s["freqs"] = None if f is None else f.cuda()
    s["pos"] = None
    if case["pos"] == "start":   # each sequence goes on behind what is in its state
        s["pos"] = (uniform(B) * 131072).to(torch.int32)
    elif case["pos"] == "each":   # packed documents: positions begin again every 300 steps
        s["pos"] = (torch.arange(T, device="cuda", dtype=torch.int32) % 300).expand(B, T).contiguous()
    s["wq"] = s["wk"] = None
    if case.get("norm") == "rms":
        s["wq"], s["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
    if case["op"].endswith("train"):
        s["dyq"], s["dyk"] = normal(B, Hq, T, d).to(io), normal(B, Hk, T, d).to(io)
    return s


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        from delta_rule_linear_gated_amd import binding as dn
        if op == "scan":
            o, hT, _ = dn.gated_scan_fwd(s["x"], s["g"], s["h0"], lens=s["lens"], coupled=c["coupled"], save_states=False)
            return {"o": o, "hT": hT}
        if op == "scan_train":
            o, hT, states = dn.gated_scan_fwd(s["x"], s["g"], s["h0"], lens=s["lens"], coupled=c["coupled"])
            gr = dn.gated_scan_bwd(s["x"], s["g"], s["h0"], s["do"], s["dhT"], states, lens=s["lens"],
                                   coupled=c["coupled"])
            return {"o": o, "hT": hT, **gr}
        if op == "scan_step":
            o = dn.gated_scan_recurrent_fwd(s["x"], s["g"], s["state"], coupled=c["coupled"])
            return {"o": o, "state": s["state"]}
        turn = dict(freqs=s["freqs"], pos=s["pos"] if c["rot"] else None, interleaved=c["interleaved"], amplitude=s["amplitude"],
                    lens=s["lens"])
        if op.startswith("norm"):
            turn.update(norm=c["norm"], eps=EPS)
            yq, yk = dn.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], **turn)
            if op == "norm":
                return {"yq": yq, "yk": yk}
            gr = dn.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], **turn)
            return {"yq": yq, "yk": yk, **{n: x for n, x in gr.items() if x is not None}}
        yq, yk = dn.rotary_fwd(s["q"], s["k"], **turn)
        if op == "rotary":
            return {"yq": yq, "yk": yk}
        dq, dk = dn.rotary_bwd(s["dyq"], s["dyk"], **turn)
        return {"yq": yq, "yk": yk, "dq": dq, "dk": dk}
    return {"scan": _scan, "scan_train": _scan, "scan_step": _scan_step}.get(op, _turn)(s)


# ------------------------------------------------------------------ plain form, 32 bits


def _along(a, b):
    """h_t = a_t h_{t-1} + b_t from zero, along dim 2: neighbours joined in pairs, the half as
    long recurrence of the pairs, then the steps between them."""
    n = a.shape[2]
    if n == 1:
        return b
    m = n // 2 * 2
    a0, a1, b0, b1 = a[:, :, 0:m:2], a[:, :, 1:m:2], b[:, :, 0:m:2], b[:, :, 1:m:2]
    odd = _along(a0 * a1, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[:, :, 1:m:2] = odd
    h[:, :, 0] = b[:, :, 0]
    h[:, :, 2::2] = a[:, :, 2::2] * odd[:, :, :(n - 1) // 2] + b[:, :, 2::2]
    return h


def _valid(lens, T):
    """True for the steps before a sequence's length, [B, 1, T, 1] (None: all are)."""
    return None if lens is None else (torch.arange(T, device="cuda") < lens[:, None])[:, None, :, None]


def _kept(ok, x, other=0.0):
    return x if ok is None else torch.where(ok, x, other)


def _scan(s):
    x, g, io = s["x"].float(), s["g"], s["x"].dtype
    ok = _valid(s["lens"], x.shape[2])
    g, x = _kept(ok, g), _kept(ok, x)
    a = torch.exp(g)
    w = -torch.expm1(g) if s["case"]["coupled"] else torch.ones_like(g)
    b = w * x
    first = torch.zeros_like(b[:, :, 0]) if s["h0"] is None else s["h0"]
    b[:, :, 0] += a[:, :, 0] * first
    h = _along(a, b)
    out = {"o": _kept(ok, h).to(io), "hT": h[:, :, -1].clone()}
    if s["case"]["op"] == "scan":
        return out
    do = _kept(ok, s["do"].float()).clone()
    do[:, :, -1] += s["dhT"]
    after = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], 2)
    D = _along(after.flip(2), do.flip(2)).flip(2)
    before = torch.cat([first[:, :, None], h[:, :, :-1]], 2)
    if s["case"]["coupled"]:
        before = before - x
    out["dx"] = _kept(ok, w * D).to(io)
    out["dg"] = _kept(ok, a * D * before)
    out["dh0"] = a[:, :, 0] * D[:, :, 0]
    return out


def _scan_step(s):
    x, g, h = s["x"].float(), s["g"], s["state"]
    a = torch.exp(g)
    b = x * -torch.expm1(g) if s["case"]["coupled"] else x.clone()
    b[:, :, 0] += a[:, :, 0] * h
    o = _along(a, b)
    h.copy_(o[:, :, -1])
    return {"o": o.to(s["x"].dtype), "state": h}


def _angles(s, T):
    """cos and sin of every position, [B or 1, 1, T, rot / 2]: angles in 64 bits."""
    t = torch.arange(T, device="cuda", dtype=torch.float64)[None]
    if s["pos"] is not None:
        t = s["pos"].double() if s["pos"].dim() == 2 else s["pos"].double()[:, None] + t
    a = (t[..., None] * s["freqs"])[:, None]
    return (a.cos() * s["amplitude"]).float(), (a.sin() * s["amplitude"]).float()


def _rotate(s, x, cos, sin):
    rot = s["case"]["rot"]
    y = x.clone()
    if s["case"]["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - v * sin, v * cos + u * sin
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - v * sin, v * cos + u * sin
    return y


def _turn(s):
    c, out = s["case"], {}
    T, d, io, norm = c["T"], c["d"], s["q"].dtype, c.get("norm")
    ok = _valid(s["lens"], T)
    cos, sin = _angles(s, T) if c["rot"] else (None, None)
    share = 1.0 if norm == "l2" else 1.0 / d
    for n in ("q", "k"):
        x, w = _kept(ok, s[n].float()), s["w" + n]
        if norm:
            r = torch.rsqrt((x * x).sum(-1, keepdim=True) * share + EPS)
            unit = x * r
        else:
            unit = x
        y = unit if w is None else unit * w
        out["y" + n] = _kept(ok, _rotate(s, y, cos, sin) if c["rot"] else y).to(io)
        if not c["op"].endswith("train"):
            continue
        u = _kept(ok, s["dy" + n].float())
        if c["rot"]:
            u = _rotate(s, u, cos, -sin)
        if w is not None:
            out["dw" + n] = (unit * u).sum((0, 1, 2))
            u = u * w
        if norm:
            u = r * (u - unit * (unit * u).sum(-1, keepdim=True) * share)
        out["d" + n] = _kept(ok, u).to(io)
    return out


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_scan(s, c):
    B, H, T, d = s["x"].shape
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"].long()
    start = s["state"] if c["op"] == "scan_step" else s["h0"]
    h = torch.zeros(B, H, d, dtype=torch.float64, device="cuda") if start is None else start.double()
    hs = torch.zeros(B, H, T + 1, d, dtype=torch.float64, device="cuda")
    hs[:, :, 0] = h
    for t in range(T):
        g, x = s["g"][:, :, t].double(), s["x"][:, :, t].double()
        new = g.exp() * h + (x * -g.expm1() if c["coupled"] else x)
        h = new if s["lens"] is None else torch.where((t < lens)[:, None, None], new, h)
        hs[:, :, t + 1] = h
    live = (torch.arange(T, device="cuda") < lens[:, None])[:, None, :, None]
    o = hs[:, :, 1:] * live
    if c["op"] == "scan_step":
        return {"o": o, "state": h}
    out = {"o": o, "hT": h}
    if c["op"] == "scan":
        return out
    D = s["dhT"].double()
    Ds = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")   # cotangent of each step's state
    for t in range(T - 1, -1, -1):
        on = (t < lens)[:, None, None]
        total = D + s["do"][:, :, t].double()
        Ds[:, :, t] = torch.where(on, total, 0.0)
        D = torch.where(on, s["g"][:, :, t].double().exp() * total, D)
    g = s["g"].double()
    out["dx"] = Ds * -g.expm1() if c["coupled"] else Ds
    out["dg"] = Ds * g.exp() * (hs[:, :, :-1] - (s["x"].double() if c["coupled"] else 0.0))
    out["dh0"] = D
    return out


def _exact_rows(s, c, n):
    """One of q and k: rotations as complex factors, rows whole."""
    x = s[n].double()
    B, H, T, d = x.shape
    rot, norm = c["rot"], c.get("norm")
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"].long()
    live = (torch.arange(T, device="cuda") < lens[:, None])[:, None, :, None].double()

    def turned(y, way):
        if not rot:
            return y
        p = torch.arange(T, device="cuda").expand(B, T).double()
        if s["pos"] is not None:
            p = s["pos"].double() if s["pos"].dim() == 2 else p + s["pos"].double()[:, None]
        f = torch.polar(torch.full_like(p, s["amplitude"])[..., None], way * p[..., None] * s["freqs"])[:, None]
        z = y[..., :rot]
        z = z.reshape(B, H, T, rot // 2, 2) if c["interleaved"] else z.reshape(B, H, T, 2, rot // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * f)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(B, H, T, rot), y[..., rot:]], -1)

    w = 1.0 if s["w" + n] is None else s["w" + n].double()
    size = 1.0
    if norm:
        size = ((x.square().sum(-1, keepdim=True) if norm == "l2" else x.square().mean(-1, keepdim=True)) + EPS).sqrt()
    out = {"y" + n: turned(x / size * w, 1.0) * live}
    if not c["op"].endswith("train"):
        return out
    u = turned(s["dy" + n].double(), -1.0) * live
    if s["w" + n] is not None:
        out["dw" + n] = (x / size * u).flatten(0, 2).sum(0)
    e = u * w
    if norm:
        share = 1.0 if norm == "l2" else 1.0 / d
        e = e / size - x * (x * e).sum(-1, keepdim=True) * share / size ** 3
    out["d" + n] = e
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("scan"):
        return _exact_scan(s, case)
    return {**_exact_rows(s, case, "q"), **_exact_rows(s, case, "k")}


# ------------------------------------------------------------------ work


def work(case):
    """Bytes: each input read once and each output written once.  Operations: of the
    definitions, an exponential, root or rotation factor as one."""
    B, T, d, op = case["B"], case["T"], case["d"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("scan"):
        rows = B * case["H"] * d
        n = rows * T
        if op == "scan_step":
            return {"bytes": (2 * e + 4) * n + 8 * rows, "flops": 5 * n}
        ends = 4 * rows * (2 if case["h0"] else 1)
        if op == "scan":
            return {"bytes": (2 * e + 4) * n + ends, "flops": 5 * n}
        return {"bytes": (2 * e + 4) * n + ends + (3 * e + 8) * n + 8 * rows, "flops": 13 * n}
    n = B * (case["Hq"] + case["Hk"]) * T * d
    turn = 3 * n * case["rot"] / d
    some = 4 * B * T + 8 * case["rot"]
    if op in ("norm", "rotary"):
        return {"bytes": 2 * e * n + some, "flops": (4 * n if op == "norm" else 0) + turn}
    if op == "rotary_train":   # the backward reads the cotangents alone
        return {"bytes": 4 * e * n + 2 * some, "flops": 2 * turn}
    return {"bytes": 5 * e * n + 2 * some, "flops": 13 * n + 2 * turn}
