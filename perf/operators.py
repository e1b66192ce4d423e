"""Cases that measure the linear-attention and draft-tree operators.

Five operators, on the layouts of ``include/dn.h``:

prompt  linear attention with a decay per head over whole prompts (``linear_fwd``):
        S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t, from h0, with ragged lengths
train   the same and its gradients (``linear_fwd`` then ``linear_bwd``)
step    one token for each sequence, the state updated in place (``linear_recurrent_fwd``)
verify  the nodes of a tree of drafted tokens, each read from the state that its path
        from the root leaves (``tree_fwd``: the gated delta rule, or linear attention)
commit  the state moved along the accepted path (``tree_commit``), in place

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits
(chunks of 64 for the long axis, no Python loop over steps); with ``own`` true it calls
the framework.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the smallest prompt: one head of width 16, where only the call's latency counts
        {"name": "prompt_one_chunk", "op": "prompt", "B": 1, "H": 1, "T": 64, "dk": 16, "dv": 16, "dtype": "fp32",
         "gate": "none", "ragged": False, "h0": False},
        # a padded batch of prompts of different lengths, each going on from a cached state
        {"name": "prompt_batch_ragged", "op": "prompt", "B": 8, "H": 16, "T": 4096, "dk": 128, "dv": 128,
         "dtype": "bf16", "gate": "head", "ragged": True, "h0": True},
        # one long document on a layer of few heads: the work has to be split over the steps
        {"name": "prompt_few_heads_long", "op": "prompt", "B": 1, "H": 4, "T": 32768, "dk": 128, "dv": 128,
         "dtype": "bf16", "gate": "scalar", "ragged": False, "h0": True},
        # training at the widths and batch of the repository's headline workload, gate learned per step
        {"name": "train_batch", "op": "train", "B": 8, "H": 16, "T": 4096, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "scalar", "ragged": False, "h0": False},
        # long-context training, constant decays
        {"name": "train_long", "op": "train", "B": 1, "H": 32, "T": 32768, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "head", "ragged": False, "h0": True},
        # full-precision training of odd, ragged sizes with values wider than keys
        {"name": "train_fp32_odd", "op": "train", "B": 3, "H": 5, "T": 777, "dk": 64, "dv": 128, "dtype": "fp32",
         "gate": "scalar", "ragged": True, "h0": True},
        # serving: one token for each of 64 sequences
        {"name": "step_batch", "op": "step", "B": 64, "H": 16, "T": 1, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "scalar"},
        # serving: one token for one sequence
        {"name": "step_one", "op": "step", "B": 1, "H": 32, "T": 1, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "head"},
        # speculative decoding of a serving batch: 16 drafted tokens for each sequence
        {"name": "verify_batch", "op": "verify", "B": 64, "H": 16, "T": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "scalar", "delta": True, "ragged": False},
        # wide trees with a gate per key channel, fewer nodes in some sequences
        {"name": "verify_wide_channels", "op": "verify", "B": 16, "H": 16, "T": 61, "dk": 128, "dv": 128,
         "dtype": "bf16", "gate": "vector", "delta": True, "ragged": True},
        # the accepted paths of the batch written into the states
        {"name": "commit_batch", "op": "commit", "B": 64, "H": 16, "T": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "gate": "scalar"},
        # one sequence, full precision, a gate per channel
        {"name": "commit_one", "op": "commit", "B": 1, "H": 16, "T": 33, "dk": 64, "dv": 64, "dtype": "fp32",
         "gate": "vector"},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "train", "step", "verify", "commit"])
    d = [16, 32, 64, 128, 128]
    c = {"op": op, "dk": rng.choice(d), "dv": rng.choice(d), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("prompt", "train"):
        c["T"] = _spread(rng, 1, 8192)
        bh = _spread(rng, 1, max(1, min(256, 262144 // c["T"])))
        c["H"] = min(bh, rng.choice([1, 3, 4, 8, 16, 32]))
        c["B"] = max(1, bh // c["H"])
        c["gate"] = rng.choice(["none", "head", "scalar", "scalar"])
        c["ragged"] = rng.random() < 0.5
        c["h0"] = rng.random() < 0.5
    else:
        bh = _spread(rng, 1, 1024)
        c["H"] = min(bh, rng.choice([1, 3, 4, 8, 16, 32]))
        c["B"] = max(1, bh // c["H"])
        if op == "step":
            c["T"] = rng.choice([1, 1, 1, 2, 5])
            c["gate"] = rng.choice(["none", "head", "scalar"])
        else:
            c["T"] = _spread(rng, 1, 64 if c["B"] * c["H"] <= 256 else 24)
            c["gate"] = rng.choice(["none", "head", "scalar", "vector"])
        if op == "verify":
            c["delta"] = rng.random() < 0.7
            c["ragged"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    """Inputs on the GPU: unit queries and keys, normal values, sigmoid step sizes,
    log-decays -softplus(N(0,1)) / 16 (per step or channel) or one in 1/512 .. 1/4 per head."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    B, H, T, dk, dv, io = case["B"], case["H"], case["T"], case["dk"], case["dv"], IO[case["dtype"]]

    def normal(*dims):
        return torch.randn(dims, generator=gen, device="cuda")

    def uniform(*dims):
        return torch.rand(dims, generator=gen, device="cuda")

    def unit(*dims):
        x = normal(*dims)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)).to(io)

    s = {"case": case, "k": unit(B, H, T, dk), "lens": None}
    if case["gate"] == "none":
        s["g"] = None
    elif case["gate"] == "head":
        s["g"] = -torch.exp(math.log(1 / 512) + uniform(H) * math.log(128.0))
    else:
        dims = (B, H, T) + ((dk,) if case["gate"] == "vector" else ())
        s["g"] = -torch.log1p(torch.exp(normal(*dims))) / 16
    if case.get("ragged"):
        lens = (uniform(B) * (T + 1)).to(torch.int32).clamp_max(T)
        lens[0] = T
        s["lens"] = lens
    if case["op"] == "commit":
        s["u"] = normal(B, H, T, dv)
    else:
        s["q"] = unit(B, H, T, dk)
        s["v"] = normal(B, H, T, dv).to(io)
    if case["op"] in ("prompt", "train"):
        s["h0"] = 0.5 * normal(B, H, dv, dk) if case["h0"] else None
        if case["op"] == "train":
            s["do"] = normal(B, H, T, dv).to(io)
            s["dhT"] = normal(B, H, dv, dk)
    else:
        s["state"] = 0.5 * normal(B, H, dv, dk)
    if case["op"] in ("verify", "commit"):
        # node n hangs on one of the 4 nodes before it, or on the root
        n = torch.arange(T, device="cuda", dtype=torch.int32)
        back = 1 + (uniform(B, T) * 4).to(torch.int32).clamp_max(3)
        s["parent"] = (n - back).clamp_min(-1).contiguous()
        s["accept"] = (uniform(B) * (T + 1)).to(torch.int32).clamp_max(T) - 1
        if case["op"] == "verify":
            s["beta"] = torch.sigmoid(normal(B, H, T)) if case["delta"] else None
    return s


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from delta_rule_linear_gated_amd import binding as dn
        if op == "prompt":
            o, hT = dn.linear_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], lens=s["lens"])
            return {"o": o, "hT": hT}
        if op == "train":
            o, hT = dn.linear_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], lens=s["lens"])
            gr = dn.linear_bwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["do"], s["dhT"], lens=s["lens"])
            return {"o": o, "hT": hT, **{n: x for n, x in gr.items() if x is not None}}
        if op == "step":
            o = dn.linear_recurrent_fwd(s["q"], s["k"], s["v"], s["g"], s["state"])
            return {"o": o, "state": s["state"]}
        if op == "verify":
            o, u = dn.tree_fwd(s["q"], s["k"], s["v"], s["beta"], s["g"], s["parent"], s["state"], counts=s["lens"])
            return {"o": o, "u": u}
        dn.tree_commit(s["k"], s["u"], s["g"], s["parent"], s["accept"], s["state"])
        return {"state": s["state"]}
    return {"prompt": _prompt, "train": _train, "step": _step, "verify": _verify, "commit": _commit}[op](s)


# ------------------------------------------------------------------ plain form, 32 bits


def _gates(s, like):
    """Log-decay of every step, [B, H, T] in 64 bits (0 without a gate)."""
    g = s["g"]
    if g is None:
        return torch.zeros(like.shape[:3], dtype=torch.float64, device=like.device)
    g = g.double()
    return g[None, :, None].expand(like.shape[:3]) if g.dim() == 1 else g


def _valid(s, like):
    """1 for the steps before a sequence's length, [B, 1, T, 1]."""
    B, _, T = like.shape[:3]
    if s["lens"] is None:
        return torch.ones(B, 1, T, 1, device=like.device)
    return (torch.arange(T, device=like.device)[None, :] < s["lens"][:, None]).float()[:, None, :, None]


def _chunks(x, fill=0.0):
    """[B, H, T, ...] padded to whole chunks, [B, H, NT, CHUNK, ...]."""
    T = x.shape[2]
    NT = -(-T // CHUNK)
    pad = torch.full((*x.shape[:2], NT * CHUNK - T, *x.shape[3:]), fill, dtype=x.dtype, device=x.device)
    return torch.cat([x, pad], 2).reshape(*x.shape[:2], NT, CHUNK, *x.shape[3:])


def _attend(x, y, z, g, s0):
    """out_i = sum_{j <= i} e^{G_i - G_j} (x_i . y_j) z_j + e^{G_i} s0 x_i over chunked inputs
    (g in 64 bits).  Returns out, its part from earlier chunks, the states entering the
    chunks and the last state (rows over z's channels)."""
    B, H, NT = x.shape[:3]
    G = g.cumsum(-1)                                     # in the chunk
    tot = G[..., -1]
    end = tot.cumsum(-1)                                 # up to and with each chunk
    start = end - tot
    low = torch.ones(CHUNK, CHUNK, device=x.device).tril() > 0
    w = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp_max(700), -math.inf).exp().float()
    intra = ((x @ y.transpose(-1, -2)) * w) @ z
    add = (z * (tot[..., None] - G).exp().float()[..., None]).transpose(-1, -2) @ y
    before = torch.ones(NT, NT, device=x.device).tril(-1) > 0
    a = torch.where(before, start[..., :, None] - end[..., None, :], -math.inf).exp().float()
    states = (a @ add.flatten(-2)).reshape(add.shape)
    if s0 is not None:
        states = states + start.exp().float()[..., None, None] * s0[:, :, None]
    last = tot[..., -1].exp().float()[..., None, None] * states[:, :, -1] + add[:, :, -1]
    inter = G.exp().float()[..., None] * (x @ states.transpose(-1, -2))
    return intra + inter, inter, states, last


def _unchunk(x, T):
    return x.flatten(2, 3)[:, :, :T]


def _inputs(s):
    ok = _valid(s, s["k"])
    q, k, v = (_chunks(s[n].float() * ok) for n in ("q", "k", "v"))
    return q, k, v, _chunks(_gates(s, s["k"]) * ok[..., 0].double()), ok


def _prompt(s):
    q, k, v, g, _ = _inputs(s)
    o, _, _, last = _attend(q, k, v, g, s["h0"])
    return {"o": _unchunk(o, s["q"].shape[2]).to(s["q"].dtype), "hT": last}


def _flip(x):
    return x.flip(2, 3)


def _train(s):
    io, T = s["q"].dtype, s["q"].shape[2]
    q, k, v, g, ok = _inputs(s)
    do = _chunks(s["do"].float() * ok)
    h0, dhT = s["h0"], s["dhT"]
    o, _, _, hT = _attend(q, k, v, g, h0)
    h0t = None if h0 is None else h0.transpose(-1, -2)
    dq, dq_in, S, _ = _attend(do, v, k, g, h0t)          # S: [dk, dv] for each chunk
    # from the last step back: the gate of a step follows it
    flat = g.flatten(2)
    nxt = torch.cat([flat[:, :, 1:], torch.zeros_like(flat[:, :, :1])], 2)
    gr = nxt.flip(2).reshape(g.shape)
    dv, dv_in, D, dl = _attend(_flip(k), _flip(q), _flip(do), gr, dhT)
    dk, _, _, _ = _attend(_flip(v), _flip(do), _flip(q), gr, dhT.transpose(-1, -2))
    dv, dv_in, dk, D = _flip(dv), _flip(dv_in), _flip(dk), D.flip(2)
    out = {"o": _unchunk(o, T).to(io), "hT": hT, "dq": _unchunk(dq, T).to(io), "dk": _unchunk(dk, T).to(io),
           "dv": _unchunk(dv, T).to(io), "dh0": dl * flat[:, :, 0].exp().float()[..., None, None]}
    if s["g"] is not None and s["g"].dim() == 3:
        # pairs j < t <= i: both in the chunk, i in it, j in it, neither
        G = g.cumsum(-1)
        low = torch.ones(CHUNK, CHUNK, device=q.device).tril() > 0
        w = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp_max(700), -math.inf).exp()
        e = w * (q @ k.transpose(-1, -2)).double() * (do @ v.transpose(-1, -2)).double()
        inside = torch.where(low, e.cumsum(-1) - e, 0.0).sum(-2)
        a = (q * dq_in).sum(-1).double()
        b = (v * dv_in).sum(-1).double()
        both = (G[..., -1] + nxt.reshape(g.shape)[..., -1]).exp() * (S.transpose(-1, -2) * D).sum((-1, -2), dtype=torch.float64)
        dg = inside + a.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + both[..., None]
        out["dg"] = _unchunk(dg, T).float() * ok[..., 0]
    return out


def _step(s):
    q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    if q.shape[2] == 1:
        if s["g"] is not None:
            S.mul_(torch.exp(s["g"]).reshape(-1, S.shape[1], 1, 1))
        S.add_(v[:, :, 0, :, None] * k[:, :, 0, None, :])
        o = (S * q[:, :, 0, None, :]).sum(-1)[:, :, None]
    else:   # a few tokens: one short chunk
        o, _, _, last = _attend(_chunks(q), _chunks(k), _chunks(v), _chunks(_gates(s, k)), S)
        o = _unchunk(o, q.shape[2])
        S.copy_(last)
    return {"o": o.to(s["q"].dtype), "state": S}


def _nilpotent_inverse(a):
    """(I - a)^-1 for a strictly lower triangular a: (I + a)(I + a^2)(I + a^4)..."""
    r = torch.eye(a.shape[-1], dtype=a.dtype, device=a.device) + a
    for _ in range(max(0, a.shape[-1] - 1).bit_length() - 1):
        a = a @ a
        r = r + r @ a
    return r


def _paths(s):
    """[B, N, N]: 1 where the column is on the row's path (the row itself included)."""
    parent = s["parent"]
    n = torch.arange(parent.shape[1], device=parent.device)
    return _nilpotent_inverse((parent[..., None] == n).float())


def _path_gates(s, k, path):
    """Log-decay from the root to each node: [B, H, N, 1 or dk] in 64 bits."""
    g = s["g"]
    g = (g if g is not None and g.dim() == 4 else _gates(s, k)[..., None]).double()
    return path[:, None].double() @ g


def _verify(s):
    io, S = s["q"].dtype, s["state"]
    ok = _valid(s, s["k"])
    q, k, v = (s[n].float() * ok for n in ("q", "k", "v"))
    path = _paths(s)
    G = _path_gates(s, k, path)
    on = (path > 0)[:, None]
    if G.shape[-1] == 1:
        w = torch.where(on, G - G.transpose(-1, -2), -math.inf).exp().float()
        P, A = (q @ k.transpose(-1, -2)) * w, (k @ k.transpose(-1, -2)) * w
    else:
        w = torch.where(on[..., None], G.float()[:, :, :, None] - G.float()[:, :, None], -math.inf).exp()
        w = w * k[:, :, None]
        P, A = (w @ q[..., None])[..., 0], (w @ k[..., None])[..., 0]
    scale = G.exp().float()
    St = S.transpose(-1, -2)
    if s["beta"] is None:
        u = v
    else:
        b = s["beta"][..., None]
        u = _nilpotent_inverse(-b * (A - torch.diag_embed(A.diagonal(dim1=-2, dim2=-1)))) @ (b * (v - (k * scale) @ St))
    o = (q * scale) @ St + P @ u
    return {"o": (o * ok).to(io), "u": u * ok}


def _commit(s):
    k, S, at = s["k"].float(), s["state"], s["accept"]
    path = _paths(s)
    some = (at >= 0)
    row = at.clamp_min(0).long()
    on = path.gather(1, row[:, None, None].expand(-1, 1, path.shape[-1]))[:, 0] * some[:, None]     # [B, N]
    G = _path_gates(s, k, path)
    Ge = G.gather(2, row[:, None, None, None].expand(-1, G.shape[1], 1, G.shape[-1])) * some[:, None, None, None]
    w = torch.where(on[:, None, :, None] > 0, Ge - G, -math.inf).exp().float()
    S.copy_(S * Ge.exp().float() + s["u"].transpose(-1, -2) @ (k * w))
    return {"state": S}


# ------------------------------------------------------------------ definitions in 64 bits


def _step_gates64(s, b, h, n):
    """Log-decays of n steps of one head."""
    g = s["g"]
    if g is None:
        return torch.zeros(n, dtype=torch.float64, device="cuda")
    return g[h].double().expand(n) if g.dim() == 1 else g[b, h, :n].double()


def _exact_sequences(s, grads):
    """Every head by the full matrices of pairs of steps."""
    B, H, T, dk = s["q"].shape
    dv = s["v"].shape[-1]
    like = {"o": (T, dv), "hT": (dv, dk)}
    if grads:
        like.update(dq=(T, dk), dk=(T, dk), dv=(T, dv), dh0=(dv, dk))
        if s["g"] is not None and s["g"].dim() == 3:
            like["dg"] = (T,)
    out = {n: torch.zeros((B, H) + d, dtype=torch.float64, device="cuda") for n, d in like.items()}
    for b in range(B):
        n = T if s["lens"] is None else int(s["lens"][b])
        for h in range(H):
            h0 = s["h0"][b, h].double() if s["h0"] is not None else torch.zeros(dv, dk, dtype=torch.float64,
                                                                                device="cuda")
            if n == 0:
                out["hT"][b, h] = h0
                if grads:
                    out["dh0"][b, h] = s["dhT"][b, h].double()
                continue
            q, k, v = (s[m][b, h, :n].double() for m in ("q", "k", "v"))
            c = _step_gates64(s, b, h, n).cumsum(0)
            decay = (c[:, None] - c[None, :]).tril_().exp_().tril_()
            grow, left = c.exp()[:, None], (c[-1] - c).exp()[:, None]
            p = (q @ k.T).mul_(decay)
            out["o"][b, h, :n] = p @ v + grow * (q @ h0.T)
            out["hT"][b, h] = hT = (left * v).T @ k + c[-1].exp() * h0
            if not grads:
                continue
            do, dhT = s["do"][b, h, :n].double(), s["dhT"][b, h].double()
            dp = (do @ v.T).mul_(decay)
            dq = dp @ k + grow * (do @ h0)
            dkk = dp.T @ q + left * (v @ dhT)
            out["dq"][b, h, :n], out["dk"][b, h, :n] = dq, dkk
            out["dv"][b, h, :n] = p.T @ do + left * (k @ dhT.T)
            out["dh0"][b, h] = (grow * do).T @ q + c[-1].exp() * dhT
            if "dg" in out:
                dc = (q * dq).sum(-1) - (k * dkk).sum(-1)
                dc[-1] += (hT * dhT).sum()
                out["dg"][b, h, :n] = dc.flip(0).cumsum(0).flip(0)
                if s["h0"] is None:
                    out["dg"][b, h, 0] = 0   # the first gate decays nothing: exactly zero
    return out


def _node_gate64(s, n):
    """Decay factor of node or step n, broadcast over [B, H, dv, dk]."""
    g = s["g"]
    if g is None:
        return 1.0
    if g.dim() == 1:
        return g.double().exp()[None, :, None, None]
    return g[:, :, n].double().exp()[..., None, None] if g.dim() == 3 else g[:, :, n].double().exp()[:, :, None, :]


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op in ("prompt", "train"):
        return _exact_sequences(s, op == "train")
    S = s["state"].double()
    k = s["k"].double()
    if op == "step":
        outs = []
        for t in range(T):
            S = S * _node_gate64(s, t) + s["v"][:, :, t].double()[..., None] * k[:, :, t, None]
            outs.append((S @ s["q"][:, :, t].double()[..., None])[..., 0])
        return {"o": torch.stack(outs, 2), "state": S}
    parent = s["parent"].long()
    rows = torch.arange(case["B"], device="cuda")
    if op == "commit":
        # up from the accepted node: each node's write, decayed by the nodes below it
        at, decay, add = s["accept"].long(), 1.0, torch.zeros_like(S)
        for n in range(T - 1, -1, -1):
            hit = (at == n)[:, None, None, None]
            add = torch.where(hit, add + s["u"][:, :, n].double()[..., None] * (k[:, :, n, None] * decay), add)
            decay = torch.where(hit, decay * torch.ones_like(S) * _node_gate64(s, n), decay * torch.ones_like(S))
            at = torch.where(at == n, parent[:, n], at)
        return {"state": S * decay + add}
    states = [S]                       # states[0]: the root; states[n + 1]: after node n
    outs, us = [], []
    ok = _valid(s, s["k"]).double()
    for n in range(T):
        before = torch.stack(states)[parent[:, n] + 1, rows] * _node_gate64(s, n)
        u = s["v"][:, :, n].double()
        if s["beta"] is not None:
            u = s["beta"][:, :, n].double()[..., None] * (u - (before @ k[:, :, n, :, None])[..., 0])
        states.append(before + u[..., None] * k[:, :, n, None])
        outs.append((states[-1] @ s["q"][:, :, n].double()[..., None])[..., 0])
        us.append(u)
    return {"o": torch.stack(outs, 2) * ok, "u": torch.stack(us, 2) * ok}


# ------------------------------------------------------------------ work


def work(case):
    """Bytes: each input read once and each output written once.  Operations: the
    products of the chunked form (pairs inside a chunk of 64, states between chunks) or,
    for steps and trees, of the state with every token."""
    B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "dk", "dv"))
    e = 2 if case["dtype"] == "bf16" else 4
    bh, op = B * H, case["op"]
    n = bh * T
    gate = {"none": 0, "head": 0, "scalar": 4 * n, "vector": 4 * n * dk}[case["gate"]]
    state = 4 * bh * dv * dk
    if op in ("prompt", "train"):
        pairs = min(T, CHUNK) / 2
        flops = 2 * n * (pairs * (dk + dv) + 2 * dk * dv)
        byt = e * n * (2 * dk + 2 * dv) + gate + state * (2 if case["h0"] else 1)
        if op == "train":
            flops += 2 * n * (pairs * (3 * dk + 2 * dv) + 5 * dk * dv)
            byt += e * n * (4 * dk + 3 * dv) + 2 * gate + state * (3 if case["h0"] else 2)
        return {"bytes": byt, "flops": flops}
    if op == "step":
        return {"bytes": 2 * state + e * n * (2 * dk + 2 * dv) + gate, "flops": 4 * n * dk * dv}
    if op == "verify":
        delta = 1 if case["delta"] else 0
        return {"bytes": state + e * n * (2 * dk + 2 * dv) + 4 * n * dv + 4 * n * delta + gate,
                "flops": 2 * n * ((1 + delta) * dk * dv + (T / 2) * (1 + delta) * (dk + dv))}
    return {"bytes": 2 * state + e * n * dk + 4 * n * dv + gate, "flops": 2 * n * dk * dv}
