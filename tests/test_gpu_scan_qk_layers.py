"""The gated recurrence and the norms and rotations where a model has them: in front of the delta
rule and linear attention, through autograd against the same layers in 64 bits, and from a
prompt to single tokens."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

pytestmark = pytest.mark.gpu


def plain_scan(x, g):
    h, out = torch.zeros_like(x[:, :, 0]), []
    for t in range(x.shape[2]):
        h = g[:, :, t].exp() * h - torch.expm1(g[:, :, t]) * x[:, :, t]
        out.append(h)
    return torch.stack(out, 2)


def plain_norm(x, w, share):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) * share + 1e-6) * w


def plain_turn(x, f):
    a = torch.arange(x.shape[2], device=x.device, dtype=torch.float64)[:, None] * f
    c, s = a.cos().to(x.dtype), a.sin().to(x.dtype)
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * s, v * c + u * s], -1)


def plain_mix(q, k, v, beta, g):
    """The delta rule (beta None: linear attention), step by step."""
    S, out = torch.zeros(*q.shape[:2], v.shape[-1], q.shape[-1], dtype=q.dtype, device=q.device), []
    for t in range(q.shape[2]):
        S = S * g[:, :, t].exp()[..., None, None]
        new = v[:, :, t] if beta is None else beta[:, :, t, None] * (v[:, :, t] - (S @ k[:, :, t, :, None])[..., 0])
        S = S + new[..., None] * k[:, :, t, None, :]
        out.append((S @ q[:, :, t, :, None])[..., 0])
    return torch.stack(out, 2)


def layer(p, own, delta, f):
    """A gated recurrence over the channels, a fused projection to queries, keys and values, the norm
    (and rotation) of queries and keys, then the delta rule or linear attention."""
    x, g = p["x"], p["g"]
    h = B.GatedScan.apply(x, g, None, None, True, False)[0] if own else plain_scan(x, g)
    Bn, _, T, _ = h.shape
    qkv = (h[:, 0] @ p["proj"]).view(Bn, T, 3, 2, 32)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    beta = torch.sigmoid(p["beta"]) if delta else None
    gate = -torch.nn.functional.softplus(p["gate"]) / 8
    if own:
        q, k = B.QKNorm.apply(q, k, *((None, None) if delta else (p["wq"], p["wk"])), "l2" if delta else "rms", 1e-6,
                              None if delta else f)
        v = v.contiguous()
        if delta:
            return B.DeltaRule.apply(q, k, v, beta, gate, None, 16)[0]
        return B.LinearAttention.apply(q, k, v, gate)[0]
    one = torch.ones((), dtype=q.dtype, device=q.device)
    q = plain_norm(q, one if delta else p["wq"], 1.0 if delta else 1 / 32)
    k = plain_norm(k, one if delta else p["wk"], 1.0 if delta else 1 / 32)
    if not delta:
        q, k = plain_turn(q, f), plain_turn(k, f)
    return plain_mix(q, k, v, beta, gate)


@pytest.mark.parametrize("delta", [True, False])
def test_a_layer_and_its_gradients(delta):
    gen = torch.Generator().manual_seed(7)

    def normal(*s):
        return torch.randn(s, generator=gen)

    Bn, T = 2, 50
    p = dict(x=normal(Bn, 1, T, 48), g=-torch.nn.functional.softplus(normal(Bn, 1, T, 48)) / 4, proj=normal(48, 192) / 7,
             beta=normal(Bn, 2, T), gate=normal(Bn, 2, T), wq=1 + 0.1 * normal(32), wk=1 + 0.1 * normal(32))
    f, _ = B.rotary_freqs(32, device="cuda")
    do = normal(Bn, 2, T, 32).cuda()
    got, want = ({n: t.to("cuda", dt).requires_grad_() for n, t in p.items()} for dt in (torch.float32, torch.float64))
    a, b = layer(got, True, delta, f), layer(want, False, delta, f)
    used = [n for n in p if n not in (("wq", "wk") if delta else ("beta",))]
    ga = torch.autograd.grad((a * do).sum(), [got[n] for n in used])
    gb = torch.autograd.grad((b * do.double()).sum(), [want[n] for n in used])
    # fp32 all along: a few hundred roundings of 2^-24 on the longest way, norms of the whole
    for n, x, y in (("o", a.detach(), b.detach()), *zip(used, ga, gb)):
        rel = float((x.double() - y).norm() / y.norm())
        print(n, f"{rel:.2e}", flush=True)
        assert rel <= 400 * 2.0 ** -24, (n, rel)


def test_a_prompt_then_tokens():
    """Serving: the prompt through the chunked forms, then token by token at its positions, against the
    whole sequence at once; sequences of different lengths."""
    gen = torch.Generator().manual_seed(8)
    Bn, H, T, d, cut = 2, 2, 90, 32, 80
    both = torch.randn(Bn, T, 3, H, d, generator=gen).cuda()
    q, k, v = (both[:, :, i].transpose(1, 2) for i in range(3))
    g = -torch.rand(Bn, H, T, generator=gen).cuda() / 8
    gc = -torch.rand(Bn, H, T, d, generator=gen).cuda() / 8
    f, amp = B.rotary_freqs(d, scaling="yarn", factor=4.0, trained=64, device="cuda")
    turn = dict(freqs=f, amplitude=amp, norm="rms")

    def mixed(q, k, v, g, gc, state, hidden, pos):
        """One call of each operator; pos: the position of the first step."""
        q, k = B.qk_norm_fwd(q, k, pos=torch.full((Bn,), pos, dtype=torch.int32, device="cuda"), **turn)
        v, g, gc = v.contiguous(), g.contiguous(), gc.contiguous()
        if q.shape[2] > 1:
            v, hidden, _ = B.gated_scan_fwd(v, gc, hidden, coupled=True, save_states=False)
            o, state = B.linear_fwd(q, k, v, g, state)
        else:
            v = B.gated_scan_recurrent_fwd(v, gc, hidden, coupled=True)
            o = B.linear_recurrent_fwd(q, k, v, g, state)
        return o, state, hidden

    whole = mixed(q, k, v, g, gc, None, None, 0)
    o, state, hidden = mixed(q[:, :, :cut], k[:, :, :cut], v[:, :, :cut], g[:, :, :cut], gc[:, :, :cut], None, None, 0)
    outs = [o]
    for t in range(cut, T):
        s = slice(t, t + 1)
        o, state, hidden = mixed(q[:, :, s], k[:, :, s], v[:, :, s], g[:, :, s], gc[:, :, s], state, hidden, t)
        outs.append(o)
    for x, y in ((torch.cat(outs, 2), whole[0]), (state, whole[1]), (hidden, whole[2])):
        assert float((x - y).norm() / y.norm()) <= 200 * 2.0 ** -24
