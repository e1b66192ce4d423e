"""Norms and rotations of queries and keys against their definition in 64 bits: widths, parts of
the head, layouts, positions, lengths, strides, both directions; streams, graphs, guard bands."""
import math

import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

from qk_ref import U32, check, reference

pytestmark = pytest.mark.gpu


def rows(Bn, Hq, Hk, T, d, dtype, seed=0):
    """Queries and keys as slices of a fused projection's output [B,T,heads,d], weights, cotangents."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=gen)

    both = (2 * normal(Bn, T, Hq + Hk, d)).to(dtype).cuda()
    s = dict(q=both[:, :, :Hq].transpose(1, 2), k=both[:, :, Hq:].transpose(1, 2), wq=(1 + 0.3 * normal(d)).cuda(),
             wk=(1 + 0.3 * normal(d)).cuda(), dyq=normal(Bn, Hq, T, d).to(dtype).cuda(),
             dyk=normal(Bn, Hk, T, d).to(dtype).cuda())
    return s


def positions(kind, Bn, T, seed=0):
    gen = torch.Generator().manual_seed(seed + 100)
    if kind == "step":
        return None
    if kind == "start":
        return torch.randint(-5, 1 << 20, (Bn,), generator=gen, dtype=torch.int32).cuda()
    return torch.randint(-50, 1 << 20, (Bn, T), generator=gen, dtype=torch.int32).cuda()


def both_ways(s, norm, weights, turn, lens=None, **how):
    """Everything forward and backward of the entry points, and its reference."""
    out, want = {}, ({}, {})
    wq, wk = (s["wq"], s["wk"]) if weights else (None, None)
    if norm:
        yq, yk = B.qk_norm_fwd(s["q"], s["k"], wq, wk, norm=norm, eps=1e-6, lens=lens, **turn, **how)
        gr = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], wq, wk, norm=norm, eps=1e-6, lens=lens, **turn, **how)
    else:
        yq, yk = B.rotary_fwd(s["q"], s["k"], lens=lens, **turn, **how)
        gr = dict(zip(("dq", "dk"), B.rotary_bwd(s["dyq"], s["dyk"], lens=lens, **turn, **how)))
    for n, y, w in (("q", yq, wq), ("k", yk, wk)):
        if s[n].shape[1] == 0:
            continue
        v, e = reference(s[n], w, norm, 1e-6, lens=lens, dy=s["dy" + n], **turn)
        got = {"y": y, "dx": gr["d" + n], "dw": gr.get("dw" + n)}
        for m in v:
            out[m + n], want[0][m + n], want[1][m + n] = got[m], v[m], e[m]
    return out, want


SIZES = [(1, 1, 1, 1), (2, 3, 1, 1), (1, 4, 2, 17), (3, 5, 5, 33), (2, 1, 7, 130), (1, 16, 16, 64)]


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm,weights", [("l2", False), ("l2", True), ("rms", True), (None, False)])
def test_against_the_definition(norm, weights, dtype, d):
    for i, (Bn, Hq, Hk, T) in enumerate(SIZES):
        s = rows(Bn, Hq, Hk, T, d, dtype, seed=i + d)
        if norm:
            out, want = both_ways(s, norm, weights, {})
            check(out, *want, label=f"{(Bn, Hq, Hk, T)} not rotated")
        for rot in {8, d // 2, d - 8, d}:
            for interleaved in (False, True):
                kind = ("step", "start", "each")[(i + rot // 8 + interleaved) % 3]
                f, amp = B.rotary_freqs(rot, scaling="yarn", factor=8.0, trained=4096, device="cuda")
                turn = dict(freqs=f, pos=positions(kind, Bn, T, i), interleaved=interleaved, amplitude=amp)
                out, want = both_ways(s, norm, weights, turn)
                check(out, *want, label=f"{(Bn, Hq, Hk, T)} rot {rot} {'pairs' if interleaved else 'halves'} {kind}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lengths(dtype):
    """Rows behind an end are not used, their results zero, weights' gradients without them."""
    T = 37
    lens = torch.tensor([T, 0, 1, 20, -2, T + 5], dtype=torch.int32).cuda()
    s = rows(6, 3, 2, T, 64, dtype, seed=1)
    f, _ = B.rotary_freqs(32, device="cuda")
    for b, n in enumerate(lens.tolist()):
        for m in ("q", "k", "dyq", "dyk"):
            s[m][b, :, max(n, 0):] = math.nan
    for norm, turn in (("rms", dict(freqs=f)), ("l2", {}), (None, dict(freqs=f, interleaved=True))):
        out, want = both_ways(s, norm, norm is not None, turn, lens)
        check(out, *want, label=str(norm))


def test_far_positions():
    """Angles up to 2^31 positions: reduced in 64 bits, so that cosine and sine keep fp32's bits."""
    f, _ = B.rotary_freqs(64, device="cuda")
    top = 2 ** 31 - 1
    pos = torch.tensor([[top, top - 1, -top - 1, 2 ** 24 + 1, 2 ** 20 + 3, 1, 0, -1]], dtype=torch.int32).cuda()
    s = rows(1, 2, 2, 8, 64, torch.float32, seed=2)
    yq, _ = B.rotary_fwd(s["q"], s["k"], f, pos=pos)
    val, err = reference(s["q"], freqs=f, pos=pos)
    # the 64-bit angle itself is off by half a step: 2^-53 * 2^31 rad
    check({"y": yq}, val, {"y": err["y"] + 2.0 ** -21 * s["q"].double().abs().amax(-1, keepdim=True)})
    start = torch.tensor([top - 3], dtype=torch.int32).cuda()   # runs past 2^31
    yq, _ = B.rotary_fwd(s["q"], s["k"], f, pos=start)
    val, err = reference(s["q"], freqs=f, pos=start)
    check({"y": yq}, val, {"y": err["y"] + 2.0 ** -21 * s["q"].double().abs().amax(-1, keepdim=True)})
    near = torch.arange(8, dtype=torch.int32).cuda() * 131071
    yq, _ = B.rotary_fwd(s["q"], s["k"], f, pos=near[None].contiguous())
    val, err = reference(s["q"], freqs=f, pos=near[None])
    check({"y": yq}, val, err)


@pytest.mark.parametrize("order", ["heads_first", "token_first", "batch_inside", "expanded", "slice"])
def test_orders_of_the_dimensions(order):
    """Any order of the dimensions but the last, gaps between rows, broadcast inputs; gradients come in the
    order of their inputs."""
    Bn, H, T, d = 2, 3, 19, 32
    gen = torch.Generator().manual_seed(4)
    plain = torch.randn(Bn, H, T, d, generator=gen).cuda()
    if order == "heads_first":
        q = plain.clone()
    elif order == "token_first":
        q = plain.transpose(1, 2).contiguous().transpose(1, 2)
    elif order == "batch_inside":
        q = plain.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    elif order == "expanded":
        q = plain[:1, :1].expand(Bn, H, T, d)
    else:
        q = torch.randn(Bn, T + 2, H + 4, d, generator=gen).cuda()[:, 1:-1, 2:-2].transpose(1, 2)
    s = dict(q=q, k=plain, wq=torch.ones(d).cuda(), wk=torch.ones(d).cuda() * 2, dyq=plain.flip(0).contiguous(),
             dyk=plain.flip(1).contiguous())
    f, _ = B.rotary_freqs(16, device="cuda")
    for norm in ("l2", None):
        out, want = both_ways(s, norm, norm is not None, dict(freqs=f))
        check(out, *want, label=order)
        assert out["yq"].is_contiguous()
        if norm and order != "expanded":
            assert out["dxq"].transpose(1, 2).is_contiguous() == (order in ("token_first", "slice"))


def test_one_side_only_and_nothing():
    f, _ = B.rotary_freqs(16, device="cuda")
    s = rows(2, 3, 2, 9, 16, torch.float32)
    for q, k in ((s["q"], None), (None, s["k"])):
        yq, yk = B.qk_norm_fwd(q, k, freqs=f)
        both = B.qk_norm_fwd(s["q"], s["k"], freqs=f)
        assert (yq is None) == (q is None) and (yk is None) == (k is None)
        assert torch.equal(yq if q is not None else yk, both[0] if q is not None else both[1])
        gr = B.qk_norm_bwd(q, k, s["dyq"] if q is not None else None, s["dyk"] if k is not None else None, freqs=f)
        assert (gr["dq"] is None) == (q is None) and (gr["dk"] is None) == (k is None)
        assert (B.rotary_fwd(q, k, f)[0] is None) == (q is None)
    for Bn, Hq, Hk, T in ((0, 2, 2, 4), (2, 0, 0, 4), (2, 2, 2, 0)):
        s = rows(Bn, Hq, Hk, T, 32, torch.bfloat16)
        yq, yk = B.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], freqs=f)
        gr = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], freqs=f)
        assert yq.shape == s["q"].shape and gr["dk"].shape == s["k"].shape
        assert (gr["dwq"] == 0).all() and (gr["dwk"] == 0).all()


def test_more_tokens_than_workgroups_take_at_once():
    """The backward's workgroups walk several token tiles; sums of the weights' gradients over 40000 rows."""
    s = rows(2, 2, 1, 10000, 128, torch.float32, seed=3)
    f, _ = B.rotary_freqs(128, device="cuda")
    out, want = both_ways(s, "rms", True, dict(freqs=f))
    check(out, *want)


def test_autograd_and_differences():
    """Directional differences of a loss in every input, to a hundredth."""
    s = rows(2, 3, 2, 21, 32, torch.float32, seed=5)
    f, amp = B.rotary_freqs(16, scaling="yarn", factor=4.0, trained=512, device="cuda")
    leaves = [s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_(), s["wq"].requires_grad_(),
              s["wk"].requires_grad_()]
    lens = torch.tensor([21, 13], dtype=torch.int32).cuda()

    def normed(q, k, wq, wk):
        yq, yk = B.QKNorm.apply(q, k, wq, wk, "rms", 1e-6, f, None, True, amp, lens)
        return (yq * s["dyq"]).double().sum() + (yk * s["dyk"]).double().sum()

    def turned(q, k, wq, wk):
        yq, yk = B.Rotary.apply(q * q, k * k, f, None, False, amp, lens)
        return (yq * s["dyq"]).double().sum() + (yk * s["dyk"]).double().sum()

    for loss, n in ((normed, 4), (turned, 2)):
        grads = torch.autograd.grad(loss(*leaves), leaves[:n])
        for i, gr in enumerate(grads):
            way, eps = torch.sign(gr), 1e-3
            with torch.no_grad():
                up = [z + eps * way if j == i else z for j, z in enumerate(leaves)]
                down = [z - eps * way if j == i else z for j, z in enumerate(leaves)]
                slope = float((loss(*up) - loss(*down)) / (2 * eps))
            assert abs(slope - float((gr * way).double().sum())) <= 1e-2 * abs(slope)


def test_nan_and_inf_stay_in_their_row():
    s = rows(1, 2, 2, 8, 32, torch.float32, seed=6)
    f, _ = B.rotary_freqs(16, device="cuda")
    q = s["q"].contiguous()
    clean = B.qk_norm_fwd(q, None, norm="l2", freqs=f)[0]
    turned = B.rotary_fwd(q, None, f)[0]
    q[0, 0, 3, 5], q[0, 1, 2, 20] = math.nan, math.inf
    got, turned2 = B.qk_norm_fwd(q, None, norm="l2", freqs=f)[0], B.rotary_fwd(q, None, f)[0]
    rest = torch.ones(1, 2, 8, dtype=torch.bool).cuda()
    rest[0, 0, 3], rest[0, 1, 2] = False, False
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[0, 0, 3]).all()
    some = torch.ones_like(turned, dtype=torch.bool)
    some[0, 0, 3, 5] = some[0, 0, 3, 13] = some[0, 1, 2, 20] = False   # the pair; not rotated
    assert torch.equal(turned2[some], turned[some]) and turned2[0, 1, 2, 20] == math.inf


def test_a_row_of_zeros():
    s = rows(1, 1, 1, 4, 16, torch.float32)
    q = s["q"].contiguous()
    q[0, 0, 1] = 0
    assert (B.qk_norm_fwd(q, None)[0][0, 0, 1] == 0).all()
    assert torch.isnan(B.qk_norm_fwd(q, None, eps=0.0)[0][0, 0, 1]).all()


def test_twice_the_same_bits():
    s = rows(4, 8, 8, 500, 64, torch.bfloat16, seed=8)
    first = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], norm="rms")
    second = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], norm="rms")
    for n in first:
        assert torch.equal(first[n], second[n])


def test_on_another_stream_and_captured():
    s = rows(2, 4, 4, 100, 64, torch.float32, seed=9)
    f, _ = B.rotary_freqs(64, device="cuda")
    turn = dict(freqs=f, pos=torch.tensor([3, 7], dtype=torch.int32).cuda())

    def work(**how):
        return {**both_ways(s, "rms", True, turn, **how)[0], **{"r" + n: x for n, x in both_ways(s, None, False, turn, **how)[0].items()}}

    def calls():
        a = B.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], norm="rms", **turn)
        b = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], norm="rms", **turn)
        return [*a, *b.values(), *B.rotary_fwd(s["q"], s["k"], **turn), *B.rotary_bwd(s["dyq"], s["dyk"], **turn)]

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work(stream=side)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n]), n
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        had = calls()
    for i in range(3):
        new = rows(2, 4, 4, 100, 64, torch.float32, seed=30 + i)
        for m in s:
            s[m].copy_(new[m])
        turn["pos"].add_(1000)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        copies = [x.clone() for x in had]
        for x, y in zip(copies, calls()):
            assert torch.equal(x, y)


def test_writes_stay_in_their_tensors():
    """Outputs between bands that have to stay as they are, rows with gaps between them too."""
    Bn, H, T, d = 2, 3, 21, 64
    s = rows(Bn, H, H, T, d, torch.bfloat16, seed=3)
    f, _ = B.rotary_freqs(32, device="cuda")
    whole = {n: torch.full((Bn * T * (H + 2) * d + 4096,), 7.0, dtype=torch.bfloat16, device="cuda") for n in ("q", "k")}
    # rows of a [B, T, heads + 2, d] tensor, two heads left alone
    part = {n: w[2048:-2048].view(Bn, T, H + 2, d)[:, :, 1:-1].transpose(1, 2) for n, w in whole.items()}
    sh = B.QKShape(Bn, H, H, T, d, 32, B.DN_BF16, B.DN_NORM_L2, B.DN_ROT_HALVES, B.DN_POS_STEP, 1e-6, 1.0,
                   *(x for t in (s["q"], s["k"], part["q"], part["k"]) for x in t.stride()[:3]))
    dw = torch.full((2, 3 * d), 7.0, device="cuda")
    ws = torch.full((B.dn_qk_workspace_bytes(sh) + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    n = ws.numel() - 4096
    B._check(B.dn_qk_bwd(sh, s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], f, None, None, part["q"], part["k"],
                         dw[0, d:2 * d], dw[1, d:2 * d], ws, n))
    torch.cuda.synchronize()
    for m, w in (("q", s["wq"]), ("k", s["wk"])):
        val, err = reference(s[m], w, "l2", 1e-6, freqs=f, dy=s["dy" + m])
        check({"y": val["y"], "dx": part[m], "dw": dw["qk".index(m), d:2 * d]}, val, err)
        grid = whole[m][2048:-2048].view(Bn, T, H + 2, d)
        assert (whole[m][:2048] == 7).all() and (whole[m][-2048:] == 7).all()
        assert (grid[:, :, 0] == 7).all() and (grid[:, :, -1] == 7).all()
    assert (dw[:, :d] == 7).all() and (dw[:, 2 * d:] == 7).all() and (ws[n:] == 0x5a).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows against a call on them alone."""
    T, H, d = 1 << 18, 33, 128
    both = torch.empty(1, T, 2 * H, d, dtype=torch.bfloat16, device="cuda").normal_()
    q, k = both[:, :, :H].transpose(1, 2), both[:, :, H:].transpose(1, 2)
    f, _ = B.rotary_freqs(d, device="cuda")
    yq, yk = B.qk_norm_fwd(q, k, freqs=f)
    gr = B.qk_norm_bwd(q, k, yq, yk, freqs=f)
    tail = slice(T - 5, T)
    pos = torch.tensor([T - 5], dtype=torch.int32, device="cuda")
    q1, k1 = q[:, -1:, tail], k[:, -1:, tail]
    zq, zk = B.qk_norm_fwd(q1, k1, freqs=f, pos=pos)
    g1 = B.qk_norm_bwd(q1, k1, zq, zk, freqs=f, pos=pos)
    for whole, part in ((yq, zq), (yk, zk), (gr["dq"], g1["dq"]), (gr["dk"], g1["dk"])):
        assert torch.equal(whole[:, -1:, tail], part)
    assert float(zk.abs().max()) > 0


def test_one_weight_for_both_and_one_gradient():
    """The same weight for queries and keys gets both gradients; a weight of one side alone."""
    s = rows(2, 3, 2, 40, 64, torch.float32, seed=12)
    w = s["wq"].requires_grad_()
    yq, yk = B.QKNorm.apply(s["q"], s["k"], w, w, "rms")
    (gw,) = torch.autograd.grad((yq * s["dyq"]).sum() + (yk * s["dyk"]).sum(), [w])
    w = w.detach()
    total, bound = 0, 0
    for n in "qk":
        v, e = reference(s[n], w, "rms", 1e-6, dy=s["dy" + n])
        total, bound = total + v["dw"], bound + e["dw"] + U32 * v["dw"].abs()
    assert ((gw.double() - total).abs() <= bound).all()
    gr = B.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], None, w, norm="rms")
    assert gr["dwq"] is None
    v, e = reference(s["k"], w, "rms", 1e-6, dy=s["dyk"])
    check({"dw": gr["dwk"], "dx": gr["dk"]}, {n: v[n] for n in ("dw", "dx")}, e)
    v, e = reference(s["q"], None, "rms", 1e-6, dy=s["dyq"])
    check({"dx": gr["dq"]}, {"dx": v["dx"]}, e)
