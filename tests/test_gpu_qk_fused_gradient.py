"""Gradients of queries and keys written as slices of one tensor, the gradient of the projection that
they are slices of: the bits of separate tensors, everything between the rows left alone."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

pytestmark = pytest.mark.gpu

Bn, T, d = 3, 67, 64


def slices(order, Hq, Hk, Hv, whole):
    """Queries, keys and what else there is, [B, heads, T, d], of one tensor."""
    if order == "pairs":   # a head's query next to its key
        x = whole.view(Bn, T, Hq, 2, d)
        return x[:, :, :, 0].transpose(1, 2), x[:, :, :, 1].transpose(1, 2), whole[:0]
    x = whole.view(Bn, T, Hq + Hk + Hv, d).transpose(1, 2) if order == "tokens" else whole.view(Bn, Hq + Hk + Hv, T, d)
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order,Hq,Hk,Hv", [("tokens", 3, 2, 2), ("tokens", 1, 1, 0), ("tokens", 4, 1, 1), ("heads", 3, 2, 1),
                                            ("pairs", 3, 3, 0)])
def test_into_one_tensor(order, Hq, Hk, Hv, dtype):
    gen = torch.Generator().manual_seed(Hq)
    n = Bn * T * (Hq + Hk + Hv) * d

    def normal(*s):
        return torch.randn(s, generator=gen).to(dtype).cuda()

    q, k, _ = slices(order, Hq, Hk, Hv, normal(n))
    dyq, dyk = normal(Bn, Hq, T, d), normal(Bn, Hk, T, d)
    wq, wk = (normal(d).float() for _ in range(2))
    lens = torch.tensor([T, 0, 20], dtype=torch.int32).cuda()
    f, amp = B.rotary_freqs(32, device="cuda")
    for norm in (B.DN_NORM_RMS, B.DN_NORM_NONE):
        grad = torch.full((n,), 7.0, dtype=dtype, device="cuda")
        dq, dk, rest = slices(order, Hq, Hk, Hv, grad)
        io = B.DN_BF16 if dtype == torch.bfloat16 else B.DN_F32
        strides = [x for t in (q, k, dq, dk) for x in t.stride()[:3]]
        sh = B.QKShape(Bn, Hq, Hk, T, d, 32, io, norm, B.DN_ROT_HALVES, B.DN_POS_STEP, 1e-6, amp, *strides)
        dw = torch.empty(2, d, device="cuda")
        ws = torch.empty(max(B.dn_qk_workspace_bytes(sh), 16), dtype=torch.uint8, device="cuda")
        if norm:
            B._check(B.dn_qk_bwd(sh, q, k, dyq, dyk, wq, wk, f, None, lens, dq, dk, dw[0], dw[1], ws, ws.numel()))
            want = B.qk_norm_bwd(q, k, dyq, dyk, wq, wk, norm="rms", freqs=f, amplitude=amp, lens=lens)
            assert torch.equal(dw[0], want["dwq"]) and torch.equal(dw[1], want["dwk"])
            want = want["dq"], want["dk"]
        else:
            B._check(B.dn_qk_bwd(sh, None, None, dyq, dyk, None, None, f, None, lens, dq, dk, None, None, None, 0))
            want = B.rotary_bwd(dyq, dyk, f, amplitude=amp, lens=lens)
        assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
        assert (rest == 7).all()
