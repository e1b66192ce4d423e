"""The weights' gradients of the norms over many rows: sums whose error does not grow with the rows
that a thread takes, and of padded batches whose workgroups walk many tiles."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

from qk_ref import U32, check, reference

pytestmark = pytest.mark.gpu

# Half steps of fp32 that a weight's gradient may be off, of the sum of its terms' absolute values: a term
# 24 (as in qk_ref); 8 rows of a token in a row, the compensated sum of a thread's tokens 2, threads of the
# same elements 5, waves 4, 2048 workgroups' sums 32 and 64.  Together 139, whatever the rows.
SUM = 139


def test_equal_rows():
    """2^24 rows, 1024 and more of a thread, of the same values: in a plain sum every addition is rounded the same
    way, which puts a channel a third of a half step a row off."""
    H, T, d = 8, 1 << 21, 128
    gen = torch.Generator().manual_seed(3)
    row = torch.randn(d, generator=gen).bfloat16().cuda()
    u = torch.randn(d, generator=gen).bfloat16().cuda()
    q = row.expand(1, H, T, d)
    dy = u.expand(1, H, T, d).contiguous()
    w = torch.ones(d, device="cuda")
    for norm, share in (("l2", 1.0), ("rms", 1.0 / d)):
        dw = B.qk_norm_bwd(q, None, dy, None, w, None, norm=norm)["dwq"]
        x = row.double()
        want = x * (x.square().sum() * share + 1e-6).rsqrt() * u.double() * (H * T)
        off = float(((dw.double() - want).abs() / (want.abs() * U32 + 1e-30)).max())
        print(f"{norm}: {off:.1f} half steps", flush=True)
        assert off <= SUM


def test_padded_batch_over_many_tiles():
    """Sequences of other lengths, each workgroup on 9 and more tiles, a thread on 72 and more rows."""
    Bn, H, T, d = 9, 32, 4097, 128
    gen = torch.Generator(device="cuda").manual_seed(5)

    def normal(*s):
        return torch.randn(s, generator=gen, device="cuda")

    q, k = (normal(Bn, T, H, d).transpose(1, 2) for _ in range(2))
    dyq, dyk = normal(Bn, H, T, d), normal(Bn, H, T, d)
    wq, wk = 1 + 0.3 * normal(d), 1 + 0.3 * normal(d)
    lens = torch.tensor([T, 0, 1, 2000, 4096, 17, 3333, -4, T + 3], dtype=torch.int32).cuda()
    f, amp = B.rotary_freqs(d, device="cuda")
    turn = dict(freqs=f, interleaved=True, amplitude=amp)
    yq, yk = B.qk_norm_fwd(q, k, wq, wk, norm="rms", lens=lens, **turn)
    gr = B.qk_norm_bwd(q, k, dyq, dyk, wq, wk, norm="rms", lens=lens, **turn)
    for x, w, dy, y, dx, dw in ((q, wq, dyq, yq, gr["dq"], gr["dwq"]), (k, wk, dyk, yk, gr["dk"], gr["dwk"])):
        total, terms = 0, 0
        for h in range(0, H, 4):   # a few heads at a time: 64 bits
            s = slice(h, h + 4)
            val, err = reference(x[:, s], w, "rms", 1e-6, lens=lens, dy=dy[:, s], **turn)
            total, terms = total + val.pop("dw"), terms + err.pop("dw") / (150 * U32)
            check({"y": y[:, s], "dx": dx[:, s]}, val, err, label=f"heads {h} on")
        off = float(((dw.double() - total).abs() / (terms * U32)).max())
        print(f"weights: {off:.2f} half steps", flush=True)
        assert off <= SUM


@pytest.mark.parametrize("what", ["infinite", "overflowing"])
def test_infinite_sums(what):
    """A cotangent's infinity, or finite terms whose sum overflows, give an infinite gradient of that channel's weight, as
    a plain sum does, wherever the row lies; the other channels keep their bits."""
    H, T, d = 1, 40000, 128
    gen = torch.Generator().manual_seed(9)
    q = torch.randn(1, H, T, d, generator=gen).cuda()
    q[..., 7] = torch.copysign(q[..., 7].abs() * 1e3 + 1e3, q[..., 7])   # the unit row's other elements are small
    dy = torch.randn(1, H, T, d, generator=gen).cuda()
    w = torch.ones(d, device="cuda")
    clean = B.qk_norm_bwd(q, None, dy, None, w, None)["dwq"]
    for t in (0, 5, 20001, T - 1):
        bad = dy.clone()
        if what == "infinite":
            bad[0, 0, t, 7] = torch.copysign(torch.tensor(float("inf")).cuda(), q[0, 0, t, 7])
        else:   # of every row: two terms of a thread overflow
            bad[..., 7] = torch.copysign(torch.tensor(3e38).cuda(), q[..., 7])
        dw = B.qk_norm_bwd(q, None, bad, None, w, None)["dwq"]
        assert float(dw[7]) == float("inf"), (t, float(dw[7]))
        rest = torch.arange(d, device="cuda") != 7
        assert torch.equal(dw[rest], clean[rest])
