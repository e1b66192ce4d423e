"""The gated linear recurrence against its definition in 64 bits: forward, backward (saved and
recomputed states), single tokens; lengths, widths, gates, segments; streams, graphs, guard
bands."""
import math

import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

from scan_ref import check, reference

pytestmark = pytest.mark.gpu


def inputs(Bn, H, T, d, dtype=torch.float32, seed=0, gates="soft"):
    gen = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=gen)

    g = -torch.nn.functional.softplus(normal(Bn, H, T, d)) / 16
    if gates == "mixed":   # resets, strong and no decay, some growth
        pick = torch.rand(Bn, H, T, d, generator=gen)
        g = torch.where(pick < 0.02, -math.inf, torch.where(pick < 0.1, -30 * pick, torch.where(pick < 0.2, 0.0, g)))
        g = torch.where(pick > 0.97, 0.3 * pick, g)
    t = dict(x=normal(Bn, H, T, d).to(dtype), g=g, h0=normal(Bn, H, d), do=normal(Bn, H, T, d).to(dtype),
             dhT=normal(Bn, H, d))
    return {n: z.cuda() for n, z in t.items()}


def run(s, lens=None, coupled=False, h0=True, dhT=True, saved=True, **how):
    h0, dhT = s["h0"] if h0 else None, s["dhT"] if dhT else None
    o, hT, st = B.gated_scan_fwd(s["x"], s["g"], h0, lens=lens, coupled=coupled, save_states=saved, **how)
    gr = B.gated_scan_bwd(s["x"], s["g"], h0, s["do"], dhT, st, lens=lens, coupled=coupled, **how)
    return {"o": o, "hT": hT, **gr}


SIZES = [(1, 1, 1, 1), (2, 3, 1, 16), (1, 1, 64, 16), (2, 3, 15, 5), (2, 3, 127, 67), (3, 2, 128, 64), (1, 2, 129, 100),
         (2, 1, 255, 128), (1, 1, 256, 200), (1, 1, 257, 63), (2, 2, 700, 3), (1, 70, 130, 65), (1, 1, 1024, 64),
         (3, 5, 777, 67), (2, 60, 600, 24), (3, 100, 140, 67), (2, 3, 16, 70), (1, 1, 17, 128), (5, 2, 65, 9),
         (8, 64, 270, 64)]


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_against_the_definition(size, dtype, coupled):
    s = inputs(*size, dtype=dtype, seed=sum(size))
    ref = reference(s["x"], s["g"], s["h0"], None, coupled, s["do"], s["dhT"])
    check(run(s, coupled=coupled), *ref, label=f"{size} saved")
    check(run(s, coupled=coupled, saved=False), *ref, label=f"{size} recomputed")
    ref = reference(s["x"], s["g"], None, None, coupled, s["do"], None)
    check(run(s, coupled=coupled, h0=False, dhT=False), *ref, label=f"{size} without ends")


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("size", [(1, 1, 1025, 1), (1, 1, 5000, 33), (2, 1, 4097, 70), (1, 3, 1025, 64), (3, 1, 16384, 64),
                                  (2, 70, 1030, 130), (3, 120, 1030, 67)], ids=str)
def test_chained_tiles(size, coupled):
    """Channels that do not fill the chip by themselves: the tiles of the steps run at once."""
    Bn, H, T, d = size
    sh = B.make_shape(Bn, H, T, d, d, 64, "fp32", "vector")
    assert B.dn_gated_scan_workspace_bytes(sh, B.DN_PASS_FWD) > 0 and B.dn_gated_scan_workspace_bytes(sh, B.DN_PASS_BWD) > 0
    for dtype in (torch.float32, torch.bfloat16):
        s = inputs(*size, dtype=dtype, seed=T)
        lens = torch.tensor([T, 0, T // 3][:Bn], dtype=torch.int32).cuda() if Bn > 1 else None
        ref = reference(s["x"], s["g"], s["h0"], lens, coupled, s["do"], s["dhT"])
        check(run(s, lens, coupled), *ref, label=f"{size} saved")
        check(run(s, lens, coupled, saved=False), *ref, label=f"{size} recomputed")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_channels(dtype):
    """A workgroup for each strip of channels, several tiles."""
    s = inputs(4, 64, 600, 64, dtype=dtype, seed=12)
    assert B.dn_gated_scan_workspace_bytes(B.make_shape(4, 64, 600, 64, 64, 64, "fp32", "vector"), B.DN_PASS_BWD) == 0
    lens = torch.tensor([600, 511, 100, 0], dtype=torch.int32).cuda()
    ref = reference(s["x"], s["g"], s["h0"], lens, True, s["do"], s["dhT"])
    check(run(s, lens, True), *ref, label="saved")
    check(run(s, lens, True, saved=False), *ref, label="recomputed")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(3, 50, 600, 24), (2, 65, 300, 100), (4, 70, 300, 67), (2, 3, 1500, 100), (3, 40, 1100, 5),
                                  (3, 1, 140, 1000), (4, 40, 300, 64), (3, 10, 700, 64),
                                  (2, 40, 600, 64), (1, 40, 700, 64)], ids=str)
def test_strips_of_one_and_of_all_heads(size, dtype):
    """Widths that leave lanes of a strip to the next head's channels or idle, in every form of the scan, with
    sequences that end inside it; the results that are not wanted left out."""
    s = inputs(*size, dtype=dtype, seed=sum(size))
    T = size[2]
    lens = torch.tensor([T, T - 130, 3, T][:size[0]], dtype=torch.int32).cuda()
    ref = reference(s["x"], s["g"], s["h0"], lens, True, s["do"], s["dhT"])
    got = run(s, lens, True)
    check(got, *ref)
    o, hT, st = B.gated_scan_fwd(s["x"], s["g"], s["h0"], lens=lens, coupled=True, want_hT=False)
    gr = B.gated_scan_bwd(s["x"], s["g"], s["h0"], s["do"], s["dhT"], st, lens=lens, coupled=True, want_dh0=False)
    assert hT is None and gr["dh0"] is None
    assert torch.equal(o, got["o"]) and torch.equal(gr["dx"], got["dx"]) and torch.equal(gr["dg"], got["dg"])


@pytest.mark.parametrize("T", [420, 530, 1100])
@pytest.mark.parametrize("d", [7, 64, 100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lengths(dtype, d, T):
    """Every kind of length in one batch, several sequences in a strip of 64 channels too; what lies
    behind an end is not used and its results are zero."""
    lens = [T, 0, 1, 127, 128, 129, 256, 400, T - 1, -3, T + 9]
    s = inputs(len(lens), 2, T, d, dtype=dtype, seed=d)
    for b, n in enumerate(lens):
        for m in ("x", "g", "do"):
            s[m][b, :, max(n, 0):] = math.nan
    lens = torch.tensor(lens, dtype=torch.int32).cuda()
    for coupled in (False, True):
        ref = reference(s["x"], s["g"], s["h0"], lens, coupled, s["do"], s["dhT"])
        check(run(s, lens, coupled), *ref, label="saved")
        check(run(s, lens, coupled, saved=False), *ref, label="recomputed")


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("size", [(2, 2, 300, 40), (1, 1, 3000, 64)], ids=str)
def test_resets_and_other_gates(size, coupled):
    s = inputs(*size, seed=5, gates="mixed")
    ref = reference(s["x"], s["g"], s["h0"], None, coupled, s["do"], s["dhT"])
    got = run(s, coupled=coupled)
    check(got, *ref)
    off = torch.isinf(s["g"])
    assert (got["dg"][off] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing_to_do(dtype):
    for Bn, H, T, d in ((0, 2, 10, 8), (2, 0, 10, 8), (2, 2, 0, 8)):
        s = inputs(Bn, H, T, d, dtype=dtype)
        for saved in (True, False):
            got = run(s, saved=saved)
            assert torch.equal(got["hT"], s["h0"]) and torch.equal(got["dh0"], s["dhT"])
            assert got["o"].shape == got["dx"].shape == got["dg"].shape == (Bn, H, T, d)
        B.gated_scan_recurrent_fwd(s["x"], s["g"], s["h0"])


def test_rows_too_far_apart_for_one_buffer():
    """Strips of one head's row: the definition as a tree of joined steps in 64 bits."""
    T = 2 ** 23
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = -torch.rand(3, 1, T, 1, generator=gen, device="cuda") / 4
    x, do = torch.randn(3, 1, T, 1, generator=gen, device="cuda"), torch.randn(3, 1, T, 1, generator=gen, device="cuda")

    def along(a, b):
        n = a.shape[2]
        if n == 1:
            return b
        m = n // 2 * 2
        a0, a1, b0, b1 = a[:, :, 0:m:2], a[:, :, 1:m:2], b[:, :, 0:m:2], b[:, :, 1:m:2]
        odd, h = along(a0 * a1, a1 * b0 + b1), torch.empty_like(b)
        h[:, :, 1:m:2], h[:, :, 0] = odd, b[:, :, 0]
        h[:, :, 2::2] = a[:, :, 2::2] * odd[:, :, :(n - 1) // 2] + b[:, :, 2::2]
        return h

    o, hT, st = B.gated_scan_fwd(x, g)
    gr = B.gated_scan_bwd(x, g, None, do, None, st)
    a = g.double().exp()
    h = along(a, x.double())
    D = along(torch.cat([a[:, :, 1:], a[:, :, :1]], 2).flip(2), do.double().flip(2)).flip(2)
    # 20 half steps a step over a memory of some 8 to 60 steps
    for got, want in ((o, h), (hT, h[:, :, -1]), (gr["dx"], D)):
        assert float((got.double() - want).abs().max()) <= 20 * 60 * 2.0 ** -24 * float(want.abs().max())


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(1, 1, 1, 1), (3, 5, 1, 67), (2, 2, 5, 128), (1, 1, 40, 3)], ids=str)
def test_tokens(size, dtype, coupled):
    s = inputs(*size, dtype=dtype, seed=9)
    state = s["h0"].clone()
    o = B.gated_scan_recurrent_fwd(s["x"], s["g"], state, coupled=coupled)
    val, err = reference(s["x"], s["g"], s["h0"], None, coupled)
    check({"o": o, "hT": state}, val, err)


def test_a_prompt_then_tokens_is_one_sequence():
    s = inputs(2, 3, 300, 70, seed=4)
    whole, hT, _ = B.gated_scan_fwd(s["x"], s["g"], s["h0"], coupled=True)
    cut = 290
    x, g = s["x"], s["g"]
    _, state, _ = B.gated_scan_fwd(x[:, :, :cut].contiguous(), g[:, :, :cut].contiguous(), s["h0"], coupled=True)
    for t in range(cut, 300):
        o = B.gated_scan_recurrent_fwd(x[:, :, t:t + 1].contiguous(), g[:, :, t:t + 1].contiguous(), state, coupled=True)
        assert float((o - whole[:, :, t:t + 1]).abs().max()) <= 1e-5 * float(whole.abs().max())
    assert float((state - hT).abs().max()) <= 1e-5 * float(hT.abs().max())


@pytest.mark.parametrize("coupled", [False, True])
def test_autograd_and_differences(coupled):
    """Directional differences of a loss in every input, to a hundredth."""
    s = inputs(2, 2, 150, 20, seed=6)
    lens = torch.tensor([150, 90], dtype=torch.int32).cuda()
    leaves = [s["x"].requires_grad_(), s["g"].requires_grad_(), s["h0"].requires_grad_()]

    def loss(x, g, h0, recompute=False):
        o, hT = B.GatedScan.apply(x, g, h0, lens, coupled, recompute)
        return (o * s["do"]).double().sum() + (hT * s["dhT"]).double().sum()

    first = torch.autograd.grad(loss(*leaves), leaves)
    again = torch.autograd.grad(loss(*leaves, True), leaves)
    for i, (leaf, gr, g2) in enumerate(zip(leaves, first, again)):
        assert torch.equal(gr, g2)
        way = torch.sign(gr)
        eps = 1e-2
        with torch.no_grad():
            up = [z + eps * way if j == i else z for j, z in enumerate(leaves)]
            down = [z - eps * way if j == i else z for j, z in enumerate(leaves)]
            slope = float((loss(*up) - loss(*down)) / (2 * eps))
        assert abs(slope - float((gr * way).double().sum())) <= 1e-2 * abs(slope)


def test_twice_the_same_bits():
    s = inputs(2, 1, 3000, 64, dtype=torch.bfloat16, seed=8)
    first, second = run(s, coupled=True), run(s, coupled=True)
    for n in first:
        assert torch.equal(first[n], second[n])


def test_nan_and_inf_stay_in_their_channel():
    s = inputs(1, 2, 600, 40, seed=2)
    clean = run(s)
    s["x"][0, 0, 300, 7], s["x"][0, 1, 20, 3], s["do"][0, 0, 500, 9] = math.nan, math.inf, math.nan
    got = run(s)
    for n in clean:
        same = torch.ones_like(clean[n], dtype=torch.bool)
        for h, c in ((0, 7), (1, 3), (0, 9)):
            same[:, h, ..., c] = False
        assert torch.equal(got[n][same], clean[n][same]), n
    assert torch.isfinite(got["o"][0, 0, :300, 7]).all() and torch.isnan(got["o"][0, 0, 300:, 7]).all()
    assert torch.isfinite(got["dx"][0, 0, 501:, 9]).all() and torch.isnan(got["dx"][0, 0, :501, 9]).all()


def test_on_another_stream():
    s = inputs(1, 1, 4000, 64, seed=1)
    want = run(s, coupled=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = run(s, coupled=True, stream=stream)
        side.synchronize()
        for n in want:
            assert torch.equal(want[n], got[n])
    with torch.cuda.stream(side):
        got = run(s, coupled=True)
    side.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n])


def test_captured_and_replayed():
    """Forward, backward and tokens in one graph; replays between eager work, with other inputs."""
    s = inputs(1, 2, 2600, 64, seed=1)
    tok = inputs(1, 2, 1, 64, seed=7)
    lens = torch.tensor([2600], dtype=torch.int32).cuda()
    state = torch.zeros(1, 2, 64, device="cuda")

    def work():
        got = run(s, lens, True)
        state.copy_(got["hT"])
        got["tok"] = B.gated_scan_recurrent_fwd(tok["x"], tok["g"], state, coupled=True)
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i, n in enumerate((2600, 1300, 0)):
        new = inputs(1, 2, 2600, 64, seed=20 + i)
        for m in s:
            s[m].copy_(new[m])
        lens.fill_(n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        had = {m: z.clone() for m, z in got.items()}
        want = work()
        torch.cuda.synchronize()
        for m in want:
            assert torch.equal(had[m], want[m]), (n, m)


def test_writes_stay_in_their_tensors():
    """Outputs between bands that have to stay as they are, workspace of the exact size."""
    Bn, H, T, d = 1, 3, 1100, 67
    sh = B.make_shape(Bn, H, T, d, d, 64, "bf16", "vector")
    sh.flags = B.DN_FLAG_COUPLED
    s = inputs(Bn, H, T, d, dtype=torch.bfloat16, seed=3)

    def banded(nbytes):
        whole = torch.full((nbytes + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
        return whole, whole[4096:4096 + nbytes]

    n = Bn * H * T * d
    sizes = dict(o=2 * n, hT=4 * Bn * H * d, states=B.dn_gated_scan_states_bytes(sh), dx=2 * n, dg=4 * n, dh0=4 * Bn * H * d,
                 wf=B.dn_gated_scan_workspace_bytes(sh, B.DN_PASS_FWD), wb=B.dn_gated_scan_workspace_bytes(sh, B.DN_PASS_BWD),
                 wr=B.dn_gated_scan_workspace_bytes(sh, B.DN_PASS_BWD_RECOMPUTE))
    buf = {m: banded(z) for m, z in sizes.items()}
    p = {m: b[1] for m, b in buf.items()}
    B._check(B.dn_gated_scan_fwd(sh, s["x"], s["g"], None, s["h0"], p["o"], p["hT"], p["states"], p["wf"], sizes["wf"]))
    B._check(B.dn_gated_scan_bwd(sh, s["x"], s["g"], None, s["h0"], s["do"], s["dhT"], p["states"], p["dx"], p["dg"], p["dh0"],
                                 p["wb"], sizes["wb"]))
    first = p["dg"].clone()
    B._check(B.dn_gated_scan_bwd(sh, s["x"], s["g"], None, s["h0"], s["do"], s["dhT"], None, p["dx"], p["dg"], p["dh0"],
                                 p["wr"], sizes["wr"]))
    torch.cuda.synchronize()
    assert torch.equal(first, p["dg"])
    for m, (whole, _) in buf.items():
        assert (whole[:4096] == 0x5a).all() and (whole[-4096:] == 0x5a).all(), m
    val, err = reference(s["x"], s["g"], s["h0"], None, True, s["do"], s["dhT"])
    got = dict(o=p["o"].view(torch.bfloat16), dx=p["dx"].view(torch.bfloat16), dg=p["dg"].view(torch.float32),
               hT=p["hT"].view(torch.float32), dh0=p["dh0"].view(torch.float32))
    check({m: got[m].reshape(val[m].shape) for m in got}, val, err)


def test_two_calls_at_once():
    """Chained calls on two streams, their workgroups on the chip together, again and again."""
    a, b = inputs(1, 2, 9000, 64, seed=21), inputs(1, 3, 7000, 100, dtype=torch.bfloat16, seed=22)
    want = [run(a, coupled=True), run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, (s, c) in enumerate(((a, True), (b, False))):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(s, coupled=c))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for n in g:
                assert torch.equal(g[n], want[i][n]), n


def test_one_workspace_for_calls_in_turn():
    """A workspace given by the caller, full of what other calls left in it."""
    s, other = inputs(1, 2, 3000, 64, seed=31), inputs(1, 1, 5000, 130, seed=32)
    n = max(B.dn_gated_scan_workspace_bytes(B.make_shape(1, H, T, d, d, 64, "fp32", "vector"), p)
            for H, T, d in ((2, 3000, 64), (1, 5000, 130)) for p in (B.DN_PASS_FWD, B.DN_PASS_BWD_RECOMPUTE))
    ws = torch.full((n,), 0x41, dtype=torch.uint8, device="cuda")
    want = run(s, saved=False)
    for _ in range(3):
        run(other, saved=False, ws=ws)
        got = run(s, saved=False, ws=ws)
        for m in want:
            assert torch.equal(got[m], want[m])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last head's results against a call on that head alone."""
    H, T, d = 33, 1 << 20, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(1, H, T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    do = torch.empty(1, H, T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g = torch.empty(1, H, T, d, device="cuda").uniform_(-0.3, -0.01, generator=gen)
    o, hT, st = B.gated_scan_fwd(x, g)
    gr = B.gated_scan_bwd(x, g, None, do, None, st)
    last = [t[:, -1:].contiguous() for t in (x, g, do)]
    o1, hT1, st1 = B.gated_scan_fwd(last[0], last[1])
    gr1 = B.gated_scan_bwd(last[0], last[1], None, last[2], None, st1)
    for whole, alone in ((o, o1), (hT, hT1), (gr["dx"], gr1["dx"]), (gr["dg"], gr1["dg"]), (gr["dh0"], gr1["dh0"])):
        part = whole[:, -1:].float()
        tol = 2.0 ** -7 if whole.dtype == torch.bfloat16 else 24 * 100 * 2.0 ** -24   # both rounded; 100 steps of memory
        assert float((part - alone.float()).abs().max()) <= tol * float(alone.float().abs().max())
        assert float(part.abs().max()) > 0
