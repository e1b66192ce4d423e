"""Linear attention with a decay per head on the GPU against the 64-bit definition:
whole sequences (forward and gradients) and single tokens, every gate, both I/O types,
lengths from none to several segments, ragged batches."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
import linear_ref as R

pytestmark = pytest.mark.gpu
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}


def draw(dtype, gate, Bn, H, T, dk, dv, h0=True, lens=None, seed=1, scale=1 / 16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rn = lambda *d: torch.randn(d, generator=gen, device="cuda")
    unit = lambda *d: torch.nn.functional.normalize(rn(*d), dim=-1).to(IO[dtype])
    d = {"q": unit(Bn, H, T, dk), "k": unit(Bn, H, T, dk), "v": rn(Bn, H, T, dv).to(IO[dtype]),
         "do": rn(Bn, H, T, dv).to(IO[dtype]), "dhT": rn(Bn, H, dv, dk),
         "h0": 0.5 * rn(Bn, H, dv, dk) if h0 else None,
         "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")}
    d["g"] = {"none": None, "head": -torch.rand(H, generator=gen, device="cuda") * 0.3,
              "scalar": -scale * torch.nn.functional.softplus(rn(Bn, H, T))}[gate]
    return d


def run(d, no_scan=False):
    o, hT = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], lens=d["lens"], no_scan=no_scan)
    gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], lens=d["lens"], no_scan=no_scan)
    torch.cuda.synchronize()
    return {"o": o, "hT": hT, **{n: t for n, t in gr.items() if t is not None}}


def verify(d, got, label):
    val, mag = R.reference(d["q"], d["k"], d["v"], d["g"], d["h0"], d["lens"], d["do"], d["dhT"])
    assert set(val) == set(got), (set(val), set(got))
    R.check(got, val, mag, d["q"].dtype, label)


SHAPES = [
    # B, H, T, dk, dv, lens
    (1, 1, 1, 16, 16, None),
    (1, 2, 5, 16, 64, None),
    (2, 3, 64, 32, 32, None),
    (1, 9, 65, 64, 16, None),
    (3, 2, 130, 128, 128, [130, 0, 67]),
    (2, 4, 191, 16, 128, [-3, 500]),
    (1, 8, 256, 128, 32, None),
    (2, 2, 333, 64, 128, [1, 333]),
    (1, 3, 700, 128, 64, [641]),
]


@pytest.mark.parametrize("gate", ["none", "head", "scalar"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:5])))
def test_sequences(shape, dtype, gate):
    Bn, H, T, dk, dv, lens = shape
    d = draw(dtype, gate, Bn, H, T, dk, dv, h0=T % 2 == 0, lens=lens)
    verify(d, run(d), f"{dtype} {gate} {shape}")


LONG = [
    # B, H, T, dk, dv, lens: parallel segments of 4 to 32 chunks, kept states every 16 and fewer
    (1, 1, 3100, 128, 128, None),
    (2, 1, 2049, 64, 64, [2049, 700]),
    (1, 2, 4096, 32, 128, None),
    (1, 16, 7680, 128, 128, [7600]),
]


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("dtype,gate", [("bf16", "scalar"), ("bf16", "head"), ("fp32", "scalar")])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s[:5])))
def test_long_sequences(shape, dtype, gate, no_scan):
    Bn, H, T, dk, dv, lens = shape
    d = draw(dtype, gate, Bn, H, T, dk, dv, lens=lens, seed=2)
    verify(d, run(d, no_scan), f"{dtype} {gate} {shape} no_scan={no_scan}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_resets_and_extreme_gates(dtype):
    """-inf (and the type's lowest value) cut the sequence: nothing crosses, nothing is NaN."""
    d = draw(dtype, "scalar", 1, 2, 300, 64, 64, seed=3)
    d["g"][0, 0, 0] = -torch.inf
    d["g"][0, 0, 100] = -torch.inf
    d["g"][0, 0, 101] = torch.finfo(torch.float32).min
    d["g"][0, 1, 63:66] = -torch.inf
    d["g"][0, 1, 200] = -300.0
    d["g"][0, 1, 250] = 2.0
    verify(d, run(d), f"{dtype} resets")


def test_steep_gates():
    d = draw("fp32", "scalar", 1, 2, 260, 64, 64, seed=4, scale=6.0)
    verify(d, run(d), "steep")


def test_no_cotangent_of_the_state_and_unwanted_outputs():
    d = draw("bf16", "scalar", 1, 2, 150, 64, 64, seed=5)
    d["dhT"] = None
    verify(d, run(d), "no dhT")
    o, hT = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], want_hT=False)
    gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], want_dh0=False)
    assert hT is None and gr["dh0"] is None
    both = run(d)
    assert torch.equal(o, both["o"]) and torch.equal(gr["dg"], both["dg"])


def test_empty():
    for T, Bn in ((0, 2), (4, 0)):
        d = draw("bf16", "scalar", Bn, 2, T, 32, 64, seed=6)
        got = run(d)
        if Bn:
            assert torch.equal(got["hT"], d["h0"]) and torch.equal(got["dh0"], d["dhT"])


def test_past_the_length_nothing_is_read():
    """What stands past a sequence's length (NaN here) reaches no result; there they are zero."""
    d = draw("bf16", "scalar", 2, 2, 200, 64, 64, lens=[77, 128], seed=7)
    ref = run(d)
    for n in ("q", "k", "v", "do", "g"):
        d[n][0, :, 77:] = torch.nan
        d[n][1, :, 128:] = torch.nan
    got = run(d)
    for n in ref:
        assert torch.equal(got[n], ref[n]), n
    assert not got["o"][0, :, 77:].any() and not got["dg"][1, :, 128:].any()


def test_same_bits_every_time():
    d = draw("bf16", "scalar", 2, 4, 1500, 128, 128, seed=8)
    a, b = run(d), run(d)
    for n in a:
        assert torch.equal(a[n], b[n]), n


STEPS = [
    # B, H, T, dk, dv
    (1, 1, 1, 16, 16),
    (3, 5, 1, 128, 128),
    (2, 2, 4, 64, 48),
    (1, 3, 9, 32, 256),
    (2, 4, 2, 128, 64),
]


@pytest.mark.parametrize("gate", ["none", "head", "scalar"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", STEPS, ids=lambda s: "x".join(map(str, s)))
def test_tokens(shape, dtype, gate):
    d = draw(dtype, gate, *shape, seed=9)
    state = d["h0"].clone()
    o = B.linear_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], state)
    torch.cuda.synchronize()
    val, mag = R.reference(d["q"], d["k"], d["v"], d["g"], d["h0"])
    R.check({"o": o, "hT": state}, val, mag, d["q"].dtype, f"step {dtype} {gate} {shape}")


def test_no_tokens_leave_the_state():
    d = draw("bf16", "scalar", 1, 2, 0, 64, 64)
    state = d["h0"].clone()
    B.linear_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], state)
    torch.cuda.synchronize()
    assert torch.equal(state, d["h0"])


def test_prompt_then_tokens():
    """A ragged prompt, then one token for each sequence from the state it left."""
    d = draw("bf16", "scalar", 3, 4, 200, 128, 128, lens=[200, 64, 3], seed=10)
    _, state = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], lens=d["lens"])
    t = draw("bf16", "scalar", 3, 4, 1, 128, 128, seed=11)
    o = B.linear_recurrent_fwd(t["q"], t["k"], t["v"], t["g"], state)
    torch.cuda.synchronize()
    for b, n in enumerate([200, 64, 3]):
        cat = {m: torch.cat([d[m][b:b + 1, :, :n], t[m][b:b + 1]], 2) for m in ("q", "k", "v", "g")}
        val, mag = R.reference(cat["q"], cat["k"], cat["v"], cat["g"], d["h0"][b:b + 1])
        val["o"], mag["o"] = val["o"][:, :, n:], mag["o"][:, :, n:]
        R.check({"o": o[b:b + 1], "hT": state[b:b + 1]}, val, mag, torch.bfloat16, f"prompt {n} then a token")


@pytest.mark.parametrize("gate", ["head", "scalar"])
def test_autograd(gate):
    d = draw("fp32", gate, 2, 2, 100, 32, 64, lens=[100, 31], seed=12)
    names = ["q", "k", "v", "h0"] + (["g"] if gate == "scalar" else [])
    for n in names:
        d[n].requires_grad_(True)
    o, hT = B.LinearAttention.apply(d["q"], d["k"], d["v"], d["g"], d["h0"], d["lens"])
    (o * d["do"]).sum().backward(retain_graph=True)
    got = {("d" + n): d[n].grad.clone() for n in names}
    with torch.no_grad():
        plain = {n: (t.detach() if torch.is_tensor(t) else t) for n, t in d.items()}
        val, mag = R.reference(plain["q"], plain["k"], plain["v"], plain["g"], plain["h0"], plain["lens"],
                               plain["do"], None)
    R.check(got, {n: val[n] for n in got}, {n: mag[n] for n in got}, torch.float32, f"autograd {gate}")


def test_gradient_against_differences():
    """fp32: central differences of L = <o, do> + <hT, dhT> along random directions, L summed in 64 bits."""
    d = draw("fp32", "scalar", 1, 2, 150, 32, 32, seed=13)
    gr = run(d)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(14)

    def loss(e):
        o, hT = B.linear_fwd(e["q"], e["k"], e["v"], e["g"], e["h0"])
        return float((o.double() * d["do"].double()).sum() + (hT.double() * d["dhT"].double()).sum())

    for n in ("q", "k", "v", "g", "h0"):
        x = d[n]
        u = torch.randn(x.shape, generator=gen, device="cuda")
        # fp32 results: each of N values off by some 2^-22 of its size, a difference quotient by
        # 2^-22 sqrt(N) |o| |do| / step; the third order term is step^2 of the quotient
        step = 1e-2 if n != "g" else 1e-3
        hi, lo = loss({**d, n: x + step * u}), loss({**d, n: x - step * u})
        want = float((gr["d" + n].double() * u.double()).sum())
        scale = float(gr["d" + n].double().norm() * u.double().norm())
        print(n, (hi - lo) / (2 * step), want, scale, flush=True)
        assert abs((hi - lo) / (2 * step) - want) <= 2e-3 * scale


def test_graph_capture():
    """Forward, backward and a token captured once; replays with new inputs and eager work
    between them give the eager results."""
    shape = ("bf16", "scalar", 1, 2, 1100, 64, 128)
    static = draw(*shape, seed=20)
    state = torch.zeros(1, 2, 128, 64, device="cuda")

    def step(d, st):
        out = {}
        out["o"], out["hT"] = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"])
        out.update(B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"]))
        st.copy_(out["hT"])
        sl = {n: d[n][:, :, :1].contiguous() for n in ("q", "k", "v", "g")}
        out["tok"] = B.linear_recurrent_fwd(sl["q"], sl["k"], sl["v"], sl["g"], st)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static, state)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static, state)
    for seed in (21, 22, 23):
        fresh = draw(*shape, seed=seed)
        for n, t in fresh.items():
            if t is not None:
                static[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        st = torch.zeros_like(state)
        ref = step(fresh, st)
        torch.cuda.synchronize()
        for n, t in ref.items():
            assert torch.equal(out[n], t), (seed, n)
        assert torch.equal(state, st)


def test_other_stream_and_shared_workspace():
    d = draw("bf16", "scalar", 1, 2, 2100, 64, 64, seed=30)
    ref = run(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sh = B.make_shape(1, 2, 2100, 64, 64, 64, "bf16", "scalar")
    ws = torch.empty(max(B.dn_linear_workspace_bytes(sh, B.DN_PASS_BWD), B.dn_linear_workspace_bytes(sh, B.DN_PASS_FWD)),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)   # NaN patterns: scratch is never read before it is written
    side.wait_stream(torch.cuda.current_stream())
    o, hT = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], ws=ws, stream=side)
    gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], ws=ws, stream=side)
    side.synchronize()
    for n, t in {"o": o, "hT": hT, **gr}.items():
        assert torch.equal(t, ref[n]), n


def test_guard_bands():
    """Outputs and workspace inside pattern-filled margins through the raw calls: nothing is
    written outside them, and inputs stay as they are."""
    for dtype, (Bn, H, T, dk, dv), lens in (("bf16", (2, 1, 1300, 128, 64), [1300, 90]), ("fp32", (1, 3, 77, 16, 128), None)):
        d = draw(dtype, "scalar", Bn, H, T, dk, dv, lens=lens, seed=40)
        keep = {n: t.clone() for n, t in d.items() if t is not None}
        ref = run(d)
        sh = B.make_shape(Bn, H, T, dk, dv, 64, dtype, "scalar")
        margin = 4096
        bufs, views = [], {}

        def banded(name, like=None, nbytes=None):
            n = nbytes if like is None else like.numel() * like.element_size()
            buf = torch.full((n + 2 * margin,), 0xA5, dtype=torch.uint8, device="cuda")
            bufs.append((name, buf, n))
            mid = buf[margin:margin + n]
            views[name] = mid if like is None else mid.view(like.dtype).view(like.shape)
            return views[name]

        nf, nb = B.dn_linear_workspace_bytes(sh, B.DN_PASS_FWD), B.dn_linear_workspace_bytes(sh, B.DN_PASS_BWD)
        st = B.dn_linear_fwd(sh, d["q"], d["k"], d["v"], d["g"], d["lens"], d["h0"], banded("o", ref["o"]),
                             banded("hT", ref["hT"]), banded("wf", nbytes=nf) if nf else None, nf)
        assert st == B.DN_OK
        outs = [banded(n, ref[n]) for n in ("dq", "dk", "dv", "dg", "dh0")]
        st = B.dn_linear_bwd(sh, d["q"], d["k"], d["v"], d["g"], d["lens"], d["h0"], d["do"], d["dhT"], *outs,
                             banded("wb", nbytes=nb), nb)
        assert st == B.DN_OK
        torch.cuda.synchronize()
        for name, buf, n in bufs:
            assert bool((buf[:margin] == 0xA5).all()) and bool((buf[margin + n:] == 0xA5).all()), name
        for n in ref:
            assert torch.equal(views[n], ref[n]), n
        for n, t in keep.items():
            assert torch.equal(d[n], t), n


def test_memory_of_a_call_on_another_stream():
    """Workspace that the wrapper allocates for a call on a side stream is not handed out to the
    current stream's tensors while that call runs."""
    d = draw("bf16", "scalar", 1, 2, 4000, 64, 64, seed=41)
    ref = run(d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(16)]
        side.synchronize()
        for n, t in gr.items():
            assert torch.equal(t, ref[n]), n
        del junk, gr


def test_memory_of_a_call_on_the_default_stream_by_its_handle():
    """stream=0 names the default stream: what the wrapper allocates for it is that stream's memory,
    not another's, which would hand it out again while the default stream still works on it."""
    d = draw("fp32", "head", 1, 2, 2048, 64, 64, seed=42)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        o, _ = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], None, want_hT=False, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(o, B.linear_fwd(d["q"], d["k"], d["v"], d["g"], None, want_hT=False)[0])
    own = [s for s in torch.cuda.memory_snapshot() if 0 <= o.data_ptr() - s["address"] < s["total_size"]]
    assert [s["stream"] for s in own] == [0]
