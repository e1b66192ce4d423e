"""Trees of drafted tokens on the recurrent state against a node-by-node evaluation in 64
bits: every gate, delta rule and linear attention, both I/O types, chains, bushes and
empty trees; the commit of an accepted path; a serving run through all of it."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
from delta_rule_linear_gated_amd import workloads as W

pytestmark = pytest.mark.gpu
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}
# fp32 rounding of a node's sums: products of up to 128 terms, a system of up to 64 nodes
# whose rows sum to O(1) (unit keys, beta <= 1) and exponentials good to a few 2^-24 of a
# path's sum: under 400 half steps in a row.
U32, ROUNDINGS = 2.0 ** -24, 400


def draw(dtype, gate, delta, Bn, H, N, dk, dv, shape="bush", counts=None, seed=1, scale=1 / 16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rn = lambda *d: torch.randn(d, generator=gen, device="cuda")
    unit = lambda *d: torch.nn.functional.normalize(rn(*d), dim=-1).to(IO[dtype])
    d = {"q": unit(Bn, H, N, dk), "k": unit(Bn, H, N, dk), "v": rn(Bn, H, N, dv).to(IO[dtype]),
         "beta": torch.sigmoid(rn(Bn, H, N)) if delta else None, "state": 0.5 * rn(Bn, H, dv, dk),
         "counts": None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")}
    soft = torch.nn.functional.softplus
    d["g"] = {"none": None, "head": -torch.rand(H, generator=gen, device="cuda") * 0.3,
              "scalar": -scale * soft(rn(Bn, H, N)), "vector": -scale * soft(rn(Bn, H, N, dk))}[gate]
    n = torch.arange(N, device="cuda")
    if shape == "chain":
        parent = (n - 1).expand(Bn, N)
    elif shape == "star":
        parent = torch.full((Bn, N), -1, device="cuda")
    else:
        parent = (torch.rand(Bn, N, generator=gen, device="cuda") * (n + 1)).long() - 1
    d["parent"] = parent.to(torch.int32).contiguous()
    return d


def factor(g, n):
    """Decay of node n over [B, H, dv, dk]."""
    if g is None:
        return 1.0
    if g.dim() == 1:
        return g.double().clamp_min(-1000).exp()[None, :, None, None]
    x = g[:, :, n].double().clamp_min(-1000).exp()
    return x[..., None, None] if g.dim() == 3 else x[:, :, None, :]


def reference(d, kz=None):
    """(o, u, states after each node), and the magnitudes of their terms, node by node in fp64."""
    Bn, H, N, dk = d["q"].shape
    rows = torch.arange(Bn, device="cuda")
    cnt = torch.full((Bn,), N, device="cuda") if d["counts"] is None else d["counts"].clamp(0, N).long()
    S, A = [d["state"].double()], [d["state"].double().abs()]
    O, Uo, MO, MU = [], [], [], []
    for n in range(N):
        p = d["parent"][:, n].long()
        p = torch.where((p >= 0) & (p < n), p, -1) + 1
        f = factor(d["g"], n)
        s, a = torch.stack(S)[p, rows] * f, torch.stack(A)[p, rows] * f
        k, q, v = (d[m][:, :, n].double()[..., None] for m in ("k", "q", "v"))
        if d["beta"] is None:
            u, mu = v, v.abs()
        else:
            b = d["beta"][:, :, n].double()[..., None, None]
            if kz is not None:
                b = b / ((k * k).sum(2, keepdim=True) + kz)
            u, mu = b * (v - s @ k), b * (v.abs() + a @ k.abs())
        S.append(s + u @ k.transpose(-1, -2))
        A.append(a + mu @ k.transpose(-1, -2).abs())
        ok = (n < cnt).double()[:, None, None]
        O.append((S[-1] @ q)[..., 0] * ok)
        MO.append((A[-1] @ q.abs())[..., 0] * ok)
        Uo.append(u[..., 0] * ok)
        MU.append(mu[..., 0] * ok)
    st = lambda x: torch.stack(x, 2) if x else torch.zeros(Bn, H, 0, d["v"].shape[3], dtype=torch.float64, device="cuda")
    return {"o": st(O), "u": st(Uo)}, {"o": st(MO), "u": st(MU)}, S, A


def close(got, ref, mag, label):
    assert got.shape == ref.shape, label
    if not ref.numel():
        return
    lim = ROUNDINGS * U32 * mag + 1e-30
    if got.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * ref.abs()   # one rounding of the result
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), label
    over, rel = float((err / lim).max()), float(err.norm() / ref.norm().clamp_min(1e-30))
    print(f"{label}: rel {rel:.2e}, worst element at {over:.3f} of its bound", flush=True)
    assert over <= 1, label
    # as a whole: one rounding moves each value by at most 2^-8 of it, so their 2-norm by at most
    # 2^-8 of the results'; 100 half steps for the fp32 sums
    assert rel <= (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0) + 100 * U32, label


def verify(d, label, kz=None):
    before = d["state"].clone()
    o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"], counts=d["counts"],
                      kaczmarz_eps=kz)
    torch.cuda.synchronize()
    ref, mag, S, A = reference(d, kz)
    close(o, ref["o"], mag["o"], label + " o")
    close(u, ref["u"], mag["u"], label + " u")
    assert torch.equal(d["state"], before)
    return u, S, A


SHAPES = [
    # B, H, N, dk, dv, form, counts
    (1, 1, 1, 16, 16, "bush", None),
    (2, 3, 7, 32, 64, "bush", [7, 0]),
    (1, 8, 16, 128, 128, "bush", None),
    (3, 2, 17, 64, 48, "bush", [17, 1, 16]),
    (2, 4, 32, 128, 64, "chain", None),
    (1, 3, 33, 16, 128, "star", None),
    (2, 2, 64, 128, 128, "bush", [64, 50]),
    (1, 2, 64, 64, 80, "chain", [-5]),
    (1, 3, 61, 32, 272, "chain", None),
]


@pytest.mark.parametrize("delta", [True, False], ids=["delta", "linear"])
@pytest.mark.parametrize("gate", ["none", "head", "scalar", "vector"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_nodes(shape, dtype, gate, delta):
    Bn, H, N, dk, dv, form, counts = shape
    verify(draw(dtype, gate, delta, Bn, H, N, dk, dv, form, counts), f"{dtype} {gate} {shape}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["scalar", "vector"])
def test_steep_gates_and_resets(gate, dtype):
    """Paths whose decay leaves the range of an exponential, and -inf (the type's lowest value
    too): a reset."""
    d = draw(dtype, gate, True, 2, 2, 40, 64, 64, "chain", seed=3, scale=6.0)
    d["g"][0, 0, 5] = -torch.inf
    d["g"][1, 1, 0] = torch.finfo(torch.float32).min
    verify(d, f"steep {gate} {dtype}")
    d = draw(dtype, gate, True, 1, 2, 20, 64, 64, "bush", seed=4, scale=1 / 16)
    d["g"][0, 1, 3:5] = -torch.inf
    verify(d, f"reset {gate} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.6, 1.1, 1.4, 1.8, 2.5])
def test_long_decays_of_channels(scale, dtype):
    """Paths whose channels decay by e^-20 to e^-90, on both sides of where the pairs' decays
    stop being products of two factors."""
    for N in (16, 40):
        d = draw(dtype, "vector", True, 2, 2, N, 64, 64, "chain", seed=30, scale=scale * 40 / N)
        verify(d, f"long decay {scale} {N} {dtype}")


@pytest.mark.parametrize("gate", ["scalar", "vector"])
def test_kaczmarz_steps(gate):
    d = draw("bf16", gate, True, 2, 2, 24, 64, 64, seed=5)
    d["k"] = (d["k"].float() * 3).to(torch.bfloat16)
    verify(d, f"kaczmarz {gate}", kz=1e-3)


def test_parents_that_are_no_earlier_node_are_the_root():
    d = draw("fp32", "scalar", True, 2, 2, 20, 32, 32, seed=6)
    d["parent"][0, 3], d["parent"][0, 7], d["parent"][1, 5] = 3, 1000, -7
    u, _, _ = verify(d, "bad parents")
    e = {**d, "parent": d["parent"].clone()}
    e["parent"][0, 3] = e["parent"][0, 7] = e["parent"][1, 5] = -1
    o2, u2 = B.tree_fwd(e["q"], e["k"], e["v"], e["beta"], e["g"], e["parent"], e["state"])
    assert torch.equal(u, u2)


@pytest.mark.parametrize("delta", [True, False], ids=["delta", "linear"])
@pytest.mark.parametrize("gate", ["none", "head", "scalar", "vector"])
@pytest.mark.parametrize("shape", [(3, 2, 16, 128, 128), (4, 3, 64, 64, 80), (3, 1, 9, 16, 272), (3, 5, 33, 32, 16)],
                         ids=lambda s: "x".join(map(str, s)))
def test_commit(shape, gate, delta):
    """Paths of every length, nothing accepted and indexes outside the tree."""
    for dtype, form in (("bf16", "bush"), ("fp32", "chain")):
        d = draw(dtype, gate, delta, *shape, form, seed=7)
        Bn, N = shape[0], shape[2]
        u, S, A = verify(d, f"{dtype} {gate} {form}")
        for accept in ([-1, N - 1, N // 2, 0], [0, N, -2 ** 31, N - 1], [N - 1, N - 2, 1, 2 ** 31 - 1]):
            at = torch.tensor(accept[:Bn], dtype=torch.int32, device="cuda")
            state = d["state"].clone()
            B.tree_commit(d["k"], u, d["g"], d["parent"], at, state)
            torch.cuda.synchronize()
            for b in range(Bn):
                a = accept[b]
                if 0 <= a < N:
                    close(state[b], S[a + 1][b], A[a + 1][b], f"commit {accept} {b}")
                else:
                    assert torch.equal(state[b], d["state"][b])


def test_commit_of_nothing_reads_nothing():
    d = draw("bf16", "scalar", True, 2, 2, 8, 32, 32, seed=8)
    u = torch.full((2, 2, 8, 32), torch.nan, device="cuda")
    state = d["state"].clone()
    state[1] = torch.nan
    at = torch.tensor([-1, -1], dtype=torch.int32, device="cuda")
    B.tree_commit(d["k"], u, d["g"], d["parent"], at, state)
    assert torch.equal(state[0], d["state"][0])


def test_empty():
    for Bn, N in ((2, 0), (0, 5)):
        d = draw("bf16", "vector", True, Bn, 2, N, 32, 32, seed=9)
        o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
        state = d["state"].clone()
        B.tree_commit(d["k"], u, d["g"], d["parent"], torch.zeros(Bn, dtype=torch.int32, device="cuda"), state)
        assert o.shape == (Bn, 2, N, 32) and torch.equal(state, d["state"])


def test_chain_equals_the_recurrent_kernel():
    """A chain of drafted tokens, all accepted, against decoding them one after the other."""
    d = draw("fp32", "vector", True, 2, 4, 12, 128, 128, "chain", seed=10)
    o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
    state = d["state"].clone()
    at = torch.full((2,), 11, dtype=torch.int32, device="cuda")
    B.tree_commit(d["k"], u, d["g"], d["parent"], at, state)
    want = d["state"].clone()
    ow = B.recurrent_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], want)
    # two fp32 evaluations of the same sums
    for x, y in ((o, ow), (state, want)):
        assert float((x - y).norm() / y.norm()) <= 200 * U32


@pytest.mark.parametrize("kind", ["delta", "linear"])
def test_serving_run(kind):
    """Prompt, drafted tree, commit of a branch, then single tokens: the same as the branch's
    tokens decoded one by one after the prompt."""
    Bn, H, T, dk, dv, N = 2, 4, 150, 64, 64, 16
    d = draw("fp32", "scalar", kind == "delta", Bn, H, N, dk, dv, "bush", seed=11)
    w = W.custom(Bn, H, T, dk, dv, 64, "scalar", "fp32", h0_std=0.5, seed=12)
    p = {n: (None if t is None else t.cuda()) for n, t in W.make_inputs(w, cotangents=False).items()}
    if kind == "delta":
        _, state, _ = B.chunk_fwd(p["q"], p["k"], p["v"], p["beta"], p["g"], p["h0"], C=32, save_states=False)
        token = lambda x, st: B.recurrent_fwd(x["q"], x["k"], x["v"], x["beta"], x["g"], st)
    else:
        _, state = B.linear_fwd(p["q"], p["k"], p["v"], p["g"], p["h0"])
        token = lambda x, st: B.linear_recurrent_fwd(x["q"], x["k"], x["v"], x["g"], st)
    want = state.clone()
    o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], state)
    at = torch.tensor([N - 1, N // 2], dtype=torch.int32, device="cuda")
    B.tree_commit(d["k"], u, d["g"], d["parent"], at, state)
    one = {n: (t[:, :, :1].contiguous() if torch.is_tensor(t) and t.dim() >= 3 else t) for n, t in
           draw("fp32", "scalar", kind == "delta", Bn, H, 1, dk, dv, seed=13).items() if n not in ("state", "parent")}
    o1 = token(one, state)
    for b in range(Bn):
        path, n = [], int(at[b])
        while n >= 0:
            path.insert(0, n)
            n = int(d["parent"][b, n])
        st = want[b:b + 1].clone()
        for n in path:
            x = {m: (None if d[m] is None else d[m][b:b + 1, :, n:n + 1].contiguous()) for m in ("q", "k", "v", "beta", "g")}
            on = token(x, st)
            assert float((on[:, :, 0] - o[b:b + 1, :, n]).norm() / on.norm()) <= 400 * U32
        x = {m: (None if t is None else t[b:b + 1].contiguous()) for m, t in one.items() if m in ("q", "k", "v", "beta", "g")}
        ow = token(x, st)
        assert float((o1[b:b + 1] - ow).norm() / ow.norm()) <= 400 * U32
        assert float((state[b:b + 1] - st).norm() / st.norm()) <= 400 * U32


def test_graph_capture():
    """Verify, commit and a token captured once and replayed with new inputs and trees."""
    args = ("bf16", "vector", True, 2, 4, 20, 64, 64)
    static = draw(*args, seed=20)
    at = torch.tensor([3, 19], dtype=torch.int32, device="cuda")

    def step(d, at):
        o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
        B.tree_commit(d["k"], u, d["g"], d["parent"], at, d["state"])
        return o, u

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step({**static, "state": static["state"].clone()}, at)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, u = step(static, at)
    for seed in (21, 22, 23):
        fresh = draw(*args, seed=seed)
        for n, t in fresh.items():
            if t is not None:
                static[n].copy_(t)
        at.copy_(torch.tensor([seed % 20, -1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ro, ru = step(fresh, at)
        torch.cuda.synchronize()
        assert torch.equal(o, ro) and torch.equal(u, ru) and torch.equal(static["state"], fresh["state"]), seed


def test_guard_bands():
    for dtype, gate, shape in (("bf16", "vector", (2, 3, 19, 64, 80)), ("fp32", "scalar", (1, 2, 64, 128, 16))):
        d = draw(dtype, gate, True, *shape, seed=40)
        Bn, H, N, dk, dv = shape
        keep = {n: t.clone() for n, t in d.items() if t is not None}
        o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
        at = torch.full((Bn,), N - 1, dtype=torch.int32, device="cuda")
        want = B.tree_commit(d["k"], u, d["g"], d["parent"], at, d["state"].clone())
        margin, bufs = 4096, []

        def banded(like):
            n = like.numel() * like.element_size()
            buf = torch.full((n + 2 * margin,), 0xA5, dtype=torch.uint8, device="cuda")
            bufs.append((buf, n))
            return buf[margin:margin + n].view(like.dtype).view(like.shape)

        sh = B.make_shape(Bn, H, N, dk, dv, 64, dtype, gate)
        o2, u2, st = banded(o), banded(u), banded(want)
        st.copy_(d["state"])
        assert B.dn_tree_fwd(sh, d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], None, d["state"], o2, u2) == B.DN_OK
        assert B.dn_tree_commit(sh, d["k"], u2, d["g"], d["parent"], at, st) == B.DN_OK
        torch.cuda.synchronize()
        for buf, n in bufs:
            assert bool((buf[:margin] == 0xA5).all()) and bool((buf[margin + n:] == 0xA5).all())
        assert torch.equal(o, o2) and torch.equal(u, u2) and torch.equal(st, want)
        for n, t in keep.items():
            assert torch.equal(d[n], t), n
