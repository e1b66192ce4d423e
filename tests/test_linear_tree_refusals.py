"""What the linear-attention and tree entry points refuse, on the host (no GPU): the C
ABI by status, before anything is launched, and the wrappers by ValueError."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

FAKE = 1 << 30   # distinct, aligned addresses that are never read


def sh(**over):
    a = dict(B=2, H=3, T=40, dk=64, dv=32, C=64, dtype="bf16", gate="scalar", kaczmarz_eps=None, no_scan=False)
    a.update(over)
    return B.make_shape(**a)


def lin_fwd(s, ws_bytes=1 << 28, **over):
    a = dict(q=FAKE, k=FAKE * 2, v=FAKE * 3, g=FAKE * 4, lens=None, h0=FAKE * 5, o=FAKE * 6, hT=FAKE * 7, ws=FAKE * 8)
    a.update(over)
    return B.dn_linear_fwd(s, a["q"], a["k"], a["v"], a["g"], a["lens"], a["h0"], a["o"], a["hT"], a["ws"], ws_bytes, 0)


def lin_bwd(s, ws_bytes=1 << 28, **over):
    n = ("q", "k", "v", "g", "lens", "h0", "dout", "dhT", "dq", "dk", "dv", "dg", "dh0", "ws")
    a = {m: FAKE * (i + 1) for i, m in enumerate(n)}
    a["lens"] = None
    a.update(over)
    return B.dn_linear_bwd(s, *(a[m] for m in n), ws_bytes, 0)


def lin_rec(s, **over):
    n = ("q", "k", "v", "g", "state", "o")
    a = {m: FAKE * (i + 1) for i, m in enumerate(n)}
    a.update(over)
    return B.dn_linear_recurrent_fwd(s, *(a[m] for m in n), 0)


def tree(s, **over):
    n = ("q", "k", "v", "beta", "g", "parent", "counts", "state", "o", "u")
    a = {m: FAKE * (i + 1) for i, m in enumerate(n)}
    a.update(over)
    return B.dn_tree_fwd(s, *(a[m] for m in n), 0)


def commit(s, **over):
    n = ("k", "u", "g", "parent", "accept", "state")
    a = {m: FAKE * (i + 1) for i, m in enumerate(n)}
    a.update(over)
    return B.dn_tree_commit(s, *(a[m] for m in n), 0)


INVALID, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = (B.DN_ERR_INVALID, B.DN_ERR_SHAPE, B.DN_ERR_DTYPE, B.DN_ERR_WORKSPACE,
                                                 B.DN_ERR_UNSUPPORTED)


@pytest.mark.parametrize("call", [lin_fwd, lin_bwd, lin_rec])
def test_linear_shapes(call):
    assert call(sh(T=-1)) == SHAPE
    assert call(sh(dv=0)) == SHAPE
    assert call(sh(dtype=9)) == DTYPE
    assert call(sh(gate=4)) == INVALID and call(sh(gate=-1)) == INVALID
    assert call(sh(gate="vector")) == UNSUPPORTED
    assert call(sh(kaczmarz_eps=1e-6)) == UNSUPPORTED
    assert call(sh(dk=48)) == UNSUPPORTED
    assert call(sh(dk=256)) == UNSUPPORTED
    s = sh()
    s.flags = 64
    assert call(s) == INVALID


def test_linear_limits():
    for call in (lin_fwd, lin_bwd):
        assert call(sh(B=65536, H=1, T=1)) == UNSUPPORTED
        assert call(sh(dv=48)) == UNSUPPORTED
        assert call(sh(B=1, H=1, T=2 ** 31 - 1)) == UNSUPPORTED
    assert lin_rec(sh(dv=24)) == UNSUPPORTED


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "o"])
def test_linear_pointers(name):
    for call in (lin_fwd, lin_rec):
        assert call(sh(), **{name: None}) == INVALID and name in B.dn_last_error()
        assert call(sh(), **{name: FAKE * 20 + 8}) == INVALID and "aligned" in B.dn_last_error()
    if name != "o":
        assert lin_bwd(sh(), **{name: None}) == INVALID and name in B.dn_last_error()


def test_linear_overlaps_and_gates():
    assert lin_fwd(sh(), o=FAKE) == INVALID and "overlaps" in B.dn_last_error()
    assert lin_fwd(sh(), hT=FAKE * 5) == INVALID                       # in place on h0
    assert lin_fwd(sh(), lens=FAKE * 6) == INVALID                     # o over lens
    assert lin_rec(sh(), o=FAKE * 5) == INVALID                        # over the state
    assert lin_bwd(sh(), dq=FAKE * 10) == INVALID
    assert lin_fwd(sh(gate="none")) == INVALID                         # g given without a gate
    assert lin_bwd(sh(gate="none"), g=None) == INVALID                 # dg given without a gate
    assert lin_bwd(sh(gate="head")) == INVALID and "dg" in B.dn_last_error()
    assert lin_bwd(sh(gate="scalar"), dg=None) == INVALID and "dg" in B.dn_last_error()


def test_linear_workspace():
    few = sh(B=1, H=1, T=8192, dk=64, dv=64)
    for pass_, call in ((B.DN_PASS_FWD, lin_fwd), (B.DN_PASS_BWD, lin_bwd)):
        n = B.dn_linear_workspace_bytes(few, pass_)
        assert n > 0
        assert call(few, ws_bytes=n - 1) == WORKSPACE
        assert call(few, ws=None, ws_bytes=n) == INVALID
    # one run of the steps keeps no boundary states; many heads need none
    assert B.dn_linear_workspace_bytes(sh(B=1, H=1, T=8192, dk=64, dv=64, gate="head", no_scan=True), B.DN_PASS_BWD) == 0
    assert B.dn_linear_workspace_bytes(sh(B=8, H=64, T=8192, gate="none"), B.DN_PASS_FWD) == 0
    assert B.dn_linear_workspace_bytes(sh(gate="vector"), B.DN_PASS_FWD) == 0
    assert B.dn_linear_workspace_bytes(sh(), B.DN_PASS_BWD_RECOMPUTE) == 0


@pytest.mark.parametrize("call", [tree, commit])
def test_tree_shapes(call):
    assert call(sh(T=65)) == UNSUPPORTED and "nodes" in B.dn_last_error()
    assert call(sh(T=-2)) == SHAPE
    assert call(sh(dtype=2)) == DTYPE
    assert call(sh(gate=5)) == INVALID
    assert call(sh(dk=24)) == UNSUPPORTED
    assert call(sh(dv=40)) == UNSUPPORTED and call(sh(dv=0)) == UNSUPPORTED
    assert call(sh(gate="none")) == INVALID                            # g given without a gate
    assert call(sh(kaczmarz_eps=-1.0)) == INVALID
    assert call(sh(), state=None) == INVALID
    assert call(sh(), parent=None) == INVALID
    assert call(sh(), g=None) == INVALID
    assert call(sh(), g=FAKE * 30 + 4) == INVALID


def test_tree_pointers():
    assert tree(sh(), o=None) == INVALID
    assert tree(sh(), o=FAKE * 8) == INVALID                           # over the state
    assert tree(sh(), u=FAKE * 9) == INVALID                           # over o
    assert tree(sh(kaczmarz_eps=1e-6), beta=None) == INVALID           # a step size without eta
    assert commit(sh(), accept=None) == INVALID
    assert commit(sh(), u=None) == INVALID
    assert commit(sh(), state=FAKE * 2) == INVALID                     # over u


def test_more_heads_than_a_launch_holds():
    """A launch has less than 2^32 threads: calls past that are refused for it, the one before is not."""
    for B_, H in ((2 ** 23, 1), (4096, 2048), (2 ** 31 - 1, 2 ** 31 - 1)):
        s = sh(B=B_, H=H, T=1, dk=16, dv=16)
        for call in (tree, commit):
            assert call(s, state=None) == UNSUPPORTED and "B*H" in B.dn_last_error()
    for call in (tree, commit):
        assert call(sh(B=2 ** 23 - 1, H=1, T=1, dk=16, dv=16), state=None) == INVALID
        assert call(sh(B=2 ** 22, H=1, T=1, dk=16, dv=80), state=None) == UNSUPPORTED
    assert lin_rec(sh(B=2 ** 24, H=1, T=1, dk=16, dv=16), state=None) == UNSUPPORTED and "B*H" in B.dn_last_error()
    assert lin_rec(sh(B=2 ** 12, H=2 ** 8, T=1, dk=16, dv=256), state=None) == UNSUPPORTED
    assert lin_rec(sh(B=2 ** 24 - 1, H=1, T=1, dk=16, dv=16), state=None) == INVALID


def _tensors(dtype=torch.bfloat16, Bn=2, H=3, T=10, dk=32, dv=64):
    z = torch.zeros
    return dict(q=z(Bn, H, T, dk, dtype=dtype), k=z(Bn, H, T, dk, dtype=dtype), v=z(Bn, H, T, dv, dtype=dtype),
                g=z(Bn, H, T), h0=z(Bn, H, dv, dk), state=z(Bn, H, dv, dk), do=z(Bn, H, T, dv, dtype=dtype),
                dhT=z(Bn, H, dv, dk), lens=z(Bn, dtype=torch.int32), beta=z(Bn, H, T),
                parent=z(Bn, T, dtype=torch.int32), counts=z(Bn, dtype=torch.int32), u=z(Bn, H, T, dv),
                accept=z(Bn, dtype=torch.int32))


CALLS = {
    "fwd": lambda d: B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], lens=d["lens"]),
    "bwd": lambda d: B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], lens=d["lens"]),
    "step": lambda d: B.linear_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["state"]),
    "tree": lambda d: B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"], counts=d["counts"]),
    "commit": lambda d: B.tree_commit(d["k"], d["u"], d["g"], d["parent"], d["accept"], d["state"]),
}
USES = {"fwd": "q k v g h0 lens", "bwd": "q k v g h0 do dhT lens", "step": "q k v g state",
        "tree": "q k v beta g parent state counts", "commit": "k u g parent accept state"}


@pytest.mark.parametrize("call", CALLS)
def test_wrappers_refuse_wrong_tensors(call):
    for name in USES[call].split():
        for bad in (lambda t: t.double(), lambda t: t[..., :-1].contiguous(), lambda t: t.unsqueeze(0)):
            d = _tensors()
            d[name] = bad(d[name])
            with pytest.raises(ValueError):
                CALLS[call](d)
        d = _tensors()
        if d[name].dim() >= 2:
            d[name] = d[name].transpose(-1, -2).contiguous().transpose(-1, -2)
            with pytest.raises(ValueError, match="contiguous"):
                CALLS[call](d)
    with pytest.raises(ValueError, match="CUDA device"):
        CALLS[call](_tensors())


def test_a_gate_per_channel_is_for_trees_only():
    d = _tensors()
    d["g"] = torch.zeros(2, 3, 10, 32)
    for call in ("fwd", "bwd", "step"):
        with pytest.raises(ValueError, match="g must have shape"):
            CALLS[call](d)
    with pytest.raises(ValueError, match="CUDA device"):
        CALLS["tree"](d)


def test_a_constant_decay_gets_no_gradient():
    d = _tensors()
    with pytest.raises(ValueError, match="constant"):
        B.LinearAttention.apply(d["q"], d["k"], d["v"], torch.zeros(3, requires_grad=True), d["h0"], None)
