"""What the gated recurrence and the norms and rotations of queries and keys refuse, on the host
(no GPU): the C ABI by status, before anything is launched, and the wrappers by ValueError; the
frequencies of scaled positions."""
import math

import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

FAKE = 1 << 34   # distinct, aligned addresses that are never read
INVALID, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = (B.DN_ERR_INVALID, B.DN_ERR_SHAPE, B.DN_ERR_DTYPE, B.DN_ERR_WORKSPACE,
                                                 B.DN_ERR_UNSUPPORTED)


def sh(flags=0, **over):
    a = dict(B=2, H=3, T=40, dk=64, dv=33, C=64, dtype="bf16", gate="vector")
    a.update(over)
    s = B.make_shape(**a)
    s.flags = flags
    return s


def call(fn, names, s, ws_bytes=None, **over):
    a = {m: FAKE * (i + 1) for i, m in enumerate(names)}
    a["lens"] = None
    a.update(over)
    tail = () if ws_bytes is None else (ws_bytes,)
    return fn(s, *(a[m] for m in names), *tail, 0)


def fwd(s, ws_bytes=1 << 28, **over):
    return call(B.dn_gated_scan_fwd, ("x", "g", "lens", "h0", "o", "hT", "states", "ws"), s, ws_bytes, **over)


def bwd(s, ws_bytes=1 << 28, **over):
    return call(B.dn_gated_scan_bwd, ("x", "g", "lens", "h0", "dout", "dhT", "states", "dx", "dg", "dh0", "ws"), s, ws_bytes,
                **over)


def rec(s, **over):
    return call(B.dn_gated_scan_recurrent_fwd, ("x", "g", "state", "o"), s, None, **over)


@pytest.mark.parametrize("f", [fwd, bwd, rec])
def test_scan_shapes(f):
    assert f(sh(T=-1)) == SHAPE and f(sh(B=-1)) == SHAPE and f(sh(dv=0)) == SHAPE
    assert f(sh(dtype=7)) == DTYPE
    assert f(sh(gate=4)) == INVALID and f(sh(gate=-1)) == INVALID
    for gate in ("none", "scalar", "head"):
        assert f(sh(gate=gate)) == UNSUPPORTED
    for flags in (B.DN_FLAG_KACZMARZ, B.DN_FLAG_NO_SCAN, 8):
        assert f(sh(flags=flags)) == INVALID
    assert f(sh(T=2 ** 30 + 1)) == UNSUPPORTED and f(sh(dv=2 ** 21 + 1)) == UNSUPPORTED
    for B_, H, d in ((2 ** 28, 1, 1), (2 ** 22, 1, 64), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 21), (1, 128, 2 ** 21)):
        assert f(sh(B=B_, H=H, dv=d, T=1)) == UNSUPPORTED and "B*H*dv" in B.dn_last_error()
    assert f(sh(B=2 ** 28 - 64, H=1, dv=1, T=1), x=None) == INVALID   # the most that one launch holds


@pytest.mark.parametrize("f,names", [(fwd, "x g o"), (bwd, "x g dout dx dg"), (rec, "x g state o")])
def test_scan_pointers(f, names):
    for n in names.split():
        assert f(sh(), **{n: None}) == INVALID and n in B.dn_last_error()
        assert f(sh(), **{n: FAKE * 30 + 8}) == INVALID and "aligned" in B.dn_last_error()


def test_scan_overlaps():
    assert fwd(sh(), o=FAKE) == INVALID and "overlaps" in B.dn_last_error()      # in place on x
    assert fwd(sh(), hT=FAKE * 4) == INVALID and fwd(sh(), states=FAKE * 5) == INVALID
    assert fwd(sh(), lens=FAKE * 5) == INVALID
    assert bwd(sh(), dx=FAKE * 5) == INVALID and bwd(sh(), dg=FAKE * 2) == INVALID and bwd(sh(), dh0=FAKE * 6) == INVALID
    assert rec(sh(), o=FAKE * 3) == INVALID and rec(sh(), state=FAKE) == INVALID


def test_scan_workspace():
    few = sh(B=1, H=1, T=8192, dv=64)
    for pass_, f, more in ((B.DN_PASS_FWD, fwd, {}), (B.DN_PASS_BWD, bwd, {}), (B.DN_PASS_BWD_RECOMPUTE, bwd, {"states": None})):
        n = B.dn_gated_scan_workspace_bytes(few, pass_)
        assert n > 0
        assert f(few, ws_bytes=n - 1, **more) == WORKSPACE
        assert f(few, ws_bytes=n, ws=None, **more) == INVALID
    many = sh(B=8, H=16, T=4096, dv=128)
    assert B.dn_gated_scan_workspace_bytes(many, B.DN_PASS_FWD) == B.dn_gated_scan_workspace_bytes(many, B.DN_PASS_BWD) == 0
    assert B.dn_gated_scan_states_bytes(sh(T=129)) == 2 * 3 * 2 * 33 * 4
    assert B.dn_gated_scan_workspace_bytes(many, 3) == B.dn_gated_scan_workspace_bytes(sh(gate="none"), 0) == 0
    assert B.dn_gated_scan_states_bytes(sh(gate="none")) == 0


def test_other_operators_refuse_the_coupled_flag():
    s = sh(flags=B.DN_FLAG_COUPLED, dv=64, gate="scalar")
    p = [FAKE * (i + 1) for i in range(12)]
    assert B.dn_chunk_fwd(s, *p[:10], 1 << 40, 0) == INVALID
    assert B.dn_recurrent_fwd(s, *p[:7], 0) == INVALID
    assert B.dn_linear_fwd(s, *p[:4], None, p[5], p[6], p[7], p[8], 1 << 40, 0) == INVALID
    assert B.dn_tree_fwd(s, *p[:10], 0) == INVALID


def qk(**over):
    a = dict(B=2, Hq=3, Hk=2, T=5, d=64, rot=32, dtype=B.DN_BF16, norm=B.DN_NORM_RMS, layout=0, pos_kind=0, eps=1e-6,
             amplitude=1.0, q_stride=(5 * 320, 64, 320), k_stride=(5 * 320, 64, 320), dq_stride=(960, 64, 192),
             dk_stride=(640, 320, 64))
    a.update(over)
    strides = [a.pop(n + "_stride") for n in ("q", "k", "dq", "dk")]
    return B.QKShape(*a.values(), *(x for s in strides for x in s))


def qfwd(s, **over):
    n = ("q", "k", "wq", "wk", "freqs", "pos", "lens", "yq", "yk")
    return call(B.dn_qk_fwd, n, s, None, **over)


def qbwd(s, ws_bytes=1 << 28, **over):
    n = ("q", "k", "dyq", "dyk", "wq", "wk", "freqs", "pos", "lens", "dq", "dk", "dwq", "dwk", "ws")
    return call(B.dn_qk_bwd, n, s, ws_bytes, **over)


BARE = dict(q=None, k=None, wq=None, wk=None, dwq=None, dwk=None)   # the backward of a rotation alone


@pytest.mark.parametrize("f", [qfwd, qbwd])
def test_qk_shapes(f):
    for over in (dict(B=-1), dict(Hq=-1), dict(Hk=-1), dict(T=-1), dict(d=0), dict(rot=-8), dict(rot=72)):
        assert f(qk(**over)) == SHAPE, over
    assert f(qk(dtype=2)) == DTYPE
    for over in (dict(norm=3), dict(norm=-1), dict(layout=2), dict(layout=-1), dict(pos_kind=3), dict(pos_kind=-1),
                 dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(amplitude=math.inf)):
        assert f(qk(**over)) == INVALID, over
    for over in (dict(d=48), dict(d=256, rot=0), dict(rot=4), dict(rot=30), dict(rot=0, norm=0), dict(B=2 ** 20, T=2 ** 11),
                 dict(q_stride=(-1600, 64, 320)), dict(k_stride=(1600, 68, 320)), dict(q_stride=(2 ** 57, 64, 320)),
                 dict(B=2 ** 15, Hq=2 ** 15, T=2 ** 10)):
        assert f(qk(**over)) == UNSUPPORTED, over
    assert f(qk(norm=0)) == INVALID   # weights without a norm


def test_qk_strides():
    # a dimension of size 1 may have any stride; the rows of an output may not share memory
    assert qbwd(qk(B=1, dq_stride=(3, 64, 192), dk_stride=(7, 320, 64)), q=None) == INVALID and "q is NULL" in B.dn_last_error()
    for over in (dict(dq_stride=(960, 32, 192)), dict(dq_stride=(960, 64, 128)), dict(dq_stride=(0, 64, 192)),
                 dict(dk_stride=(640, 312, 64)), dict(dk_stride=(632, 320, 64))):
        assert qbwd(qk(**over)) == INVALID and "overlap" in B.dn_last_error(), over
        assert qfwd(qk(**over), q=None) == INVALID and "q is NULL" in B.dn_last_error()   # not read there


@pytest.mark.parametrize("f,names", [(qfwd, "q k freqs yq yk"), (qbwd, "q k dyq dyk freqs dq dk")])
def test_qk_pointers(f, names):
    for n in names.split():
        assert f(qk(), **{n: None}) == INVALID and n in B.dn_last_error()
        assert f(qk(), **{n: FAKE * 30 + 8}) == INVALID and "aligned" in B.dn_last_error()
    for kind in (1, 2):
        assert f(qk(pos_kind=kind), pos=None) == INVALID and "pos" in B.dn_last_error()
    assert f(qk(), **{names.split()[-1]: FAKE * 2}) == INVALID and "overlaps" in B.dn_last_error()


def test_qk_weights_and_workspace():
    assert qbwd(qk(), wq=None) == INVALID and "gradient without the weight" in B.dn_last_error()
    n = B.dn_qk_workspace_bytes(qk())
    assert n > 0 and qbwd(qk(), ws_bytes=n - 1) == WORKSPACE and qbwd(qk(), ws_bytes=n, ws=None) == INVALID
    assert qbwd(qk(), ws_bytes=0, ws=None, dwq=None, dwk=None, q=None) == INVALID and "q is NULL" in B.dn_last_error()
    assert qbwd(qk(norm=0), **{**BARE, "q": FAKE}) == INVALID
    assert qbwd(qk(norm=0), **{**BARE, "dq": None}) == INVALID and "dq" in B.dn_last_error()
    assert B.dn_qk_workspace_bytes(qk(norm=0)) == 0 and B.dn_qk_workspace_bytes(qk(d=24)) == 0


def tensors():
    z = torch.zeros
    q, k = z(2, 3, 5, 32), z(2, 2, 5, 32)
    return dict(x=z(2, 3, 5, 7), g=z(2, 3, 5, 7), h0=z(2, 3, 7), state=z(2, 3, 7), do=z(2, 3, 5, 7), dhT=z(2, 3, 7),
                states=z(2, 3, 1, 7), lens=z(2, dtype=torch.int32), q=q, k=k, wq=z(32), wk=z(32), dyq=z(2, 3, 5, 32),
                dyk=z(2, 2, 5, 32), freqs=z(8, dtype=torch.float64), pos=z(2, 5, dtype=torch.int32))


CALLS = {
    "fwd": (lambda d: B.gated_scan_fwd(d["x"], d["g"], d["h0"], lens=d["lens"]), "x g h0 lens"),
    "bwd": (lambda d: B.gated_scan_bwd(d["x"], d["g"], d["h0"], d["do"], d["dhT"], d["states"], lens=d["lens"]),
            "x g h0 do dhT states lens"),
    "step": (lambda d: B.gated_scan_recurrent_fwd(d["x"], d["g"], d["state"]), "x g state"),
    "norm": (lambda d: B.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], freqs=d["freqs"], pos=d["pos"], lens=d["lens"]),
             "q k wq wk freqs pos lens"),
    "norm_bwd": (lambda d: B.qk_norm_bwd(d["q"], d["k"], d["dyq"], d["dyk"], d["wq"], d["wk"], freqs=d["freqs"],
                                         pos=d["pos"], lens=d["lens"]), "q k dyq dyk wq wk freqs pos lens"),
    "rotary": (lambda d: B.rotary_fwd(d["q"], d["k"], d["freqs"], pos=d["pos"], lens=d["lens"]), "q k freqs pos lens"),
    "rotary_bwd": (lambda d: B.rotary_bwd(d["dyq"], d["dyk"], d["freqs"], pos=d["pos"], lens=d["lens"]),
                   "dyq dyk freqs pos lens"),
}


@pytest.mark.parametrize("name", CALLS)
def test_wrappers_refuse_wrong_tensors(name):
    f, uses = CALLS[name]
    for n in uses.split():
        if n in ("freqs",):
            bads = (lambda t: t.float(), lambda t: t[None])
        else:
            bads = (lambda t: t.half() if t.is_floating_point() else t.long(), lambda t: t[..., :-1].contiguous(),
                    lambda t: t.unsqueeze(0).unsqueeze(0))
        for bad in bads:
            d = tensors()
            d[n] = bad(d[n])
            with pytest.raises(ValueError):
                f(d)
        d = tensors()
        if d[n].dim() >= 2 and d[n].shape[-2] > 1:
            d[n] = d[n].transpose(-1, -2).contiguous().transpose(-1, -2)
            with pytest.raises(ValueError, match="contiguous|dense"):
                f(d)
    with pytest.raises(ValueError, match="CUDA device"):
        f(tensors())


def test_wrappers_refuse_what_cannot_be_meant():
    d = tensors()
    with pytest.raises(ValueError, match="must be given"):
        B.rotary_fwd(None, None, d["freqs"])
    with pytest.raises(ValueError, match="without freqs"):
        B.qk_norm_fwd(d["q"], d["k"], pos=d["pos"])
    with pytest.raises(ValueError, match="norm must be"):
        B.qk_norm_fwd(d["q"], d["k"], norm="layer")
    with pytest.raises(ValueError, match="no gradient"):
        B.Rotary.apply(d["q"], d["k"], d["freqs"].requires_grad_())


def test_frequencies():
    f, a = B.rotary_freqs(64)
    want = [10000.0 ** (-2 * m / 64) for m in range(32)]
    assert a == 1.0 and f.dtype == torch.float64 and f.tolist() == pytest.approx(want, rel=1e-14)
    f2, a = B.rotary_freqs(64, scaling="linear", factor=4.0)
    assert a == 1.0 and f2.tolist() == pytest.approx([x / 4 for x in want], rel=1e-14)
    f3, a = B.rotary_freqs(64, scaling="ntk", factor=4.0)
    assert a == 1.0 and float(f3[0]) == 1.0 and float(f3[-1]) == pytest.approx(want[-1] / 4, rel=1e-12)
    f4, a = B.rotary_freqs(64, scaling="yarn", factor=8.0, trained=4096)
    assert a == pytest.approx(0.1 * math.log(8) + 1)
    for x, y in zip(want, f4.tolist()):
        turns = 4096 * x / (2 * math.pi)
        keep = min(max((turns - 1) / 31, 0.0), 1.0)
        assert y == pytest.approx(x * keep + x / 8 * (1 - keep), rel=1e-14)
    assert f4.tolist()[0] == want[0] and f4.tolist()[-1] == pytest.approx(want[-1] / 8)
    for bad in (dict(rot=0), dict(rot=7), dict(rot=8, scaling="other"), dict(rot=8, factor=0.5), dict(rot=8, base=0.0),
                dict(rot=8, scaling="yarn", factor=2.0), dict(rot=8, scaling="yarn", factor=2.0, trained=64, fast=1.0)):
        with pytest.raises(ValueError):
            B.rotary_freqs(**bad)
