"""The gate's gradient of packed sequences: a gate of a zero factor (a reset) has none, and what
one document holds enters no other's, exactly."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
from gate_ref import gate_gradient
from test_gpu_linear import draw

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
LOWEST = torch.finfo(torch.float32).min


def packed(dtype, H, T, dk, dv, starts, silent, h0, lens=None, seed=70):
    """Documents that start at `starts` (a reset there); those in `silent` have no cotangent."""
    d = draw(dtype, "scalar", 1, H, T, dk, dv, h0=h0, lens=lens, seed=seed)
    resets = [-torch.inf, LOWEST, -1001.0, -200.0]
    for i, t in enumerate(starts):
        d["g"][:, :, t] = resets[i % 4]
    edges = [0, *starts, T]
    for i in silent:
        d["do"][:, :, edges[i]:edges[i + 1]] = 0
    if len(edges) - 2 in silent:
        d["dhT"].zero_()
    return d, edges


CASES = [
    # H, T, starts, silent documents
    (2, 200, [100], [0]),
    (2, 200, [100], [1]),
    (1, 700, [1, 63, 64, 65, 128, 300, 301, 302, 511, 640], [0, 2, 4, 6, 8, 10]),
    (1, 700, [1, 63, 64, 65, 128, 300, 301, 302, 511, 640], [1, 3, 5, 7, 9]),
    (2, 2500, [5, 1000, 1024, 1025, 1990, 2400], [0, 2, 4, 6]),
    (2, 2500, [5, 1000, 1024, 1025, 1990, 2400], [1, 3, 5]),
    (1, 300, [], [0]),
]


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}-{len(c[2])}-{c[3][0]}")
def test_documents_keep_their_gate_gradients(case, dtype, no_scan):
    H, T, starts, silent = case
    d, edges = packed(dtype, H, T, 64, 32, starts, silent, h0=T % 200 == 0)
    gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], no_scan=no_scan)
    torch.cuda.synchronize()
    dg = gr["dg"]
    for t in starts:
        assert not dg[:, :, t].any(), t
    for i in silent:
        assert not dg[:, :, edges[i]:edges[i + 1]].any(), (i, edges[i], edges[i + 1])
    for h in range(H):
        val, mag, run = gate_gradient(d["q"][0, h], d["k"][0, h], d["v"][0, h], d["g"][0, h],
                                      None if d["h0"] is None else d["h0"][0, h], d["do"][0, h], d["dhT"][0, h])
        # at most 400 fp32 roundings on the way of each step's part (dots of up to 128 channels,
        # chunks of 64, a few dozen chunk updates), which add up over the run between two resets
        err, lim = (dg[0, h].double() - val).abs(), 400 * U32 * (mag + run) + 1e-30
        over = float((err / lim).max())
        print(f"{dtype} {case[1:]} head {h}: worst at {over:.3f} of its bound", flush=True)
        assert over <= 1
    if len(silent) == len(edges) - 1:
        assert not dg.any()


def test_a_reset_past_the_length_cuts_nothing():
    """Gates behind a sequence's length are no part of it, resets there either."""
    d, _ = packed("fp32", 2, 300, 64, 64, [], [], h0=True, lens=[200], seed=71)
    ref = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], lens=d["lens"])
    d["g"][:, :, 200:] = -torch.inf
    got = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], lens=d["lens"])
    for n in ref:
        assert torch.equal(got[n], ref[n]), n
