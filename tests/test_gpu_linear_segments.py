"""Parallel segments longer than the distance of the kept states (the gate's gradient), whose last
is shorter, over batches whose lengths end inside a segment's stretches, leave whole segments
empty, or are zero: against the 64-bit definition, as one run of the steps too."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
import linear_ref as R
from gate_ref import gate_gradient
from test_gpu_linear import draw, run
from test_linear_plan import plan

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24

SHAPES = [
    # dtype, B, H, T, dk, dv, segments, chunks of each, chunks between kept states, lens
    ("bf16", 4, 15, 4268, 32, 16, (4, 18, 9), [4268, 1152 + 500, 1052, 0]),
    ("bf16", 2, 30, 5040, 16, 32, (4, 20, 10), None),
    ("fp32", 4, 20, 3130, 16, 16, (3, 18, 9), [3130, 2304, 577, 1]),
]


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_segments_of_several_stretches(shape, no_scan):
    dtype, Bn, H, T, dk, dv, want, lens = shape
    assert plan(Bn * H, T, dv, dtype, "dots") == want
    d = draw(dtype, "scalar", Bn, H, T, dk, dv, lens=lens, seed=90)
    got = run(d, no_scan)
    val, mag = R.reference(d["q"], d["k"], d["v"], d["g"], d["h0"], d["lens"], d["do"], d["dhT"])
    R.check(got, val, mag, d["q"].dtype, f"{shape} no_scan={no_scan}")
    for b in range(Bn):
        n = T if lens is None else lens[b]
        assert not got["dg"][b, :, n:].any()
        if n:
            cut = lambda t: t[b, H - 1, :n]
            ref, m, size = gate_gradient(*(cut(d[x]) for x in ("q", "k", "v", "g")), d["h0"][b, H - 1], cut(d["do"]),
                                         d["dhT"][b, H - 1])
            assert bool(((cut(got["dg"]).double() - ref).abs() <= 400 * U32 * (m + size)).all()), b
