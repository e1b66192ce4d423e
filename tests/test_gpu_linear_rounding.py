"""bf16 results of linear attention against the 64-bit definition, element by element: what
stands between them is the result's own rounding and operands held to 16 bits.

The kernel's value before its rounding, y, is off the definition's r by at most e: a term's
two factors with two bf16 parts each (what both parts of x leave is at most 2^-16 |x|) and
400 fp32 roundings of partial sums of the terms, whose absolute values sum to `mag`.  The
distance of a value to the nearest bf16 changes by no more than the value does, so that
    |bf16(y) - r| <= |bf16(y) - y| + e <= |bf16(r) - r| + 2 e.
(An operand rounded to one bf16, 2^-8 of a term, breaks this bound by far.)"""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
import linear_ref as R
from test_gpu_linear import draw

pytestmark = pytest.mark.gpu
OPERAND, SUMS = 2 * 2.0 ** -16 * (1 + 2.0 ** -16), 400 * 2.0 ** -24


def close(got, val, mag, label):
    bad = []
    for n in ("o", "dq", "dk", "dv"):
        r = val[n]
        lim = (r.bfloat16().double() - r).abs() + 2 * (OPERAND + SUMS) * mag[n] + 1e-30
        over = float(((got[n].double() - r).abs() / lim).max())
        print(f"{label} {n}: worst element at {over:.3f} of its bound", flush=True)
        if not over <= 1:
            bad.append((n, over))
    assert not bad, (label, bad)


SHAPES = [
    # B, H, T, dk, dv, lens
    (2, 3, 300, 128, 128, [300, 130]),
    (1, 2, 197, 64, 128, None),
    (1, 3, 333, 16, 32, None),
    (1, 2, 2100, 128, 64, None),      # parallel segments: the same bound wherever a chunk is in its run
]


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("gate", ["none", "head", "scalar"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:5])))
def test_outputs_carry_one_rounding(shape, gate, no_scan):
    Bn, H, T, dk, dv, lens = shape
    d = draw("bf16", gate, Bn, H, T, dk, dv, lens=lens, seed=60)
    o, hT = B.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], lens=d["lens"], no_scan=no_scan)
    gr = B.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], lens=d["lens"], no_scan=no_scan)
    torch.cuda.synchronize()
    val, mag = R.reference(d["q"], d["k"], d["v"], d["g"], d["h0"], d["lens"], d["do"], d["dhT"])
    close({"o": o, **gr}, val, mag, f"{gate} {shape} no_scan={no_scan}")
