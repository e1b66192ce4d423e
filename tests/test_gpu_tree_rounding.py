"""bf16 outputs of trees: rounded from values held to fp32, whatever the gate.

A value y off the definition's r by e, much less than the distance s of bf16 values there, rounds
to another bf16 than r with a chance of e / s (r falls anywhere between two of them).  y is a sum
of terms S_c q_c (S the state after the node): with p their 2-norm, some 50 independent fp32
roundings of 0.58 half steps each leave e = 4 half steps of p in root mean square; three times that
is allowed, 12 * 2^-24 p.  The number of outputs that differ from the rounded definition is then at
most the sum of 12 * 2^-24 p / s, with five times its square root for chance.  (Operands held to 16
bits, off by 2^-17.8 of a term in root mean square, would give five times as many.)"""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
from test_gpu_tree import draw, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("delta", [True, False], ids=["delta", "linear"])
@pytest.mark.parametrize("gate,scale", [("none", 0), ("head", 0), ("scalar", 1 / 16), ("vector", 1 / 16), ("vector", 0.5),
                                        ("vector", 2.5)])
@pytest.mark.parametrize("N,dk", [(61, 128), (16, 64)])
def test_outputs_carry_one_rounding(N, dk, gate, scale, delta):
    d = draw("bf16", gate, delta, 8, 16, N, dk, 128, "chain", seed=57, scale=scale)
    o, _ = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
    torch.cuda.synchronize()
    val, _, S, _ = reference(d)
    r, q = val["o"], d["q"].double()
    p = torch.stack([(S[n + 1] * q[:, :, n, None]).square().sum(-1).sqrt() for n in range(N)], 2)
    s = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(1e-30))) - 7)
    most = float((12 * 2.0 ** -24 * p / s).clamp_max(1).sum())
    differ = int((o != r.bfloat16()).sum())
    print(f"{gate} {scale} N {N} dk {dk}: {differ} of {o.numel()} differ, {most:.0f} allowed", flush=True)
    assert differ <= most + 5 * most ** 0.5
