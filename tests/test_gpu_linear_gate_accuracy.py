"""How exact the gate's gradient is over a long sequence, as a whole (2-norm).

dg_t is summed between ends that are known from kept states, W steps apart, and what the sum
misses is spread along it: a bridge, off by sqrt(W / 6) of a step's error in root mean square.
A step's part of the sum is two dots x . y, q_s . dq_s and v_s . dv_s, over d channels.  With p the
2-norm of the products x_c y_c: the channels' values have some 20 roundings each (products of up
to 128 and chunks of 64 in three operand parts), independent and 0.58 half steps in root mean
square, together 0.58 sqrt(20) p = 2.6 p; some 30 partial sums, whose size is p / sqrt(2) in
root mean square, add 0.58 sqrt(30) / sqrt(2) p = 2.2 p: 3.4 half steps of p.  The ends are sums of
d^2 products in 64 bits; they and the result's rounding count as 2 half steps of dg.
(Without the known ends and what they take off, the error of the sum over all T steps is
sqrt(T / 2) of a step's: 7 times as much here in one run.)"""
import pytest
import torch

from gate_ref import gate_gradient
from test_gpu_linear import draw, run
from test_linear_plan import plan

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 128), ("fp32", 64)])
def test_long_sequences(dtype, d, no_scan):
    T = 16384
    x = draw(dtype, "scalar", 1, 1, T, d, d, seed=95)
    got = run(x, no_scan)
    W = 64 * (16 if no_scan else plan(1, T, d, dtype, "dots")[2])
    ref, _, _ = gate_gradient(*(x[n][0, 0] for n in ("q", "k", "v", "g", "h0", "do", "dhT")))
    p = sum((x[n][0, 0].double() * got["d" + n][0, 0].double()).square().sum(-1) for n in ("q", "v")).sqrt()
    lim = U32 * float(3.4 * (W / 6) ** 0.5 * p.norm() / ref.norm()) + 2 * U32
    rel = float((got["dg"][0, 0].double() - ref).norm() / ref.norm())
    print(f"{dtype} {d} W {W}: dg off by {rel:.2e} of its norm, {rel / lim:.3f} of the bound", flush=True)
    assert rel <= lim
