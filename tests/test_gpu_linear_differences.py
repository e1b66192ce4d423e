"""Linear attention's gradients against central differences of L = <o, do> + <hT, dhT> (fp32),
along the gradient itself and along random directions, all of norm 1.

L is linear in each of q, k, v and h0, so that a difference quotient over a step as long as the
input has no error but L's rounding.  An output's rounding: some 50 independent roundings of
partial sums of its terms, 0.58 half steps each in root mean square, 4 half steps of the terms'
absolute sum `mag`; L, summed in 64 bits, is off by that times the 2-norm of mag * do; five times
it is allowed.  In g the quotient over step s is off by s^2 / 6 of the third derivative, at most
the sum over pairs of |term| |direction summed between them|^3."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
import linear_ref as R
from test_gpu_linear import draw, run

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def third(d, u):
    """Bound of |d^3 L / ds^3| along g + s u: every pair of a step, h0 or dhT with a later one."""
    total = 0.0
    for h in range(d["g"].shape[1]):
        q, k, v, e = (d[n][0, h].double().abs() for n in ("q", "k", "v", "do"))
        S, D = d["h0"][0, h].double().abs(), d["dhT"][0, h].double().abs()
        c, s = d["g"][0, h].double().cumsum(0), u[0, h].double().cumsum(0)
        n = len(c)
        far = lambda x: x.abs() ** 3
        w = torch.where(torch.ones(n, n, device=c.device).tril() > 0, c[:, None] - c[None, :], -torch.inf).exp()
        total += (w * (q @ k.T) * (e @ v.T) * far(s[:, None] - s[None, :])).sum()
        total += (c.exp() * ((q @ S.T) * e).sum(-1) * far(s)).sum()
        total += ((c[-1] - c).exp() * ((k @ D.T) * v).sum(-1) * far(s[-1] - s)).sum()
        total += c[-1].exp() * (S * D).sum() * far(s[-1])
    return float(total)


@pytest.mark.parametrize("T,no_scan", [(150, True), (1100, False)])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "h0"])
def test_gradients(name, T, no_scan):
    d = draw("fp32", "scalar", 1, 2, T, 32, 32, seed=13)
    grad = run(d, no_scan)["d" + name].double()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(14)
    do, dhT = d["do"].double(), d["dhT"].double()

    def loss(e):
        o, hT = B.linear_fwd(e["q"], e["k"], e["v"], e["g"], e["h0"], no_scan=no_scan)
        _, mag = R.reference(e["q"], e["k"], e["v"], e["g"], e["h0"])
        off = 5 * 4 * U32 * ((mag["o"] * do).square().sum() + (mag["hT"] * dhT).square().sum()).sqrt()
        return float((o.double() * do).sum() + (hT.double() * dhT).sum()), float(off)

    x, size = d[name], float(grad.norm())
    step = 1e-2 if name == "g" else float(x.double().norm())
    for along in range(3):
        u = grad if along == 0 else torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        u = u / u.norm()
        up, down = (x.double() + step * u).float(), (x.double() - step * u).float()
        real = (up.double() - down.double()) / 2            # the step as rounded
        (hi, a), (lo, b) = loss({**d, name: up}), loss({**d, name: down})
        want = float((grad * real).sum()) / step
        lim = (a + b) / (2 * step) + (step ** 2 / 6 * third(d, u) if name == "g" else 0.0) + 16 * U32 * size
        got = (hi - lo) / (2 * step)
        print(f"{name} T {T} direction {along}: {got:.6f} against {want:.6f}, off by {abs(got - want) / lim:.3f} of "
              f"{lim / size:.2e} |grad|", flush=True)
        assert abs(got - want) <= lim
        assert lim <= 1e-2 * size                           # a bound that sees a hundredth of the gradient
