"""NaN in one step of a sequence: it reaches its chunk of 64 steps and, beyond, only what the
formulas let it reach; everything else is what it is without it."""
import pytest
import torch

from gate_ref import gate_gradient
from test_gpu_linear import draw, run

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
@pytest.mark.parametrize("T,at", [(900, 500), (2500, 1023), (2500, 1100)])
def test_one_bad_step(T, at, name, dtype, no_scan):
    d = draw(dtype, "scalar", 1, 2, T, 64, 64, seed=80)
    clean = run(d, no_scan)
    bad = {**d, name: d[name].clone()}
    bad[name][0, 0, at, 3] = torch.nan
    got = run(bad, no_scan)
    for n in clean:
        assert torch.equal(got[n][:, 1], clean[n][:, 1]), n      # the other head
    c0, c1 = at // 64 * 64, min(T, at // 64 * 64 + 64)
    before, behind = slice(0, c0), slice(c1, T)
    same = lambda n, part: torch.equal(got[n][0, 0, part], clean[n][0, 0, part])
    if name in ("k", "v"):
        assert same("o", before) and same("dq", before)
        assert got["o"][0, 0, behind].isnan().any() and got["dg"][0, 0, behind].isnan().all()
        free = "dk" if name == "k" else "dv"                      # no term of it holds this input
        own = "dv" if name == "k" else "dk"
        assert torch.equal(got[free], clean[free]) and same(own, before) and same(own, behind)
        assert torch.equal(got["dh0"], clean["dh0"]) and got["hT"][0, 0].isnan().any()
        part = before
    else:
        assert same("dk", behind) and same("dv", behind)
        assert got["dg"][0, 0, before].isnan().all()
        own, free = ("o", "dq") if name == "q" else ("dq", "o")
        assert torch.equal(got[free], clean[free]) and same(own, before) and same(own, behind)
        assert torch.equal(got["hT"], clean["hT"]) and got["dh0"][0, 0].isnan().any()
        part = behind
    # the gate's gradient, summed to its other end: within the bounds of its sum all the same
    val, mag, size = gate_gradient(d["q"][0, 0], d["k"][0, 0], d["v"][0, 0], d["g"][0, 0], d["h0"][0, 0], d["do"][0, 0],
                                   d["dhT"][0, 0])
    err = (got["dg"][0, 0, part].double() - val[part]).abs()
    assert torch.isfinite(err).all()
    assert bool((err <= 400 * U32 * (mag + size)[part]).all())
