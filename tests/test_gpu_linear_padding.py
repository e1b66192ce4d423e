"""What stands behind a sequence's length (NaN here) reaches no result: fp32 and bf16, one run
and parallel segments, every gate."""
import pytest
import torch

from test_gpu_linear import draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("no_scan", [False, True], ids=["segments", "one-run"])
@pytest.mark.parametrize("gate", ["none", "head", "scalar"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,lens", [(200, [77, 128, 0]), (2500, [1300, 64, 2499])])
def test_behind_the_length_nothing_is_read(T, lens, dtype, gate, no_scan):
    d = draw(dtype, gate, 3, 2, T, 64, 128, lens=lens, seed=52)
    ref = run(d, no_scan)
    for b, n in enumerate(lens):
        for x in ("q", "k", "v", "do") + (("g",) if gate == "scalar" else ()):
            d[x][b, :, n:] = torch.nan
    got = run(d, no_scan)
    for x in ref:
        assert torch.equal(got[x], ref[x]), x
    for b, n in enumerate(lens):
        for x in ("o", "dq", "dk", "dv") + (("dg",) if gate == "scalar" else ()):
            assert not got[x][b, :, n:].any(), (x, b)
