"""Norms of rows at the ends of fp32's range, as the contract has them: down to 1e-18 with eps 0, and of any
size with an eps; far smaller ones without one are Inf or NaN, in their row alone."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

from qk_ref import check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("d", [16, 128])
def test_scales(norm, d):
    gen = torch.Generator().manual_seed(d)
    unit = torch.randn(1, 1, 9, d, generator=gen).cuda()
    unit = unit + unit.sign()   # no element far below its row
    dy = torch.randn(1, 1, 9, d, generator=gen).cuda()
    for scale in (1e-18, 1e-9, 1.0, 1e9, 1e17):
        x = unit * scale
        y = B.qk_norm_fwd(x, None, norm=norm, eps=0.0)[0]
        dx = B.qk_norm_bwd(x, None, dy, None, norm=norm, eps=0.0)["dq"]
        check({"y": y, "dx": dx}, *reference(x, norm=norm, eps=0.0, dy=dy), label=f"{scale}")
    for scale in (1e-30, 1e-25, 1e-21):
        x = unit * scale
        y = B.qk_norm_fwd(x, None, norm=norm, eps=1e-6)[0]
        check({"y": y}, *reference(x, norm=norm, eps=1e-6), label=f"{scale} with eps")


def test_rows_whose_squares_underflow():
    """eps 0: a row with elements of 1e-25 is Inf, one of zeros NaN; its neighbours and the other tensor do not notice."""
    x = torch.randn(1, 2, 5, 32, generator=torch.Generator().manual_seed(1)).cuda()
    clean = B.qk_norm_fwd(x, x, eps=0.0)
    small = x.clone()
    small[0, 1, 2] = torch.where(x[0, 1, 2] < 0, -1e-25, 1e-25)
    small[0, 0, 4] = 0
    yq, yk = B.qk_norm_fwd(small, x, eps=0.0)
    assert torch.equal(yk, clean[1])
    assert torch.isinf(yq[0, 1, 2]).all() and torch.isnan(yq[0, 0, 4]).all()
    rest = torch.ones(1, 2, 5, dtype=torch.bool).cuda()
    rest[0, 1, 2] = rest[0, 0, 4] = False
    assert torch.equal(yq[rest], clean[0][rest])
