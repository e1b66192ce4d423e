"""A workspace given to the linear-attention wrappers: memory of another device or with holes is
refused before anything is launched (no GPU)."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B


def call(which, ws):
    z = torch.zeros
    q, v, g, h = z(1, 2, 10, 32), z(1, 2, 10, 64), z(1, 2, 10), z(1, 2, 64, 32)
    if which == "fwd":
        return B.linear_fwd(q, q, v, g, h, ws=ws)
    return B.linear_bwd(q, q, v, g, h, v, h, ws=ws)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_refused(which):
    for ws in (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), torch.zeros(64, 64).t()[::2],
               torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws must be"):
            call(which, ws)
    with pytest.raises(ValueError, match="CUDA device"):   # a sound one: the tensors themselves are refused
        call(which, torch.zeros(1 << 12, dtype=torch.uint8))
