"""Trees of fewer nodes than the batch's: whatever stands behind a batch element's count reaches
no result; nothing accepted leaves every state's bits."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
from test_gpu_tree import draw

pytestmark = pytest.mark.gpu


def fwd(d):
    o, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"], counts=d["counts"])
    torch.cuda.synchronize()
    return o, u


@pytest.mark.parametrize("scale", [1 / 16, 2.5], ids=["", "deep"])
@pytest.mark.parametrize("delta", [True, False], ids=["delta", "linear"])
@pytest.mark.parametrize("gate", ["none", "head", "scalar", "vector"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,counts", [(16, [16, 0, 5]), (30, [17, 1, -3]), (64, [40, 63, 16])])
def test_behind_the_count_nothing_is_read(N, counts, dtype, gate, delta, scale):
    d = draw(dtype, gate, delta, 3, 2, N, 64, 48, "chain", counts=counts, seed=50, scale=scale)
    o, u = fwd(d)
    bad = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in d.items()}
    for b, c in enumerate(counts):
        c = max(0, c)
        for n in ("q", "k", "v", "beta", "g"):
            if bad[n] is not None and bad[n].dim() >= 3:
                bad[n][b, :, c:] = torch.nan
        bad["parent"][b, c:] = torch.tensor([2 ** 31 - 1, -2 ** 31, N + 3, 0, c][b % 5], dtype=torch.int32)
    o2, u2 = fwd(bad)
    assert torch.equal(o, o2) and torch.equal(u, u2)
    for b, c in enumerate(counts):
        assert not o2[b, :, max(0, c):].any() and not u2[b, :, max(0, c):].any()


def test_nothing_accepted_leaves_every_bit():
    d = draw("bf16", "scalar", True, 3, 2, 8, 32, 32, seed=51)
    u = torch.full((3, 2, 8, 32), torch.nan, device="cuda")
    state = d["state"].clone()
    state[1] = torch.nan
    state[2, 1, 3] = -torch.inf
    before = state.view(torch.int32).clone()
    B.tree_commit(d["k"], u, d["g"], d["parent"], torch.tensor([-1, 8, -2 ** 31], dtype=torch.int32, device="cuda"), state)
    torch.cuda.synchronize()
    assert torch.equal(state.view(torch.int32), before)
