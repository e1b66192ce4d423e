"""The commit of trees of fewer nodes than the batch's: a node behind a tree's count is none of
it, whatever its key, gate and parent hold."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B
from test_gpu_tree import draw, reference, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["none", "head", "scalar", "vector"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,counts", [(16, [16, 0, 5, 9]), (33, [33, 1, -3, 500])])
def test_nodes_behind_the_count(N, counts, dtype, gate):
    d = draw(dtype, gate, True, 4, 2, N, 64, 80, "bush", counts=counts, seed=55)
    for b, c in enumerate(counts):
        c = max(0, min(N, c))
        for n in ("q", "k", "v", "beta", "g"):
            if d[n] is not None and d[n].dim() >= 3:
                d[n][b, :, c:] = torch.nan
        d["parent"][b, c:] = 0
    _, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"], counts=d["counts"])
    clean = {n: (torch.nan_to_num(t) if torch.is_tensor(t) and t.is_floating_point() else t) for n, t in d.items()}
    _, _, S, A = reference(clean)
    for accept in ([N - 1, 0, 5, 8], [0, 1, 4, 9], [3, -1, 0, N]):
        at = torch.tensor(accept, dtype=torch.int32, device="cuda")
        state = d["state"].clone()
        B.tree_commit(d["k"], u, d["g"], d["parent"], at, state, counts=d["counts"])
        torch.cuda.synchronize()
        for b, (a, c) in enumerate(zip(accept, counts)):
            if 0 <= a < min(N, c):
                close(state[b], S[a + 1][b], A[a + 1][b], f"{accept} {b}")
            else:
                assert torch.equal(state[b], d["state"][b]), (accept, b)


def test_all_counted_is_the_commit_without_counts():
    d = draw("bf16", "scalar", True, 3, 2, 20, 32, 32, seed=56)
    _, u = B.tree_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"], d["parent"], d["state"])
    at = torch.tensor([19, 7, 20], dtype=torch.int32, device="cuda")
    full = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    a, b, c = (d["state"].clone() for _ in range(3))
    B.tree_commit(d["k"], u, d["g"], d["parent"], at, a)
    B.tree_commit(d["k"], u, d["g"], d["parent"], at, b, counts=full)
    sh = B.make_shape(3, 2, 20, 32, 32, 64, "bf16", "scalar")
    assert B.dn_tree_commit(sh, d["k"], u, d["g"], d["parent"], at, c) == B.DN_OK
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
