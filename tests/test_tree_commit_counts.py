"""What the commit of trees of fewer nodes refuses, on the host (no GPU)."""
import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

FAKE = 1 << 30   # distinct, aligned addresses that are never read


def commit(s, **over):
    n = ("k", "u", "g", "parent", "counts", "accept", "state")
    a = {m: FAKE * (i + 1) for i, m in enumerate(n)}
    a.update(over)
    return B.dn_tree_commit_counts(s, *(a[m] for m in n), 0)


def sh(**over):
    a = dict(B=2, H=3, T=40, dk=64, dv=32, C=64, dtype="bf16", gate="scalar")
    a.update(over)
    return B.make_shape(*(a[n] for n in ("B", "H", "T", "dk", "dv", "C", "dtype", "gate")))


def test_raw_call():
    assert commit(sh(T=65)) == B.DN_ERR_UNSUPPORTED and "nodes" in B.dn_last_error()
    assert commit(sh(dk=24)) == B.DN_ERR_UNSUPPORTED
    for name in ("k", "u", "g", "parent", "accept", "state"):
        assert commit(sh(), **{name: None}) == B.DN_ERR_INVALID and name in B.dn_last_error()
    assert commit(sh(), counts=FAKE * 30 + 4) == B.DN_ERR_INVALID and "counts" in B.dn_last_error()
    assert commit(sh(), state=FAKE * 5) == B.DN_ERR_INVALID                # over counts
    assert commit(sh(), state=FAKE * 6) == B.DN_ERR_INVALID                # over accept


def test_wrapper():
    z = torch.zeros
    args = (z(2, 3, 10, 32), z(2, 3, 10, 64), z(2, 3, 10), z(2, 10, dtype=torch.int32), z(2, dtype=torch.int32),
            z(2, 3, 64, 32))
    for bad in (z(2), z(3, dtype=torch.int32), z(2, 10, dtype=torch.int32), z(2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="counts"):
            B.tree_commit(*args, counts=bad)
    with pytest.raises(ValueError, match="CUDA device"):
        B.tree_commit(*args, counts=z(2, dtype=torch.int32))
