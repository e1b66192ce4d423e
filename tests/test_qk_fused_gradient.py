"""Gradients of queries and keys as slices of one tensor, the gradient of a fused projection, on the host
(no GPU, nothing is launched): rows that lie between one another's are taken, rows that share memory
refused, over random layouts against the addresses themselves."""
import random

import pytest

from delta_rule_linear_gated_amd import binding as B

BASE = 1 << 40   # addresses that are never read


def refused(Bn, Hq, Hk, T, d, dq, dk, delta, dtype=B.DN_BF16):
    """Whether dq (batch, head, step strides) and dk, delta elements behind it, are refused for sharing memory: the
    error is theirs, or that of the weights' gradient over the workspace, which is looked for after it."""
    E = 2 if dtype == B.DN_BF16 else 4
    dense = [(H * T * d, T * d, d) for H in (Hq, Hk)]
    sh = B.QKShape(Bn, Hq, Hk, T, d, 0, dtype, B.DN_NORM_L2, 0, 0, 1e-6, 1.0, *dense[0], *dense[1], *dq, *dk)
    n = B.dn_qk_workspace_bytes(sh)
    far = [i << 50 for i in range(1, 9)]
    st = B.dn_qk_bwd(sh, far[0], far[1], far[2], far[3], far[4], far[5], None, None, None, BASE, BASE + delta * E,
                     far[6], far[7], far[6], n, 0)
    assert st == B.DN_ERR_INVALID, st
    if B.dn_last_error() == "dq overlaps dk":
        return True
    assert B.dn_last_error() == "dwq overlaps workspace", B.dn_last_error()
    return False


@pytest.mark.parametrize("dtype", [B.DN_F32, B.DN_BF16])
def test_slices_of_one_tensor(dtype):
    d, T = 64, 7
    for Hq, Hk, Hv in ((3, 2, 0), (1, 1, 0), (1, 4, 2), (4, 1, 1), (2, 2, 2)):
        H = Hq + Hk + Hv
        by_token = (T * H * d, d, H * d)          # [B][T][H][d]
        by_head = (H * T * d, T * d, d)           # [B][H][T][d]
        pairs = (T * 2 * Hq * d, 2 * d, 2 * Hq * d)   # [B][T][H][2][d], as many keys as queries
        for Bn in (1, 3):
            assert not refused(Bn, Hq, Hk, T, d, by_token, by_token, Hq * d, dtype)
            assert not refused(Bn, Hk, Hq, T, d, by_token, by_token, -Hq * d, dtype)   # keys first
            assert not refused(Bn, Hq, Hk, T, d, by_head, by_head, Hq * T * d, dtype)
            assert not refused(Bn, Hq, Hq, T, d, pairs, pairs, d, dtype)
            for delta in (0, d // 2, -d // 2):
                assert refused(Bn, Hq, Hk, T, d, by_token, by_token, delta, dtype)
                assert refused(Bn, Hq, Hk, T, d, by_head, by_head, delta, dtype)
            if Hq > 1:
                assert refused(Bn, Hq, Hk, T, d, by_token, by_token, (Hq - 1) * d, dtype)
            assert refused(Bn, Hq, Hk, T, d, by_token, by_token, H * d, dtype)   # a step further
            assert refused(Bn, Hq, Hk, T, d, by_token, by_token, Hq * d + 8, dtype) == (Hv == 0)
    # other strides: not looked into
    assert refused(2, 2, 2, T, d, (T * 4 * d, d, 4 * d), (T * 4 * d, 2 * d, 4 * d), 2 * d, dtype)
    assert not refused(2, 2, 2, T, d, (T * 4 * d, d, 4 * d), (T * 4 * d, 2 * d, 4 * d), 2 * T * 4 * d, dtype)


def rows(n, stride, at, d):
    """The elements of all rows."""
    return {at + i * stride[0] + j * stride[1] + t * stride[2] + e
            for i in range(n[0]) for j in range(n[1]) for t in range(n[2]) for e in range(0, d, 4)}


def test_random_layouts():
    """Same strides in both, any order of the dimensions, gaps, any distance: refused if and only if an element is both's."""
    rng = random.Random(7)
    d, seen = 16, [0, 0]
    for _ in range(4000):
        Bn, T = rng.randint(1, 3), rng.randint(1, 4)
        Hq, Hk = rng.randint(1, 3), rng.randint(1, 3)
        size = (Bn, max(Hq, Hk), T)
        stride, step = [0, 0, 0], d
        for i in rng.sample(range(3), 3):
            stride[i] = step + 8 * rng.choice([0, 0, 0, 1, 2, 3, 4, 8])
            step = stride[i] * size[i]
        reach = sum(s * (n - 1) for s, n in zip(stride, size)) + d
        delta = 8 * rng.randint(-reach // 8 - 2, reach // 8 + 2)
        shared = bool(rows((Bn, Hq, T), stride, 0, d) & rows((Bn, Hk, T), stride, delta, d))
        assert refused(Bn, Hq, Hk, T, d, stride, stride, delta) == shared, (Bn, Hq, Hk, T, stride, delta)
        seen[shared] += 1
    assert min(seen) > 500
