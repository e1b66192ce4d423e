"""The split of linear attention's steps into parallel segments, restated here and compared with
the library's through the bytes of its workspace (no GPU): where it changes, and that one more
chunk or head never costs much more."""
import numpy as np
import pytest

from delta_rule_linear_gated_amd import binding as B

UNITS, XCDS = 256, 8
cd = lambda a, b: -(-a // b)


def plan(BH, T, dv, dtype, kind):
    """(segments, chunks of each, chunks between kept states): kind "fwd", "bwd" (no gate per step) or "dots"."""
    bf, dots = dtype == "bf16", kind == "dots"
    NT, nblk, nops = cd(T, 64), cd(dv, 64 if bf else 32), {"fwd": 1, "bwd": 3, "dots": 2}[kind]
    wgs = BH * nblk * nops
    full, cost = (216 if dots else 144, 6 if dots else 9) if bf else (256 if dots else 208, 4)
    w = wgs // 2 if wgs <= UNITS < cd(BH, XCDS) * XCDS * nblk * nops else wgs
    best = (None, 1, max(NT, 1), 16 if dots else max(NT, 1))
    if wgs and NT * (full - w) >= cost * full:
        for ns in range(2, min(64, NT // 2, 8 * UNITS // wgs) + 1):
            n = cd(NT, ns)
            snap = cd(n, cd(n, 16)) if dots else n
            n = cd(n, snap) * snap
            nseg = cd(NT, n)
            if nseg < 2 or (n < 4 and nseg * wgs > UNITS):
                continue
            t = time(BH, nseg, n, nblk, nops)
            if best[0] is None or t < best[0]:
                best = (t, nseg, n, snap)
    return best[1:]


def time(BH, nseg, n, nblk, nops):
    """The rule's estimate, in chunks of one workgroup alone (fp32, as the library)."""
    f = np.float32
    k = cd(cd(BH * nseg, XCDS) * nblk * nops, UNITS // XCDS)
    state = BH * (nseg - 1) * nblk * (2 if nops > 1 else 1)
    outs = f(1.7) * f(k // 2) + f(k % 2)
    return f(n + 1) * (outs + f(0.5) * max(f(1), f(state) / f(2 * UNITS)))


def workspace(BH, T, dk, dv, dtype, kind):
    nseg, _, snap = plan(BH, T, dv, dtype, kind)
    NT = cd(T, 64)
    al = lambda x: cd(x, 256) * 256
    nent = cd(NT, snap) if NT else 1
    keep = nseg > 1 or kind == "dots"
    n = (1 if kind == "fwd" else 2) * al(BH * (nent + 1) * dk * dv * 4) if keep else 0
    n += al((1 if kind == "fwd" else 2) * BH * nseg * 4) if nseg > 1 else 0
    if kind == "dots":
        vb = 64 if dtype == "bf16" else 32
        n += al(2 * cd(dk, vb) * BH * T * 4) + al(2 * cd(dv, vb) * BH * T * 4)
    return n


def library(BH, T, dk, dv, dtype, kind):
    sh = B.make_shape(1, BH, T, dk, dv, 64, dtype, "scalar" if kind == "dots" else "head")
    return B.dn_linear_workspace_bytes(sh, B.DN_PASS_FWD if kind == "fwd" else B.DN_PASS_BWD)


@pytest.mark.parametrize("kind", ["fwd", "bwd", "dots"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (16, 32)])
def test_plan_and_workspace(dk, dv, dtype, kind):
    for BH in (1, 2, 4, 5, 11, 16, 20, 32, 50, 64, 100, 128, 300):
        for T in (0, 1, 64, 512, 1025, 4096, 8192 + 1, 16384, 65536, 65600):
            assert library(BH, T, dk, dv, dtype, kind) == workspace(BH, T, dk, dv, dtype, kind), (BH, T)


def cost(BH, T, dv, dtype, kind):
    """Chunk times of the plan, one run included."""
    nseg, n, _ = plan(BH, T, dv, dtype, kind)
    nblk, nops = cd(dv, 64 if dtype == "bf16" else 32), {"fwd": 1, "bwd": 3, "dots": 2}[kind]
    if nseg > 1:
        return float(time(BH, nseg, n, nblk, nops))
    k = cd(cd(BH, XCDS) * nblk * nops, UNITS // XCDS)
    return (n + 1) * (1.7 * (k // 2) + k % 2)


def test_one_more_chunk_costs_little():
    """The same number of segments of a chunk more, and a chunk more for each kept state between
    its ends (rounding to whole numbers of those), is always there to be taken: segments of 17
    chunks are not made 32 long."""
    for BH in (1, 2, 4, 16, 50):
        for T in (16384, 32768, 65536, 131072):
            for kind in ("fwd", "bwd", "dots"):
                n = plan(BH, T, 128, "bf16", kind)[1]
                more = 1 + (cd(n + 1, 16) - 1 if kind == "dots" else 0)
                a, b = (cost(BH, t, 128, "bf16", kind) for t in (T, T + 64))
                # times are fp32: at most four roundings on each side
                assert b <= a * (n + 1 + more) / (n + 1) * (1 + 8 * 2.0 ** -24), (BH, T, kind, a, b)
    # 2 heads: segments of 16 chunks at 65536 steps, of 17 (kept states 9 and 9 apart) one chunk later
    assert plan(2, 65600, 128, "bf16", "dots")[1] <= 18


def test_a_fuller_xcd_counts():
    """20 heads x 12 workgroups are 240, but three (b, h) on one XCD are 36 on its 32 units."""
    assert plan(20, 16384, 128, "fp32", "bwd")[0] > 1
    assert plan(16, 16384, 128, "fp32", "bwd")[0] > 1      # 192: below the threshold all the same
    assert plan(24, 16384, 128, "fp32", "bwd")[0] == 1     # 288: two turns anyway
