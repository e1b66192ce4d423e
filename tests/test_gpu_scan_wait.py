"""The chained scan where messages of tiles never come: launched from the host so that the first tiles
are left out, the call ends, what depends on them is NaN, and everything else is as it was or NaN."""
import ctypes
import time

import pytest
import torch

from delta_rule_linear_gated_amd import binding as B

pytestmark = pytest.mark.gpu


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "T", "d", "bf16", "coupled")]


class Fwd(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "g", "lens", "h0", "o", "hT", "states")] + [("first_tile", ctypes.c_int)]


class Bwd(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "g", "lens", "h0", "dout", "dhT", "states", "dx", "dg", "dh0")] + [
        ("first_tile", ctypes.c_int)]


FWD = "_ZN2dn21launch_gated_scan_fwdERKNS_9GsProblemERKNS_5GsFwdEPcP12ihipStream_t"
BWD = "_ZN2dn21launch_gated_scan_bwdERKNS_9GsProblemERKNS_5GsBwdEPcP12ihipStream_t"


def launch(name, problem, args, ws):
    f = getattr(B.lib(), name)
    f.argtypes, f.restype = [ctypes.c_void_p] * 4, ctypes.c_int
    start = time.time()
    assert f(ctypes.addressof(problem), ctypes.addressof(args), ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    print(f"{time.time() - start:.3f} s", flush=True)
    assert time.time() - start < 30


def ptr(*tensors):
    return [None if t is None else t.data_ptr() for t in tensors]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,T,d,left", [(1, 30000, 64, 0), (1, 30000, 64, 1), (5, 9000, 100, 1), (1, 30000, 64, 3)])
def test_messages_that_never_come(H, T, d, left, dtype):
    """left: tiles of the first strip (head 0's first 64 channels) that are left out, in the order in which they are
    handed out; tiles of 192 steps from the first one forward, of 128 steps from the last one backward."""
    gen = torch.Generator().manual_seed(T)
    x, do = (torch.randn(1, H, T, d, generator=gen).to(dtype).cuda() for _ in range(2))
    g = (-torch.rand(1, H, T, d, generator=gen) / 8).cuda()
    h0, dhT = (torch.randn(1, H, d, generator=gen).cuda() for _ in range(2))
    o, hT, st = B.gated_scan_fwd(x, g, h0, coupled=True)
    gr = B.gated_scan_bwd(x, g, h0, do, dhT, st, coupled=True)
    sh = B.make_shape(1, H, T, d, d, 64, "bf16" if dtype == torch.bfloat16 else "fp32", "vector")
    ws = torch.empty(max(B.dn_gated_scan_workspace_bytes(sh, p) for p in (B.DN_PASS_FWD, B.DN_PASS_BWD)), dtype=torch.uint8,
                     device="cuda")
    pr = Problem(1, H, T, d, dtype == torch.bfloat16, 1)
    got = {n: torch.full_like(t, 7) for n, t in (("o", o), ("hT", hT), *gr.items())}
    launch(FWD, pr, Fwd(*ptr(x, g, None, h0, got["o"], got["hT"], None), left), ws)
    launch(BWD, pr, Bwd(*ptr(x, g, None, h0, do, dhT, st, got["dx"], got["dg"], got["dh0"]), left), ws)
    cut, back = 192 * left, (-(-T // 128) - left) * 128
    for n, want in (("o", o), ("hT", hT), *gr.items()):
        part = got[n][0, 0, ..., :64]   # the first strip: nothing where tiles are left out, else NaN
        kept = slice(cut, None) if n == "o" else slice(0, back) if n in ("dx", "dg") else slice(None)
        if left:
            assert torch.isnan(part[kept]).all(), n
            part[kept] = 7
            assert (part == 7).all(), n
            part[...] = want[0, 0, ..., :64]
        # the others: right, or NaN where a workgroup that waited for the first strip kept them waiting
        wrong = got[n] != want
        assert torch.isnan(got[n][wrong]).all() if left else not wrong.any(), n
    again = B.gated_scan_fwd(x, g, h0, coupled=True)   # a call after it is whole
    assert torch.equal(again[0], o) and torch.equal(again[1], hT)
