"""The gated scan's choice of a form and its sizes under the sanitizers (g++, host code only): directly,
and through the entry points, whose own test has it from the built library."""
import os
import subprocess

import pytest

from test_sanitizers import HERE, PKG, _run
from test_sanitizers_qk_plan import BASE, PLAN as QK_PLAN

PLAN = os.path.join(PKG, "csrc", "dn_gated_scan_plan.cpp")


@pytest.mark.skipif(not os.path.isdir("/opt/rocm/include"), reason="needs the ROCm headers")
def test_plan_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "scan_plan_driver")
    subprocess.run([*BASE, os.path.join(HERE, "scan_plan_driver.cpp"), PLAN, "-o", exe], check=True)
    _run(exe, leaks=True)


@pytest.mark.skipif(not os.path.exists(os.path.join(PKG, "libdn.so")) or not os.path.isdir("/opt/rocm/include"),
                    reason="needs the built library and the ROCm headers")
def test_entry_points_with_the_plans_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "scan_qk_driver")
    subprocess.run([*BASE, os.path.join(HERE, "scan_qk_driver.cpp"), os.path.join(PKG, "csrc", "dn_api.cpp"), PLAN, QK_PLAN,
                    "-L", PKG, "-ldn", f"-Wl,-rpath,{PKG}", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True)
    _run(exe, leaks=False)
