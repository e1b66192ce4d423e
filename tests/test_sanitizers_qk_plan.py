"""How the queries' and keys' calls are split over workgroups, under the sanitizers (g++, host
code only): directly, and through the entry points over sizes up to the largest integers."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import HERE, PKG, ROOT, SAN, _run

BASE = [shutil.which("g++"), "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc")]
PLAN = os.path.join(PKG, "csrc", "dn_qk_plan.cpp")


@pytest.mark.skipif(not os.path.isdir("/opt/rocm/include"), reason="needs the ROCm headers")
def test_split_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "qk_plan_driver")
    subprocess.run([*BASE, os.path.join(HERE, "qk_plan_driver.cpp"), PLAN, "-o", exe], check=True)
    _run(exe, leaks=True)


@pytest.mark.skipif(not os.path.exists(os.path.join(PKG, "libdn.so")) or not os.path.isdir("/opt/rocm/include"),
                    reason="needs the built library and the ROCm headers")
def test_entry_points_with_the_split_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "scan_qk_driver")
    subprocess.run([*BASE, os.path.join(HERE, "scan_qk_driver.cpp"), os.path.join(PKG, "csrc", "dn_api.cpp"), PLAN,
                    "-L", PKG, "-ldn", f"-Wl,-rpath,{PKG}", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True)
    _run(exe, leaks=False)
