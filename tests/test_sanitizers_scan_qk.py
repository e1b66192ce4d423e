"""The host side of the gated scan's and the queries' and keys' entry points under the sanitizers
(g++, host code only), as test_sanitizers.py has the others."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import HERE, PKG, ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists(os.path.join(PKG, "libdn.so")) or not os.path.isdir("/opt/rocm/include"),
                    reason="needs the built library and the ROCm headers")
def test_scan_qk_validation_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "scan_qk_driver")
    subprocess.run([shutil.which("g++"), "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
                    os.path.join(HERE, "scan_qk_driver.cpp"), os.path.join(PKG, "csrc", "dn_api.cpp"),
                    "-L", PKG, "-ldn", f"-Wl,-rpath,{PKG}", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True)
    _run(exe, leaks=False)
