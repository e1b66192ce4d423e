"""The chained scan's wait for messages of other tiles, on the host: it ends after a given number of
looks."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import HERE, PKG, SAN, _run


@pytest.mark.skipif(not os.path.isdir("/opt/rocm/include"), reason="needs the ROCm headers")
def test_waits_end(tmp_path):
    exe = str(tmp_path / "wait_driver")
    subprocess.run([shutil.which("g++"), "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(PKG, "csrc"), os.path.join(HERE, "wait_driver.cpp"), "-o", exe], check=True)
    _run(exe, leaks=True)


def test_every_wait_of_the_scan_is_one_of_these():
    """No loop of the scan's kernels reads another tile's message but through wait_until."""
    text = open(os.path.join(PKG, "csrc", "dn_gated_scan.hip")).read()
    assert "while (!__all" not in text and text.count("wait_until(") == 2
