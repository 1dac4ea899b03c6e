"""tests/c/per_device_check.cpp: a set-up that failed is made again by the next call."""
import os
import shutil
import subprocess

import pytest

from blockwise_fp8_weight_b200 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_failed_set_up_is_not_kept(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "include")
    exe = str(tmp_path / "per_device_check")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-O1", "-I", B.CSRC,
                    "-I", os.path.join(B.ROOT, "include"), "-I", cuda,
                    os.path.join(HERE, "c", "per_device_check.cpp"), "-o", exe, "-lpthread"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert "per device ok" in r.stdout
