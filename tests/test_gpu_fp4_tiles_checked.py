"""The forced kernels, the gate and the lists of weights again under the bounds-checked library: a
skipped out-of-range access fails the status check after each test."""
import os
import subprocess
import sys

import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from blockwise_fp8_weight_b200 import build as cuda_build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(fq.CHECKED, reason="this process is the checked child")
def test_under_the_checked_library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_fp4_tiles.py", "tests/test_gpu_fp4_gate.py",
                        "tests/test_gpu_fp4_weights.py"],
                       cwd=ROOT, env=dict(os.environ, FP8BQ_CHECKED="1"), capture_output=True, text=True,
                       timeout=1800)
    tail = r.stdout[-6000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
