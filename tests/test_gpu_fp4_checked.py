"""The bounds-checked build (libfp8bq_checked.so) on the 4-bit operators: their GPU tests run again in
a child process that loads it, where a skipped out-of-range access fails the status check after each
test; and with outputs taken one byte short, the last store of each kernel is reported and skipped."""
import os
import subprocess
import sys

import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from blockwise_fp8_weight_b200 import build as cuda_build
from tests.gpu_util import CANARY, Guarded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
checked_only = pytest.mark.skipif(not fq.CHECKED, reason="needs the checked library "
                                  "(run by the child process of the suite test)")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()


@pytest.mark.skipif(fq.CHECKED, reason="this process is the checked child")
def test_fp4_suite_under_the_checked_library():
    cuda_build.build(checked=True)
    env = dict(os.environ, FP8BQ_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_fp4.py", "tests/test_gpu_fp4_checked.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    tail = r.stdout[-6000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail


@pytest.fixture
def trimmed():
    assert fq.fp8bq_debug_take_bounds()[0] == fq.FP8BQ_OK
    assert fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_TRIM_OUTPUTS) == fq.FP8BQ_OK
    yield
    fq.fp8bq_debug_set_inject(0)
    fq.fp8bq_debug_take_bounds()


def caught(*buffers):
    assert fq.fp8bq_sync_status() == fq.FP8BQ_ERR_DEVICE_BOUNDS
    st, count, first = fq.fp8bq_debug_take_bounds()
    assert st == fq.FP8BQ_OK and count >= len(buffers)
    assert any(b.ptr + b.nbytes - 32 <= first < b.ptr + b.nbytes for b in buffers)
    for b in buffers:
        assert b.canaries_intact() and b.view[-1] == CANARY   # the skipped store left the fill byte


@checked_only
@pytest.mark.parametrize("fmt", [fq.FP8BQ_MXFP4, fq.FP8BQ_NVFP4])
@pytest.mark.parametrize("K", [512, 500, 501])
def test_trimmed_quantise_and_dequantise_outputs_are_caught(trimmed, fmt, K):
    x = torch.randn(128, K, device="cuda").to(torch.bfloat16)
    codes = Guarded(128 * 16 * (-(-K // 32)))
    scales = Guarded(-(-K // (128 if fmt == fq.FP8BQ_MXFP4 else 64)) * 512)
    assert fq.fp8bq_fp4_quantize(x, fq.FP8BQ_BF16, 128, K, K, fmt, None, codes.ptr, scales.ptr) == \
        fq.FP8BQ_OK
    caught(codes, scales)
    out = Guarded(128 * K * 2)
    assert fq.fp8bq_fp4_dequantize(codes.ptr, scales.ptr, 1, 128, K, fmt, None, 0, out.ptr,
                                   fq.FP8BQ_BF16, K, 0) == fq.FP8BQ_OK
    caught(out)


@checked_only
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 256), (40, 256), (128, 40000), (700, 515)])
def test_trimmed_product_outputs_are_caught(trimmed, gated, dtype, M, N):
    fq.fp8bq_debug_set_inject(0)
    a, sa = fq.scaled_fp4_blockwise(torch.randn(M, 512, device="cuda"))
    b, sb = fq.scaled_fp4_blockwise(torch.randn(N, 512, device="cuda"))
    fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_TRIM_OUTPUTS)
    buf = Guarded(M * N * (2 if dtype == torch.bfloat16 else 4))
    out = buf.view.view(dtype).view(M, N)
    if gated:
        fq.gated_matmul_fp4(a, sa, b, sb, b, sb, out=out)
    else:
        fq.matmul_fp4(a, sa, b, sb, out=out)
    caught(buf)
