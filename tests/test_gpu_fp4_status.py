"""What the status check costs a process that makes no 4-bit product, and that it still sees the
products of one that does."""
import os
import subprocess
import sys

import pytest
import torch

import blockwise_fp8_weight_b200 as fq

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


CHILD = """
import torch, blockwise_fp8_weight_b200 as fq
from torch.profiler import profile, ProfilerActivity
x = torch.randn(256, 384, device="cuda").bfloat16()

def copies(calls):
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        x.add_(1)
        for _ in range(calls):
            assert fq.fp8bq_sync_status() == fq.FP8BQ_OK
    ev = [e.name for e in p.events()]
    assert any("add" in n for n in ev), "no trace"
    return sum("DtoH" in n for n in ev)

fq.scaled_fp8_blockwise(x)
c, s = fq.scaled_fp4_blockwise(x)
a = copies(5)
fq.matmul_fp4(c, s, c, s)
b = copies(5)
print("copies", a, b)
"""


@pytest.mark.skipif(fq.CHECKED, reason="checked builds read the bounds records as well")
def test_a_status_check_reads_one_word_until_a_product_was_launched():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, cwd=ROOT)
    if "no trace" in r.stderr:
        pytest.skip("the profiler traces nothing here")
    assert r.returncode == 0, r.stderr[-3000:]
    assert "copies 5 10" in r.stdout, r.stdout


CAPTURED = """
import torch, blockwise_fp8_weight_b200 as fq
x = torch.randn(40, 1024, device="cuda")
c, s = fq.scaled_fp4_blockwise(x)
assert fq.fp8bq_debug_set_wait_limit_ns(5_000_000) == 0
assert fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_DROP_FIRST_LOAD) == 0
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = fq.matmul_fp4(c, s, c, s)
assert fq.fp8bq_sync_status() == fq.FP8BQ_OK
graph.replay()
assert fq.fp8bq_sync_status() == fq.FP8BQ_ERR_DEVICE_TIMEOUT
assert fq.fp8bq_sync_status() == fq.FP8BQ_OK
"""


def test_a_product_that_was_only_captured_is_seen():
    r = subprocess.run([sys.executable, "-c", CAPTURED], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
