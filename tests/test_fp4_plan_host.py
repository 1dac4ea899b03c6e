"""How a 4-bit product would be launched: the library's own rule, and the Python package's."""
import math
import os
import subprocess
import sys

import pytest

import blockwise_fp8_weight_b200 as fq
from tests.test_fp4_host import mm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _settings():
    yield
    fq.fp8bq_set_pdl(1)
    fq.fp8bq_set_pdl_min_us(6.5)
    fq.fp8bq_debug_set_fp4_tokens(-1)


def product(M, N, K, batch=1):
    d = mm(M=M, N=N, K=K, batch=batch, ld_out=N, out_batch_stride=M * N)
    for o in (d.a, d.b, d.up):
        o.codes_batch_stride = o.scales_batch_stride = 1 << 24
    return d


PLAIN_C = """
import ctypes, sys
L = ctypes.CDLL(sys.argv[1])
L.fp8bq_get_pdl_min_us.restype = ctypes.c_double
assert L.fp8bq_get_pdl() == 1 and L.fp8bq_get_pdl_min_us() == 0.0
"""


def test_a_c_program_overlaps_every_launch():
    """fp8bq_set_pdl is on and means every kernel, as its documentation says."""
    r = subprocess.run([sys.executable, "-c", PLAIN_C, fq.lib()._name], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    fq.fp8bq_set_pdl_min_us(0.0)
    for gated in (False, True):
        for size in ((1, 64, 64), (1, 6144, 4096), (8192, 6144, 4096)):
            st, _, overlap = fq.fp8bq_fp4_plan(product(*size), gated)
            assert (st, overlap) == (fq.FP8BQ_OK, 1)
    fq.fp8bq_set_pdl(0)
    assert fq.fp8bq_fp4_plan(product(8192, 6144, 4096))[2] == 0


def test_the_package_leaves_out_what_is_shorter_than_its_own_call():
    assert fq.fp8bq_get_pdl_min_us() == 6.5
    assert fq.fp8bq_fp4_plan(product(1, 64, 64))[2] == 0
    assert fq.fp8bq_fp4_plan(product(8192, 6144, 4096))[2] == 1
    for us in (-1.0, math.nan):
        assert fq.fp8bq_set_pdl_min_us(us) == fq.FP8BQ_ERR_ARG
    assert fq.fp8bq_get_pdl_min_us() == 6.5
    assert fq.fp8bq_set_pdl_min_us(math.inf) == fq.FP8BQ_OK
    assert fq.fp8bq_fp4_plan(product(8192, 6144, 4096))[2] == 0


def test_plans_and_their_refusals():
    assert fq.fp8bq_fp4_plan(product(1, 256, 512))[:2] == (fq.FP8BQ_OK, 16)
    assert fq.fp8bq_fp4_plan(product(17, 256, 512), True)[:2] == (fq.FP8BQ_OK, 32)
    assert fq.fp8bq_fp4_plan(product(8192, 6144, 4096))[:2] == (fq.FP8BQ_OK, 0)
    assert fq.fp8bq_fp4_plan(product(0, 256, 512)) == (fq.FP8BQ_OK, -1, -1)
    assert fq.fp8bq_fp4_plan(product(8, 256, 512, batch=0)) == (fq.FP8BQ_OK, -1, -1)
    assert fq.fp8bq_fp4_plan(mm(K=0))[0] == fq.FP8BQ_ERR_SHAPE
    assert fq.fp8bq_fp4_plan(mm(up__codes=0), True)[0] == fq.FP8BQ_ERR_NULL
    assert fq.fp8bq_fp4_plan(mm(up__codes=0), False)[0] == fq.FP8BQ_OK
    L = fq.lib()
    assert L.fp8bq_fp4_plan(None, 0, None, None) == fq.FP8BQ_ERR_NULL
    assert L.fp8bq_fp4_plan(product(1, 256, 512), 0, None, None) == fq.FP8BQ_OK


def test_forced_kernels():
    """A forced width is taken by every product it can serve."""
    for bad in (-2, 1, 48, 512):
        assert fq.fp8bq_debug_set_fp4_tokens(bad) == fq.FP8BQ_ERR_ARG
    for M in (1, 16, 17, 32, 33, 700):
        for gated in (False, True):
            assert fq.fp8bq_debug_set_fp4_tokens(-1) == fq.FP8BQ_OK
            own = fq.fp8bq_fp4_plan(product(M, 300, 512), gated)
            for t in (0, 16, 32, 64, 128, 256):
                assert fq.fp8bq_debug_set_fp4_tokens(t) == fq.FP8BQ_OK
                serves = t == 0 or (M <= t if t < 64 else t <= (128 if gated else 256))
                got = fq.fp8bq_fp4_plan(product(M, 300, 512), gated)
                assert got[:2] == (fq.FP8BQ_OK, t if serves else own[1])
