"""Host-side checks of the NVFP4 tensor scales' entry point."""
import pytest
import torch

import blockwise_fp8_weight_b200 as fq

X, S = 0x7000_0000_0000, 0x7100_0000_0000


@pytest.mark.parametrize("kw,out,n,status", [
    ({}, S, -1, fq.FP8BQ_ERR_ARG),
    ({}, S, 0, fq.FP8BQ_OK),
    ({}, 0, 1, fq.FP8BQ_ERR_NULL),
    ({}, S + 2, 1, fq.FP8BQ_ERR_ALIGN),
    (dict(dtype_in=5), S, 1, fq.FP8BQ_ERR_DTYPE),
    (dict(numel=-1), S, 1, fq.FP8BQ_ERR_SHAPE),
    (dict(x=0), S, 1, fq.FP8BQ_ERR_NULL),
    (dict(x=X + 1), S, 1, fq.FP8BQ_ERR_ALIGN),
    (dict(x=S - 100), S, 1, fq.FP8BQ_ERR_OVERLAP),
])
def test_refusals(kw, out, n, status):
    d = fq.fp8bq_scale_desc()
    for k, v in (dict(x=X, numel=4096, dtype_in=fq.FP8BQ_BF16) | kw).items():
        setattr(d, k, v)
    assert fq.fp8bq_fp4_tensor_scale([d], out, n_tensors=n) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_a_valid_call_without_a_device():
    d = fq.fp8bq_scale_desc()
    d.x, d.numel, d.dtype_in = X, 4096, fq.FP8BQ_F32
    assert fq.fp8bq_fp4_tensor_scale([d], S) == fq.FP8BQ_ERR_DEVICE
