"""Lists of weights quantised to 4 bits (quant_weights_fp4): the tensor scales."""
import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert fq.fp8bq_sync_status() == fq.FP8BQ_OK


def scale_of(amax):
    """max(amax, eps) / 448 / 6, both IEEE fp32 divisions."""
    return np.maximum(amax, np.float32(1e-10)) / np.float32(448) / np.float32(6)


def test_the_tensor_scale_is_divided_by_six():
    """Not multiplied by the rounded reciprocal, which is another number for a third of these."""
    amax = (0.5 + np.random.default_rng(1).random(512)).astype(np.float32)
    want = scale_of(amax)
    by_448 = amax / np.float32(448)
    assert (want != by_448 * (np.float32(1) / np.float32(6))).sum() > 100
    named = [(f"w{i}", torch.full((1, 1), float(a), device="cuda")) for i, a in enumerate(amax)]
    out = dict(fq.quant_weights_fp4(named, "nvfp4"))
    got = torch.cat([out[f"w{i}_scale_2"] for i in range(amax.size)]).cpu().numpy()
    assert np.array_equal(got, want)
