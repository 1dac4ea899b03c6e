"""The 4-bit conveniences where their call module cannot be built."""
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


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_the_same_results_without_the_call_module(monkeypatch, fmt):
    x, w = torch.randn(20, 200, device="cuda"), torch.randn(150, 200, device="cuda")

    def all_of_them():
        a, b = fq.scaled_fp4_blockwise(x, fmt), fq.scaled_fp4_blockwise(w, fmt)
        return (*a, *b, fq.dequantize_fp4_blockwise(*a, fmt, columns=200), fq.matmul_fp4(*a, *b, fmt),
                fq.gated_matmul_fp4(*a, *b, *b, fmt, out_dtype=torch.float32))

    want = all_of_them()
    monkeypatch.setattr(fq, "_calls", False)
    for p, q in zip(want, all_of_them()):
        assert p.dtype == q.dtype and torch.equal(p, q)
    with pytest.raises(ValueError, match="do not go with"):
        fq.matmul_fp4(want[0], want[3], want[2], want[3], fmt)
