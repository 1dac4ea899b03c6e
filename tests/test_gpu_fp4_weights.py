"""Lists of weights quantised to 4 bits (quant_weights_fp4): the tensor scales."""
import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from tests import fp4_reference as ref
from tests.gpu_util import Guarded

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


NOT_FINITE = [np.inf, -np.inf, np.nan, -np.nan]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("start", [0, 1])               # rows of 16-byte vectors, and of elements
@pytest.mark.parametrize("bad", NOT_FINITE)
def test_a_value_that_is_not_finite_costs_its_block_alone(dtype, start, bad):
    M, K = 70, 640
    x = np.random.default_rng(3).standard_normal((M, K)).astype(np.float32)
    w = torch.empty(M * K + 8, dtype=dtype, device="cuda")[start:start + M * K].view(M, K)
    w.copy_(torch.from_numpy(x))
    at = [(0, 0), (0, 1), (3, 5), (40, 333), (69, 639)]
    for r, c in at:
        w[r, c] = bad
    x = w.float().cpu().numpy()
    named = [("w", w), ("clean", torch.ones(3, 64, dtype=dtype, device="cuda"))]
    out = dict(fq.quant_weights_fp4(named, "nvfp4"))
    t = out["w_scale_2"].cpu().numpy()[0]
    assert t == scale_of(np.abs(x[np.isfinite(x)]).max())
    code, sc = ref.quantize(x, "nvfp4", t)
    assert np.array_equal(out["w"].cpu().numpy(), ref.pack(code))
    assert np.array_equal(out["w_scale"].cpu().numpy(), ref.tile(sc))
    v = fq.dequantize_fp4_blockwise(out["w"], out["w_scale"], "nvfp4", columns=K,
                                    tensor_scale=out["w_scale_2"])
    nan = np.zeros((M, K), bool)
    for r, c in at:
        nan[r, c // 16 * 16:c // 16 * 16 + 16] = True
    assert np.array_equal(v.isnan().cpu().numpy(), nan)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensor_scales_over_finite_values(dtype):
    """Vectors and tails, values of one kind only, subnormals, the largest value, empty tensors."""
    big = torch.finfo(dtype).max
    rng = np.random.default_rng(4)
    lists = [np.full(n, v, np.float32) for n in (1, 8, 33, 4096, 70000) for v in (np.inf, np.nan)]
    lists += [np.array([big, -np.inf], np.float32), np.full(40, 1e-39, np.float32),
              np.array([], np.float32), np.zeros(9, np.float32)]
    for n in (7, 64, 100000):
        for k in (1, n // 2, n - 1):
            x = rng.standard_normal(n).astype(np.float32)
            x[rng.permutation(n)[:k]] = rng.choice(np.array(NOT_FINITE, np.float32), k)
            lists.append(x)
    dev = [torch.from_numpy(x).cuda().to(dtype) for x in lists]
    descs = []
    for d in dev:
        r = fq.fp8bq_scale_desc()
        r.x, r.numel = d.data_ptr(), d.numel()
        r.dtype_in = fq.FP8BQ_BF16 if dtype == torch.bfloat16 else fq.FP8BQ_F32
        descs.append(r)
    got = Guarded(4 * len(descs))
    assert fq.fp8bq_fp4_tensor_scale(descs, got.ptr) == fq.FP8BQ_OK
    torch.cuda.synchronize()
    assert got.canaries_intact()
    want = []
    for d in dev:
        x = d.float().cpu().numpy()
        want.append(scale_of(np.abs(x[np.isfinite(x)]).max(initial=np.float32(0))))
    assert np.array_equal(got.numpy().view(np.float32), np.array(want, np.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_weights_and_stacks(dtype):
    """A weight whose rows lie apart, one that is a slice of columns, and a stack."""
    g = torch.Generator(device="cuda").manual_seed(5)
    big = torch.randn(80, 400, generator=g, device="cuda").to(dtype)
    big[:, 300] = 1e4                                    # outside the slices
    named = [("rows", big[::2, :96]), ("cols", big[:, 101:229]),
             ("stack", torch.randn(3, 20, 64, generator=g, device="cuda").to(dtype))]
    out = dict(fq.quant_weights_fp4(named, "nvfp4"))
    for name, w in named:
        x = w.float().cpu().numpy()
        t = out[name + "_scale_2"].cpu().numpy()[0]
        assert t == scale_of(np.abs(x).max())
        c, s = fq.scaled_fp4_blockwise(w.contiguous(), "nvfp4", out[name + "_scale_2"])
        assert torch.equal(c, out[name]) and torch.equal(s, out[name + "_scale"])
