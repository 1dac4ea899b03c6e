"""Host-side tests of the 4-bit operators: argument checks (before any device
is touched), structure layouts, and the 64-bit reference the GPU tests use.
No GPU is needed: pointers are fake and never dereferenced."""
import ctypes

import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from tests import fp4_reference as ref

NO_GPU = not torch.cuda.is_available()
X, C, S, T = 0x7000_0000_0000, 0x7100_0000_0000, 0x7200_0000_0000, 0x7300_0000_0000


def q(**kw):
    a = dict(x=X, dtype_in=fq.FP8BQ_BF16, M=256, K=384, ld=384, format=fq.FP8BQ_NVFP4,
             tensor_scale=T, codes=C, scales=S, stream=0)
    a.update(kw)
    return fq.fp8bq_fp4_quantize(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype_in=2), fq.FP8BQ_ERR_DTYPE),
    (dict(format=2), fq.FP8BQ_ERR_ARG),
    (dict(format=-1), fq.FP8BQ_ERR_ARG),
    (dict(format=fq.FP8BQ_MXFP4), fq.FP8BQ_ERR_ARG),            # a tensor scale with mxfp4
    (dict(M=-1), fq.FP8BQ_ERR_SHAPE),
    (dict(K=-1, ld=0), fq.FP8BQ_ERR_SHAPE),
    (dict(ld=383), fq.FP8BQ_ERR_SHAPE),
    (dict(M=(1 << 31) - 255), fq.FP8BQ_ERR_SHAPE),
    (dict(M=1 << 30, ld=1 << 40), fq.FP8BQ_ERR_SHAPE),          # offsets beyond 2^62
    (dict(x=0), fq.FP8BQ_ERR_NULL),
    (dict(codes=0), fq.FP8BQ_ERR_NULL),
    (dict(scales=0), fq.FP8BQ_ERR_NULL),
    (dict(x=X + 1), fq.FP8BQ_ERR_ALIGN),
    (dict(dtype_in=fq.FP8BQ_F32, x=X + 2), fq.FP8BQ_ERR_ALIGN),
    (dict(codes=C + 8), fq.FP8BQ_ERR_ALIGN),
    (dict(scales=S + 8), fq.FP8BQ_ERR_ALIGN),
    (dict(tensor_scale=T + 2), fq.FP8BQ_ERR_ALIGN),
    (dict(codes=X + 1024), fq.FP8BQ_ERR_OVERLAP),
    (dict(scales=C + 256 * 192 - 16), fq.FP8BQ_ERR_OVERLAP),
    (dict(tensor_scale=S + 16), fq.FP8BQ_ERR_OVERLAP),
])
def test_quantise_refusals(kw, status):
    assert q(**kw) == status


def test_empty_and_lists():
    assert q(M=0, x=0, codes=0) == fq.FP8BQ_OK
    assert q(K=0, ld=0) == fq.FP8BQ_OK
    assert fq.fp8bq_fp4_quantize_batched([]) == fq.FP8BQ_OK
    assert fq.fp8bq_fp4_quantize_batched([], n_tensors=-1) == fq.FP8BQ_ERR_ARG
    assert fq.lib().fp8bq_fp4_quantize_batched(None, 1, 0) == fq.FP8BQ_ERR_NULL


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), fq.FP8BQ_ERR_SHAPE),
    (dict(K=0, ld_out=0), fq.FP8BQ_OK),
    (dict(dtype_out=7), fq.FP8BQ_ERR_DTYPE),
    (dict(out=0), fq.FP8BQ_ERR_NULL),
    (dict(out=X + 1), fq.FP8BQ_ERR_ALIGN),
    (dict(ld_out=383), fq.FP8BQ_ERR_SHAPE),
    (dict(out_batch_stride=255 * 384), fq.FP8BQ_ERR_OVERLAP),   # the stack's outputs overlap
    (dict(out=C), fq.FP8BQ_ERR_OVERLAP),
])
def test_dequantise_refusals(kw, status):
    a = dict(codes=C, scales=S, batch=2, M=256, K=384, format=fq.FP8BQ_MXFP4, tensor_scale=0,
             tensor_scale_stride=0, out=X, dtype_out=fq.FP8BQ_BF16, ld_out=384,
             out_batch_stride=256 * 384, stream=0)
    a.update(kw)
    assert fq.fp8bq_fp4_dequantize(**a) == status


def mm(**kw):
    d = fq.fp8bq_fp4_matmul_desc()
    for i, o in enumerate((d.a, d.b, d.up)):
        o.codes, o.scales = C + (i << 32), S + (i << 32)
        o.codes_batch_stride, o.scales_batch_stride = 256 * 192, 1 << 20
    d.out, d.M, d.N, d.K, d.batch, d.ld_out = X, 100, 256, 384, 2, 256
    d.out_batch_stride, d.dtype_out = 25600, fq.FP8BQ_F32
    for k, v in kw.items():
        o = d
        for part in k.split("__")[:-1]:
            o = getattr(o, part)
        setattr(o, k.split("__")[-1], v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype_out=3), fq.FP8BQ_ERR_DTYPE),
    (dict(format=5), fq.FP8BQ_ERR_ARG),
    (dict(a__tensor_scale=T), fq.FP8BQ_ERR_ARG),
    (dict(K=0), fq.FP8BQ_ERR_SHAPE),
    (dict(M=-1), fq.FP8BQ_ERR_SHAPE),
    (dict(N=-5), fq.FP8BQ_ERR_SHAPE),
    (dict(batch=1 << 30, M=128, N=1, ld_out=1, out_batch_stride=128), fq.FP8BQ_ERR_SHAPE),
    (dict(M=(1 << 31) - 255, ld_out=256, out_batch_stride=1 << 40), fq.FP8BQ_ERR_SHAPE),
    (dict(ld_out=255), fq.FP8BQ_ERR_SHAPE),
    (dict(a__codes_batch_stride=-16), fq.FP8BQ_ERR_SHAPE),
    (dict(b__scales_batch_stride=1 << 40), fq.FP8BQ_ERR_SHAPE),
    (dict(a__codes=0), fq.FP8BQ_ERR_NULL),
    (dict(b__scales=0), fq.FP8BQ_ERR_NULL),
    (dict(out=0), fq.FP8BQ_ERR_NULL),
    (dict(a__codes=C + 8), fq.FP8BQ_ERR_ALIGN),
    (dict(b__codes_batch_stride=24), fq.FP8BQ_ERR_ALIGN),
    (dict(out=X + 2), fq.FP8BQ_ERR_ALIGN),
    (dict(rows=T + 1), fq.FP8BQ_ERR_ALIGN),
    (dict(out_batch_stride=25599), fq.FP8BQ_ERR_OVERLAP),
    (dict(out=C), fq.FP8BQ_ERR_OVERLAP),
    (dict(rows=X + 4), fq.FP8BQ_ERR_OVERLAP),
    (dict(M=0, out=0), fq.FP8BQ_OK),
    (dict(batch=0), fq.FP8BQ_OK),
])
@pytest.mark.parametrize("call", [fq.fp8bq_fp4_matmul, fq.fp8bq_fp4_gated_matmul])
def test_product_refusals(call, kw, status):
    assert call(mm(**kw), 0) == status


def test_only_the_gated_product_looks_at_up():
    assert fq.fp8bq_fp4_gated_matmul(mm(up__codes=0), 0) == fq.FP8BQ_ERR_NULL
    if NO_GPU:
        assert fq.fp8bq_fp4_matmul(mm(up__codes=0), 0) == fq.FP8BQ_ERR_DEVICE
    assert fq.lib().fp8bq_fp4_matmul(None, 0) == fq.FP8BQ_ERR_NULL


@pytest.mark.skipif(not NO_GPU, reason="checks the no-device path")
def test_valid_calls_without_a_device():
    assert q() == fq.FP8BQ_ERR_DEVICE
    assert fq.fp8bq_fp4_matmul(mm(), 0) == fq.FP8BQ_ERR_DEVICE
    assert fq.fp8bq_fp4_gated_matmul(mm(rows=T), 0) == fq.FP8BQ_ERR_DEVICE


def test_packed_descriptors_match_the_structures():
    assert ctypes.sizeof(fq.fp8bq_fp4_desc) == fq._FP4_DESC.size == 88
    assert ctypes.sizeof(fq.fp8bq_fp4_operand) == 48
    assert ctypes.sizeof(fq.fp8bq_fp4_matmul_desc) == fq._FP4_MATMUL_DESC.size == 216
    d = fq.fp8bq_fp4_matmul_desc.from_buffer_copy(fq._FP4_MATMUL_DESC.pack(*range(1, 29)))
    flat = [getattr(o, n) for o in (d.a, d.b, d.up) for n, _ in o._fields_]
    flat += [getattr(d, n) for n, _ in d._fields_[3:]]
    assert flat == list(range(1, 29))
    d = fq.fp8bq_fp4_desc.from_buffer_copy(fq._FP4_DESC.pack(*range(1, 13)))
    assert [getattr(d, n) for n, _ in d._fields_] == list(range(1, 13))


def test_conveniences_refuse_host_tensors_and_unknown_formats():
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 16, dtype=torch.uint8)
    for call in (lambda f: fq.scaled_fp4_blockwise(x, f),
                 lambda f: fq.quant_weights_fp4([("w", x)], f),
                 lambda f: fq.dequantize_fp4_blockwise(c, s, f),
                 lambda f: fq.matmul_fp4(c, s, c, s, f),
                 lambda f: fq.gated_matmul_fp4(c, s, c, s, c, s, f)):
        with pytest.raises(ValueError, match="CUDA"):
            call("mxfp4")
        with pytest.raises(ValueError, match="format"):
            call("fp4")


@pytest.mark.parametrize("rows,columns", [(1, 1), (130, 300), (128, 256), (257, 96)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_scale_rows_undo_the_tiles(rows, columns, fmt):
    nb = -(-columns // ref.BLOCK[fmt])
    sc = np.random.default_rng(1).integers(0, 255, (rows, nb)).astype(np.uint8)
    t = torch.from_numpy(ref.tile(sc))
    assert np.array_equal(fq.fp4_scale_rows(t, rows, columns, fmt).numpy(), sc)
    stack = torch.stack([t, t.flip(-1)])
    assert np.array_equal(fq.fp4_scale_rows(stack, rows, columns, fmt)[0].numpy(), sc)
    assert np.array_equal(ref.untile(ref.tile(sc), rows, nb), sc)


# ------------------------------------------------------------------ the reference itself


def test_reference_grid_ties_and_saturation():
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, -0.25, -5, -0.1, 0.3, 2.6]
    code, sc = ref.quantize(x, "mxfp4")
    assert sc[0, 0] == 127                       # absmax in [4, 8): scale 1
    want = [4, 0, 1, 1, 2, 2, 4, 4, 6, 6, 6, -0.0, -4, -0.0, 0.5, 3]
    got = ref.values(code, sc, "mxfp4")[0, :16]
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


def test_reference_e4m3_is_the_format():
    assert np.array_equal(ref.E4M3, torch.arange(127, dtype=torch.uint8).view(
        torch.float8_e4m3fn).double().numpy())
    v = np.random.default_rng(0).random(20000) * 448
    t = torch.from_numpy(v).float()
    assert np.array_equal(ref.nearest(t.double().numpy(), ref.E4M3),
                          t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scales_and_error_bound():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((50, 320)) * np.exp2(rng.integers(-30, 30, (50, 1)))).astype(np.float32)
    code, sc = ref.quantize(x, "mxfp4")
    v = ref.values(code, sc, "mxfp4")
    s = np.repeat(ref.scale_values(sc, "mxfp4"), 32, axis=1)
    inside = np.abs(x) <= 6 * s                  # half a step, at most 1 below 6; 2 to the limit 8
    assert (np.abs(v - x) <= np.where(inside, 1.0, 2.0) * s).all()
    a = np.abs(x).reshape(50, 10, 32).max(-1)
    lead = a / ref.scale_values(sc, "mxfp4")
    assert (lead >= 4).all() and (lead < 8).all()
    t = np.float32(np.abs(x).max() / 2688)
    _, sc = ref.quantize(x, "nvfp4", t)
    assert sc.max() == 126                       # 448: the largest block's scale


def test_the_call_module_leaves_what_is_not_ordinary():
    """It returns None, with nothing done and no Python error pending, for anything but contiguous
    CUDA tensors that fit each other; the conveniences then say what is wrong."""
    m = fq._load_calls()
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 16, dtype=torch.uint8)
    for call in (lambda: m.product(0, 0, 0, 0, c, s, None, c, s, None, None, None, None, None),
                 lambda: m.product(0, 0, -1, 0, c, s, None, c, s, None, None, None, None, None),
                 lambda: m.product(1, 0, 0, 0, 1, "a", None, [], s, None, None, None, None, None),
                 lambda: m.product(0, "x", 0, 0, c, s, None, c, s, None, None, None, None, None),
                 lambda: m.product(0, 0, 0), lambda: m.product(),
                 lambda: m.quantize(0, 0, 0, x, None), lambda: m.quantize(0, 0, 0, None, None),
                 lambda: m.quantize(0, 0, 1 << 80, x, None), lambda: m.quantize(),
                 lambda: m.dequantize(0, 0, 0, c, s, None, None, None),
                 lambda: m.dequantize(0, -1, 0, c, s, None, None, None), lambda: m.dequantize(1)):
        assert call() is None
    with pytest.raises(TypeError):
        m.setup(1, 2, 3)
