"""The 4-bit operators on the GPU against their formulas in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from tests import fp4_reference as ref
from tests.gpu_util import CANARY, Guarded

pytestmark = pytest.mark.gpu
FORMATS = ("mxfp4", "nvfp4")
CODE = {"mxfp4": fq.FP8BQ_MXFP4, "nvfp4": fq.FP8BQ_NVFP4}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _no_error():
    yield
    assert fq.fp8bq_sync_status() == fq.FP8BQ_OK


# ------------------------------------------------------------------ quantise


def some_values(M, K, seed, dtype):
    """Rows of very different sizes, zeros of both signs, exact midpoints, tiny and large values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-20, 20, (M, 1)).astype(float))
    x[rng.random((M, K)) < 0.05] = -0.0
    mid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -5.0], (M, K))
    x = np.where(rng.random((M, 1)) < 0.3, mid, x).astype(np.float32)
    if M > 2:
        x[1] = 0.0
        x[2] *= np.float32(1e-38)
    t = torch.from_numpy(x).to(dtype)
    return t, t.float().numpy()


def nv_scale(x, fmt):
    if fmt == "mxfp4":
        return None
    return np.float32(max(np.abs(x[np.isfinite(x)]).max(initial=0), 1e-30) / np.float32(2688))


def on_gpu(t):
    return None if t is None else torch.tensor([t], dtype=torch.float32, device="cuda")


def check_quantised(codes, scales, x, fmt, t):
    code, sc = ref.quantize(x, fmt, t)
    got = codes.cpu().numpy()
    assert np.array_equal(got, ref.pack(code)), int((got != ref.pack(code)).sum())
    assert np.array_equal(scales.cpu().numpy(), ref.tile(sc))
    return code, sc


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (3, 33), (5, 16), (128, 256), (129, 257),
                                 (33, 1000), (300, 520), (1, 4096), (97, 4100), (64, 32)])
def test_quantise_matches_the_formula(fmt, dtype, M, K):
    xt, x = some_values(M, K, M * 7 + K, dtype)
    t = nv_scale(x, fmt)
    codes, scales = fq.scaled_fp4_blockwise(xt.cuda(), fmt, tensor_scale=on_gpu(t))
    code, sc = check_quantised(codes, scales, x, fmt, t)
    assert np.array_equal(fq.fp4_scale_rows(scales, M, K, fmt).cpu().numpy(), sc)
    want = ref.values(code, sc, fmt)[:, :K]
    for out in (torch.float32, torch.bfloat16):
        got = fq.dequantize_fp4_blockwise(codes, scales, fmt, columns=K, tensor_scale=on_gpu(t),
                                          out_dtype=out)
        w = torch.from_numpy(want.astype(np.float32)) * (1.0 if t is None else float(t))
        assert torch.equal(got.cpu(), w.to(out))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_a_block_with_a_value_that_is_not_finite_is_nan(fmt, value):
    xt, x = some_values(40, 200, 5, torch.float32)
    for r, c in ((0, 0), (7, 31), (39, 199), (20, 100)):
        x[r, c] = value
    t = nv_scale(x, fmt)
    codes, scales = fq.scaled_fp4_blockwise(torch.from_numpy(x).cuda(), fmt, tensor_scale=on_gpu(t))
    code, sc = check_quantised(codes, scales, x, fmt, t)
    got = fq.dequantize_fp4_blockwise(codes, scales, fmt, columns=200, tensor_scale=on_gpu(t),
                                      out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref.values(code, sc, fmt)[:, :200]))
    assert np.isnan(got[0, 0]) and np.isnan(got[39, 199])


@pytest.mark.parametrize("fmt", FORMATS)
def test_subnormals_and_the_ends_of_the_range(fmt):
    tiny = np.float32(2.0) ** np.arange(-149, -100, dtype=np.float32)
    big = np.float32(2.0) ** np.arange(90, 128, dtype=np.float32)
    x = np.zeros((90, 64), np.float32)
    x[: tiny.size, 3] = tiny
    x[: tiny.size, 40] = -tiny * np.float32(1.5)
    x[tiny.size: tiny.size + big.size, 5] = big * np.float32(1.75)
    x[89] = np.finfo(np.float32).max
    codes, scales = fq.scaled_fp4_blockwise(torch.from_numpy(x).cuda(), fmt)
    check_quantised(codes, scales, x, fmt, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ld,offset", [(264, 0), (260, 4), (259, 1), (257, 3)])
def test_strided_and_misaligned_inputs(fmt, dtype, ld, offset):
    M, K = 70, 257
    xt, x = some_values(M, K, 11, dtype)
    buf = torch.full((M * ld + offset + 8,), 3e4, dtype=dtype, device="cuda")
    view = buf[offset:offset + M * ld].as_strided((M, K), (ld, 1), offset)
    view.copy_(xt)
    t = nv_scale(x, fmt)
    check_quantised(*fq.scaled_fp4_blockwise(view, fmt, tensor_scale=on_gpu(t)), x, fmt, t)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_list_of_weights_in_one_call(fmt):
    shapes = [(3, 64), (130, 96), (1, 1000), (64, 77), (257, 512), (9, 40), (12, 12), (5, 5),
              (128, 128), (40, 300)]
    named, xs = [], []
    for i, (M, K) in enumerate(shapes):
        xt, x = some_values(M, K, 50 + i, torch.bfloat16 if i % 3 else torch.float32)
        named.append((f"w{i}", xt.cuda()))
        xs.append(x)
    out = dict(fq.quant_weights_fp4(named, fmt))
    for (name, w), x in zip(named, xs):
        t = None
        if fmt == "nvfp4":
            t = out[name + "_scale_2"].cpu().numpy()[0]
            want = max(np.abs(x).max(), np.float32(1e-10)) / np.float32(448) / np.float32(6)
            assert t == want
        check_quantised(out[name], out[name + "_scale"], x, fmt, t)


@pytest.mark.parametrize("fmt", FORMATS)
def test_stacks_with_a_scale_each_and_nothing_written_beside(fmt):
    E, M, K = 5, 131, 96
    xt, x = some_values(E * M, K, 77, torch.bfloat16)
    x = x.reshape(E, M, K)
    ts = None
    if fmt == "nvfp4":
        ts = np.array([nv_scale(x[e], fmt) for e in range(E)], np.float32)
    KT = -(-K // (4 * ref.BLOCK[fmt]))
    codes, scales = Guarded(E * M * 48), Guarded(E * 2 * KT * 512)
    d = fq.fp8bq_fp4_desc()
    dev = xt.cuda()
    tt = None if ts is None else torch.from_numpy(ts).cuda()
    d.x, d.codes, d.scales = dev.data_ptr(), codes.ptr, scales.ptr
    d.tensor_scale, d.tensor_scale_stride = (0, 0) if tt is None else (tt.data_ptr(), 1)
    d.M, d.K, d.ld, d.batch, d.x_batch_stride = M, K, K, E, M * K
    d.dtype_in, d.format = fq.FP8BQ_BF16, CODE[fmt]
    assert fq.fp8bq_fp4_quantize_batched([d]) == fq.FP8BQ_OK
    torch.cuda.synchronize()
    assert codes.canaries_intact() and scales.canaries_intact()
    c = codes.view.view(E, M, 48)
    s = scales.view.view(E, 2, KT, 32, 16)
    out = Guarded(E * M * (K + 3) * 2)
    st = fq.fp8bq_fp4_dequantize(codes.ptr, scales.ptr, E, M, K, CODE[fmt],
                                 tt, 0 if tt is None else 1, out.ptr, fq.FP8BQ_BF16, K + 3,
                                 M * (K + 3))
    assert st == fq.FP8BQ_OK
    torch.cuda.synchronize()
    assert out.canaries_intact()
    got = out.view.view(torch.bfloat16).view(E, M, K + 3).cpu()
    assert (out.view.view(E, M, K + 3, 2)[:, :, K:] == CANARY).all()
    for e in range(E):
        t = None if ts is None else ts[e]
        code, sc = check_quantised(c[e], s[e], x[e], fmt, t)
        w = torch.from_numpy(ref.values(code, sc, fmt).astype(np.float32)) * (
            1.0 if t is None else float(t))
        assert torch.equal(got[e, :, :K], w.to(torch.bfloat16))


# ------------------------------------------------------------------ products


def exact_operand(rows, K, seed, fmt, E=0):
    """Random codes with scales 1 or 2: products are multiples of 1/4 of at most 36 * 4, so up to
    2^14 of them add up to less than 2^24 quarters, and fp32 sums are exact in any order."""
    rng = np.random.default_rng(seed)
    B = ref.BLOCK[fmt]
    n = max(E, 1)
    Kp = -(-K // 32) * 32
    code = rng.integers(0, 16, (n, rows, Kp)).astype(np.uint8)
    code[rng.random(code.shape) < 0.5] = 0
    code[:, :, K:] = 0
    one = 127 if fmt == "mxfp4" else 0x38
    step = 1 if fmt == "mxfp4" else 8
    sc = (one + step * rng.integers(0, 2, (n, rows, -(-K // B)))).astype(np.uint8)
    val = np.stack([ref.values(code[e], sc[e], fmt) for e in range(n)])
    codes = np.stack([ref.pack(c) for c in code])
    tiles = np.stack([ref.tile(s) for s in sc])
    if not E:
        val, codes, tiles = val[0], codes[0], tiles[0]
    return torch.from_numpy(codes).cuda(), torch.from_numpy(tiles).cuda(), val


def as_float(t):
    return t.float().cpu().numpy().astype(np.float64)


def rounded(y, dtype):
    return torch.from_numpy(y.astype(np.float32)).to(dtype).float().numpy().astype(np.float64)


SHAPES = [(1, 1, 1), (1, 128, 256), (16, 128, 64), (1, 300, 4096), (7, 129, 96), (17, 256, 1000),
          (33, 64, 2048), (64, 500, 320), (65, 128, 128), (100, 260, 544), (128, 128, 512),
          (129, 384, 256), (256, 200, 800), (257, 256, 1056), (300, 1000, 96), (515, 130, 4100),
          (1000, 640, 288), (1, 8, 8192), (515, 1000, 4100), (200, 4096, 512), (90, 3000, 768),
          (300, 256, 8192), (40, 136, 2080)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_is_exact_where_its_sums_are(M, N, K, fmt, out):
    a, sa, va = exact_operand(M, K, 1, fmt)
    b, sb, vb = exact_operand(N, K, 2, fmt)
    y = fq.matmul_fp4(a, sa, b, sb, fmt, out_dtype=out)
    assert y.shape == (M, N) and y.dtype == out
    assert np.array_equal(as_float(y), rounded(va @ vb.T, out))
    assert torch.equal(y, fq.matmul_fp4(a, sa, b, sb, fmt, out_dtype=out))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 77, 2048), (9, 400, 64), (40, 129, 512), (100, 1030, 256),
                                   (200, 131, 1024), (40, 40000, 32), (700, 515, 64)])
def test_outputs_of_every_alignment(M, N, K, out):
    """Row strides and starts that allow 32-, 16-, 8-, 4-byte stores or the element's only; nothing
    beside the output is written."""
    a, sa, va = exact_operand(M, K, 1, "mxfp4")
    b, sb, vb = exact_operand(N, K, 2, "mxfp4")
    want = rounded(va @ vb.T, out)
    es = 2 if out == torch.bfloat16 else 4
    for ld, start in ((N + -N % 16, 0), (N + -N % 16 + 8, 0), (N + -N % 4 + 4, 0), (N + -N % 2 + 2, 2),
                      (N, 0), (N + 1 - N % 2, 1)):
        buf = Guarded((M * ld + start) * es)
        flat = buf.view.view(out)
        y = flat.as_strided((M, N), (ld, 1), flat.storage_offset() + start)
        fq.matmul_fp4(a, sa, b, sb, "mxfp4", out=y)
        assert np.array_equal(as_float(y), want), (ld, start)
        assert buf.canaries_intact()
        rows = buf.view[start * es:].view(M, ld, es)
        assert (rows[:, N:] == CANARY).all() and (buf.view[:start * es] == CANARY).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,E", [(2300, 5000, 288, 0), (700, 1100, 1600, 9), (16500, 330, 96, 0)])
def test_products_of_many_tiles(fmt, M, N, K, E):
    """More tiles than SMs: every pair walks over several, the sums' buffers alternating."""
    a, sa, va = exact_operand(M, K, 1, fmt, E)
    b, sb, vb = exact_operand(N, K, 2, fmt, E)
    want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().transpose(-1, -2)
    y = fq.matmul_fp4(a, sa, b, sb, fmt, out_dtype=torch.float32)
    assert torch.equal(y, want.float())
    assert torch.equal(fq.matmul_fp4(a, sa, b, sb, fmt), want.to(torch.float32).to(torch.bfloat16))
    low = sa.int() - (6 if fmt == "mxfp4" else 48)
    sa = torch.where(sa > 0, low, 0).to(torch.uint8)
    y = fq.gated_matmul_fp4(a, sa, b, sb, b, sb, fmt, out_dtype=torch.float32)
    g = (want / 64).cpu().numpy()
    gated_close(y, g, g, torch.float32)


# Gated outputs are not exact.  With g, u the exact sums, the fast exponential is off by up to
# 2 + |1.173 g| ulp (CUDA's documentation; an ulp is at most 2^-23 of the value), 1 + e by half an
# ulp, the fast division by 2 ulp, the two products by half an ulp each: under
# (6 + 1.2 |g|) 2^-23 of the value, and bf16's own rounding is eps / 2 = 2^-8.  Beyond |g| = 87
# the exponential may overflow (and the division by more than 2^126 gives 0) where
# |silu(g)| < 88 exp(-87) < 2e-36.
def gated_tol(want, g, u, out):
    tol = np.abs(want) * ((6 + 1.2 * np.abs(g)) * 2.0**-23
                          + (2.0**-8 if out == torch.bfloat16 else 0))
    return tol + np.where(g < -86, 2e-36 * np.abs(u), 0) + 1e-37


def gated_close(y, g, u, out):
    want = ref.silu(g) * u
    err = np.abs(as_float(y) - want)
    assert (err <= gated_tol(want, g, u, out)).all(), (err / (np.abs(want) + 1e-30)).max()


GATED = [(1, 1, 1), (1, 128, 256), (16, 64, 512), (5, 300, 1100), (32, 129, 96), (50, 256, 320),
         (64, 128, 128), (77, 1000, 64), (128, 140, 288), (129, 256, 256), (300, 130, 1000),
         (1, 24, 4096), (700, 384, 544), (515, 1000, 2048), (100, 2500, 512), (40, 72, 2080)]


def gated_operands(M, N, K, fmt, E=0):
    """Scales of 2^-6 on the tokens keep the pre-activations of the order of one to a hundred."""
    a, sa, va = exact_operand(M, K, 3, fmt, E)
    low = sa.cpu().numpy()
    low = np.where(low > 0, low - (6 if fmt == "mxfp4" else 6 * 8), 0).astype(np.uint8)
    return (a, torch.from_numpy(low).cuda(), va / 64.0, *exact_operand(N, K, 4, fmt, E),
            *exact_operand(N, K, 5, fmt, E))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", GATED)
def test_gated_product(M, N, K, fmt, out):
    a, sa, va, g, sg, vg, u, su, vu = gated_operands(M, N, K, fmt)
    y = fq.gated_matmul_fp4(a, sa, g, sg, u, su, fmt, out_dtype=out)
    assert y.shape == (M, N) and y.dtype == out
    gated_close(y, va @ vg.T, va @ vu.T, out)
    assert torch.equal(y, fq.gated_matmul_fp4(a, sa, g, sg, u, su, fmt, out_dtype=out))


@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (40, 200, 1504), (300, 260, 2048)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_nvfp4_tensor_scales_multiply_the_result(M, N, K, out):
    a, sa, va = exact_operand(M, K, 1, "nvfp4")
    b, sb, vb = exact_operand(N, K, 2, "nvfp4")
    u, su, vu = exact_operand(N, K, 6, "nvfp4")
    ta, tb, tu = (np.float32(v) for v in (0.0123, 0.37, 0.0071))
    y = fq.matmul_fp4(a, sa, b, sb, "nvfp4", on_gpu(ta), on_gpu(tb), out_dtype=out)
    want = (va @ vb.T).astype(np.float32) * (ta * tb)          # fp32, as the formula rounds
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(out))
    y = fq.gated_matmul_fp4(a, sa, b, sb, u, su, "nvfp4", on_gpu(ta), on_gpu(tb), on_gpu(tu),
                            out_dtype=out)
    # the pre-activations' own rounding, 2^-24 of each, moves silu(g) u by up to (2 + |g|) 2^-24 more
    g, up = (va @ vb.T) * float(ta * tb), (va @ vu.T) * float(ta * tu)
    want = ref.silu(g) * up
    tol = gated_tol(want, g, up, out) + np.abs(want) * (2 + np.abs(g)) * 2.0**-24
    assert (np.abs(as_float(y) - want) <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (96, 384, 2048), (300, 512, 3008)])
def test_product_of_quantised_values(fmt, M, N, K):
    """Scales over the whole range of real ones.  K sums of fp32, each of at most K additions that
    round by at most 2^-23 of a partial sum, which |a| |b| bounds."""
    rng = np.random.default_rng(9)
    x = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(np.float32)
    w = (rng.standard_normal((N, K)) * 0.02 * np.exp(rng.standard_normal((N, 1)))).astype(np.float32)
    tx, tw = nv_scale(x, fmt), nv_scale(w, fmt)
    a, sa = fq.scaled_fp4_blockwise(torch.from_numpy(x).cuda(), fmt, on_gpu(tx))
    b, sb = fq.scaled_fp4_blockwise(torch.from_numpy(w).cuda(), fmt, on_gpu(tw))
    y = as_float(fq.matmul_fp4(a, sa, b, sb, fmt, on_gpu(tx), on_gpu(tw), out_dtype=torch.float32))
    va, vb = ref.values(*ref.quantize(x, fmt, tx), fmt), ref.values(*ref.quantize(w, fmt, tw), fmt)
    t = 1.0 if tx is None else float(tx) * float(tw)
    tol = K * 2.0**-23 * (np.abs(va) @ np.abs(vb).T) * t
    assert (np.abs(y - (va @ vb.T) * t) <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 20, 64, 130, 300])
def test_stacks_with_rows_leave_the_rest_as_it_was(fmt, gated, M):
    E, N, K, ld = 6, 200, 352, 203
    a, sa, va, g, sg, vg, u, su, vu = gated_operands(M, N, K, fmt, E)
    counts = np.array([M, 0, M // 2, -3, M + 9, min(M, 129)])
    rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    buf = Guarded(E * (M + 2) * ld * 4)
    out = buf.view.view(torch.float32).as_strided((E, M, N), ((M + 2) * ld, ld, 1))
    if gated:
        y = fq.gated_matmul_fp4(a, sa, g, sg, u, su, fmt, rows=rows, out=out)
    else:
        y = fq.matmul_fp4(a, sa, g, sg, fmt, rows=rows, out=out)
    assert y.data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    assert buf.canaries_intact()
    assert (buf.view.view(E, M + 2, ld, 4)[:, :, N:] == CANARY).all()
    assert (buf.view.view(E, M + 2, ld, 4)[:, M:] == CANARY).all()
    for e, c in enumerate(np.clip(counts, 0, M)):
        if gated:
            gated_close(y[e, :c], va[e, :c] @ vg[e].T, va[e, :c] @ vu[e].T, torch.float32)
        else:
            assert np.array_equal(as_float(y[e, :c]), va[e, :c] @ vg[e].T)
        assert (out[e, c:].contiguous().view(torch.uint8) == CANARY).all()
    made = fq.matmul_fp4(a, sa, g, sg, fmt, rows=rows)        # an output made here: zeros behind
    for e, c in enumerate(np.clip(counts, 0, M)):
        assert (made[e, c:] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_halves_of_a_fused_weight_and_one_matrix_for_a_stack(fmt):
    E, M, F, K = 3, 40, 128, 224
    a, sa, va = exact_operand(M, K, 3, fmt, E)
    w, sw, vw = exact_operand(2 * F, K, 4, fmt, E)
    y = fq.matmul_fp4(a, sa, w[:, F:], sw[:, 1:], fmt, out_dtype=torch.float32)
    for e in range(E):
        assert np.array_equal(as_float(y[e]), va[e] @ vw[e, F:].T)
    one, s1, v1 = exact_operand(F, K, 8, fmt)
    y = fq.matmul_fp4(a, sa, one.expand(E, F, -1), s1.expand(E, *s1.shape), fmt,
                      out_dtype=torch.float32)
    for e in range(E):
        assert np.array_equal(as_float(y[e]), va[e] @ v1.T)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [3, 300])
def test_nan_scales_stay_in_their_rows(fmt, M):
    N, K = 150, 200
    a, sa, va = exact_operand(M, K, 1, fmt)
    b, sb, vb = exact_operand(N, K, 2, fmt)
    nan = 0xFF if fmt == "mxfp4" else 0x7F
    sa[0, 0, 2, 1] = nan                    # token 2, block 1
    sb[(N - 1) // 128, 0, (N - 1) % 32, 4 * ((N - 1) % 128 // 32)] = nan
    y = as_float(fq.matmul_fp4(a, sa, b, sb, fmt, out_dtype=torch.float32))
    want = va @ vb.T
    want[2] = np.nan
    want[:, N - 1] = np.nan
    assert np.array_equal(y, want, equal_nan=True)


@pytest.mark.parametrize("M", [1, 48, 300])
def test_streams_graphs_and_the_feed_forward_block(M):
    """quantise -> gated product -> quantise -> product on a side stream, then captured once and
    replayed on new inputs: the same outputs as call by call."""
    fmt, F, K = "mxfp4", 384, 256
    rng = np.random.default_rng(3)
    wg, wu, wd = (torch.from_numpy((rng.standard_normal(s) * 0.06).astype(np.float32)).cuda()
                  .to(torch.bfloat16) for s in ((F, K), (F, K), (K, F)))
    g, u, d = (fq.scaled_fp4_blockwise(w, fmt) for w in (wg, wu, wd))

    def block(x):
        h = fq.gated_matmul_fp4(*fq.scaled_fp4_blockwise(x, fmt), *g, *u, fmt)
        return h, fq.matmul_fp4(*fq.scaled_fp4_blockwise(h, fmt), *d, fmt)

    xs = [torch.randn(M, K, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    want = [block(x) for x in xs]
    # each product against its own inputs in 64 bits
    vals = [ref.values(*ref.quantize(w.float().cpu().numpy(), fmt), fmt) for w in (wg, wu, wd)]
    for x, (h, y) in zip(xs, want):
        vx = ref.values(*ref.quantize(x.float().cpu().numpy(), fmt), fmt)
        a, b = vx @ vals[0].T, vx @ vals[1].T
        s = np.abs(vx) @ np.abs(vals[0]).T, np.abs(vx) @ np.abs(vals[1]).T
        # sums off by K 2^-23 s, |silu'| <= 1.1; the activation by (6 + 1.2 |a|) 2^-23 < 2^-17
        # here (|a| < 40); then the output's half step
        lost = K * 2.0**-23 * (1.1 * s[0] * np.abs(b) + np.abs(ref.silu(a)) * s[1])
        hv = ref.silu(a) * b
        assert (np.abs(as_float(h) - hv) <= (2.0**-8 + 2.0**-17) * np.abs(hv) + 1.01 * lost).all()
        vh = ref.values(*ref.quantize(h.float().cpu().numpy(), fmt), fmt)
        yv = vh @ vals[2].T
        lost = F * 2.0**-23 * (np.abs(vh) @ np.abs(vals[2]).T)
        assert (np.abs(as_float(y) - yv) <= 2.0**-8 * np.abs(yv) + 1.01 * lost).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [block(x) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    for (h, y), (h2, y2) in zip(want, got):
        assert torch.equal(h, h2) and torch.equal(y, y2)
    x = xs[0].clone()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y = block(x)
    with torch.cuda.graph(other):
        h2, y2 = block(x)
    for k in (1, 2, 0):
        x.copy_(xs[k])
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k][1]) and torch.equal(y2, want[k][1])
        assert torch.equal(h, want[k][0]) and torch.equal(h2, want[k][0])


@pytest.mark.parametrize("pdl", [0, 1])
def test_calls_on_several_streams_at_once(pdl):
    """Products of several shapes in flight together: CTAs that share an SM share its tensor memory."""
    cases = []
    for i, (M, N, K) in enumerate([(1, 4096, 2048), (16, 1024, 4096), (64, 2048, 1024),
                                   (128, 1000, 2048), (300, 512, 1024), (600, 1024, 512)]):
        fmt = FORMATS[i % 2]
        a, b = exact_operand(M, K, i, fmt), exact_operand(N, K, 90 + i, fmt)
        cases.append((fmt, a, b, rounded(a[2] @ b[2].T, torch.float32)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    assert fq.fp8bq_set_pdl(pdl) == fq.FP8BQ_OK
    try:
        outs = []
        for rep in range(12):
            for i, (fmt, a, b, want) in enumerate(cases):
                st = streams[(i + rep) % 4]
                outs.append((fq.matmul_fp4(a[0], a[1], b[0], b[1], fmt, out_dtype=torch.float32,
                                           stream=st), want))
        torch.cuda.synchronize()
    finally:
        fq.fp8bq_set_pdl(1)
    for y, want in outs:
        assert np.array_equal(as_float(y), want)


@pytest.mark.parametrize("M", [1, 300])
def test_a_wait_that_runs_out_is_reported(M):
    a, sa, va = exact_operand(M, 1024, 1, "mxfp4")
    b, sb, vb = exact_operand(256, 1024, 2, "mxfp4")
    assert fq.fp8bq_debug_set_wait_limit_ns(5_000_000) == fq.FP8BQ_OK
    assert fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_DROP_FIRST_LOAD) == fq.FP8BQ_OK
    try:
        fq.matmul_fp4(a, sa, b, sb, "mxfp4")
        assert fq.fp8bq_sync_status() == fq.FP8BQ_ERR_DEVICE_TIMEOUT
    finally:
        fq.fp8bq_debug_set_inject(0)
        fq.fp8bq_debug_set_wait_limit_ns(0)
    y = fq.matmul_fp4(a, sa, b, sb, "mxfp4", out_dtype=torch.float32)
    assert np.array_equal(as_float(y), va @ vb.T)


def test_conveniences_refuse_what_does_not_fit():
    x = torch.zeros(40, 96, device="cuda", dtype=torch.bfloat16)
    c, s = fq.scaled_fp4_blockwise(x, "mxfp4")
    c3, s3 = fq.scaled_fp4_blockwise(torch.stack([x, x]), "mxfp4")
    t = torch.ones(1, device="cuda")
    bad = [
        (ValueError, lambda: fq.scaled_fp4_blockwise(x.t(), "mxfp4")),          # strided columns
        (ValueError, lambda: fq.scaled_fp4_blockwise(x[0], "mxfp4")),
        (ValueError, lambda: fq.scaled_fp4_blockwise(x[:1].expand(40, 96), "mxfp4")),   # rows overlap
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s, out=torch.empty(1, 40, device="cuda").expand(
            40, 40))),
        (TypeError, lambda: fq.scaled_fp4_blockwise(x.half(), "mxfp4")),
        (ValueError, lambda: fq.scaled_fp4_blockwise(x, "mxfp4", tensor_scale=t)),
        (TypeError, lambda: fq.scaled_fp4_blockwise(x, "nvfp4", tensor_scale=t.double())),
        (ValueError, lambda: fq.scaled_fp4_blockwise(x, "nvfp4", tensor_scale=t.expand(2))),
        (ValueError, lambda: fq.dequantize_fp4_blockwise(c, s, "mxfp4", columns=97)),
        (ValueError, lambda: fq.dequantize_fp4_blockwise(c, s, "mxfp4", columns=64)),
        (ValueError, lambda: fq.dequantize_fp4_blockwise(c, s, "nvfp4")),       # other tiles
        (TypeError, lambda: fq.dequantize_fp4_blockwise(c, s, out_dtype=torch.float16)),
        (TypeError, lambda: fq.dequantize_fp4_blockwise(c.view(torch.int8), s)),
        (ValueError, lambda: fq.matmul_fp4(c, s, c[:, :32], s)),
        (ValueError, lambda: fq.matmul_fp4(c, s, c3, s3)),                      # a stack with a matrix
        (ValueError, lambda: fq.matmul_fp4(c[::2], s, c, s)),                   # rows apart
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s[:, :, :16])),
        (ValueError, lambda: fq.gated_matmul_fp4(c, s, c, s, c[:32], s)),       # gate and up differ
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s, rows=torch.ones(1, device="cuda").int())),
        (ValueError, lambda: fq.matmul_fp4(c3, s3, c3, s3, rows=torch.ones(2, device="cuda"))),
        (ValueError, lambda: fq.matmul_fp4(c3, s3, c3, s3, rows=torch.ones(2).int())),
        (TypeError, lambda: fq.matmul_fp4(c, s, c, s, out_dtype=torch.float16)),
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s, out=x)),
        (TypeError, lambda: fq.matmul_fp4(c, s, c, s, out=torch.empty(40, 40, device="cuda").half())),
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s, out=torch.empty(40, 80, device="cuda")[:, ::2])),
        (ValueError, lambda: fq.matmul_fp4(c, s, c, s, "mxfp4", a_tensor_scale=t)),
        (fq.Fp8bqError, lambda: fq.matmul_fp4(c3, s3, c3, s3, out=torch.empty(
            1, 40, 40, device="cuda").expand(2, 40, 40))),                      # outputs overlap
        (fq.Fp8bqError, lambda: fq.matmul_fp4(c[:, :0], s[:, :0], c[:, :0], s[:, :0])),   # empty sums
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")


def test_empty_stacks_with_a_scale_for_each_matrix():
    x = torch.empty(0, 130, 96, device="cuda")
    t = torch.empty(0, device="cuda")
    c, s = fq.scaled_fp4_blockwise(x, "nvfp4", t)
    assert fq.dequantize_fp4_blockwise(c, s, "nvfp4", tensor_scale=t).shape == x.shape
    for ts in (t, torch.ones(1, device="cuda"), None):
        assert fq.matmul_fp4(c, s, c, s, "nvfp4", ts, ts).shape == (0, 130, 130)
        assert fq.gated_matmul_fp4(c, s, c, s, c, s, "nvfp4", ts, ts, ts).shape == (0, 130, 130)
    c, s = fq.scaled_fp4_blockwise(torch.ones(2, 96, device="cuda"), "nvfp4")
    with pytest.raises(ValueError):
        fq.matmul_fp4(c, s, c, s, "nvfp4", t)


def test_empty_inputs():
    for shape in ((0, 64), (3, 0), (0, 5, 64), (2, 0, 64)):
        x = torch.zeros(shape, device="cuda")
        c, s = fq.scaled_fp4_blockwise(x, "nvfp4")
        y = fq.dequantize_fp4_blockwise(c, s, "nvfp4", columns=shape[-1])
        assert y.shape == shape
    c, s = fq.scaled_fp4_blockwise(torch.zeros(0, 64, device="cuda"))
    w, ws = fq.scaled_fp4_blockwise(torch.ones(16, 64, device="cuda"))
    assert fq.matmul_fp4(c, s, w, ws).shape == (0, 16)
    assert fq.matmul_fp4(w, ws, c, s).shape == (16, 0)
    assert fq.quant_weights_fp4([]) == []


def test_offsets_beyond_32_bits():
    """A weight whose codes, and a product whose outputs, pass 4 GiB: the last rows are right."""
    M, K = 600_000, 16384                                     # 19.7 GB of bf16, 4.9 GB of codes
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(300, K, device="cuda").to(torch.bfloat16)
    x[-300:] = tail
    c, s = fq.scaled_fp4_blockwise(x)
    del x
    ct, st = fq.scaled_fp4_blockwise(torch.cat([torch.zeros(M % 128 + 128 * 3 - 300, K, device="cuda",
                                                            dtype=torch.bfloat16), tail]))
    assert torch.equal(c[-300:], ct[-300:]) and not c[:-300].any()
    assert torch.equal(s[-3:], st[-3:])
    v = fq.dequantize_fp4_blockwise(c, s, out_dtype=torch.bfloat16)
    assert torch.equal(v[-300:], fq.dequantize_fp4_blockwise(ct, st)[-300:])
    del v
    w, ws = fq.scaled_fp4_blockwise(torch.randn(4000, K, device="cuda").to(torch.bfloat16))
    y = fq.matmul_fp4(c, s, w, ws)                            # 600,000 x 4000 bf16: 4.8 GB
    yt = fq.matmul_fp4(ct, st, w, ws)
    assert torch.equal(y[-300:], yt[-300:]) and not y[:-300].any()
    y1 = fq.matmul_fp4(w[:7], ws[:1], c, s)                   # 600,000 outputs of 7 tokens
    assert torch.equal(y1[:, -300:].t(), y[-300:, :7])


def test_the_call_module_and_the_python_path_agree(monkeypatch):
    """The ordinary call goes through the call module; a stream, rows or an output given goes
    through Python: the same outputs."""
    now = torch.cuda.current_stream()
    t = torch.tensor([0.01], device="cuda")
    for fmt in FORMATS:
        ts = t if fmt == "nvfp4" else None
        for shape in ((3, 100), (2, 40, 96)):
            for dtype in (torch.bfloat16, torch.float32):
                x = torch.randn(shape, device="cuda").to(dtype)
                quick, slow = (fq.scaled_fp4_blockwise(x, fmt, ts, **k) for k in ({}, {"stream": now}))
                assert all(torch.equal(a, b) for a, b in zip(quick, slow))
                for k in (dict(columns=shape[-1]), dict(out_dtype=torch.float32), dict()):
                    a, b = (fq.dequantize_fp4_blockwise(*quick, fmt, tensor_scale=ts, **k, **e)
                            for e in ({}, {"stream": now}))
                    assert a.dtype == b.dtype and torch.equal(a, b)
                for out in (None, torch.float32):
                    a, b = (fq.matmul_fp4(*quick, *quick, fmt, ts, ts, out_dtype=out, **e)
                            for e in ({}, {"stream": now}))
                    assert a.dtype == b.dtype and torch.equal(a, b)
                    a, b = (fq.gated_matmul_fp4(*quick, *quick, *quick, fmt, ts, ts, ts, out_dtype=out,
                                                **e) for e in ({}, {"stream": now}))
                    assert a.dtype == b.dtype and torch.equal(a, b)
    w = torch.nn.Parameter(torch.randn(5, 64, device="cuda"))     # a subclass of Tensor
    assert torch.equal(fq.scaled_fp4_blockwise(w)[0], fq.scaled_fp4_blockwise(w.detach())[0])
    with monkeypatch.context() as m:
        m.setattr(fq, "_fp4_product", None)
        m.setattr(fq, "_fp4_setup", None)
        c, s = fq.scaled_fp4_blockwise(x[0], "mxfp4")
        fq.dequantize_fp4_blockwise(c, s)
        fq.matmul_fp4(c, s, c, s)
        fq.gated_matmul_fp4(c, s, c, s, c, s)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [5, 60, 600])
def test_no_valid_rows_at_all(M, gated):
    E, N, K = 3, 300, 512
    a, sa, _, g, sg, _, u, su, _ = gated_operands(M, N, K, "mxfp4", E)
    rows = torch.zeros(E, dtype=torch.int32, device="cuda")
    out = torch.full((E, M, N), 7.0, device="cuda")
    if gated:
        fq.gated_matmul_fp4(a, sa, g, sg, u, su, rows=rows, out=out)
    else:
        fq.matmul_fp4(a, sa, g, sg, rows=rows, out=out)
    assert (out == 7.0).all()


def test_a_long_list_of_weights():
    """More weights of one kind than one launch's descriptors hold."""
    g = torch.Generator().manual_seed(5)
    named = [(f"w{i}", torch.randn(1 + i % 7, 1 + (i * 13) % 90, generator=g).cuda()) for i in range(700)]
    named += [(f"s{i}", torch.randn(2, 3, 64, generator=g).cuda().to(torch.bfloat16)) for i in range(9)]
    out = dict(fq.quant_weights_fp4(named, "mxfp4"))
    for name, w in named:
        c, s = fq.scaled_fp4_blockwise(w, "mxfp4")
        assert torch.equal(out[name], c) and torch.equal(out[name + "_scale"], s)


FIRST_CALL = """
import torch, blockwise_fp8_weight_b200 as fq
x = torch.randn(%d, 512, device="cuda")
w = torch.randn(300, 512, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    c, s = fq.scaled_fp4_blockwise(x)
    d, t = fq.scaled_fp4_blockwise(w)
    y = fq.matmul_fp4(c, s, d, t)
    h = fq.gated_matmul_fp4(c, s, d, t, d, t)
    v = fq.dequantize_fp4_blockwise(c, s)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, fq.matmul_fp4(c, s, d, t))
assert torch.equal(h, fq.gated_matmul_fp4(c, s, d, t, d, t))
assert torch.equal(v, fq.dequantize_fp4_blockwise(*fq.scaled_fp4_blockwise(x)))
assert fq.fp8bq_sync_status() == fq.FP8BQ_OK
"""


@pytest.mark.parametrize("M", [2, 700])
def test_the_first_call_of_a_process_may_be_captured(M):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % M], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-3000:]


def test_calls_from_several_host_threads():
    import threading
    a, sa, va = exact_operand(20, 512, 1, "mxfp4")
    b, sb, vb = exact_operand(400, 512, 2, "mxfp4")
    want = torch.from_numpy(va @ vb.T).cuda().float()
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    if not torch.equal(fq.matmul_fp4(a, sa, b, sb, out_dtype=torch.float32), want):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001 -- reported by the test
            bad.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]
