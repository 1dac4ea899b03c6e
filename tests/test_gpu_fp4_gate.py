"""The gate of the gated product: silu over the range of fp32."""
import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert fq.fp8bq_sync_status() == fq.FP8BQ_OK


def gated_once(g_scale, u_scale, M, out):
    """(outputs, g, u in 64 bits) of M equal tokens: g = g_scale * (k + f / 16) for columns of every
    k of -6..6 in the grid's steps and f of 0..15, u = u_scale.  One product each of exact sums: token
    values 1 and 1/16 against codes k and f."""
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6])
    fine = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    k, f = (a.reshape(-1) for a in np.meshgrid(grid, fine, indexing="ij"))
    x = np.zeros((M, 32), np.float32)
    x[:, 0], x[:, 16] = 6.0, 6.0 / 16                 # blocks with scales of 1 and 1/16
    w = np.zeros((k.size, 32), np.float32)
    w[:, 0], w[:, 16] = k, f
    w[:, 15], w[:, 31] = 6.0, 6.0                     # every block's scale is 1; x is 0 there
    up = np.zeros((k.size, 32), np.float32)
    up[:, 0] = 6.0
    one = torch.ones(1, device="cuda")
    a = fq.scaled_fp4_blockwise(torch.from_numpy(x).cuda(), "nvfp4", one)
    b = fq.scaled_fp4_blockwise(torch.from_numpy(w).cuda(), "nvfp4", one)
    c = fq.scaled_fp4_blockwise(torch.from_numpy(up).cuda(), "nvfp4", one)
    for q, v in ((a, x), (b, w), (c, up)):
        assert np.array_equal(fq.dequantize_fp4_blockwise(
            *q, "nvfp4", columns=32, out_dtype=torch.float32).cpu().numpy(), v)
    tg, tu = (torch.tensor([s], dtype=torch.float32, device="cuda") for s in (g_scale, u_scale))
    y = fq.gated_matmul_fp4(*a, *b, *c, "nvfp4", None, tg, tu, out_dtype=out)
    assert torch.equal(y[0].expand_as(y), y)
    # sums are exact; each is rounded once by its tensor scale
    g = ((6 * k + 6 / 16 * f).astype(np.float32) * np.float32(g_scale)).astype(np.float64)
    return y[0].float().cpu().numpy().astype(np.float64), g, float(np.float32(36) * np.float32(u_scale))


@pytest.mark.parametrize("M", [1, 100, 600])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g_scale", [0.01, 0.11, 0.5, 1.3, 1.7, 2.1, 2.43])
def test_silu_is_as_exact_far_out_as_near_zero(g_scale, out, M):
    """In units of 2^-23 of the value: expf 2, v e and 1 + e a half each, the fast division 2, the
    product with u a half: 5.5.  (bf16: the fast exponential's 2 + 1.173 |g| in place of 2, and the
    output's half step of 2^-8.)  Below the normal range, beyond |g| = 87.3, the exponential's units
    are of 2^-149; v e and the product round by half of one more at most."""
    for u_scale in (1.0, 3e4):
        y, g, u = gated_once(g_scale, u_scale, M, out)
        want = ref.silu(g) * u
        tol = 5.5 * 2.0**-23 * np.abs(want)
        if out == torch.bfloat16:
            tol += (1.173 * np.abs(g) * 2.0**-23 + 2.0**-8) * np.abs(want) * 1.001
        units = 2 if out == torch.float32 else 2 + 1.173 * np.abs(g)
        tol += (units + 1) * 2.0**-149 * (1 + np.abs(g)) * (1 + u)
        err = np.abs(y - want)
        assert (err <= tol).all(), (g[err > tol][:4], (err / np.abs(want))[err > tol][:4] * 2.0**24)
        assert (y[g < -87.3] != 0).all()                  # exp(87.4) is beyond 2^126


@pytest.mark.parametrize("M", [1, 100, 600])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_beyond_the_exponential(M, out):
    """Gates of thousands: silu is the gate itself, or zero; nothing is NaN."""
    y, g, u = gated_once(300.0, 1.0, M, out)
    far = np.abs(g) > 150
    want = torch.from_numpy((np.where(g > 0, g, 0) * u)[far]).to(torch.float32).to(out).double().numpy()
    eps = 2.0**-21 if out == torch.float32 else 2.0**-7
    assert far.any() and (np.abs(y[far] - want) <= eps * want).all()
    assert np.isfinite(y).all()
