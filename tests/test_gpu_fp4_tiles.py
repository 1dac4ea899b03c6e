"""Every kernel and tile width of the 4-bit products, forced: which one a shape reaches by itself is
an estimate of times, and moves with it."""
import contextlib

import numpy as np
import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from tests.gpu_util import CANARY, Guarded
from tests.test_gpu_fp4 import exact_operand

pytestmark = pytest.mark.gpu
FORMATS = ("mxfp4", "nvfp4")
TYPES = (torch.float32, torch.bfloat16)
checked_only = pytest.mark.skipif(not fq.CHECKED, reason="needs the checked library")

# (gated, tokens): 0 is the many-token kernel
KERNELS = [(False, t) for t in (0, 16, 32, 64, 128, 256)] + [(True, t) for t in (0, 16, 32, 64, 128)]
kernels = pytest.mark.parametrize("gated,tokens", KERNELS,
                                  ids=[("gated-" if g else "") + str(t) for g, t in KERNELS])


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


@contextlib.contextmanager
def forced(tokens, M):
    """The kernel forced for products of M tokens."""
    assert tokens == 0 or tokens >= 64 or M <= tokens
    assert fq.fp8bq_debug_set_fp4_tokens(tokens) == fq.FP8BQ_OK
    try:
        yield
    finally:
        fq.fp8bq_debug_set_fp4_tokens(-1)


def fit(tokens, M):
    """M, or as many tokens as the width holds."""
    return min(M, tokens) if tokens in (16, 32) else M


class Case:
    """Operands whose sums are exact in fp32, and the expected outputs in 64 bits (on the GPU)."""

    def __init__(self, gated, M, N, K, fmt, E=0):
        self.gated, self.fmt = gated, fmt
        a, sa, va = exact_operand(M, K, 3, fmt, E)
        if gated:                                   # pre-activations of the order of one to a hundred
            low = sa.int() - (6 if fmt == "mxfp4" else 48)
            sa, va = torch.where(sa > 0, low, 0).to(torch.uint8), va / 64.0
        self.a = (a, sa)
        ws = [exact_operand(N, K, 4 + i, fmt, E) for i in range(2 if gated else 1)]
        self.w = [(w, s) for w, s, _ in ws]
        v = torch.from_numpy(va).cuda()
        self.sums = [v @ torch.from_numpy(x).cuda().transpose(-1, -2) for _, _, x in ws]

    def run(self, scales=(None, None, None), **kw):
        if self.gated:
            return fq.gated_matmul_fp4(*self.a, *self.w[0], *self.w[1], self.fmt, scales[0], scales[1],
                                       scales[2], **kw)
        return fq.matmul_fp4(*self.a, *self.w[0], self.fmt, scales[0], scales[1], **kw)

    def check(self, y, alpha=None, at=...):
        """y[at] against the formula; alpha: the fp32 products of the tensor scales, [E, 1, 1] each."""
        s = [x if alpha is None else x * al.double() for x, al in zip(self.sums, alpha or (1, 1))]
        if not self.gated:
            want = s[0].float() if alpha is None else self.sums[0].float() * alpha[0]
            assert torch.equal(y[at], want.to(y.dtype)[at])
            return
        g, u = (x[at] for x in s)
        want = g / (1 + torch.exp(-g)) * u
        # the fast exponential 2 + 1.173 |g| units of 2^-23 (expf 2), the fast division 2, four roundings
        # of half a unit; with tensor scales each pre-activation rounds once, which moves silu(g) u
        # by (2 + |g|) 2^-24; bf16's own half step.  Beyond exp(-87) steps of 2^-149.
        tol = want.abs() * ((6 + 1.2 * g.abs()) * 2.0**-23 + (2.0**-8 if y.dtype == torch.bfloat16 else 0)
                            + (0 if alpha is None else (2 + g.abs()) * 2.0**-24))
        tol += 2.0**-149 * (4 + 1.2 * g.abs()) * (1 + g.abs()) * (1 + u.abs())
        err = (y[at].double() - want).abs()
        assert (err <= tol).all(), (err / (want.abs() + 1e-30)).max()


# a cluster that splits K, one tile, several tiles for each CTA, and more rounds than one
SHAPES = [(1, 130, 8192), (40, 257, 4100), (129, 64, 64), (300, 500, 1056), (515, 1000, 288),
          (300, 40000, 96), (700, 25001, 544)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
@kernels
def test_sums_are_exact(gated, tokens, M, N, K, fmt, out):
    M = fit(tokens, M)
    c = Case(gated, M, N, K, fmt)
    with forced(tokens, M):
        y = c.run(out_dtype=out)
        again = c.run(out_dtype=out)
    c.check(y)
    assert torch.equal(y, again)


# row strides and starts for stores of 32, 16, 8, 4 bytes and by element
def layouts(N):
    return ((N + -N % 16, 0), (N + -N % 16 + 8, 0), (N + -N % 4 + 4, 0), (N + -N % 2 + 2, 2), (N, 0),
            (N + 1 - N % 2, 1))


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 77, 2048), (100, 1030, 64), (300, 515, 544), (600, 9001, 64)])
@kernels
def test_outputs_of_every_alignment(gated, tokens, M, N, K, out):
    M, es = fit(tokens, M), 2 if out == torch.bfloat16 else 4
    c = Case(gated, M, N, K, "mxfp4")
    for ld, start in layouts(N):
        buf = Guarded((M * ld + start) * es)
        flat = buf.view.view(out)
        y = flat.as_strided((M, N), (ld, 1), flat.storage_offset() + start)
        with forced(tokens, M):
            c.run(out=y)
        c.check(y)
        assert buf.canaries_intact(), (ld, start)
        rows = buf.view[start * es:].view(M, ld, es)
        assert (rows[:, N:] == CANARY).all() and (buf.view[:start * es] == CANARY).all(), (ld, start)


@pytest.mark.parametrize("fmt,out", [("mxfp4", torch.float32), ("nvfp4", torch.bfloat16)])
@pytest.mark.parametrize("ld", [1024, 1003])
@pytest.mark.parametrize("M", [20, 300, 600])
@kernels
def test_stacks_with_counts_of_rows(gated, tokens, M, ld, fmt, out):
    """More tiles than the device runs at once; matrices without rows, with parts of a tile, with
    one row more than a tile, and with counts out of range; then no rows at all."""
    M, N, K = fit(tokens, M), 1000, 352
    counts = [M, 0, M // 2, -3, M + 9, min(M, 129), 0, 1, min(M, 257), M, 0, M - 1]
    E = len(counts)
    c = Case(gated, M, N, K, fmt, E)
    rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    es = 2 if out == torch.bfloat16 else 4
    buf = Guarded(E * (M + 1) * ld * es)
    y = buf.view.view(out).as_strided((E, M, N), ((M + 1) * ld, ld, 1), buf.view.view(out).storage_offset())
    with forced(tokens, M):
        c.run(rows=torch.zeros_like(rows), out=y)
        torch.cuda.synchronize()
        assert buf.canaries_intact() and (buf.view == CANARY).all()
        c.run(rows=rows, out=y)
    assert buf.canaries_intact()
    bytes_ = buf.view.view(E, M + 1, ld, es)
    assert (bytes_[:, :, N:] == CANARY).all() and (bytes_[:, M:] == CANARY).all()
    for e, n in enumerate(np.clip(counts, 0, M)):
        assert (bytes_[e, n:] == CANARY).all(), e
        c.check(y, at=(e, slice(0, int(n))))


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,K", [(7, 2080), (140, 96)])
@kernels
def test_a_tensor_scale_for_each_matrix(gated, tokens, M, K, out):
    """Of the tokens, of the weights, of both, one of them shared; in a stack of one too."""
    M, N = fit(tokens, M), 500
    for E in (5, 1):
        c = Case(gated, M, N, K, "nvfp4", E)
        rng = np.random.default_rng(E)
        each = [torch.from_numpy((0.3 + rng.random(E)).astype(np.float32)).cuda() for _ in range(3)]
        one = [t[:1].clone() for t in each]
        for picks in ((each[0], each[1], each[2]), (each[0], one[1], None), (one[0], each[1], one[2]),
                      (None, one[1], each[2])):
            with forced(tokens, M):
                y = c.run(scales=picks, out_dtype=out)
            t = [torch.ones(1, 1, 1, device="cuda") if s is None else s.view(-1, 1, 1) for s in picks]
            c.check(y, alpha=[t[0] * t[1], t[0] * t[2]])


@pytest.mark.parametrize("M,N,K", [(20, 300, 2048), (300, 1000, 96), (200, 60000, 288)])
@kernels
def test_a_load_that_never_comes_is_reported(gated, tokens, M, N, K):
    """The first CTA leaves its first load out, so its waits run out (5 ms here): the call is
    reported, and the next one is right."""
    M = fit(tokens, M)
    c = Case(gated, M, N, K, "mxfp4")
    assert fq.fp8bq_debug_set_wait_limit_ns(5_000_000) == fq.FP8BQ_OK
    assert fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_DROP_FIRST_LOAD) == fq.FP8BQ_OK
    try:
        with forced(tokens, M):
            c.run()
            assert fq.fp8bq_sync_status() == fq.FP8BQ_ERR_DEVICE_TIMEOUT
    finally:
        fq.fp8bq_debug_set_inject(0)
        fq.fp8bq_debug_set_wait_limit_ns(0)
    with forced(tokens, M):
        y = c.run(out_dtype=torch.float32)
    c.check(y)


@pytest.mark.parametrize("pdl", [0, 1])
def test_every_kernel_at_once(pdl):
    """All of them on four streams: CTAs of different kernels share SMs and their tensor memory."""
    cases = [(t, Case(g, fit(t, 200), 700, 1056, FORMATS[i % 2])) for i, (g, t) in enumerate(KERNELS)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    assert fq.fp8bq_set_pdl(pdl) == fq.FP8BQ_OK
    try:
        outs = []
        for rep in range(8):
            for i, (t, c) in enumerate(cases):
                with forced(t, fit(t, 200)):
                    outs.append((c, c.run(out_dtype=torch.float32, stream=streams[(i + rep) % 4])))
        torch.cuda.synchronize()
    finally:
        fq.fp8bq_set_pdl(1)
    first = {}
    for c, y in outs:
        if c not in first:
            c.check(y)
            first[c] = y
        assert torch.equal(y, first[c])


# ------------------------------------------------------------------ the bounds-checked build


@checked_only
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,N", [(9, 130), (300, 515), (129, 40001)])
@kernels
def test_trimmed_outputs_are_caught(gated, tokens, M, N, out):
    """With the output taken one byte short, the last store is reported and skipped."""
    M, es = fit(tokens, M), 2 if out == torch.bfloat16 else 4
    c = Case(gated, M, N, 64, "mxfp4")
    for ld, start in layouts(N):
        nbytes = ((M - 1) * ld + N + start) * es
        buf = Guarded(nbytes)
        flat = buf.view.view(out)
        y = flat.as_strided((M, N), (ld, 1), flat.storage_offset() + start)
        assert fq.fp8bq_debug_take_bounds()[0] == fq.FP8BQ_OK
        assert fq.fp8bq_debug_set_inject(fq.FP8BQ_INJECT_TRIM_OUTPUTS) == fq.FP8BQ_OK
        try:
            with forced(tokens, M):
                c.run(out=y)
            assert fq.fp8bq_sync_status() == fq.FP8BQ_ERR_DEVICE_BOUNDS
            st, count, first = fq.fp8bq_debug_take_bounds()
        finally:
            fq.fp8bq_debug_set_inject(0)
            fq.fp8bq_debug_take_bounds()
        assert st == fq.FP8BQ_OK and count >= 1 and buf.ptr + nbytes - 32 <= first < buf.ptr + nbytes
        assert buf.canaries_intact() and buf.view[-1] == CANARY
