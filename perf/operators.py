"""The 4-bit operators' workloads: quantisation to microscaled 4-bit floating
point and back, the product of two such matrices, and the gated product of a
feed-forward block (both projections, the activation and the product).

With ``own`` false, ``run`` computes the operators in elementary torch
operations; with ``own`` true it makes the calls a user makes of
``blockwise_fp8_weight_b200``.

Layouts (made here by plain torch, the ones the library reads and writes):
codes ``[(E,) M, 16 * ceil(K / 32)]`` bytes, two e2m1 codes per byte, the even
column in the low half, columns beyond K zero; block scales in tiles of 128
rows by four blocks, ``[(E,) ceil(M / 128), ceil(K / (4 bs)), 32, 16]`` bytes,
row r of a tile at ``[r % 32, 4 * (r // 32) + block]``, zero beyond the matrix.
"""
import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a trainer's gate projection on its way into the rollout engine
        dict(name="quant_gate_proj_mx", kind="quant", E=1, M=12288, K=4096, fmt="mxfp4", dtype="bf16"),
        # fp32 master weights with ragged edges, with a scale for the tensor
        dict(name="quant_ragged_nv_f32", kind="quant", E=1, M=4000, K=4100, fmt="nvfp4", dtype="f32"),
        # one token's activations ahead of a product: latency
        dict(name="quant_token_mx", kind="quant", E=1, M=1, K=4096, fmt="mxfp4", dtype="bf16"),
        # the fused q, k, v projection of one decoded token
        dict(name="mm_token_mx", kind="mm", E=1, M=1, N=6144, K=4096, fmt="mxfp4", out="bf16"),
        # the down projection of a decode batch
        dict(name="mm_batch48_nv", kind="mm", E=1, M=48, N=4096, K=12288, fmt="nvfp4", out="bf16"),
        # the fused q, k, v projection of a prefill
        dict(name="mm_prefill_mx", kind="mm", E=1, M=8192, N=6144, K=4096, fmt="mxfp4", out="bf16"),
        # odd sizes, fp32 out
        dict(name="mm_ragged_nv_f32", kind="mm", E=1, M=515, N=1000, K=4100, fmt="nvfp4", out="f32"),
        # the experts' down projections of a padded batch of routed tokens
        dict(name="mm_experts_mx", kind="mm", E=128, M=64, N=2048, K=768, fmt="mxfp4", out="bf16"),
        # the feed-forward's gated half for one decoded token
        dict(name="gated_token_mx", kind="gated", E=1, M=1, N=12288, K=4096, fmt="mxfp4", out="bf16"),
        # ... for a prefill
        dict(name="gated_prefill_nv", kind="gated", E=1, M=2048, N=12288, K=4096, fmt="nvfp4", out="bf16"),
        # ... for the experts of a decode batch
        dict(name="gated_experts_nv", kind="gated", E=128, M=16, N=768, K=2048, fmt="nvfp4", out="bf16"),
        # ... odd sizes, fp32 out
        dict(name="gated_ragged_mx_f32", kind="gated", E=1, M=77, N=1000, K=2000, fmt="mxfp4", out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("quant", "mm", "mm", "gated"))
    fmt = rng.choice(("mxfp4", "nvfp4"))
    if kind == "quant":
        K = _log_int(rng, 32, 14000)
        return dict(kind=kind, E=1, M=_log_int(rng, 1, min(16384, 50_000_000 // K)), K=K, fmt=fmt,
                    dtype=rng.choice(("bf16", "f32")))
    out = rng.choice(("bf16", "bf16", "f32"))
    K, N = _log_int(rng, 64, 12288), _log_int(rng, 64, 12288)
    weights = 1 if kind == "mm" else 2
    if rng.random() < 0.25:  # a stack of experts
        E = _log_int(rng, 2, min(128, max(2, 200_000_000 // (K * N * weights))))
        M = _log_int(rng, 1, 128)
    else:
        E, M = 1, _log_int(rng, 1, 8192)
    M = min(M, max(1, 200_000_000_000 // (E * K * N * weights)))
    return dict(kind=kind, E=E, M=M, N=N, K=K, fmt=fmt, out=out)


def work(case):
    E, M, K, bs = case["E"], case["M"], case["K"], BLOCK[case["fmt"]]
    held = 0.5 + 1.0 / bs  # bytes for each 4-bit value
    if case["kind"] == "quant":  # x read, codes and scales written and read, values written
        n = E * M * K
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2 * held + 2), "flops": 4 * n}
    w = 1 if case["kind"] == "mm" else 2
    rows = sum(_rows(case)) if E > 1 else M
    outs = rows * case["N"] * (2 if case["out"] == "bf16" else 4)
    return {"bytes": (rows + E * w * case["N"]) * K * held + outs,
            "flops": 2 * rows * w * case["N"] * K}


def _rows(case):
    """Valid rows of each expert: a fixed spread over 0..M, the same for every seed."""
    E, M = case["E"], case["M"]
    return [(e * 7919 + 13) % (M + 1) for e in range(E)]


# ------------------------------------------------------------------ plain forms


def _untile(scales, rows, blocks):
    """[(E,) MT, KT, 32, 16] -> [(E,) rows, blocks]."""
    s = scales.reshape(*scales.shape[:-2], 32, 4, 4)
    mt, kt = s.shape[-5], s.shape[-4]
    s = s.movedim(-4, -2).movedim(-4, -3)  # [(E,) MT, 4, 32, KT, 4]
    return s.reshape(*s.shape[:-5], mt * 128, kt * 4)[..., :rows, :blocks]


def _tile(s):
    """[(E,) M, blocks] bytes -> [(E,) MT, KT, 32, 16], zero beyond."""
    M, nb = s.shape[-2:]
    mt, kt = -(-M // 128), -(-nb // 4)
    s = torch.nn.functional.pad(s, (0, kt * 4 - nb, 0, mt * 128 - M))
    s = s.reshape(*s.shape[:-2], mt, 4, 32, kt, 4).movedim(-2, -4).movedim(-3, -2)
    return s.reshape(*s.shape[:-5], mt, kt, 32, 16).contiguous()


def _blocks(x, bs):
    """fp32 blocks [..., nb, bs] of the last axis, zero beyond it (a multiple of 32 columns)."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % 32))
    return x.reshape(*x.shape[:-1], -1, bs)


def _e2m1(v):
    """Round to the e2m1 grid, to nearest, ties to even, beyond 6 to 6."""
    a = v.abs().clamp(max=6.0)
    step = 0.5 + 0.5 * (a >= 2.0) + 1.0 * (a >= 4.0)
    return torch.copysign(torch.round(a / step) * step, v)


def _quantise(x, fmt, tensor_scale):
    """(grid values [..., nb, bs], scales [..., nb] in fp32, scale bytes)."""
    b = _blocks(x, BLOCK[fmt])
    a = b.abs().amax(-1)
    if fmt == "mxfp4":
        e = (torch.frexp(a).exponent - 3).clamp(-127, 127)
        e = torch.where(a == 0, -127, e)
        q = _e2m1(torch.ldexp(torch.ldexp(b, -(e // 2)[..., None]), -(e - e // 2)[..., None]))
        s = torch.ldexp(torch.ldexp(torch.ones_like(a), e // 2), e - e // 2)
        code = (e + 127).to(torch.uint8)
    else:
        s8 = (a / 6.0 / tensor_scale).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float()
        d = s * tensor_scale
        r = torch.where(d > 0, 1.0 / d, 0.0).clamp(max=torch.finfo(torch.float32).max)
        q = _e2m1(b * r[..., None])
        code = s8.view(torch.uint8)
    bad = ~torch.isfinite(a)
    q = torch.where(bad[..., None], 0.0, q)
    return q, torch.where(bad, math.nan, s), torch.where(bad, 0xFF if fmt == "mxfp4" else 0x7F, code)


def _pack(q):
    """Grid values [..., nb, bs] -> code bytes [..., nb * bs / 2]."""
    a = q.abs()
    c = (2 * a).clamp(max=4) + (a - 2).clamp(0, 2) + (a - 4).clamp(0, 2) / 2
    c = (c.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _held(x, fmt, tensor_scale):
    """What a program has in hand: (codes, tiled scales)."""
    q, _, code = _quantise(x, fmt, tensor_scale)
    return _pack(q).contiguous(), _tile(code)


def _decode(codes, scales, fmt):
    """fp32 values [..., M, K] without the tensor's scale."""
    bs = BLOCK[fmt]
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1).flatten(-2)
    s = _untile(scales, codes.shape[-2], v.shape[-1] // bs)
    if fmt == "mxfp4":
        e = s.int() - 127
        f = torch.ldexp(torch.ldexp(torch.ones_like(e, dtype=torch.float32), e // 2), e - e // 2)
        f = torch.where(s == 255, math.nan, f)
    else:
        f = s.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, bs)) * f[..., None]).flatten(-2)


def _keep(state, y):
    """Rows behind an expert's last stay as they were in the output buffer."""
    if state["rows"] is None:
        return y
    at = torch.arange(y.shape[-2], device=y.device)
    return torch.where((at < state["rows"][:, None])[..., None], y, state["before"])


# ------------------------------------------------------------------ the passes

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    fmt, E, M, K = case["fmt"], case["E"], case["M"], case["K"]
    nv = fmt == "nvfp4"
    lead = (E,) if E > 1 else ()

    def scale(x):  # of a whole tensor, so that the blocks' scales span e4m3
        return (x.abs().amax().float() / (6.0 * 448.0)).reshape(1) if nv else None

    def spread(*shape):  # weights: rows of different sizes, some values far out
        w = normal(*shape) * 0.02 * torch.exp(0.5 * normal(*shape[:-1], 1))
        far = torch.rand(shape, generator=g, device="cuda") < 1e-3
        return torch.where(far, w * 20, w)

    state = {"case": case, "fmt": fmt}
    if case["kind"] == "quant":
        x = (spread if M > 64 else normal)(*lead, M, K).to(DTYPE[case["dtype"]])
        state |= {"x": x, "t": scale(x)}
        return state
    x = (normal(*lead, M, K) * torch.exp(0.5 * normal(*lead, M, 1))).to(torch.bfloat16)
    state["xt"] = scale(x)
    state["x"], state["xs"] = _held(x, fmt, state["xt"])
    for k in ("w",) if case["kind"] == "mm" else ("g", "u"):
        w = spread(*lead, case["N"], K).to(torch.bfloat16)
        if k != "w":  # pre-activations of order one, as a trained block has
            w = w * (2.0 / math.sqrt(K) / 0.02)
        state[k + "t"] = scale(w)
        state[k], state[k + "s"] = _held(w, fmt, state[k + "t"])
        del w
    state["out_dtype"] = DTYPE[case["out"]]
    state["rows"] = state["before"] = None
    if E > 1:
        state["rows"] = torch.tensor(_rows(case), dtype=torch.int32, device="cuda")
        state["before"] = normal(E, M, case["N"]).to(state["out_dtype"])
        state["buffer"] = state["before"].clone()
    return state


def run(state):
    kind, fmt = state["case"]["kind"], state["fmt"]
    if own:
        import blockwise_fp8_weight_b200 as fq

        if kind == "quant":
            codes, scales = fq.scaled_fp4_blockwise(state["x"], fmt, tensor_scale=state["t"])
            return fq.dequantize_fp4_blockwise(codes, scales, fmt, columns=state["x"].shape[-1],
                                               tensor_scale=state["t"])
        kw = dict(a_tensor_scale=state["xt"], out_dtype=state["out_dtype"], rows=state["rows"],
                  out=state.get("buffer"))
        if kind == "mm":
            return fq.matmul_fp4(state["x"], state["xs"], state["w"], state["ws"], fmt,
                                 b_tensor_scale=state["wt"], **kw)
        return fq.gated_matmul_fp4(state["x"], state["xs"], state["g"], state["gs"], state["u"],
                                   state["us"], fmt, gate_tensor_scale=state["gt"],
                                   up_tensor_scale=state["ut"], **kw)
    if kind == "quant":
        x, t = state["x"], state["t"]
        q, s, _ = _quantise(x, fmt, t)
        v = q * s[..., None] if t is None else q * s[..., None] * t
        return v.flatten(-2)[..., : x.shape[-1]].to(torch.bfloat16)
    x = _decode(state["x"], state["xs"], fmt)

    def product(k):
        y = x @ _decode(state[k], state[k + "s"], fmt).transpose(-1, -2)
        return y if state["xt"] is None else y * (state["xt"] * state[k + "t"])

    if kind == "mm":
        return _keep(state, product("w").to(state["out_dtype"]))
    a = product("g")
    return _keep(state, (a / (1.0 + torch.exp(-a)) * product("u")).to(state["out_dtype"]))


# ------------------------------------------------------------------ in 64 bits


def _value64(codes, scales, fmt):
    """The codes' values in 64 bits, from the formats' fields."""
    rows, kb = codes.shape[-2:]
    cols = torch.arange(2 * kb, device=codes.device)
    c = ((codes[..., cols // 2].int() >> (4 * (cols % 2)).int()) & 15).double()
    sign, c = 1.0 - 2.0 * (c >= 8), c % 8
    ex, man = torch.floor(c / 2), c % 2
    v = sign * torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * 2.0 ** (ex - 1.0))
    r, b = torch.arange(rows, device=codes.device)[:, None], (cols // BLOCK[fmt])[None]
    s = scales[..., r // 128, b // 4, r % 32, 4 * (r % 128 // 32) + b % 4].double()
    if fmt == "mxfp4":
        return v * torch.where(s == 255, math.nan, 2.0 ** (s - 127.0))
    ex, man = torch.floor(s / 8), s % 8
    f = torch.where(ex == 0, man * 2.0**-9, (1.0 + man / 8.0) * 2.0 ** (ex - 7.0))
    return v * torch.where(s == 127, math.nan, f)


def exact(case, seed):
    w = work(case)
    if case["kind"] != "quant" and w["flops"] > 5e11:
        return None
    state = prepare(case, seed)
    fmt, bs = case["fmt"], BLOCK[case["fmt"]]
    if case["kind"] == "quant":
        x = state["x"].double()
        K = x.shape[-1]
        x = torch.nn.functional.pad(x, (0, -K % bs)).unflatten(-1, (-1, bs))
        a = x.abs().amax(-1, keepdim=True)
        if fmt == "mxfp4":
            power = torch.tensor([2.0**k for k in range(-125, 129)], device=x.device,
                                 dtype=torch.float64)  # the largest that a reaches
            d = power[(torch.searchsorted(power, a, right=True) - 1).clamp(min=0)] / 4.0
        else:  # the nearest of the 127 values of e4m3, in the even code's favour at ties
            code = torch.arange(127, device=x.device, dtype=torch.float64)
            e4m3 = torch.where(code < 8, code * 2.0**-9,
                               (1 + code % 8 / 8) * 2.0 ** (torch.floor(code / 8) - 7))
            want = torch.clamp(a / 6.0 / state["t"].double(), max=448.0)
            hi = torch.searchsorted(e4m3, want).clamp(max=126)
            lo = (hi - 1).clamp(min=0)
            up, down = e4m3[hi] - want, want - e4m3[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            d = e4m3[pick] * state["t"].double()
        v = torch.where(d > 0, x / d, 0.0)
        n = v.abs()
        near = torch.zeros_like(n)  # a midpoint goes to the even code
        for k, (low, high) in enumerate(zip(GRID, GRID[1:])):
            mid = (low + high) / 2
            near = torch.where((n > mid) | ((n == mid) & (k % 2 == 1)), high, near)
        return (torch.sign(v) * near * d).flatten(-2)[..., :K]
    x = _value64(state["x"], state["xs"], fmt)

    def product(k):
        y = torch.einsum("...mk,...nk->...mn", x, _value64(state[k], state[k + "s"], fmt))
        return y if state["xt"] is None else y * state["xt"].double() * state[k + "t"].double()

    y = product("w") if case["kind"] == "mm" else None
    if y is None:
        a = product("g")
        y = a * torch.sigmoid(a) * product("u")
    if state["rows"] is not None:
        past = torch.arange(y.shape[-2], device=y.device) >= state["rows"][:, None]
        y = torch.where(past[..., None], state["before"].double(), y)
    return y
