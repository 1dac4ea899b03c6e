"""Blockwise FP8 (float8_e4m3fn) weight quantizer for NVIDIA B200 (sm_100a).

A thin ctypes binding of the C ABI in ``include/fp8bq.h`` (library
``libfp8bq.so``, built in-tree by ``blockwise_fp8_weight_b200.build``).  The
functions named ``fp8bq_*`` mirror the C entry points one to one and only
marshal arguments; every step of the quantization runs in the library's CUDA
kernels.  There is no CPU or PyTorch fallback: if the library cannot be
loaded, every call raises.

On top of the raw entry points, two conveniences keep the call shapes of the
pages' Python API (verl docs "fp8_kernel.py -- FP8 量化内核", section 1 and
"vllm_fp8_utils.py", section 3):

    scaled_fp8_blockwise(data_hp, weight_block_size) -> (fp8_data, descale)
    quant_weights(named_weights, weight_block_size)  -> [(name, fp8), (name + "_scale_inv", s), ...]

and the same for microscaled 4-bit floating point ("mxfp4", "nvfp4"), with the
products that read it:

    scaled_fp4_blockwise(data_hp, format)            -> (codes, scales)
    quant_weights_fp4(named_weights, format)         -> [(name, codes), (name + "_scale", s), ...]
    dequantize_fp4_blockwise(codes, scales, format)  -> values
    matmul_fp4(a, a_scales, b, b_scales, format)     -> a b^T
    gated_matmul_fp4(a, a_scales, gate, gate_scales, up, up_scales, format)
                                                     -> silu(a gate^T) * (a up^T)

They allocate the outputs with PyTorch (device memory and streams are
PyTorch's job here) and hand the pointers to the library.

With the environment variable ``FP8BQ_CHECKED=1`` set before the first call,
the process loads ``libfp8bq_checked.so`` instead: the same library with every
plain global access of its kernels bounds-checked (``fp8bq_checked_build``,
``fp8bq_debug_take_bounds``).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Iterable, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
CHECKED = os.environ.get("FP8BQ_CHECKED", "0") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libfp8bq_checked.so" if CHECKED else "libfp8bq.so")

# fp8bq_dtype
FP8BQ_BF16 = 0
FP8BQ_F32 = 1
# fp8bq_status
FP8BQ_OK = 0
FP8BQ_ERR_NULL = 1
FP8BQ_ERR_SHAPE = 2
FP8BQ_ERR_BLOCK = 3
FP8BQ_ERR_DTYPE = 4
FP8BQ_ERR_OVERLAP = 5
FP8BQ_ERR_DEVICE = 6
FP8BQ_ERR_DEVICE_TIMEOUT = 7
FP8BQ_ERR_ALIGN = 8
FP8BQ_ERR_ARG = 9
FP8BQ_ERR_DEVICE_UNSAFE = 10
FP8BQ_ERR_DEVICE_BOUNDS = 11
# fp8bq_path
FP8BQ_PATH_AUTO = 0
FP8BQ_PATH_VECTOR = 1
FP8BQ_PATH_TMA = 2
FP8BQ_PATH_GENERIC = 3
FP8BQ_INJECT_DROP_FIRST_LOAD = 1
FP8BQ_INJECT_TRIM_OUTPUTS = 2
# fp8bq_fp4_format
FP8BQ_MXFP4 = 0
FP8BQ_NVFP4 = 1

DEFAULT_BLOCK = (128, 128)


class fp8bq_desc(ctypes.Structure):
    """Mirror of ``struct fp8bq_desc`` (96 bytes)."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("y_u8", ctypes.c_void_p),
        ("descale_f32", ctypes.c_void_p),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("ld", ctypes.c_int64),
        ("batch", ctypes.c_int64),
        ("x_batch_stride", ctypes.c_int64),
        ("y_batch_stride", ctypes.c_int64),
        ("s_batch_stride", ctypes.c_int64),
        ("dtype_in", ctypes.c_int32),
        ("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class fp8bq_dequant_desc(ctypes.Structure):
    """Mirror of ``struct fp8bq_dequant_desc`` (80 bytes)."""
    _fields_ = [
        ("y_u8", ctypes.c_void_p),
        ("descale_f32", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("batch", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
        ("ld_out", ctypes.c_int64),
        ("out_batch_stride", ctypes.c_int64),
        ("dtype_out", ctypes.c_int32),
        ("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class fp8bq_scale_desc(ctypes.Structure):
    """Mirror of ``struct fp8bq_scale_desc`` (24 bytes)."""
    _fields_ = [("x", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype_in", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class fp8bq_fp4_desc(ctypes.Structure):
    """Mirror of ``struct fp8bq_fp4_desc`` (88 bytes)."""
    _fields_ = [
        ("x", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("tensor_scale", ctypes.c_void_p),
        ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("ld", ctypes.c_int64),
        ("batch", ctypes.c_int64), ("x_batch_stride", ctypes.c_int64),
        ("tensor_scale_stride", ctypes.c_int64),
        ("dtype_in", ctypes.c_int32), ("format", ctypes.c_int32),
    ]


class fp8bq_fp4_operand(ctypes.Structure):
    """Mirror of ``struct fp8bq_fp4_operand`` (48 bytes)."""
    _fields_ = [
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
        ("codes_batch_stride", ctypes.c_int64), ("scales_batch_stride", ctypes.c_int64),
        ("tensor_scale_stride", ctypes.c_int64),
    ]


class fp8bq_fp4_matmul_desc(ctypes.Structure):
    """Mirror of ``struct fp8bq_fp4_matmul_desc`` (216 bytes)."""
    _fields_ = [
        ("a", fp8bq_fp4_operand), ("b", fp8bq_fp4_operand), ("up", fp8bq_fp4_operand),
        ("out", ctypes.c_void_p), ("rows", ctypes.c_void_p),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("batch", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("out_batch_stride", ctypes.c_int64),
        ("format", ctypes.c_int32), ("dtype_out", ctypes.c_int32),
    ]


class Fp8bqError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = fp8bq_status_string(status)
        super().__init__(f"{what}: {msg}" if what else msg)


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load ``libfp8bq.so`` (``libfp8bq_checked.so`` under FP8BQ_CHECKED=1),
    building it first with nvcc if it is missing or older than its sources.
    Raises if it cannot be built or loaded."""
    global _lib
    with _lock:
        if _lib is None:
            from . import build as _build
            if not _build.up_to_date(LIB_PATH):
                _build.build(checked=CHECKED)
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            L.fp8bq_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp]
            L.fp8bq_quantize.restype = i32
            L.fp8bq_quantize_batched.argtypes = [ctypes.POINTER(fp8bq_desc), i32, vp]
            L.fp8bq_quantize_batched.restype = i32
            L.fp8bq_dequantize.argtypes = [vp, vp, i64, i64, i64, i32, i32, vp, i32, i64, i64, vp]
            L.fp8bq_dequantize.restype = i32
            L.fp8bq_dequantize_batched.argtypes = [ctypes.POINTER(fp8bq_dequant_desc), i32, vp]
            L.fp8bq_dequantize_batched.restype = i32
            L.fp8bq_tensor_scale.argtypes = [ctypes.POINTER(fp8bq_scale_desc), i32, vp, vp]
            L.fp8bq_tensor_scale.restype = i32
            L.fp8bq_status_string.argtypes = [i32]
            L.fp8bq_status_string.restype = ctypes.c_char_p
            L.fp8bq_sync_status.argtypes = [vp]
            L.fp8bq_sync_status.restype = i32
            L.fp8bq_version.argtypes = []
            L.fp8bq_version.restype = i32
            L.fp8bq_set_path.argtypes = [i32]
            L.fp8bq_set_path.restype = i32
            L.fp8bq_get_path.argtypes = []
            L.fp8bq_get_path.restype = i32
            L.fp8bq_set_pdl.argtypes = [i32]
            L.fp8bq_set_pdl.restype = i32
            L.fp8bq_get_pdl.argtypes = []
            L.fp8bq_get_pdl.restype = i32
            L.fp8bq_set_pdl_min_us.argtypes = [ctypes.c_double]
            L.fp8bq_set_pdl_min_us.restype = i32
            L.fp8bq_get_pdl_min_us.argtypes = []
            L.fp8bq_get_pdl_min_us.restype = ctypes.c_double
            L.fp8bq_path_for.argtypes = [ctypes.POINTER(fp8bq_desc)]
            L.fp8bq_path_for.restype = i32
            L.fp8bq_launch_count.argtypes = [ctypes.POINTER(fp8bq_desc), i32]
            L.fp8bq_launch_count.restype = i32
            L.fp8bq_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.fp8bq_debug_set_wait_limit_ns.restype = i32
            L.fp8bq_debug_set_inject.argtypes = [ctypes.c_uint32]
            L.fp8bq_debug_set_inject.restype = i32
            L.fp8bq_checked_build.argtypes = []
            L.fp8bq_checked_build.restype = i32
            L.fp8bq_debug_take_bounds.argtypes = [ctypes.POINTER(ctypes.c_uint64),
                                                  ctypes.POINTER(ctypes.c_uint64)]
            L.fp8bq_debug_take_bounds.restype = i32
            L.fp8bq_fp4_quantize.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp]
            L.fp8bq_fp4_quantize.restype = i32
            L.fp8bq_fp4_quantize_batched.argtypes = [vp, i32, vp]
            L.fp8bq_fp4_quantize_batched.restype = i32
            L.fp8bq_fp4_dequantize.argtypes = [vp, vp, i64, i64, i64, i32, vp, i64, vp, i32, i64,
                                               i64, vp]
            L.fp8bq_fp4_dequantize.restype = i32
            L.fp8bq_fp4_tensor_scale.argtypes = [ctypes.POINTER(fp8bq_scale_desc), i32, vp, vp]
            L.fp8bq_fp4_tensor_scale.restype = i32
            # the descriptor: a fp8bq_fp4_matmul_desc by reference, or its bytes
            L.fp8bq_fp4_matmul.argtypes = [vp, vp]
            L.fp8bq_fp4_matmul.restype = i32
            L.fp8bq_fp4_gated_matmul.argtypes = [vp, vp]
            L.fp8bq_fp4_gated_matmul.restype = i32
            L.fp8bq_fp4_plan.argtypes = [ctypes.POINTER(fp8bq_fp4_matmul_desc), i32,
                                         ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.fp8bq_fp4_plan.restype = i32
            L.fp8bq_debug_set_fp4_tokens.argtypes = [i32]
            L.fp8bq_debug_set_fp4_tokens.restype = i32
            # A call through Python takes about 9 us.  With the launch overlap for every
            # call, one token's product takes 1.6 us more of them.
            L.fp8bq_set_pdl_min_us(6.5)
            _lib = L
    return _lib


def _ptr(a) -> int:
    """Pointer value of an int, None, or a tensor-like with data_ptr()."""
    if a is None:
        return 0
    if isinstance(a, int):
        return a
    return int(a.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        if not torch.cuda.is_available():
            return 0  # no device: the library reports FP8BQ_ERR_DEVICE itself
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ----------------------------------------------------------------- C entry points


def fp8bq_quantize(x, dtype_in: int, M: int, N: int, ld: int, block_m: int, block_n: int,
                   y_u8, descale_f32, stream=None) -> int:
    """``fp8bq_quantize`` of the C ABI; pointers may be ints or tensors.
    Returns the fp8bq_status code."""
    return lib().fp8bq_quantize(_ptr(x), dtype_in, M, N, ld, block_m, block_n, _ptr(y_u8),
                                _ptr(descale_f32), _stream(stream))


def fp8bq_quantize_batched(desc_table: Sequence[fp8bq_desc] | ctypes.Array, n_tensors=None,
                           stream=None) -> int:
    """``fp8bq_quantize_batched`` of the C ABI.  Returns the status code."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_quantize_batched(desc_table, n, _stream(stream))


def fp8bq_dequantize(y_u8, descale_f32, batch: int, M: int, N: int, block_m: int, block_n: int,
                     out, dtype_out: int, ld_out: int, out_batch_stride: int, stream=None) -> int:
    """``fp8bq_dequantize`` of the C ABI.  Returns the status code."""
    return lib().fp8bq_dequantize(_ptr(y_u8), _ptr(descale_f32), batch, M, N, block_m, block_n,
                                  _ptr(out), dtype_out, ld_out, out_batch_stride,
                                  _stream(stream))


def fp8bq_dequantize_batched(desc_table, n_tensors=None, stream=None) -> int:
    """``fp8bq_dequantize_batched`` of the C ABI.  Returns the status code."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_dequant_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_dequantize_batched(desc_table, n, _stream(stream))


def fp8bq_tensor_scale(desc_table, scale_out, n_tensors=None, stream=None) -> int:
    """``fp8bq_tensor_scale`` of the C ABI.  Returns the status code."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_scale_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_tensor_scale(desc_table, n, _ptr(scale_out), _stream(stream))


def fp8bq_fp4_quantize(x, dtype_in: int, M: int, K: int, ld: int, format: int, tensor_scale, codes,
                       scales, stream=None) -> int:
    """``fp8bq_fp4_quantize`` of the C ABI.  Returns the status code."""
    return lib().fp8bq_fp4_quantize(_ptr(x), dtype_in, M, K, ld, format, _ptr(tensor_scale),
                                    _ptr(codes), _ptr(scales), _stream(stream))


def fp8bq_fp4_quantize_batched(desc_table, n_tensors=None, stream=None) -> int:
    """``fp8bq_fp4_quantize_batched`` of the C ABI.  Returns the status code."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_fp4_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_fp4_quantize_batched(desc_table, n, _stream(stream))


def fp8bq_fp4_tensor_scale(desc_table, scale_out, n_tensors=None, stream=None) -> int:
    """``fp8bq_fp4_tensor_scale`` of the C ABI.  Returns the status code."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_scale_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_fp4_tensor_scale(desc_table, n, _ptr(scale_out), _stream(stream))


def fp8bq_fp4_dequantize(codes, scales, batch: int, M: int, K: int, format: int, tensor_scale,
                         tensor_scale_stride: int, out, dtype_out: int, ld_out: int,
                         out_batch_stride: int, stream=None) -> int:
    """``fp8bq_fp4_dequantize`` of the C ABI.  Returns the status code."""
    return lib().fp8bq_fp4_dequantize(_ptr(codes), _ptr(scales), batch, M, K, format,
                                      _ptr(tensor_scale), tensor_scale_stride, _ptr(out),
                                      dtype_out, ld_out, out_batch_stride, _stream(stream))


def fp8bq_fp4_matmul(desc: fp8bq_fp4_matmul_desc, stream=None) -> int:
    """``fp8bq_fp4_matmul`` of the C ABI.  Returns the status code."""
    return lib().fp8bq_fp4_matmul(ctypes.byref(desc), _stream(stream))


def fp8bq_fp4_gated_matmul(desc: fp8bq_fp4_matmul_desc, stream=None) -> int:
    """``fp8bq_fp4_gated_matmul`` of the C ABI.  Returns the status code."""
    return lib().fp8bq_fp4_gated_matmul(ctypes.byref(desc), _stream(stream))


def fp8bq_fp4_plan(desc: fp8bq_fp4_matmul_desc, gated: bool = False) -> tuple[int, int, int]:
    """``fp8bq_fp4_plan`` of the C ABI: (status, tokens, overlap)."""
    t, o = ctypes.c_int(-1), ctypes.c_int(-1)
    st = lib().fp8bq_fp4_plan(ctypes.byref(desc), int(gated), ctypes.byref(t), ctypes.byref(o))
    return st, t.value, o.value


def fp8bq_status_string(status: int) -> str:
    return lib().fp8bq_status_string(status).decode()


def fp8bq_sync_status(stream=None) -> int:
    return lib().fp8bq_sync_status(_stream(stream))


def fp8bq_version() -> int:
    return lib().fp8bq_version()


def fp8bq_set_path(path: int) -> int:
    return lib().fp8bq_set_path(path)


def fp8bq_get_path() -> int:
    return lib().fp8bq_get_path()


def fp8bq_set_pdl(enable: int) -> int:
    return lib().fp8bq_set_pdl(int(enable))


def fp8bq_get_pdl() -> int:
    return lib().fp8bq_get_pdl()


def fp8bq_set_pdl_min_us(us: float) -> int:
    return lib().fp8bq_set_pdl_min_us(us)


def fp8bq_get_pdl_min_us() -> float:
    return lib().fp8bq_get_pdl_min_us()


def fp8bq_path_for(desc: fp8bq_desc) -> int:
    return lib().fp8bq_path_for(ctypes.byref(desc))


def fp8bq_launch_count(desc_table, n_tensors=None) -> int:
    """``fp8bq_launch_count`` of the C ABI: kernel launches the grouped call
    would enqueue (-1 if it would fail)."""
    if not isinstance(desc_table, ctypes.Array):
        desc_table = (fp8bq_desc * len(desc_table))(*desc_table)
    n = len(desc_table) if n_tensors is None else n_tensors
    return lib().fp8bq_launch_count(desc_table, n)


def fp8bq_debug_set_wait_limit_ns(ns: int) -> int:
    return lib().fp8bq_debug_set_wait_limit_ns(ns)


def fp8bq_debug_set_inject(flags: int) -> int:
    return lib().fp8bq_debug_set_inject(flags)


def fp8bq_debug_set_fp4_tokens(tokens: int) -> int:
    return lib().fp8bq_debug_set_fp4_tokens(tokens)


def fp8bq_checked_build() -> int:
    return lib().fp8bq_checked_build()


def fp8bq_debug_take_bounds() -> tuple[int, int, int]:
    """``fp8bq_debug_take_bounds``: (status, count, first_address)."""
    c, f = ctypes.c_uint64(0), ctypes.c_uint64(0)
    st = lib().fp8bq_debug_take_bounds(ctypes.byref(c), ctypes.byref(f))
    return st, int(c.value), int(f.value)


def check(status: int, what: str = "") -> None:
    if status != FP8BQ_OK:
        raise Fp8bqError(status, what)


# ----------------------------------------------------------------- PyTorch conveniences


def _check_cuda(t, what: str) -> None:
    """The library reads and writes device memory of the current device: refuse
    anything else here, before a kernel could touch a host address."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{what} is on {t.device}, not on the current device cuda:{cur}")


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FP8BQ_BF16
    if t.dtype == torch.float32:
        return FP8BQ_F32
    raise TypeError(f"input must be bfloat16 or float32, got {t.dtype}")


def make_desc(x, y, s, block=DEFAULT_BLOCK) -> fp8bq_desc:
    """Descriptor for a CUDA tensor ``x`` of shape [M, N] or [E, M, N] (unit
    stride along N), its e4m3fn output ``y`` (contiguous, same shape) and its
    descale ``s`` (contiguous [(E,) ceil(M/bm), ceil(N/bn)])."""
    if x.dim() not in (2, 3):
        raise ValueError("expected a 2-D weight or a 3-D stack of expert weights")
    _check_cuda(x, "the input")
    _check_cuda(y, "the e4m3fn output")
    _check_cuda(s, "the descale output")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError("the last dimension of the input must have unit stride")
    d = fp8bq_desc()
    d.x, d.y_u8, d.descale_f32 = _ptr(x), _ptr(y), _ptr(s)
    d.M, d.N = int(x.shape[-2]), int(x.shape[-1])
    d.ld = int(x.stride(-2)) if x.shape[-2] > 1 else max(int(x.shape[-1]), 1)
    d.ld = max(d.ld, d.N)
    d.batch = int(x.shape[0]) if x.dim() == 3 else 1
    gm, gn = -(-d.M // block[0]), -(-d.N // block[1])
    d.x_batch_stride = int(x.stride(0)) if x.dim() == 3 else 0
    d.y_batch_stride = d.M * d.N if x.dim() == 3 else 0
    d.s_batch_stride = gm * gn if x.dim() == 3 else 0
    d.dtype_in = _dtype_code(x)
    d.block_m, d.block_n = int(block[0]), int(block[1])
    return d


def _on_stream(stream):
    """Context in which PyTorch allocates for ``stream``: outputs the library
    writes on a stream other than the current one are allocated on that
    stream, so the caching allocator cannot hand their memory to another
    stream's work while the kernel still writes it."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _outputs(x, block):
    import torch
    M, N = x.shape[-2], x.shape[-1]
    gm, gn = -(-M // block[0]), -(-N // block[1])
    y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty((*x.shape[:-2], gm, gn), dtype=torch.float32, device=x.device)
    return y, s


def scaled_fp8_blockwise(data_hp, weight_block_size=DEFAULT_BLOCK, stream=None):
    """Quantize one bf16/fp32 CUDA weight ([M, N], or [E, M, N] for a stack of
    experts) to e4m3fn with one fp32 descale per block.

    Returns ``(fp8_data, descale)``: ``fp8_data`` has the input's shape and
    dtype ``torch.float8_e4m3fn``; ``descale`` is [(E,) ceil(M/bm), ceil(N/bn)]
    fp32 (the "weight_scale_inv" of the rollout engine).
    """
    block = tuple(int(b) for b in weight_block_size)
    _check_cuda(data_hp, "data_hp")
    with _on_stream(stream):
        y, s = _outputs(data_hp, block)
    if data_hp.dim() == 2 and (data_hp.shape[-1] <= 1 or data_hp.stride(-1) == 1):
        M, N = data_hp.shape
        ld = max(data_hp.stride(0) if M > 1 else max(N, 1), N)
        st = lib().fp8bq_quantize(data_hp.data_ptr(), _dtype_code(data_hp), M, N, ld, block[0],
                                  block[1], y.data_ptr(), s.data_ptr(), _stream(stream))
    else:
        st = fp8bq_quantize_batched([make_desc(data_hp, y, s, block)], stream=stream)
    check(st, "scaled_fp8_blockwise")
    return y, s


def dequantize_fp8_blockwise(fp8_data, descale, weight_block_size=DEFAULT_BLOCK,
                             out_dtype=None, stream=None):
    """Reverse map of ``scaled_fp8_blockwise``: decode(fp8_data) * descale per
    block, as bf16 (default) or fp32, same shape as ``fp8_data``."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    _check_cuda(fp8_data, "fp8_data")
    _check_cuda(descale, "descale")
    if not fp8_data.is_contiguous() or not descale.is_contiguous():
        raise ValueError("fp8_data and descale must be contiguous")
    bm, bn = (int(b) for b in weight_block_size)
    M, N = fp8_data.shape[-2], fp8_data.shape[-1]
    batch = fp8_data.shape[0] if fp8_data.dim() == 3 else 1
    with _on_stream(stream):
        out = torch.empty(fp8_data.shape, dtype=out_dtype, device=fp8_data.device)
    check(fp8bq_dequantize(fp8_data, descale, batch, M, N, bm, bn, out,
                           FP8BQ_BF16 if out_dtype == torch.bfloat16 else FP8BQ_F32, N, M * N,
                           stream), "dequantize_fp8_blockwise")
    return out


def tensor_scales(tensors, stream=None):
    """Per-tensor FP8 scales max(max|x|, eps) / 448 of contiguous bf16/fp32
    CUDA tensors (e.g. this step's Q, K and V), in one grouped call; returns a
    float32 CUDA tensor of len(tensors) scales."""
    return _tensor_scales(fp8bq_tensor_scale, "tensor_scales", tensors, stream)


def _tensor_scales(call, what: str, tensors, stream):
    import torch
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    _check_cuda(tensors[0], "every tensor")
    with _on_stream(stream):
        out = torch.empty(len(tensors), dtype=torch.float32, device=tensors[0].device)
    descs = []
    for t in tensors:
        _check_cuda(t, "every tensor")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        d = fp8bq_scale_desc()
        d.x, d.numel, d.dtype_in, d.reserved = _ptr(t), t.numel(), _dtype_code(t), 0
        descs.append(d)
    check(call(descs, out, stream=stream), what)
    return out


# fp8bq_desc as a numpy record (the same 96-byte layout), so that a whole
# table is built from one list of tuples instead of field by field.
_DESC_RECORD = [("x", "<u8"), ("y_u8", "<u8"), ("descale_f32", "<u8"), ("M", "<i8"),
                ("N", "<i8"), ("ld", "<i8"), ("batch", "<i8"), ("x_batch_stride", "<i8"),
                ("y_batch_stride", "<i8"), ("s_batch_stride", "<i8"), ("dtype_in", "<i4"),
                ("block_m", "<i4"), ("block_n", "<i4"), ("reserved", "<i4")]


def _plan_weights(named, bm: int, bn: int, stream=None):
    """Descriptor table (a numpy record array) and output views of
    quant_weights: the fp8 weights are views of one allocation and the
    descales of another, each piece at a 256-byte aligned offset."""
    import numpy as np
    import torch
    cur = torch.cuda.current_device() if torch.cuda.is_available() else -1
    rows = []
    yo = so = 0
    for name, w in named:
        if not isinstance(w, torch.Tensor) or not w.is_cuda or w.device.index != cur:
            _check_cuda(w, name)  # raises with the reason
        shape = w.shape
        if len(shape) not in (2, 3):
            raise ValueError(f"{name}: expected a 2-D weight or a 3-D stack of expert weights")
        M, N = shape[-2], shape[-1]
        if N > 1 and w.stride(-1) != 1:
            raise ValueError(f"{name}: the last dimension of the input must have unit stride")
        dt = FP8BQ_BF16 if w.dtype == torch.bfloat16 else _dtype_code(w)
        gm, gn = -(-M // bm), -(-N // bn)
        stack = len(shape) == 3
        E = shape[0] if stack else 1
        rows.append((w, shape, yo, so, gm, gn, E, M, N, stack, dt))
        yo += (E * M * N + 255) & ~255
        so += (E * gm * gn + 63) & ~63
    dev = named[0][1].device
    with _on_stream(stream):
        ybuf = torch.empty(max(yo, 1), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        sbuf = torch.empty(max(so, 1), dtype=torch.float32, device=dev)
    yp, sp = ybuf.data_ptr(), sbuf.data_ptr()
    recs, outs = [], []
    for (name, _w), (w, shape, yoff, soff, gm, gn, E, M, N, stack, dt) in zip(named, rows):
        ld = max(w.stride(-2) if M > 1 else max(N, 1), N)
        recs.append((w.data_ptr(), yp + yoff, sp + 4 * soff, M, N, ld, E,
                     w.stride(0) if stack else 0, M * N if stack else 0,
                     gm * gn if stack else 0, dt, bm, bn, 0))
        if stack:
            y = ybuf.as_strided((E, M, N), (M * N, N, 1), yoff)
            s = sbuf.as_strided((E, gm, gn), (gm * gn, gn, 1), soff)
        else:
            y = ybuf.as_strided((M, N), (N, 1), yoff)
            s = sbuf.as_strided((gm, gn), (gn, 1), soff)
        outs.append((name, y))
        outs.append((name + "_scale_inv", s))
    return np.array(recs, dtype=_DESC_RECORD), outs


def quant_weights(weights: Iterable, weight_block_size=DEFAULT_BLOCK, stream=None):
    """Quantize every (name, tensor) pair in one grouped call and return the
    list the rollout engine loads: (name, fp8 weight) followed by
    (name + "_scale_inv", descale) for each input, in input order.

    The fp8 weights are views of one device allocation and the descales of
    another (each piece at a 256-byte aligned offset), so a whole model costs
    two allocations; the memory is returned when the last view is freed."""
    bm, bn = (int(b) for b in weight_block_size)
    named = list(weights)
    if not named:
        return []
    table, out = _plan_weights(named, bm, bn, stream)
    st = lib().fp8bq_quantize_batched(table.ctypes.data_as(ctypes.POINTER(fp8bq_desc)),
                                      len(named), _stream(stream))
    check(st, "quant_weights")
    return out


# ----------------------------------------------------------------- 4-bit conveniences
#
# A product of one token takes the GPU a few microseconds, so what these
# functions do on the host is most of such a call.  The ordinary call (contiguous
# CUDA tensors that fit each other, on the current stream) is made by the module
# `_calls` (csrc/fp8bq_calls.c), which returns None for any other; the code here
# then takes it, checks it and says what is wrong with it.  It takes every call
# where that module cannot be built.

_FP4_FORMATS = {"mxfp4": (FP8BQ_MXFP4, 32), "nvfp4": (FP8BQ_NVFP4, 16)}
# fp8bq_fp4_desc and fp8bq_fp4_matmul_desc as packed bytes
_FP4_DESC = struct.Struct("<4Q6q2i")
_FP4_MATMUL_DESC = struct.Struct("<" + 3 * "3Q3q" + "2Q6q2i")


_calls = None  # the call module; False where it can be neither built nor loaded


def _load_calls():
    """The call module, built if it is missing or older than its source; False,
    with a warning, where that fails (no C compiler, no headers of Python)."""
    global _calls
    L = lib()
    with _lock:
        if _calls is None:
            import subprocess
            try:
                _calls = _make_calls(L)
            except (ImportError, OSError, RuntimeError, subprocess.SubprocessError) as e:
                import warnings
                warnings.warn("the 4-bit conveniences' call module cannot be built; their calls go "
                              f"through Python, several microseconds slower: {e}", RuntimeWarning,
                              stacklevel=2)
                _calls = False
    return _calls


def _make_calls(L):
    import importlib.machinery
    import importlib.util

    import torch

    from . import build as _build
    spec = importlib.util.spec_from_file_location(__name__ + "._calls", _build.build_calls())
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.setup(torch.Tensor, torch.uint8, torch.bfloat16, torch.float32,
            *(ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.fp8bq_fp4_matmul, L.fp8bq_fp4_gated_matmul, L.fp8bq_fp4_quantize_batched,
                L.fp8bq_fp4_dequantize)))
    return m


def _fp4_quick(name: str, what: str, like, format: str, lead, args):
    """The call by the call module, or None where it is not an ordinary one."""
    f = _FP4_FORMATS.get(format) if type(format) is str else None
    if f is None or not getattr(like, "is_cuda", False):
        return None
    calls = _load_calls() if _calls is None else _calls
    if not calls:
        return None
    import torch
    dev = torch._C._cuda_getDevice()
    r = getattr(calls, name)(
        *lead, f[0], dev, torch._C._cuda_getCurrentRawStream(dev), *args)
    if type(r) is int:
        check(r, what)
    return r


def _fp4_format(format: str) -> tuple[int, int]:
    """(fp8bq_fp4_format, values a scale) of a format's name."""
    try:
        return _FP4_FORMATS[format]
    except (KeyError, TypeError):
        raise ValueError(f"format must be 'mxfp4' or 'nvfp4', got {format!r}") from None


def _fp4_setup(tensor, what: str):
    """(torch, current device, its current stream, the library) of a call on ``tensor``."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    if not isinstance(tensor, torch.Tensor) or tensor.get_device() != dev:
        _check_cuda(tensor, what)
        dev = tensor.get_device()
    return torch, dev, torch._C._cuda_getCurrentRawStream(dev), _lib or lib()


def _fp4_empty(shape, dtype, like, stream):
    """An output on ``like``'s device, allocated on ``stream`` (see _on_stream)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on_stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _fp4_tensor_scale(t, batch: int, format: str, what: str) -> tuple[int, int]:
    """(pointer, stride) of a tensor scale: None, one fp32 value, or one for
    each matrix of a stack."""
    if t is None:
        return 0, 0
    import torch
    _check_cuda(t, what)
    if format == "mxfp4":
        raise ValueError(f"{what}: mxfp4 has no tensor scale")
    if t.dtype != torch.float32:
        raise TypeError(f"{what} must be float32, got {t.dtype}")
    n = t.numel()
    if n == 1:
        return t.data_ptr(), 0
    if n != batch:
        raise ValueError(f"{what} must hold one value, or one for each of the {batch} matrices")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr(), 1


def _fp4_record(w, name: str, format: str, block: int, tensor_scale):
    """(shape of the codes, shape of the scale tiles, the other fields of an
    ``fp8bq_fp4_desc``) for the CUDA tensor ``w``."""
    shape = w.shape
    if len(shape) == 2:
        (M, K), E, xbs, lead = shape, 1, 0, ()
    elif len(shape) == 3:
        E, M, K = shape
        xbs, lead = w.stride(0), (E,)
    else:
        raise ValueError(f"{name}: expected a 2-D weight or a 3-D stack of expert weights")
    if K > 1 and w.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension of the input must have unit stride")
    ld = w.stride(-2) if M > 1 else K
    if ld < K:
        raise ValueError(f"{name}: the rows of the input overlap")
    t, ts = _fp4_tensor_scale(tensor_scale, E, format, f"{name}'s tensor scale")
    return ((*lead, M, 16 * (-(-K // 32))), (*lead, -(-M // 128), -(-K // (4 * block)), 32, 16),
            (t, M, K, ld, E, xbs, ts, _dtype_code(w),
             _FP4_FORMATS[format][0]))


def scaled_fp4_blockwise(data_hp, format="mxfp4", tensor_scale=None, stream=None):
    """Quantize one bf16/fp32 CUDA tensor ([M, K], or [E, M, K] for a stack) to
    4 bits: ``"mxfp4"`` (a power-of-two scale for each 32 values of a row) or
    ``"nvfp4"`` (an e4m3 scale for each 16, times ``tensor_scale``, an fp32 CUDA
    tensor of one value or of one for each matrix of the stack; None is 1).

    Returns ``(codes, scales)``, both uint8: codes [(E,) M, 16 * ceil(K / 32)],
    two e2m1 codes a byte; scales [(E,) ceil(M / 128), ceil(K / 4B), 32, 16], B
    the block length, in the tiles that the products read (``fp4_scale_rows``
    gives them row by row).  Both are padded with zeros.
    """
    if stream is None:
        r = _fp4_quick("quantize", "scaled_fp4_blockwise", data_hp, format, (),
                       (data_hp, tensor_scale))
        if r is not None:
            return r
    _, block = _fp4_format(format)
    torch, _, current, L = _fp4_setup(data_hp, "data_hp")
    cs, ss, rec = _fp4_record(data_hp, "data_hp", format, block, tensor_scale)
    codes = _fp4_empty(cs, torch.uint8, data_hp, stream)
    scales = _fp4_empty(ss, torch.uint8, data_hp, stream)
    st = L.fp8bq_fp4_quantize_batched(
        _FP4_DESC.pack(data_hp.data_ptr(), codes.data_ptr(), scales.data_ptr(), *rec), 1,
        current if stream is None else _stream(stream))
    if st:
        check(st, "scaled_fp4_blockwise")
    return codes, scales


def fp4_scale_rows(scales, rows: int, columns: int, format="mxfp4"):
    """The scale bytes of ``scaled_fp4_blockwise`` as [(E,) rows, ceil(columns / B)],
    the order of a checkpoint (a copy)."""
    _, block = _fp4_format(format)
    mt, kt = scales.shape[-4], scales.shape[-3]
    s = scales.reshape(*scales.shape[:-2], 32, 4, 4).movedim(-4, -2).movedim(-4, -3)
    return s.reshape(*s.shape[:-5], mt * 128, kt * 4)[..., :rows, :-(-columns // block)].contiguous()


def quant_weights_fp4(weights: Iterable, format="mxfp4", stream=None):
    """Quantize every (name, tensor) pair to 4 bits in one grouped call and
    return the list a rollout engine loads: (name, codes), (name + "_scale",
    scales) and, for ``"nvfp4"``, (name + "_scale_2", tensor scale) for each
    input, in input order.  The tensor scale is max(max|w|, eps) / 448 / 6 over
    the finite values, so that the largest finite block's scale is 448; a block
    with an infinity or a NaN, and no other, becomes NaN."""
    _, block = _fp4_format(format)
    named = list(weights)
    if not named:
        return []
    recs = []
    for name, w in named:
        _check_cuda(w, name)
        recs.append(_fp4_record(w, name, format, block, None))
    import torch
    ts = None
    with _on_stream(stream):
        if format == "nvfp4":
            ts = _tensor_scales(fp8bq_fp4_tensor_scale, "quant_weights_fp4",
                                [w if w.is_contiguous() else w.contiguous() for _, w in named],
                                stream)
        made = [(torch.empty(cs, dtype=torch.uint8, device=w.device),
                 torch.empty(ss, dtype=torch.uint8, device=w.device))
                for (cs, ss, _), (_, w) in zip(recs, named)]
    packed, out = [], []
    for i, ((name, w), (codes, scales), (_, _, rec)) in enumerate(zip(named, made, recs)):
        if ts is not None:
            rec = (ts.data_ptr() + 4 * i, *rec[1:])
        packed.append(_FP4_DESC.pack(w.data_ptr(), codes.data_ptr(), scales.data_ptr(), *rec))
        out += [(name, codes), (name + "_scale", scales)]
        if ts is not None:
            out.append((name + "_scale_2", ts[i:i + 1]))
    check(lib().fp8bq_fp4_quantize_batched(b"".join(packed), len(packed), _stream(stream)),
          "quant_weights_fp4")
    return out


def _fp4_operand(torch, dev, codes, scales, tensor_scale, format: str, block: int, what: str):
    """The fields of an ``fp8bq_fp4_operand``, then its batch (0 for a plain
    matrix), rows, bytes a row and dimensions."""
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and
            codes.get_device() == scales.get_device() == dev):
        _check_cuda(codes, what)
        _check_cuda(scales, f"{what}'s scales")
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TypeError(f"{what}: codes and scales must be uint8")
    shape, ss = codes.shape, scales.shape
    dim, E, Es = len(shape), 0, 0
    try:
        if dim == 2:
            (rows, kb), (mt, kt, r, c) = shape, ss
        else:
            (E, rows, kb), (Es, mt, kt, r, c) = shape, ss
    except ValueError:
        raise ValueError(f"{what}: expected codes [(E,) M, K / 2] and scales "
                         "[(E,) M tiles, K tiles, 32, 16]") from None
    if kb & 15 or E != Es or r != 32 or c != 16 or mt != (rows + 127) // 128 or \
            kt != (kb + 2 * block - 1) // (2 * block):
        raise ValueError(f"{what}: codes {tuple(shape)} do not go with {format} scales {tuple(ss)}")
    if codes.is_contiguous() and scales.is_contiguous():
        cbs, sbs = rows * kb, mt * kt * 512
    else:
        cs, st = codes.stride(), scales.stride()
        if (kb > 1 and cs[-1] != 1) or (rows > 1 and cs[-2] != kb):
            raise ValueError(f"{what}: the codes' rows must be contiguous")
        if st[-1] != 1 or st[-2] != 16 or (kt > 1 and st[-3] != 512) or \
                (mt > 1 and st[-4] != 512 * kt):
            raise ValueError(f"{what}: the scale tiles must be contiguous")
        cbs, sbs = cs[0], st[0]
    t, ts = (0, 0) if tensor_scale is None else \
        _fp4_tensor_scale(tensor_scale, E if dim == 3 else 1, format, f"{what}'s tensor scale")
    return codes.data_ptr(), scales.data_ptr(), t, cbs, sbs, ts, E, rows, kb, dim


def dequantize_fp4_blockwise(codes, scales, format="mxfp4", columns=None, tensor_scale=None,
                             out_dtype=None, stream=None):
    """Reverse map of ``scaled_fp4_blockwise``: the values as bf16 (default) or
    fp32, [(E,) M, columns] (default: every column the codes have room for)."""
    if stream is None:
        r = _fp4_quick("dequantize", "dequantize_fp4_blockwise", codes, format, (),
                       (codes, scales, tensor_scale, columns, out_dtype))
        if r is not None:
            return r
    fmt, block = _fp4_format(format)
    torch, dev, current, L = _fp4_setup(codes, "codes")
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    c, s, t, cbs, sbs, ts, E, M, kb, dim = _fp4_operand(torch, dev, codes, scales, tensor_scale,
                                                        format, block, "codes")
    K = 2 * kb if columns is None else int(columns)
    if K < 0 or -(-K // 32) * 16 != kb:
        raise ValueError(f"codes of {kb} bytes a row do not hold {K} columns")
    if E > 1 and (cbs != M * kb or sbs != scales[0].numel()):
        raise ValueError("a stack's codes and scales must be contiguous")
    out = _fp4_empty((M, K) if dim == 2 else (E, M, K), out_dtype, codes, stream)
    st = L.fp8bq_fp4_dequantize(c, s, E if dim == 3 else 1, M, K, fmt, t, ts, out.data_ptr(),
                                    FP8BQ_BF16 if out_dtype == torch.bfloat16 else FP8BQ_F32, K,
                                    M * K, current if stream is None else _stream(stream))
    if st:
        check(st, "dequantize_fp4_blockwise")
    return out


def _fp4_product(what, a, b, up, format, out_dtype, rows, out, stream):
    fmt, block = _fp4_format(format)
    torch, dev, current, L = _fp4_setup(a[0], "a")
    *fa, E, M, kb, dim = _fp4_operand(torch, dev, *a, format, block, "a")
    *fb, Eb, N, kb_b, dim_b = _fp4_operand(torch, dev, *b, format, block,
                                           "b" if up is None else "gate")
    if (Eb, kb_b, dim_b) != (E, kb, dim):
        raise ValueError(f"a weight {tuple(b[0].shape)} does not match a {tuple(a[0].shape)}")
    fu = (0, 0, 0, 0, 0, 0)
    if up is not None:
        *fu, Eu, Nu, ku, dim_u = _fp4_operand(torch, dev, *up, format, block, "up")
        if (Eu, Nu, ku, dim_u) != (Eb, N, kb, dim):
            raise ValueError(f"gate {tuple(b[0].shape)} and up {tuple(up[0].shape)} differ")
    shape = (E, M, N) if dim == 3 else (M, N)
    if rows is not None:
        _check_cuda(rows, "rows")
        if dim != 3 or rows.dtype != torch.int32 or rows.shape != (E,) or not rows.is_contiguous():
            raise ValueError("rows must be int32, contiguous, one value for each matrix of a stack")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16
        elif out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        out = _fp4_empty(shape, out_dtype, a[0], stream)
        if rows is not None:
            with _on_stream(stream):
                out.zero_()
        ld, obs = N, M * N
    else:
        _check_cuda(out, "out")
        if out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be {shape} {out_dtype or ''}, got {tuple(out.shape)} "
                             f"{out.dtype}")
        out_dtype = out.dtype
        st = out.stride()
        if N > 1 and st[-1] != 1:
            raise ValueError("the last dimension of out must have unit stride")
        ld, obs = (st[-2] if M > 1 else N), (st[0] if dim == 3 else 0)
        if ld < N:
            raise ValueError("the rows of out overlap")
    st = getattr(L, "fp8bq_fp4_" + what)(_FP4_MATMUL_DESC.pack(
        *fa, *fb, *fu, out.data_ptr(), 0 if rows is None else rows.data_ptr(), M, N, 2 * kb,
        E if dim == 3 else 1, ld, obs, fmt,
        FP8BQ_BF16 if out_dtype == torch.bfloat16 else _dtype_code(out)),
        current if stream is None else _stream(stream))
    if st:
        check(st, what + "_fp4")
    return out


def matmul_fp4(a, a_scales, b, b_scales, format="mxfp4", a_tensor_scale=None, b_tensor_scale=None,
               out_dtype=None, rows=None, out=None, stream=None):
    """The product a b^T of 4-bit matrices, as ``scaled_fp4_blockwise`` makes
    them: a [(E,) M, K] (tokens), b [(E,) N, K] (a weight), both of one format.
    Returns [(E,) M, N] in bf16 (default) or fp32, or ``out`` filled.

    ``rows`` (int32 CUDA tensor, one value for each matrix of a stack): only the
    first rows[e] rows of a[e] are used, and the rows of out[e] behind them are
    left as they were (zeros in an output made here).

    The codes carry no gradient: they are what an inference engine holds.
    """
    if stream is None and rows is None and out is None:
        r = _fp4_quick("product", "matmul_fp4", a, format, (0,),
                       (a, a_scales, a_tensor_scale, b, b_scales, b_tensor_scale, None, None, None,
                        out_dtype))
        if r is not None:
            return r
    return _fp4_product("matmul", (a, a_scales, a_tensor_scale), (b, b_scales, b_tensor_scale),
                        None, format, out_dtype, rows, out, stream)


def gated_matmul_fp4(a, a_scales, gate, gate_scales, up, up_scales, format="mxfp4",
                     a_tensor_scale=None, gate_tensor_scale=None, up_tensor_scale=None,
                     out_dtype=None, rows=None, out=None, stream=None):
    """silu(a gate^T) * (a up^T), the gated half of a feed-forward block, in one
    kernel; operands and arguments as in ``matmul_fp4``.  The halves of a fused
    [(E,) 2F, K] weight may be views of it where F is a multiple of 128
    (codes[..., :F, :], scales[..., :F // 128, :, :, :], and the rest).

    The activation is fp32: off by at most 5 units of 2^-23 for an fp32 output,
    and by 1.173 |v| more, far below its rounding, for a bf16 one."""
    if stream is None and rows is None and out is None:
        r = _fp4_quick("product", "gated_matmul_fp4", a, format, (1,),
                       (a, a_scales, a_tensor_scale, gate, gate_scales, gate_tensor_scale, up,
                        up_scales, up_tensor_scale, out_dtype))
        if r is not None:
            return r
    return _fp4_product("gated_matmul", (a, a_scales, a_tensor_scale),
                        (gate, gate_scales, gate_tensor_scale), (up, up_scales, up_tensor_scale),
                        format, out_dtype, rows, out, stream)
