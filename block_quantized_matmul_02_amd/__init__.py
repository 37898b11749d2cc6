"""Python binding of libbqmm, the gfx950 block-quantized projection matmul.

Argument marshalling only: every step runs in the HIP kernels of
``libbqmm.so`` (built in-tree by ``block_quantized_matmul_02_amd.build``).
The functions carry the C ABI's names (``include/bqmm.h`` and, for the
operators around the matmul, ``include/bqmm_layer.h``), take torch
tensors that live on the GPU, enqueue on torch's current stream and never
synchronize.  There is no CPU fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbqmm.so")

BQM_OK = 0
BQM_EINVAL = 1
BQM_EUNSUPPORTED = 2
BQM_EHIP_BASE = 10000
GEMV_MAX_M = 15
E4M3_GEMV_MAX_M = 16
MXFP4_GEMV_MAX_M = 16
LOGPROBS_MAX_TOP = 32
BQM_F32 = 0
BQM_F16 = 1
BQM_BF16 = 2

_lib = None
_raw_stream = None


class BqmError(RuntimeError):
    def __init__(self, fn: str, rc: int):
        self.rc = rc
        super().__init__(f"{fn} failed: rc={rc} ({strerror(rc)})")


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m block_quantized_matmul_02_amd.build` or __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        L.bqm_q8_1_quantize.argtypes = [P, P, P, I, I, P]
        L.bqm_q8_0_gemv.argtypes = [P, I64, P, P, P, I, I, I, P]
        L.bqm_q8_0_gemm.argtypes = [P, I64, P, P, P, I, I, I, P]
        L.bqm_q8_0_gemm_f8acc.argtypes = [P, I64, P, P, P, I, I, I, P]
        L.bqm_q8_0_gemv_f32.argtypes = [P, I64, P, P, I, I, I, P]
        L.bqm_e4m3_nan_count.argtypes = [P, I64, P, P]
        L.bqm_e4m3_blk_quantize.argtypes = [P, P, P, I, I, P]
        L.bqm_e4m3_blk_gemm.argtypes = [P, P, P, P, P, I, I, I, P]
        L.bqm_e4m3_quantize_amax.argtypes = [P, P, P, F, I, I, P]
        L.bqm_e4m3_gemm.argtypes = [P, P, P, P, I, I, I, P]
        L.bqm_e4m3_gemm_exact.argtypes = [P, P, P, P, I, I, I, P]
        L.bqm_e4m3_gemv.argtypes = [P, P, F, P, I, I, I, P]
        L.bqm_q8_0_dequant_f16.argtypes = [P, I64, P, I, I, P]
        L.bqm_f16_cvt.argtypes = [P, P, I64, P]
        L.bqm_f16_gemm.argtypes = [P, P, P, I, I, I, P]
        for fn in ("bqm_q8_1_quantize", "bqm_q8_0_gemv", "bqm_q8_0_gemm", "bqm_e4m3_quantize_amax",
                   "bqm_e4m3_gemm", "bqm_e4m3_gemv", "bqm_q8_0_dequant_f16", "bqm_f16_cvt", "bqm_f16_gemm",
                   "bqm_q8_0_gemm_f8acc", "bqm_e4m3_nan_count", "bqm_e4m3_blk_quantize", "bqm_e4m3_blk_gemm",
                   "bqm_q8_0_gemv_f32", "bqm_e4m3_gemm_exact"):
            getattr(L, fn).restype = ctypes.c_int
        L.bqm_add_rmsnorm.argtypes = [P, I64, P, I64, P, F, P, I64, P, I, I, I, I, P]
        L.bqm_add_rmsnorm_q8_1.argtypes = [P, I64, P, I64, P, F, P, I64, P, P, I, I, I, P]
        L.bqm_add_rmsnorm_e4m3_blk.argtypes = [P, I64, P, I64, P, F, P, I64, P, P, I, I, I, P]
        L.bqm_mxfp4_quantize.argtypes = [P, I64, P, P, I, I, I, P]
        L.bqm_mxfp4_dequantize.argtypes = [P, P, P, I, I, I, P]
        L.bqm_mxfp4_gemm.argtypes = [P, P, P, P, P, I, I, I, P]
        L.bqm_mxfp4_gemv.argtypes = [P, P, P, P, I, I, I, P]
        L.bqm_logprobs.argtypes = [P, I64, I, P, I, P, P, P, P, P, I, P, I, I, P]
        L.bqm_logprobs_workspace.argtypes = [I, I, I]
        L.bqm_logprobs_workspace.restype = I64
        for fn in ("bqm_add_rmsnorm", "bqm_add_rmsnorm_q8_1", "bqm_add_rmsnorm_e4m3_blk", "bqm_mxfp4_quantize",
                   "bqm_mxfp4_dequantize", "bqm_mxfp4_gemm", "bqm_mxfp4_gemv", "bqm_logprobs"):
            getattr(L, fn).restype = ctypes.c_int
        L.bqm_strerror.argtypes = [I]
        L.bqm_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(rc: int) -> str:
    return lib().bqm_strerror(int(rc)).decode()


def _stream(t):
    """The handle of torch's current stream on t's device, without building a Stream object where torch allows."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(t.device.index)


def _check(t, dtype, name, shape=None):
    if t.is_cuda and t.dtype == dtype and t.is_contiguous() and (shape is None or t.shape == shape):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t):
    return t.data_ptr()


def _raise(fn, rc):
    if rc != BQM_OK:
        raise BqmError(fn, rc)


def bqm_q8_1_quantize(x, xq=None, xds=None):
    """q8_1 quantization of f32 ``x [m, k]`` -> (int8 ``xq [m, k]``, f32 ``xds [m, k/32, 2]``)."""
    import torch

    m, k = x.shape
    _check(x, torch.float32, "x")
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=x.device)
    if xds is None:
        xds = torch.empty((m, k // 32, 2), dtype=torch.float32, device=x.device)
    _check(xq, torch.int8, "xq", (m, k))
    _check(xds, torch.float32, "xds", (m, k // 32, 2))
    _raise("bqm_q8_1_quantize", lib().bqm_q8_1_quantize(_ptr(x), _ptr(xq), _ptr(xds), m, k, _stream(x)))
    return xq, xds


def _q8_0_args(w, xq, xds, y, k, n):
    import torch

    m = xq.shape[0]
    _check(w, torch.uint8, "w")
    if w.dim() != 2 or w.shape[0] != n:
        raise ValueError(f"w must be [n={n}, row_bytes], got {tuple(w.shape)}")
    _check(xq, torch.int8, "xq", (m, k))
    _check(xds, torch.float32, "xds", (m, k // 32, 2))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=xq.device)
    _check(y, torch.float32, "y", (m, n))
    return m, y


def bqm_q8_0_gemv(w, xq, xds, y=None):
    """Q8_0 GEMV, 1 <= m <= 15: ``w [n, row_bytes]`` uint8 Q8_0 rows -> f32 ``y [m, n]``."""
    n = w.shape[0]
    k = xq.shape[1]
    m, y = _q8_0_args(w, xq, xds, y, k, n)
    rc = lib().bqm_q8_0_gemv(_ptr(w), w.shape[1], _ptr(xq), _ptr(xds), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_q8_0_gemv", rc)
    return y


def bqm_q8_0_gemm(w, xq, xds, y=None):
    """Q8_0 MMQ GEMM, any m: ``w [n, row_bytes]`` uint8 Q8_0 rows -> f32 ``y [m, n]``."""
    n = w.shape[0]
    k = xq.shape[1]
    m, y = _q8_0_args(w, xq, xds, y, k, n)
    rc = lib().bqm_q8_0_gemm(_ptr(w), w.shape[1], _ptr(xq), _ptr(xds), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_q8_0_gemm", rc)
    return y


def bqm_q8_0_gemv_f32(w, x, y=None):
    """Decode step in one launch: q8_1 quantization of f32 ``x [m, k]`` and the Q8_0 GEMV against
    ``w [n, row_bytes]`` -> f32 ``y [m, n]``, bitwise equal to bqm_q8_1_quantize + bqm_q8_0_gemv."""
    import torch

    n = w.shape[0]
    m, k = x.shape
    _check(w, torch.uint8, "w")
    _check(x, torch.float32, "x")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check(y, torch.float32, "y", (m, n))
    _raise("bqm_q8_0_gemv_f32", lib().bqm_q8_0_gemv_f32(_ptr(w), w.shape[1], _ptr(x), _ptr(y), m, k, n, _stream(w)))
    return y


def bqm_q8_0_gemm_f8acc(w, xq, xds, y=None):
    """The accumulator instrument's f32 arm: bqm_q8_0_gemm with the quant bytes read as e4m3
    and multiplied on the fp8 matrix cores (f32 accumulate); same arguments."""
    n = w.shape[0]
    k = xq.shape[1]
    m, y = _q8_0_args(w, xq, xds, y, k, n)
    rc = lib().bqm_q8_0_gemm_f8acc(_ptr(w), w.shape[1], _ptr(xq), _ptr(xds), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_q8_0_gemm_f8acc", rc)
    return y


def bqm_e4m3_quantize_amax(x, w_scale: float, xq=None, scales=None):
    """Per-batch e4m3 quantization of f32 ``x [m, k]`` -> (uint8 codes ``[m, k]``, f32 ``scales[4]``)."""
    import torch

    m, k = x.shape
    _check(x, torch.float32, "x")
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(4, dtype=torch.float32, device=x.device)
    _check(xq, torch.uint8, "xq", (m, k))
    _check(scales, torch.float32, "scales", (4,))
    rc = lib().bqm_e4m3_quantize_amax(_ptr(x), _ptr(xq), _ptr(scales), ctypes.c_float(w_scale), m, k, _stream(x))
    _raise("bqm_e4m3_quantize_amax", rc)
    return xq, scales


def bqm_e4m3_gemm(w, xq, scales, y=None):
    """e4m3 GEMM: codes ``w [n, k]`` and ``xq [m, k]`` -> f32 ``y [m, n]`` scaled by ``scales[2]``."""
    import torch

    n, k = w.shape
    m = xq.shape[0]
    _check(w, torch.uint8, "w")
    _check(xq, torch.uint8, "xq", (m, k))
    _check(scales, torch.float32, "scales", (4,))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=xq.device)
    _check(y, torch.float32, "y", (m, n))
    rc = lib().bqm_e4m3_gemm(_ptr(w), _ptr(xq), _ptr(scales), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_e4m3_gemm", rc)
    return y


def bqm_e4m3_gemm_exact(w, xq, scales, y=None):
    """e4m3 GEMM with the bound (27 + k/128) * 2^-24 * sum|terms| on every output: same arguments and
    result as :func:`bqm_e4m3_gemm`."""
    import torch

    n, k = w.shape
    m = xq.shape[0]
    _check(w, torch.uint8, "w")
    _check(xq, torch.uint8, "xq", (m, k))
    _check(scales, torch.float32, "scales", (4,))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=xq.device)
    _check(y, torch.float32, "y", (m, n))
    rc = lib().bqm_e4m3_gemm_exact(_ptr(w), _ptr(xq), _ptr(scales), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_e4m3_gemm_exact", rc)
    return y


def bqm_e4m3_gemv(w, x, w_scale: float, y=None):
    """e4m3 decode GEMV, 1 <= m <= 16: codes ``w [n, k]`` against f32 ``x [m, k]`` -> f32 ``y [m, n]``
    = w_scale * x @ dec(w)^T."""
    import torch

    n, k = w.shape
    m = x.shape[0]
    _check(w, torch.uint8, "w")
    _check(x, torch.float32, "x", (m, k))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check(y, torch.float32, "y", (m, n))
    rc = lib().bqm_e4m3_gemv(_ptr(w), _ptr(x), ctypes.c_float(w_scale), _ptr(y), m, k, n, _stream(w))
    _raise("bqm_e4m3_gemv", rc)
    return y


def bqm_q8_0_dequant_f16(w, k: int, w16=None):
    """fp16 mirror of Q8_0 rows ``w [n, row_bytes]`` -> ``w16 [n, k]`` (torch.float16) = fp16(d * q)."""
    import torch

    n = w.shape[0]
    _check(w, torch.uint8, "w")
    if w16 is None:
        w16 = torch.empty((n, k), dtype=torch.float16, device=w.device)
    _check(w16, torch.float16, "w16", (n, k))
    _raise("bqm_q8_0_dequant_f16", lib().bqm_q8_0_dequant_f16(_ptr(w), w.shape[1], _ptr(w16), k, n, _stream(w)))
    return w16


def bqm_f16_cvt(x, x16=None):
    """f32 -> fp16 cast (round to nearest even) of a contiguous tensor, same shape."""
    import torch

    _check(x, torch.float32, "x")
    if x16 is None:
        x16 = torch.empty(x.shape, dtype=torch.float16, device=x.device)
    _check(x16, torch.float16, "x16", tuple(x.shape))
    _raise("bqm_f16_cvt", lib().bqm_f16_cvt(_ptr(x), _ptr(x16), x.numel(), _stream(x)))
    return x16


def bqm_f16_gemm(w16, x16, y=None):
    """fp16 GEMM: ``w16 [n, k]`` and ``x16 [m, k]`` (torch.float16) -> f32 ``y [m, n]`` = x16 @ w16^T."""
    import torch

    n, k = w16.shape
    m = x16.shape[0]
    _check(w16, torch.float16, "w16")
    _check(x16, torch.float16, "x16", (m, k))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x16.device)
    _check(y, torch.float32, "y", (m, n))
    _raise("bqm_f16_gemm", lib().bqm_f16_gemm(_ptr(w16), _ptr(x16), _ptr(y), m, k, n, _stream(w16)))
    return y


def bqm_e4m3_nan_count(w, out=None):
    """Number of e4m3 NaN codes (magnitude 0x7F) in a uint8 tensor, as a device int64 tensor of one element."""
    import torch

    _check(w, torch.uint8, "w")
    if out is None:
        out = torch.empty(1, dtype=torch.int64, device=w.device)
    _check(out, torch.int64, "out", (1,))
    _raise("bqm_e4m3_nan_count", lib().bqm_e4m3_nan_count(_ptr(w), w.numel(), _ptr(out), _stream(w)))
    return out


def bqm_e4m3_blk_quantize(x, xq=None, xs=None):
    """Per (token, 128-k block) e4m3 quantization of f32 ``x [m, k]`` -> (uint8 ``xq [m, k]``,
    f32 ``xs [m, ceil(k/128)]``); k % 16 == 0, the last block short when k % 128 != 0."""
    import torch

    m, k = x.shape
    _check(x, torch.float32, "x")
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if xs is None:
        xs = torch.empty((m, (k + 127) // 128), dtype=torch.float32, device=x.device)
    _check(xq, torch.uint8, "xq", (m, k))
    _check(xs, torch.float32, "xs", (m, (k + 127) // 128))
    _raise("bqm_e4m3_blk_quantize", lib().bqm_e4m3_blk_quantize(_ptr(x), _ptr(xq), _ptr(xs), m, k, _stream(x)))
    return xq, xs


def bqm_e4m3_blk_gemm(w, grid, xq, xs, y=None):
    """Block-128 FP8 GEMM: e4m3 ``w [n, k]`` with f32 ``grid [ceil(n/128), ceil(k/128)]``, ``xq``/``xs`` from
    bqm_e4m3_blk_quantize -> f32 ``y [m, n]``."""
    import torch

    n, k = w.shape
    m = xq.shape[0]
    _check(w, torch.uint8, "w")
    _check(grid, torch.float32, "grid", ((n + 127) // 128, (k + 127) // 128))
    _check(xq, torch.uint8, "xq", (m, k))
    _check(xs, torch.float32, "xs", (m, (k + 127) // 128))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=w.device)
    _check(y, torch.float32, "y", (m, n))
    _raise("bqm_e4m3_blk_gemm", lib().bqm_e4m3_blk_gemm(_ptr(w), _ptr(grid), _ptr(xq), _ptr(xs), _ptr(y), m, k, n,
                                                        _stream(w)))
    return y


# ------------------------------------------- the operators around the matmul


_types = {}


def _type(t, name):
    if not _types:
        import torch

        _types.update({torch.float32: BQM_F32, torch.float16: BQM_F16, torch.bfloat16: BQM_BF16})
    code = _types.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _rows(t, name, dtype=None, shape=None):
    """Checks a 2-D GPU tensor whose rows are contiguous; returns its row stride."""
    if t.is_cuda and (dtype is None or t.dtype == dtype) and (t.shape == shape if shape is not None else t.dim() == 2):
        row, column = t.stride()
        if column == 1:
            return row
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape {shape or '[rows, columns]'}, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0)


def _optr(t):
    return None if t is None else t.data_ptr()


def _norm_args(x, res, gain, h):
    """The arguments that the three norms share: x .. gain, and h with its stride."""
    import torch

    ldx = _rows(x, "x")
    _type(x, "x")
    if gain is not None:
        _check(gain, torch.float32, "gain", (x.shape[1],))
    if res is None:
        if h is not None:
            raise ValueError("h is the sum x + res: it goes with res")
        return (_ptr(x), ldx, None, 0, _optr(gain)), (None, 0), None
    ldr = _rows(res, "res", x.dtype, x.shape)
    if h is None:
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    ldh = _rows(h, "h", x.dtype, x.shape)
    return (_ptr(x), ldx, _ptr(res), ldr, _optr(gain)), (_ptr(h), ldh), h


def bqm_add_rmsnorm(x, res=None, gain=None, eps: float = 1e-6, h=None, y=None, out_dtype=None):
    """RMS norm of ``x [m, k]`` or of ``x + res`` -> (``y [m, k]``, ``h = x + res`` or None).

    x, res and h are f32, fp16 or bf16 alike, with any row stride; ``gain`` is f32 ``[k]`` or None for ones.
    y is f32 or x's type (``out_dtype``, f32 if not given); h may be x or res itself.
    """
    import torch

    m, k = x.shape
    head, tail, h = _norm_args(x, res, gain, h)
    if y is None:
        y = torch.empty((m, k), dtype=out_dtype or torch.float32, device=x.device)
    _check(y, out_dtype or y.dtype, "y", (m, k))
    _raise("bqm_add_rmsnorm", lib().bqm_add_rmsnorm(*head, eps, *tail, _ptr(y), _type(x, "x"), _type(y, "y"), m, k,
                                                    _stream(x)))
    return y, h


def bqm_add_rmsnorm_q8_1(x, res=None, gain=None, eps: float = 1e-6, h=None, xq=None, xds=None):
    """RMS norm as :func:`bqm_add_rmsnorm`, written as the q8_1 operand of bqm_q8_0_gemv / bqm_q8_0_gemm:
    (int8 ``xq [m, k]``, f32 ``xds [m, k/32, 2]``, ``h`` or None)."""
    import torch

    m, k = x.shape
    head, tail, h = _norm_args(x, res, gain, h)
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=x.device)
    if xds is None:
        xds = torch.empty((m, k // 32, 2), dtype=torch.float32, device=x.device)
    _check(xq, torch.int8, "xq", (m, k))
    _check(xds, torch.float32, "xds", (m, k // 32, 2))
    _raise("bqm_add_rmsnorm_q8_1", lib().bqm_add_rmsnorm_q8_1(*head, eps, *tail, _ptr(xq), _ptr(xds), _type(x, "x"),
                                                              m, k, _stream(x)))
    return xq, xds, h


def bqm_add_rmsnorm_e4m3_blk(x, res=None, gain=None, eps: float = 1e-6, h=None, xq=None, xs=None):
    """RMS norm as :func:`bqm_add_rmsnorm`, written as the operand of bqm_e4m3_blk_gemm:
    (e4m3 codes ``xq [m, k]``, f32 ``xs [m, ceil(k/128)]``, ``h`` or None)."""
    import torch

    m, k = x.shape
    head, tail, h = _norm_args(x, res, gain, h)
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if xs is None:
        xs = torch.empty((m, (k + 127) // 128), dtype=torch.float32, device=x.device)
    _check(xq, torch.uint8, "xq", (m, k))
    _check(xs, torch.float32, "xs", (m, (k + 127) // 128))
    _raise("bqm_add_rmsnorm_e4m3_blk",
           lib().bqm_add_rmsnorm_e4m3_blk(*head, eps, *tail, _ptr(xq), _ptr(xs), _type(x, "x"), m, k, _stream(x)))
    return xq, xs, h


def bqm_mxfp4_quantize(x, codes=None, scales=None):
    """MXFP4 quantization of ``x [m, k]`` (f32, fp16 or bf16, any row stride) -> (uint8 ``codes [m, k/2]``,
    E8M0 ``scales [m, k/32]``)."""
    import torch

    m, k = x.shape
    ldx = _rows(x, "x")
    if codes is None:
        codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((m, k // 32), dtype=torch.uint8, device=x.device)
    _check(codes, torch.uint8, "codes", (m, k // 2))
    _check(scales, torch.uint8, "scales", (m, k // 32))
    _raise("bqm_mxfp4_quantize", lib().bqm_mxfp4_quantize(_ptr(x), ldx, _ptr(codes), _ptr(scales), _type(x, "x"), m, k,
                                                          _stream(x)))
    return codes, scales


def bqm_mxfp4_dequantize(codes, scales, dtype=None, y=None):
    """The values of MXFP4 ``codes [m, k/2]`` and ``scales [m, k/32]`` -> ``y [m, k]`` (f32 if no ``dtype``)."""
    import torch

    _check(codes, torch.uint8, "codes")
    m, k = codes.shape[0], codes.shape[1] * 2
    _check(scales, torch.uint8, "scales", (m, k // 32))
    if y is None:
        y = torch.empty((m, k), dtype=dtype or torch.float32, device=codes.device)
    _check(y, dtype or y.dtype, "y", (m, k))
    _raise("bqm_mxfp4_dequantize", lib().bqm_mxfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(y), _type(y, "y"), m, k,
                                                              _stream(codes)))
    return y


def bqm_mxfp4_gemm(w, ws, xq, xs, y=None):
    """MXFP4 x MXFP4 GEMM, any m: weights ``w [n, k/2]``, ``ws [n, k/32]`` and activations ``xq [m, k/2]``,
    ``xs [m, k/32]`` -> f32 ``y [m, n]``."""
    import torch

    n, half = w.shape
    m, k = xq.shape[0], 2 * half
    _check(w, torch.uint8, "w")
    _check(ws, torch.uint8, "ws", (n, k // 32))
    _check(xq, torch.uint8, "xq", (m, half))
    _check(xs, torch.uint8, "xs", (m, k // 32))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=xq.device)
    _check(y, torch.float32, "y", (m, n))
    _raise("bqm_mxfp4_gemm", lib().bqm_mxfp4_gemm(_ptr(w), _ptr(ws), _ptr(xq), _ptr(xs), _ptr(y), m, k, n, _stream(w)))
    return y


def bqm_mxfp4_gemv(w, ws, x, y=None):
    """MXFP4 decode GEMV, 1 <= m <= 16: weights ``w [n, k/2]``, ``ws [n, k/32]`` against f32 ``x [m, k]``
    -> f32 ``y [m, n]``."""
    import torch

    n, half = w.shape
    m, k = x.shape[0], 2 * half
    _check(w, torch.uint8, "w")
    _check(ws, torch.uint8, "ws", (n, k // 32))
    _check(x, torch.float32, "x", (m, k))
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check(y, torch.float32, "y", (m, n))
    _raise("bqm_mxfp4_gemv", lib().bqm_mxfp4_gemv(_ptr(w), _ptr(ws), _ptr(x), _ptr(y), m, k, n, _stream(w)))
    return y


@functools.lru_cache(maxsize=256)
def bqm_logprobs_workspace(m: int, n: int, top_k: int) -> int:
    """Bytes of workspace that :func:`bqm_logprobs` needs for ``m`` rows of ``n`` logits."""
    size = lib().bqm_logprobs_workspace(m, n, top_k)
    if size < 0:
        valid = m >= 1 and n >= 1 and 0 <= top_k <= min(n, LOGPROBS_MAX_TOP)
        raise BqmError("bqm_logprobs_workspace", BQM_EUNSUPPORTED if valid else BQM_EINVAL)
    return size


def bqm_logprobs(logits, tokens=None, top_k: int = 0, out=None, workspace=None):
    """Log probabilities of int32 ``tokens [m, t]`` under ``logits [m, n]`` (f32, fp16 or bf16, any row stride),
    with each row's log-sum-exp, entropy and ``top_k`` alternatives.

    -> (``logp [m, t]``, ``lse [m]``, ``entropy [m]``, int32 ``top_ids [m, top_k]``, ``top_logp [m, top_k]``);
    ``out`` is such a tuple to write into, ``workspace`` uint8 of at least :func:`bqm_logprobs_workspace` bytes.
    """
    import torch

    m, n = logits.shape
    ld = _rows(logits, "logits")
    t = 0
    if tokens is not None:
        if tokens.dim() != 2:
            raise ValueError(f"tokens must be [m, t], got {tuple(tokens.shape)}")
        t = tokens.shape[1]
        _check(tokens, torch.int32, "tokens", (m, t))
    if out is None:
        f = dict(dtype=torch.float32, device=logits.device)
        out = (torch.empty((m, t), **f), torch.empty(m, **f), torch.empty(m, **f),
               torch.empty((m, max(top_k, 0)), dtype=torch.int32, device=logits.device),
               torch.empty((m, max(top_k, 0)), **f))
    logp, lse, entropy, ids, top = out
    _check(logp, torch.float32, "logp", (m, t))
    _check(lse, torch.float32, "lse", (m,))
    _check(entropy, torch.float32, "entropy", (m,))
    _check(ids, torch.int32, "top_ids", (m, max(top_k, 0)))
    _check(top, torch.float32, "top_logp", (m, max(top_k, 0)))
    need = bqm_logprobs_workspace(m, n, top_k)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
    if workspace is not None:
        _check(workspace, torch.uint8, "workspace")
        if workspace.numel() < need:
            raise ValueError(f"workspace must hold {need} bytes, got {workspace.numel()}")
    _raise("bqm_logprobs", lib().bqm_logprobs(_ptr(logits), ld, _type(logits, "logits"), _optr(tokens), t, _ptr(logp),
                                              _ptr(lse), _ptr(entropy), _ptr(ids), _ptr(top), top_k,
                                              _optr(workspace), m, n, _stream(logits)))
    return logp, lse, entropy, ids, top
