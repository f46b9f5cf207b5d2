"""fp8_scaled_quantization_reduce_amd -- FP8 scaled quantization and scaled FP8
GEMM for MI355X (gfx950).

This module is a thin ctypes binding over ``libfp8q.so``: the functions carry
the names of the C entry points in ``include/fp8q.h`` and only marshal torch
tensors (device memory) and the current HIP stream into them.  Every step of
the computation runs in the library's HIP kernels; there is no Python or CPU
fallback.  Importing the package fails if the library has not been built
(``python fp8_scaled_quantization_reduce_amd/build.py``).

Tensor conventions: high-precision inputs are ``torch.float32`` or
``torch.bfloat16``; FP8 codes are ``torch.uint8``; scalars (amax, scales) are
one-element ``torch.float32`` tensors on the device.  ``fmt`` is E4M3FN (0) or
E5M2 (1).
"""
from __future__ import annotations

import array
import ctypes
import os

import torch

E4M3FN, E5M2 = 0, 1
F32, BF16 = 0, 1
ALGO_MAX, ALGO_MOST_RECENT = 0, 1
PER_TENSOR, BLOCK_1x128_128x128, BLOCK_1x128_1x128, MXFP8 = 0, 1, 2, 3
OUT_E4M3FN, OUT_E5M2 = 2, 3
ACT_NONE, ACT_RELU, ACT_GELU = 0, 1, 2
COLSRC_ORIGINAL, COLSRC_ROWWISE_DEQUANTIZED = 0, 1
SUBQ_BLOCK_128x128, SUBQ_BLOCK_1x128, SUBQ_MXFP8, SUBQ_PER_TENSOR = 0, 1, 2, 3
OK, EINVAL, EUNSUPPORTED, EHIP = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")

# every entry point of include/fp8q.h, with its ctypes argument list
_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
SIGNATURES = {
    "fp8_amax": [_VP, _I32, _I64, _VP, _VP],
    "fp8_quantize_tensor": [_VP, _I32, _I64, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP],
    "fp8_quantize_tensor_stats": [_VP, _I32, _I64, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "fp8_dequantize": [_VP, _I32, _I64, _VP, _VP, _VP],
    "fp8_quantize_rowwise_colwise": [_VP, _I32, _I64, _I64, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "fp8_quantize_block": [_VP, _I32, _I64, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _VP],
    "fp8_quantize_mx": [_VP, _I32, _I64, _I64, _I32, _VP, _VP, _VP, _VP, _VP],
    "fp8_update_scale_delayed": [_VP, _I32, _I32, _I32, _VP, _I64, _I32, _I32, _I32, _VP, _VP, _VP],
    "fp8_quantize_delayed": [_VP, _I32, _I64, _I32, _VP, _I32, _I32, _I32, _I64, _I32, _I32, _I32, _VP, _VP, _VP, _VP,
                             _VP, _VP],
    "fp8_scaled_gemm": [_VP, _I32, _VP, _VP, _I32, _VP, _I64, _I64, _I64, _I32, _VP, _I32, _VP, _VP],
    "fp8_scaled_gemm_fused": [_VP, _I32, _VP, _VP, _I32, _VP, _I64, _I64, _I64, _I32, _VP, _I32, _VP, _I32, _VP, _VP,
                              _VP],
    "fp8_quantize_hybrid": [_VP, _I32, _I64, _I64, _I32, _I32, _I32, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                            _VP, _VP],
    "fp8_quantize_hybrid_blockwise": [_VP, _I32, _I64, _I64, _I32, _I32, _VP, _VP, _I32, _I32, _I32, _VP, _VP,
                                      _VP, _I32, _VP, _VP],
    "fp8_cast_stats": [_VP, _I32, _I64, _I32, _VP, _VP, _VP],
    "fp8_quantize_error_feedback": [_VP, _I32, _VP, _I64, _I32, _VP, _VP, _VP, _VP],
    "fp8_quantize_grouped": [_VP, _I32, _I64, _I64, _VP, _I64, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _I64, _VP],
    "fp8_grouped_gemm": [_VP, _I32, _VP, _VP, _I32, _VP, _VP, _I32, _I64, _I64, _I64, _VP, _VP],
    "fp8_grouped_gemm_wgrad": [_VP, _I32, _VP, _VP, _I32, _VP, _VP, _I32, _I64, _I64, _I64, _I64, _VP, _I32, _VP],
    "fp8q_layernorm": [_VP, _I32, _I64, _I64, _VP, _VP, _I32, ctypes.c_float, _VP, _VP, _VP, _VP],
    "fp8q_layernorm_backward": [_VP, _VP, _I32, _I64, _I64, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP],
    "fp8q_layernorm_backward_workspace": [_I32, _I64, _I64, _VP],
    "fp8q_grad_norm_clip": [_VP, _VP, _VP, _VP, _I32, ctypes.c_float, _VP, _VP, _VP],
    "fp8q_clock_monitor": [_VP, _VP, _VP],
    "fp8q_set_finish_poll_rounds": [ctypes.c_uint32, _VP],
    "fp8q_last_error": [],
}


class Fp8qError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("status %d: %s" % (status, message))
        self.status = status


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libfp8q.so is not built (%s); build it with "
                          "`python fp8_scaled_quantization_reduce_amd/build.py`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, argtypes in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_char_p if name == "fp8q_last_error" else ctypes.c_int
    return lib


lib = _load_library()


def last_error() -> str:
    return lib.fp8q_last_error().decode()


def _check(status: int) -> None:
    if status != OK:
        raise Fp8qError(status, last_error())


# ------------------------------------------------------- argument checks --
# The C ABI sees only pointers, so it cannot tell a buffer's size, type or
# device; the binding checks them before any call, so that a short output or
# a host tensor raises here instead of reaching a kernel.  Sizes and types are
# checked first and the device last.

def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _need(t, name, dtypes, numel=None, at_least=False):
    """t (or None) has one of `dtypes` and exactly `numel` elements (with
    at_least, `numel` or more: an input the kernels read a prefix of)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        _tensor(t, name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if numel is None:
        return
    if at_least and t.numel() < numel:
        raise ValueError("%s must have at least %d elements, got %d" % (name, numel, t.numel()))
    if not at_least and t.numel() != numel:
        raise ValueError("%s must have %d elements, got %d" % (name, numel, t.numel()))


def _need_scalar(t, name):
    _need(t, name, (torch.float32,), 1)


# The current device and stream without torch.cuda's Python layers (2.8 us a
# call for the stream, against 0.1 us: as long as a small kernel runs).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ptr(t, name="tensor"):
    """Device address of a contiguous tensor on the current GPU (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        _tensor(t, name)
    dev = t.get_device()  # -1 for host tensors
    if dev < 0:
        raise ValueError("%s must be a GPU tensor (device %s)" % (name, t.device))
    if dev != _current_device():
        raise ValueError("%s is on cuda:%d but the current device is cuda:%d" % (name, dev,
                                                                               torch.cuda.current_device()))
    return t.data_ptr()


_HP = (torch.float32, torch.bfloat16)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_STATS = (torch.int64, torch.uint64)
_I32T = (torch.int32,)
_BF16T = (torch.bfloat16,)


_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype(t) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("high-precision tensors must be float32 or bfloat16, got %s" % t.dtype)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _shape2(x, name="x"):
    _need(x, name, _HP)
    if x.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(x.shape)))
    return x.shape


def fp8_amax(x, amax, stream=None):
    """amax[0] = max |x|."""
    _need(x, "x", _HP)
    _need_scalar(amax, "amax")
    _check(lib.fp8_amax(_ptr(x, "x"), _dtype(x), x.numel(), _ptr(amax, "amax"), _stream(stream)))


def _scalars(**kw):
    for name, t in kw.items():
        if t is not None:
            _need_scalar(t, name)


def fp8_quantize_tensor(x, fmt, q, *, amax_in=None, margin=0, scale_inv_in=None, scale_inv_out=None,
                        scale_out=None, amax_out=None, stream=None):
    """Per-tensor scaled cast; exactly one of amax_in / scale_inv_in."""
    _need(x, "x", _HP)
    _need(q, "q", _U8, x.numel())
    _scalars(amax_in=amax_in, scale_inv_in=scale_inv_in, scale_inv_out=scale_inv_out, scale_out=scale_out,
             amax_out=amax_out)
    _check(lib.fp8_quantize_tensor(_ptr(x, "x"), _dtype(x), x.numel(), fmt, _ptr(amax_in, "amax_in"), margin,
                                   _ptr(scale_inv_in, "scale_inv_in"), _ptr(q, "q"),
                                   _ptr(scale_inv_out, "scale_inv_out"), _ptr(scale_out, "scale_out"),
                                   _ptr(amax_out, "amax_out"), _stream(stream)))


def fp8_quantize_tensor_stats(x, fmt, q, stats, *, amax_in=None, margin=0, scale_inv_in=None, scale_inv_out=None,
                              scale_out=None, amax_out=None, stream=None):
    """fp8_quantize_tensor that also writes the cast's counts to stats (int64
    [4] on the device: overflows, underflows, NaNs, nonzeros) in the same pass."""
    _need(x, "x", _HP)
    _need(q, "q", _U8, x.numel())
    _need(stats, "stats", _STATS, 4)
    _scalars(amax_in=amax_in, scale_inv_in=scale_inv_in, scale_inv_out=scale_inv_out, scale_out=scale_out,
             amax_out=amax_out)
    _check(lib.fp8_quantize_tensor_stats(_ptr(x, "x"), _dtype(x), x.numel(), fmt, _ptr(amax_in, "amax_in"), margin,
                                         _ptr(scale_inv_in, "scale_inv_in"), _ptr(q, "q"),
                                         _ptr(scale_inv_out, "scale_inv_out"), _ptr(scale_out, "scale_out"),
                                         _ptr(amax_out, "amax_out"), _ptr(stats, "stats"), _stream(stream)))


def fp8_dequantize(q, fmt, scale_inv, y, stream=None):
    """y = value(q) * scale_inv[0]."""
    _need(q, "q", _U8)
    _need_scalar(scale_inv, "scale_inv")
    _need(y, "y", _F32, q.numel())
    _check(lib.fp8_dequantize(_ptr(q, "q"), fmt, q.numel(), _ptr(scale_inv, "scale_inv"), _ptr(y, "y"),
                              _stream(stream)))


def fp8_quantize_rowwise_colwise(x, fmt, *, q_row=None, q_col=None, amax_in=None, margin=0, scale_inv_in=None,
                                 scale_inv_out=None, scale_out=None, amax_out=None, stream=None):
    """Per-tensor cast of a 2-D tensor to row-major codes and transposed codes."""
    rows, cols = _shape2(x)
    _need(q_row, "q_row", _U8, rows * cols)
    _need(q_col, "q_col", _U8, rows * cols)
    _scalars(amax_in=amax_in, scale_inv_in=scale_inv_in, scale_inv_out=scale_inv_out, scale_out=scale_out,
             amax_out=amax_out)
    _check(lib.fp8_quantize_rowwise_colwise(_ptr(x, "x"), _dtype(x), rows, cols, fmt, _ptr(amax_in, "amax_in"),
                                            margin, _ptr(scale_inv_in, "scale_inv_in"), _ptr(q_row, "q_row"),
                                            _ptr(q_col, "q_col"), _ptr(scale_inv_out, "scale_inv_out"),
                                            _ptr(scale_out, "scale_out"), _ptr(amax_out, "amax_out"),
                                            _stream(stream)))


def fp8_quantize_block(x, fmt, block_rows, q_row, s_row, q_col=None, s_col=None, stream=None):
    """Block current scaling (1x128 or 128x128) with optional columnwise copy."""
    rows, cols = _shape2(x)
    if block_rows in (1, 128):
        _need(q_row, "q_row", _U8, rows * cols)
        _need(s_row, "s_row", _F32, (rows // block_rows) * (cols // 128))
        _need(q_col, "q_col", _U8, rows * cols)
        _need(s_col, "s_col", _F32, (cols // 128 if block_rows == 128 else cols) * (rows // 128))
    _check(lib.fp8_quantize_block(_ptr(x, "x"), _dtype(x), rows, cols, fmt, block_rows, _ptr(q_row, "q_row"),
                                  _ptr(s_row, "s_row"), _ptr(q_col, "q_col"), _ptr(s_col, "s_col"), _stream(stream)))


def fp8_quantize_mx(x, fmt, q_row, s_row, q_col=None, s_col=None, stream=None):
    """MXFP8: 1x32 blocks along the rows with E8M0 scale bytes (uint8 tensors),
    optionally the columnwise copy (the same rule on x^T)."""
    rows, cols = _shape2(x)
    _need(q_row, "q_row", _U8, rows * cols)
    _need(s_row, "s_row", _U8, rows * (cols // 32))
    _need(q_col, "q_col", _U8, rows * cols)
    _need(s_col, "s_col", _U8, cols * (rows // 32))
    _check(lib.fp8_quantize_mx(_ptr(x, "x"), _dtype(x), rows, cols, fmt, _ptr(q_row, "q_row"), _ptr(s_row, "s_row"),
                               _ptr(q_col, "q_col"), _ptr(s_col, "s_col"), _stream(stream)))


def _delayed_state(hist, new_amax, scale, scale_inv):
    _need(hist, "hist", _F32)
    if hist.dim() != 2:
        raise ValueError("hist must be [history_len][n_cols], got shape %s" % (tuple(hist.shape),))
    n_cols = hist.shape[1]
    if new_amax is not None:
        _need_scalar(new_amax, "new_amax")
    _need(scale, "scale", _F32, n_cols)
    _need(scale_inv, "scale_inv", _F32, n_cols)
    return hist.shape


def fp8_update_scale_delayed(hist, col, new_amax, step, fmt, margin, algo, scale, scale_inv, stream=None):
    """Delayed-scaling update of column `col` of hist [history_len][n_cols]."""
    if new_amax is None:
        raise ValueError("new_amax is required")
    history_len, n_cols = _delayed_state(hist, new_amax, scale, scale_inv)
    _check(lib.fp8_update_scale_delayed(_ptr(hist, "hist"), history_len, n_cols, col, _ptr(new_amax, "new_amax"),
                                        step, fmt, margin, algo, _ptr(scale, "scale"), _ptr(scale_inv, "scale_inv"),
                                        _stream(stream)))


def fp8_quantize_delayed(x, fmt, hist, col, step, fmt_next, margin, algo, scale, scale_inv, q, q_scale_inv_out=None,
                         amax_out=None, stream=None):
    """One delayed-scaling step: cast with scale_inv[col], then record max|x|
    in column col of hist and update scale/scale_inv for fmt_next."""
    _need(x, "x", _HP)
    history_len, n_cols = _delayed_state(hist, None, scale, scale_inv)
    _need(q, "q", _U8, x.numel())
    _scalars(q_scale_inv_out=q_scale_inv_out, amax_out=amax_out)
    _check(lib.fp8_quantize_delayed(_ptr(x, "x"), _dtype(x), x.numel(), fmt, _ptr(hist, "hist"), history_len, n_cols,
                                    col, step, fmt_next, margin, algo, _ptr(scale, "scale"),
                                    _ptr(scale_inv, "scale_inv"), _ptr(q, "q"),
                                    _ptr(q_scale_inv_out, "q_scale_inv_out"), _ptr(amax_out, "amax_out"),
                                    _stream(stream)))


def _gemm_operands(A, sA, B, sB, mode, C):
    """Shapes of C = A B^T and the scale buffers each mode reads."""
    _need(A, "A", _U8)
    _need(B, "B", _U8)
    if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
        raise ValueError("A, B and C must be 2-D")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape), tuple(C.shape)))
    # scale buffers are read, never written: a longer one is harmless (a
    # K = 0 product reads none but still needs a buffer)
    if mode == PER_TENSOR:
        _need(sA, "sA", _F32, 1)
        _need(sB, "sB", _F32, 1)
    elif mode == BLOCK_1x128_128x128:
        _need(sA, "sA", _F32, max(1, M * (K // 128)), at_least=True)
        _need(sB, "sB", _F32, max(1, (N // 128) * (K // 128)), at_least=True)
    elif mode == BLOCK_1x128_1x128:
        _need(sA, "sA", _F32, max(1, M * (K // 128)), at_least=True)
        _need(sB, "sB", _F32, max(1, N * (K // 128)), at_least=True)
    elif mode == MXFP8:
        _need(sA, "sA", _U8, max(1, M * (K // 32)), at_least=True)
        _need(sB, "sB", _U8, max(1, N * (K // 32)), at_least=True)
    if sA is None or sB is None:
        raise ValueError("sA and sB are required")
    return M, N, K


def fp8_scaled_gemm(A, fa, sA, B, fb, sB, mode, C, amax_out=None, stream=None):
    """C = (A*sA)(B*sB)^T, A [M][K], B [N][K] codes, C [M][N] bfloat16 or float32."""
    _need(C, "C", _HP)
    M, N, K = _gemm_operands(A, sA, B, sB, mode, C)
    _scalars(amax_out=amax_out)
    _check(lib.fp8_scaled_gemm(_ptr(A, "A"), fa, _ptr(sA, "sA"), _ptr(B, "B"), fb, _ptr(sB, "sB"), M, N, K, mode,
                               _ptr(C, "C"), _dtype(C), _ptr(amax_out, "amax_out"), _stream(stream)))


def fp8_scaled_gemm_fused(A, fa, sA, B, fb, sB, mode, C, *, bias=None, act=ACT_NONE, out_fmt=None,
                          c_scale_inv=None, amax_out=None, stream=None):
    """C = out(act((A*sA)(B*sB)^T + bias)); C bfloat16 / float32, or uint8
    codes of out_fmt (E4M3FN / E5M2) cast with the dequant scale c_scale_inv."""
    _need(C, "C", (torch.float32, torch.bfloat16, torch.uint8))
    M, N, K = _gemm_operands(A, sA, B, sB, mode, C)
    if C.dtype == torch.uint8:
        if out_fmt not in (E4M3FN, E5M2):
            raise ValueError("a uint8 C needs out_fmt E4M3FN or E5M2")
        c_type = OUT_E4M3FN if out_fmt == E4M3FN else OUT_E5M2
        if c_scale_inv is None:
            raise ValueError("an FP8 output needs c_scale_inv")
    else:
        c_type = _dtype(C)
    _need(bias, "bias", _F32, N)
    _scalars(c_scale_inv=c_scale_inv, amax_out=amax_out)
    _check(lib.fp8_scaled_gemm_fused(_ptr(A, "A"), fa, _ptr(sA, "sA"), _ptr(B, "B"), fb, _ptr(sB, "sB"), M, N, K,
                                     mode, _ptr(bias, "bias"), act, _ptr(C, "C"), c_type,
                                     _ptr(c_scale_inv, "c_scale_inv"), _ptr(amax_out, "amax_out"), _stream(stream)))


def fp8_quantize_hybrid(x, row_fmt, col_fmt, col_source, *, q_row=None, q_col=None, amax_in=None, row_margin=0,
                        col_margin=0, row_scale_inv_in=None, col_scale_inv_in=None, row_scale_inv_out=None,
                        col_scale_inv_out=None, amax_out=None, stream=None):
    """Per-direction per-tensor cast: rowwise codes in row_fmt, columnwise
    (transposed) codes in col_fmt from x or from the dequantized rows."""
    rows, cols = _shape2(x)
    _need(q_row, "q_row", _U8, rows * cols)
    _need(q_col, "q_col", _U8, rows * cols)
    _scalars(amax_in=amax_in, row_scale_inv_in=row_scale_inv_in, col_scale_inv_in=col_scale_inv_in,
             row_scale_inv_out=row_scale_inv_out, col_scale_inv_out=col_scale_inv_out, amax_out=amax_out)
    _check(lib.fp8_quantize_hybrid(_ptr(x, "x"), _dtype(x), rows, cols, row_fmt, col_fmt, col_source,
                                   _ptr(amax_in, "amax_in"), row_margin, col_margin,
                                   _ptr(row_scale_inv_in, "row_scale_inv_in"),
                                   _ptr(col_scale_inv_in, "col_scale_inv_in"), _ptr(q_row, "q_row"),
                                   _ptr(q_col, "q_col"), _ptr(row_scale_inv_out, "row_scale_inv_out"),
                                   _ptr(col_scale_inv_out, "col_scale_inv_out"), _ptr(amax_out, "amax_out"),
                                   _stream(stream)))


def _subq_scales(recipe, rows, cols):
    """(dtype, element count) of the scale buffer of one direction's copy of a
    [rows][cols] tensor under a sub-quantizer."""
    if recipe == SUBQ_PER_TENSOR:
        return _F32, 1
    if recipe == SUBQ_BLOCK_128x128:
        return _F32, (rows // 128) * (cols // 128)
    if recipe == SUBQ_BLOCK_1x128:
        return _F32, rows * (cols // 128)
    return _U8, rows * (cols // 32)


def fp8_quantize_hybrid_blockwise(x, row_recipe, row_fmt, col_recipe, col_fmt, *, col_source=COLSRC_ORIGINAL,
                                  q_row=None, s_row=None, q_col=None, s_col=None, amax_in=None, margin=0,
                                  scale_inv_in=None, stream=None):
    """Per-direction quantization with block, MXFP8 or (in one direction)
    per-tensor sub-quantizers: rowwise copy by row_recipe in row_fmt (codes
    [rows][cols]), columnwise copy by col_recipe in col_fmt applied to x^T or
    to the dequantized rows (codes [cols][rows]); scales float32 (blocks; one
    float for a per-tensor direction, which takes amax_in or scale_inv_in) or
    uint8 (MXFP8)."""
    rows, cols = _shape2(x)
    recipes = (SUBQ_BLOCK_128x128, SUBQ_BLOCK_1x128, SUBQ_MXFP8, SUBQ_PER_TENSOR)
    if row_recipe in recipes:
        _need(q_row, "q_row", _U8, rows * cols)
        _need(s_row, "s_row", *_subq_scales(row_recipe, rows, cols))
    if col_recipe in recipes:
        _need(q_col, "q_col", _U8, rows * cols)
        _need(s_col, "s_col", *_subq_scales(col_recipe, cols, rows))
    _scalars(amax_in=amax_in, scale_inv_in=scale_inv_in)
    _check(lib.fp8_quantize_hybrid_blockwise(_ptr(x, "x"), _dtype(x), rows, cols, row_recipe, row_fmt,
                                             _ptr(q_row, "q_row"), _ptr(s_row, "s_row"), col_recipe, col_fmt,
                                             col_source, _ptr(q_col, "q_col"), _ptr(s_col, "s_col"),
                                             _ptr(amax_in, "amax_in"), margin, _ptr(scale_inv_in, "scale_inv_in"),
                                             _stream(stream)))


def fp8_cast_stats(x, fmt, scale_inv, stats, stream=None):
    """stats (int64 [4] on the device) = overflows, underflows, NaNs,
    nonzeros of the cast of x with dequant scale scale_inv."""
    _need(x, "x", _HP)
    _need_scalar(scale_inv, "scale_inv")
    _need(stats, "stats", _STATS, 4)
    _check(lib.fp8_cast_stats(_ptr(x, "x"), _dtype(x), x.numel(), fmt, _ptr(scale_inv, "scale_inv"),
                              _ptr(stats, "stats"), _stream(stream)))


def fp8_quantize_error_feedback(g, residual, fmt, scale_inv, q, amax_out=None, stream=None):
    """q = cast(g + residual); residual <- (g + residual) - dequant(q), in place."""
    _need(g, "g", _HP)
    _need(residual, "residual", _F32, g.numel())
    _need(q, "q", _U8, g.numel())
    _need_scalar(scale_inv, "scale_inv")
    _scalars(amax_out=amax_out)
    _check(lib.fp8_quantize_error_feedback(_ptr(g, "g"), _dtype(g), _ptr(residual, "residual"), g.numel(), fmt,
                                           _ptr(scale_inv, "scale_inv"), _ptr(q, "q"), _ptr(amax_out, "amax_out"),
                                           _stream(stream)))


def _groups(offsets):
    """Number of groups of an int32 offsets tensor [groups + 1]."""
    _required(offsets=offsets)
    _need(offsets, "offsets", _I32T)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be [groups + 1], got shape %s" % (tuple(offsets.shape),))
    return offsets.numel() - 1


def _col_copy(q, s, name, rows):
    """col_stride of a columnwise copy: codes [rows][col_stride], scales [rows][col_stride/128]."""
    _need(q, "q_" + name if name == "col" else name, _U8)
    if q.dim() != 2 or q.shape[0] != rows:
        raise ValueError("%s must be [%d][col_stride], got shape %s" % ("q_" + name if name == "col" else name, rows,
                                                                       tuple(q.shape)))
    _need(s, "s_" + name if name == "col" else "s" + name, _F32, rows * (q.shape[1] // 128))
    return q.shape[1]


def fp8_quantize_grouped(x, offsets, fmt, *, row_index=None, q_row=None, s_row=None, q_col=None, s_col=None,
                         stream=None):
    """1x128 block quantization of the rows of x in group order (row t is
    x[row_index[t]], or x[t]); offsets: int32 [groups + 1] on the device.
    q_col [cols][col_stride], s_col [cols][col_stride/128]: the columnwise copy
    with every group padded to whole blocks of 128."""
    try:
        dev = _current_device()
        x_rows, cols = x.shape
        i32, u8, f32 = torch.int32, torch.uint8, torch.float32
        groups, = offsets.shape
        rows = x_rows if row_index is None else row_index.numel()
        stride = 0
        if q_col is not None:
            c, stride = q_col.shape
            if c != cols:
                raise _Unfit
            col = _at(q_col, u8, cols * stride, dev), _at(s_col, f32, cols * (stride // 128), dev)
        else:
            col = None, _at_or_none(s_col, f32, 0, dev)
        args = (_at(x, x.dtype, x_rows * cols, dev), _CODES[x.dtype], x_rows, cols,
                _at_or_none(row_index, i32, rows, dev), rows, _at(offsets, i32, groups, dev), groups - 1, fmt,
                _at_or_none(q_row, u8, rows * cols, dev), _at_or_none(s_row, f32, rows * (cols // 128), dev), *col,
                stride)
        if groups < 1:
            raise _Unfit
    except _UNFIT:
        x_rows, cols = _shape2(x)
        _groups(offsets)
        _need(row_index, "row_index", _I32T)
        rows = x_rows if row_index is None else row_index.numel()
        _need(q_row, "q_row", _U8, rows * cols)
        _need(s_row, "s_row", _F32, rows * (cols // 128))
        if q_col is not None:
            _required(s_col=s_col)
            _col_copy(q_col, s_col, "col", cols)
        elif s_col is not None:
            raise ValueError("s_col needs q_col")
        _on_device(x=x, row_index=row_index, offsets=offsets, q_row=q_row, s_row=s_row, q_col=q_col, s_col=s_col)
        raise
    _check(lib.fp8_quantize_grouped(*args, _stream(stream)))


def fp8_grouped_gemm(A, fa, sA, B, fb, sB, offsets, C, stream=None):
    """C[t] = (A[t]*sA[t]) (B[e]*sB[e])^T for the rows t of group e: A [rows][K],
    B [groups][N][K] codes, C [rows][N] bfloat16."""
    try:
        dev = _current_device()
        u8, f32 = torch.uint8, torch.float32
        rows, K = A.shape
        groups, N, k = B.shape
        if k != K or C.shape != (rows, N):
            raise _Unfit
        args = (_at(A, u8, rows * K, dev), fa, _at(sA, f32, rows * (K // 128), dev), _at(B, u8, groups * N * K, dev), fb,
                _at(sB, f32, groups * (N // 128) * (K // 128), dev), _at(offsets, torch.int32, groups + 1, dev), groups,
                rows, N, K, _at(C, torch.bfloat16, rows * N, dev))
        if offsets.dim() != 1:
            raise _Unfit
    except _UNFIT:
        groups = _groups(offsets)
        _required(A=A, sA=sA, B=B, sB=sB, C=C)
        _need(A, "A", _U8)
        _need(B, "B", _U8)
        _need(C, "C", _BF16T)
        if A.dim() != 2 or B.dim() != 3 or C.dim() != 2:
            raise ValueError("A and C must be 2-D and B 3-D")
        rows, K = A.shape
        N = B.shape[1]
        if B.shape[0] != groups or B.shape[2] != K or tuple(C.shape) != (rows, N):
            raise ValueError("shape mismatch: A %s, B %s, C %s, %d groups" % (tuple(A.shape), tuple(B.shape),
                                                                             tuple(C.shape), groups))
        _need(sA, "sA", _F32, rows * (K // 128))
        _need(sB, "sB", _F32, groups * (N // 128) * (K // 128))
        _on_device(A=A, sA=sA, B=B, sB=sB, offsets=offsets, C=C)
        raise
    _check(lib.fp8_grouped_gemm(*args, _stream(stream)))


def fp8_grouped_gemm_wgrad(A, fa, sA, B, fb, sB, offsets, C, stream=None):
    """C[e] = (A_e*sA_e) (B_e*sB_e)^T over the tokens of group e: A
    [M][col_stride], B [N][col_stride] columnwise codes of fp8_quantize_grouped,
    C [groups][M][N] bfloat16 or float32."""
    try:
        dev = _current_device()
        u8, f32 = torch.uint8, torch.float32
        groups, M, N = C.shape
        (m, stride), (n, other) = A.shape, B.shape
        if m != M or n != N or other != stride or offsets.dim() != 1:
            raise _Unfit
        # the tokens in the groups are at most the columns that hold them
        args = (_at(A, u8, M * stride, dev), fa, _at(sA, f32, M * (stride // 128), dev), _at(B, u8, N * stride, dev),
                fb, _at(sB, f32, N * (stride // 128), dev), _at(offsets, torch.int32, groups + 1, dev), groups, stride,
                stride, M, N, _at(C, C.dtype, groups * M * N, dev), _CODES[C.dtype])
    except _UNFIT:
        groups = _groups(offsets)
        _required(A=A, sA=sA, B=B, sB=sB, C=C)
        _need(C, "C", _HP)
        if C.dim() != 3 or C.shape[0] != groups:
            raise ValueError("C must be [%d][M][N], got shape %s" % (groups, tuple(C.shape)))
        M, N = C.shape[1:]
        if _col_copy(A, sA, "A", M) != _col_copy(B, sB, "B", N):
            raise ValueError("A and B must have one col_stride")
        _on_device(A=A, sA=sA, B=B, sB=sB, offsets=offsets, C=C)
        raise
    _check(lib.fp8_grouped_gemm_wgrad(*args, _stream(stream)))


def _params(cols, x, **kw):
    """dtype of the per-column parameters (all of one type); x's when none is given."""
    got = {n: t for n, t in kw.items() if t is not None}
    for n, t in got.items():
        _need(t, n, _HP, cols)
    types = {t.dtype for t in got.values()}
    if len(types) > 1:
        raise TypeError("%s must have one dtype" % " and ".join(sorted(got)))
    return _dtype(next(iter(got.values()))) if got else _dtype(x)


class _Unfit(ValueError):
    """A tensor that a call cannot take; the checks by name say why."""


# What a call may find wrong before it has looked closer (RuntimeError: no GPU)
_UNFIT = (ValueError, AttributeError, KeyError, TypeError, RuntimeError)


def _at(t, dtype, numel, device):
    """Address of a contiguous tensor of this type and size on the device.  A
    small kernel takes as long as the checks of its arguments by name, so the
    calls below make all checks of a tensor at once and look for the reason, in
    the order types, sizes, device, only if one fails (2.3 us less a call of
    six tensors)."""
    if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    raise _Unfit


def _at_or_none(t, dtype, numel, device):
    return None if t is None else _at(t, dtype, numel, device)


def _same(t, name, x):
    """t has x's dtype and element count."""
    _need(t, name, (x.dtype,), x.numel())


def _on_device(**kw):
    """Every tensor given is on the current GPU."""
    for name, t in kw.items():
        _ptr(t, name)


def _required(**kw):
    for name, t in kw.items():
        if t is None:
            raise ValueError("%s is required" % name)


def fp8q_layernorm(x, gamma, beta, eps, y, mean=None, rstd=None, stream=None):
    """y = layer norm of the rows of x [rows][cols] with gain gamma and bias
    beta (either may be None); mean, rstd (float32 [rows]) for the backward
    pass."""
    try:
        dev = _current_device()
        rows, cols = x.shape
        t, n = x.dtype, rows * cols
        p = t if gamma is None and beta is None else (beta if gamma is None else gamma).dtype
        args = (_at(x, t, n, dev), _CODES[t], rows, cols, _at_or_none(gamma, p, cols, dev),
                _at_or_none(beta, p, cols, dev), _CODES[p], eps, _at(y, t, n, dev),
                _at_or_none(mean, torch.float32, rows, dev), _at_or_none(rstd, torch.float32, rows, dev))
    except _UNFIT:
        rows, cols = _shape2(x)
        _required(y=y)
        _params(cols, x, gamma=gamma, beta=beta)
        _same(y, "y", x)
        _need(mean, "mean", _F32, rows)
        _need(rstd, "rstd", _F32, rows)
        _on_device(x=x, gamma=gamma, beta=beta, y=y, mean=mean, rstd=rstd)
        raise
    _check(lib.fp8q_layernorm(*args, _stream(stream)))


def fp8q_layernorm_backward_workspace(dtype, rows, cols):
    """Bytes of the workspace of fp8q_layernorm_backward (dtype: F32 or BF16)."""
    n = ctypes.c_int64(0)
    _check(lib.fp8q_layernorm_backward_workspace(dtype, rows, cols, ctypes.byref(n)))
    return n.value


def fp8q_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, workspace=None, stream=None):
    """dx and (if given) dgamma, dbeta of fp8q_layernorm; workspace: a device
    tensor of at least fp8q_layernorm_backward_workspace bytes, needed with
    dgamma or dbeta."""
    try:
        dev = _current_device()
        rows, cols = x.shape
        t, n, f32 = x.dtype, rows * cols, torch.float32
        given = gamma if gamma is not None else dgamma if dgamma is not None else dbeta
        p = t if given is None else given.dtype
        ws = ws_bytes = 0
        if workspace is not None:
            ws, ws_bytes = _at(workspace, workspace.dtype, workspace.numel(), dev), workspace.nbytes
        args = (_at(dy, t, n, dev), _at(x, t, n, dev), _CODES[t], rows, cols, _at_or_none(gamma, p, cols, dev),
                _CODES[p], _at(mean, f32, rows, dev), _at(rstd, f32, rows, dev), _at(dx, t, n, dev),
                _at_or_none(dgamma, p, cols, dev), _at_or_none(dbeta, p, cols, dev), ws, ws_bytes)
    except _UNFIT:
        rows, cols = _shape2(x)
        _required(dy=dy, mean=mean, rstd=rstd, dx=dx)
        _params(cols, x, gamma=gamma, dgamma=dgamma, dbeta=dbeta)
        _same(dy, "dy", x)
        _same(dx, "dx", x)
        _need(mean, "mean", _F32, rows)
        _need(rstd, "rstd", _F32, rows)
        if workspace is not None:
            _tensor(workspace, "workspace")
        _on_device(dy=dy, x=x, gamma=gamma, mean=mean, rstd=rstd, dx=dx, dgamma=dgamma, dbeta=dbeta,
                   workspace=workspace)
        raise
    _check(lib.fp8q_layernorm_backward(*args, _stream(stream)))


_T = torch.Tensor
_dtype_of = _T.dtype.__get__


def _addresses(ts):
    """Addresses of a list of contiguous tensors on the current GPU, as a C
    array (one C call per tensor and property: the list of a model's
    gradients is long)."""
    if not all(map(_T.is_contiguous, ts)) or (len(ts) and set(map(_T.get_device, ts)) != {_current_device()}):
        raise _Unfit
    return array.array("Q", list(map(_T.data_ptr, ts)))


def _address(a):
    return a.buffer_info()[0]


def fp8q_grad_norm_clip(grads, max_norm, norm, coef, out=None, stream=None):
    """norm[0] = the 2-norm over all tensors of grads (float32 / bfloat16, any
    shapes), coef[0] = min(1, max_norm / (norm + 1e-6)); every gradient is
    multiplied by coef, in place or into the tensors of out.  An infinite
    max_norm computes the norm alone."""
    _required(norm=norm, coef=coef)
    _scalars(norm=norm, coef=coef)
    count = len(grads)
    if out is not None and len(out) != count:
        raise ValueError("out must have %d tensors, got %d" % (count, len(out)))
    try:
        types, sizes = list(map(_dtype_of, grads)), list(map(_T.numel, grads))
        if out is not None and (list(map(_dtype_of, out)) != types or list(map(_T.numel, out)) != sizes):
            raise _Unfit
        d, n = array.array("i", [_CODES[t] for t in types]), array.array("q", sizes)
        g, o = _addresses(grads), None if out is None else _addresses(out)
    except _UNFIT:
        # find what is wrong: types and sizes first, the device last
        for i, t in enumerate(grads):
            _need(t, "grads[%d]" % i, _HP)
        for i, t in enumerate(grads if out is not None else ()):
            _same(out[i], "out[%d]" % i, t)
        for i, t in enumerate(grads):
            _ptr(t, "grads[%d]" % i)
        for i, t in enumerate(out or ()):
            _ptr(t, "out[%d]" % i)
        raise
    # the arrays outlive the call, which reads them before it returns
    _check(lib.fp8q_grad_norm_clip(_address(g), None if o is None else _address(o), _address(n), _address(d), count,
                                   max_norm, _ptr(norm, "norm"), _ptr(coef, "coef"), _stream(stream)))


CLOCK_BLOCKS = 8
CLOCK_MONITOR_SECONDS = 2


def fp8q_clock_monitor(out, stop, stream=None):
    """Enqueue the clock monitor (a measurement aid): out (int64 [25] on the
    device) receives, per block b, the XCD id, the shader-clock cycles and
    the constant-rate ticks from the kernel's start until stop (int32 [1] on
    the device) becomes nonzero; out[24] = the constant rate in kHz."""
    _need(out, "out", _STATS, 3 * CLOCK_BLOCKS + 1)
    _need(stop, "stop", (torch.int32,), 1)
    _check(lib.fp8q_clock_monitor(_ptr(out, "out"), _ptr(stop, "stop"), _stream(stream)))


POLL_ROUNDS_DEFAULT = 0xFFFFFFFF


def fp8q_set_finish_poll_rounds(rounds):
    """Set the bound on a finishing block's polling rounds for later calls
    (a failure-handling knob; 0 makes every finishing block give up at once,
    POLL_ROUNDS_DEFAULT restores the default) and return the bound that was
    in force."""
    if not 0 <= int(rounds) <= 0xFFFFFFFF:
        raise ValueError("rounds must fit in 32 bits")
    prev = ctypes.c_uint32(0)
    _check(lib.fp8q_set_finish_poll_rounds(ctypes.c_uint32(int(rounds)), ctypes.byref(prev)))
    return prev.value


def clock_mhz(sample):
    """{xcd: MHz} from a host copy of a clock-monitor output (an XCD measured
    by several blocks keeps their mean); None for a monitor that ran into its
    time limit instead of seeing stop."""
    khz = int(sample[3 * CLOCK_BLOCKS])
    if khz <= 0:
        return None
    acc = {}
    for b in range(CLOCK_BLOCKS):
        cycles, ticks = int(sample[3 * b + 1]), int(sample[3 * b + 2])
        if ticks >= khz * 1000 * CLOCK_MONITOR_SECONDS or cycles <= 0 or ticks <= 0:
            return None
        acc.setdefault(int(sample[3 * b]), []).append(cycles / (ticks / (khz * 1e3)) / 1e6)
    return {x: sum(v) / len(v) for x, v in sorted(acc.items())}
