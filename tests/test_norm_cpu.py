"""Refusals of the layer norm and the gradient norm: bad arguments are
reported on the host before any HIP call, and the binding checks sizes, types
and devices before the library is called."""
import ctypes
import math

import pytest
import torch

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")

L, S = fq.lib, 0
BAD = 0x100000  # aligned fake device addresses, never dereferenced


def _expect(status, code, fragment):
    assert status == code, (status, fq.last_error())
    assert fragment in fq.last_error(), fq.last_error()


def _ln(x=BAD, dtype=fq.BF16, rows=4, cols=64, gamma=BAD + 0x10000, beta=BAD + 0x20000, pt=fq.F32, eps=1e-5,
        y=BAD + 0x30000, mean=BAD + 0x40000, rstd=BAD + 0x50000):
    return L.fp8q_layernorm(x, dtype, rows, cols, gamma, beta, pt, eps, y, mean, rstd, S)


def test_layernorm_validation():
    _expect(_ln(dtype=2), fq.EINVAL, "dtype")
    _expect(_ln(pt=-1), fq.EINVAL, "dtype")
    _expect(_ln(rows=-1), fq.EINVAL, "rows")
    _expect(_ln(cols=0), fq.EINVAL, "cols")
    _expect(_ln(cols=(1 << 31) + 1), fq.EUNSUPPORTED, "2^31")
    for eps in (-1e-5, math.nan, math.inf):
        _expect(_ln(eps=eps), fq.EINVAL, "eps")
    _expect(_ln(x=None), fq.EINVAL, "x must")
    _expect(_ln(x=BAD + 1), fq.EINVAL, "x must")
    _expect(_ln(dtype=fq.F32, x=BAD + 2), fq.EINVAL, "x must")
    _expect(_ln(y=None), fq.EINVAL, "y must")
    _expect(_ln(gamma=BAD + 0x10002), fq.EINVAL, "gamma")
    _expect(_ln(mean=BAD + 0x40002), fq.EINVAL, "mean")
    _expect(_ln(y=BAD), fq.EINVAL, "overlaps an input")
    _expect(_ln(mean=BAD + 0x20000), fq.EINVAL, "overlaps an input")
    _expect(_ln(rstd=BAD + 0x40000), fq.EINVAL, "overlap each other")


def _lnb(dy=BAD, x=BAD + 0x10000, dtype=fq.BF16, rows=4, cols=64, gamma=BAD + 0x20000, pt=fq.F32, mean=BAD + 0x30000,
         rstd=BAD + 0x40000, dx=BAD + 0x50000, dg=BAD + 0x60000, db=BAD + 0x70000, ws=BAD + 0x80000, nb=1 << 30):
    return L.fp8q_layernorm_backward(dy, x, dtype, rows, cols, gamma, pt, mean, rstd, dx, dg, db, ws, nb, S)


def test_layernorm_backward_validation():
    _expect(_lnb(dtype=5), fq.EINVAL, "dtype")
    _expect(_lnb(pt=5), fq.EINVAL, "dtype")
    _expect(_lnb(rows=-4), fq.EINVAL, "rows")
    _expect(_lnb(dy=None), fq.EINVAL, "dy, x and dx")
    _expect(_lnb(dx=BAD + 0x50001), fq.EINVAL, "dy, x and dx")
    _expect(_lnb(mean=None), fq.EINVAL, "mean and rstd")
    _expect(_lnb(ws=None), fq.EINVAL, "workspace")
    _expect(_lnb(ws=BAD + 0x80004), fq.EINVAL, "workspace")
    _expect(_lnb(nb=0), fq.EINVAL, "workspace needs")
    _expect(_lnb(dx=BAD), fq.EINVAL, "overlaps an input")
    _expect(_lnb(dg=BAD + 0x20000), fq.EINVAL, "overlaps an input")
    _expect(_lnb(db=BAD + 0x60000), fq.EINVAL, "overlap each other")
    _expect(_lnb(ws=BAD + 0x50000), fq.EINVAL, "overlap each other")


def test_layernorm_workspace():
    n = ctypes.c_int64(-1)
    _expect(L.fp8q_layernorm_backward_workspace(9, 4, 64, ctypes.byref(n)), fq.EINVAL, "dtype")
    _expect(L.fp8q_layernorm_backward_workspace(0, 4, 0, ctypes.byref(n)), fq.EINVAL, "cols")
    _expect(L.fp8q_layernorm_backward_workspace(0, 4, 64, None), fq.EINVAL, "bytes")
    sizes = [fq.fp8q_layernorm_backward_workspace(fq.BF16, r, 4096) for r in (0, 1, 100, 16384, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[1] >= 2 * 4096 * 4 and sizes[-1] <= 64 << 20


def _clip(sizes=(4,), g=BAD, out=None, dt=fq.F32, max_norm=1.0, norm=BAD + 0x80000, coef=BAD + 0x80010, count=None):
    k = len(sizes)
    gs = (ctypes.c_void_p * k)(*[g] * k)
    o = None if out is None else (ctypes.c_void_p * k)(*[out] * k)
    n = (ctypes.c_int64 * k)(*sizes)
    d = (ctypes.c_int32 * k)(*[dt] * k)
    return L.fp8q_grad_norm_clip(gs, o, n, d, k if count is None else count, max_norm, norm, coef, S)


def test_grad_norm_clip_validation():
    _expect(_clip(count=-1), fq.EINVAL, "count")
    _expect(L.fp8q_grad_norm_clip(None, None, None, None, 1, 1.0, BAD, BAD + 4, S), fq.EINVAL, "must be given")
    for m in (-1.0, math.nan):
        _expect(_clip(max_norm=m), fq.EINVAL, "max_norm")
    _expect(_clip(norm=None), fq.EINVAL, "norm and coef")
    _expect(_clip(coef=BAD + 0x80000), fq.EINVAL, "norm and coef")
    _expect(_clip(max_norm=math.inf, out=BAD + 0x1000), fq.EINVAL, "out must be null")
    _expect(_clip(dt=3), fq.EINVAL, "dtype")
    _expect(_clip(sizes=(4, -1)), fq.EINVAL, "size")
    _expect(_clip(g=None), fq.EINVAL, "tensor 0")
    _expect(_clip(g=BAD + 2), fq.EINVAL, "tensor 0")
    _expect(_clip(out=BAD + 0x1002), fq.EINVAL, "output 0")
    _expect(_clip(out=BAD + 8), fq.EINVAL, "overlaps its gradient")
    _expect(_clip(norm=BAD + 8), fq.EINVAL, "overlaps tensor")


X = torch.zeros(8, 64, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(*s)


BAD_CALLS = [
    (lambda: fq.fp8q_layernorm(X, f32(63), None, 1e-5, X.clone()), ValueError, "gamma must have 64"),
    (lambda: fq.fp8q_layernorm(X, f32(64), X[0].clone(), 1e-5, X.clone()), TypeError, "one dtype"),
    (lambda: fq.fp8q_layernorm(X, None, None, 1e-5, f32(8, 64)), TypeError, "y must be"),
    (lambda: fq.fp8q_layernorm(X, None, None, 1e-5, None), ValueError, "y is required"),
    (lambda: fq.fp8q_layernorm(X, None, None, 1e-5, X.clone(), f32(7)), ValueError, "mean must have 8"),
    (lambda: fq.fp8q_layernorm(X.t(), None, None, 1e-5, X.clone()), ValueError, "contiguous"),
    (lambda: fq.fp8q_layernorm(X[0], None, None, 1e-5, X[0].clone()), ValueError, "2-D"),
    (lambda: fq.fp8q_layernorm_backward(X[:4], X, None, f32(8), f32(8), X.clone()), ValueError, "dy must have"),
    (lambda: fq.fp8q_layernorm_backward(X, X, None, f32(8), None, X.clone()), ValueError, "rstd is required"),
    (lambda: fq.fp8q_layernorm_backward(X, X, f32(64), f32(8), f32(8), X.clone(), f32(65)), ValueError, "dgamma"),
    (lambda: fq.fp8q_grad_norm_clip([X, X.double()], 1.0, f32(1), f32(1)), TypeError, r"grads\[1\]"),
    (lambda: fq.fp8q_grad_norm_clip([X, X.t()], 1.0, f32(1), f32(1)), ValueError, "contiguous"),
    (lambda: fq.fp8q_grad_norm_clip([X], 1.0, f32(1), f32(1), out=[]), ValueError, "out must have 1"),
    (lambda: fq.fp8q_grad_norm_clip([X], 1.0, f32(1), f32(1), out=[X.float()]), TypeError, r"out\[0\]"),
    (lambda: fq.fp8q_grad_norm_clip([X], 1.0, f32(2), f32(1)), ValueError, "norm must have 1"),
    # right sizes and types, not on the GPU
    (lambda: fq.fp8q_layernorm(X, f32(64), f32(64), 1e-5, X.clone(), f32(8), f32(8)), ValueError, "GPU tensor"),
    (lambda: fq.fp8q_grad_norm_clip([X], 1.0, f32(1), f32(1)), ValueError, "GPU tensor"),
]


@pytest.mark.parametrize("i", range(len(BAD_CALLS)))
def test_binding_refuses(i):
    call, exc, fragment = BAD_CALLS[i]
    with pytest.raises(exc, match=fragment):
        call()


def test_layernorm_sizes_whose_bytes_pass_64_bits():
    """2^64 bytes would look like none to the overlap checks (here y on x, dx on x)."""
    big = 1 << 31
    _expect(_ln(dtype=fq.F32, rows=big, cols=big, y=BAD), fq.EUNSUPPORTED, "2^40")
    _expect(_ln(rows=(1 << 20) + 1, cols=1 << 20), fq.EUNSUPPORTED, "2^40")
    _expect(_lnb(dtype=fq.F32, rows=big, cols=big, dx=BAD + 0x10000), fq.EUNSUPPORTED, "2^40")
    n = ctypes.c_int64(-1)
    _expect(L.fp8q_layernorm_backward_workspace(0, big, big, ctypes.byref(n)), fq.EUNSUPPORTED, "2^40")
    assert L.fp8q_layernorm_backward_workspace(0, 1 << 20, 1 << 20, ctypes.byref(n)) == fq.OK and n.value > 0
