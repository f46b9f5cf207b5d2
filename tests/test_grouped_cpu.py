"""Refusals of the grouped calls: bad arguments are reported on the host before
any HIP call, and the binding checks sizes, types and devices first."""
import pytest
import torch

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")

L, S = fq.lib, 0
P = [0x1000000 * (i + 1) for i in range(12)]  # aligned fake device addresses, never dereferenced


def _expect(status, code, fragment):
    assert status == code, (status, fq.last_error())
    assert fragment in fq.last_error(), fq.last_error()


def _q(x=P[0], dt=fq.BF16, x_rows=64, cols=256, index=P[1], rows=64, off=P[2], groups=3, fmt=0, qr=P[3], sr=P[4],
       qc=P[5], sc=P[6], stride=512):
    return L.fp8_quantize_grouped(x, dt, x_rows, cols, index, rows, off, groups, fmt, qr, sr, qc, sc, stride, S)


def test_quantize_grouped_validation():
    _expect(_q(dt=2), fq.EINVAL, "dtype")
    _expect(_q(fmt=7), fq.EINVAL, "format")
    _expect(_q(groups=-1), fq.EINVAL, "negative")
    _expect(_q(rows=-1), fq.EINVAL, "negative")
    _expect(_q(groups=70000), fq.EUNSUPPORTED, "65536")
    _expect(_q(rows=0x7FFFFFFF), fq.EUNSUPPORTED, "2^31")
    _expect(_q(off=None), fq.EINVAL, "offsets")
    _expect(_q(off=P[2] + 2), fq.EINVAL, "offsets")
    _expect(_q(cols=100), fq.EUNSUPPORTED, "multiple of 128")
    _expect(_q(cols=-128), fq.EINVAL, "negative shape")
    _expect(_q(index=None, rows=63), fq.EINVAL, "row_index")
    _expect(_q(index=P[1] + 1), fq.EINVAL, "row_index")
    _expect(_q(sr=None), fq.EINVAL, "go together")
    _expect(_q(qc=None), fq.EINVAL, "go together")
    _expect(_q(qr=None, sr=None, qc=None, sc=None), fq.EINVAL, "at least one")
    _expect(_q(stride=500), fq.EINVAL, "col_stride")
    _expect(_q(x=None), fq.EINVAL, "x must")
    _expect(_q(x=P[0] + 8), fq.EINVAL, "x must")
    _expect(_q(qr=P[3] + 8), fq.EINVAL, "16-byte")
    _expect(_q(qr=P[0]), fq.EINVAL, "overlaps an input")
    _expect(_q(sc=P[2]), fq.EINVAL, "overlaps an input")
    _expect(_q(qc=P[3] + 256), fq.EINVAL, "overlap")


def _g(A=P[0], fa=0, sA=P[1], B=P[2], fb=0, sB=P[3], off=P[4], groups=3, rows=64, N=256, K=256, C=P[5]):
    return L.fp8_grouped_gemm(A, fa, sA, B, fb, sB, off, groups, rows, N, K, C, S)


def test_grouped_gemm_validation():
    _expect(_g(fa=2), fq.EINVAL, "format")
    _expect(_g(fb=-1), fq.EINVAL, "format")
    _expect(_g(N=200), fq.EUNSUPPORTED, "multiples of 128")
    _expect(_g(K=64), fq.EUNSUPPORTED, "multiples of 128")
    _expect(_g(K=-128), fq.EINVAL, "negative")
    _expect(_g(K=(1 << 22) + 128), fq.EUNSUPPORTED, "2^22")
    _expect(_g(groups=70000), fq.EUNSUPPORTED, "65536")
    _expect(_g(off=None), fq.EINVAL, "offsets")
    _expect(_g(A=None), fq.EINVAL, "A and B")
    _expect(_g(B=P[2] + 8), fq.EINVAL, "A and B")
    _expect(_g(sA=P[1] + 2), fq.EINVAL, "sA and sB")
    _expect(_g(C=None), fq.EINVAL, "C must")
    _expect(_g(C=P[5] + 2), fq.EINVAL, "C must")
    _expect(_g(C=P[2]), fq.EINVAL, "overlaps")
    _expect(_g(C=P[4]), fq.EINVAL, "overlaps")


def _w(A=P[0], fa=1, sA=P[1], B=P[2], fb=0, sB=P[3], off=P[4], groups=3, rows=64, stride=384, M=256, N=128, C=P[5],
       ct=fq.F32):
    return L.fp8_grouped_gemm_wgrad(A, fa, sA, B, fb, sB, off, groups, rows, stride, M, N, C, ct, S)


def test_grouped_wgrad_validation():
    _expect(_w(ct=2), fq.EINVAL, "output dtype")
    _expect(_w(fa=9), fq.EINVAL, "format")
    _expect(_w(M=100), fq.EUNSUPPORTED, "multiples of 128")
    _expect(_w(stride=100), fq.EINVAL, "col_stride")
    _expect(_w(stride=(1 << 22) + 128), fq.EUNSUPPORTED, "2^22")
    _expect(_w(rows=-1), fq.EINVAL, "negative")
    _expect(_w(A=P[0] + 4), fq.EINVAL, "A and B")
    _expect(_w(sB=None), fq.EINVAL, "sA and sB")
    _expect(_w(C=P[1]), fq.EINVAL, "overlaps")


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(*s)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


X = torch.zeros(64, 256, dtype=torch.bfloat16)
C = torch.zeros(64, 128, dtype=torch.bfloat16)
BAD_CALLS = [
    (lambda: fq.fp8_quantize_grouped(X, torch.zeros(4, dtype=torch.int64), 0, q_row=u8(64, 256), s_row=f32(64, 2)),
     TypeError, "offsets must be"),
    (lambda: fq.fp8_quantize_grouped(X, None, 0, q_row=u8(64, 256), s_row=f32(64, 2)), ValueError, "offsets is"),
    (lambda: fq.fp8_quantize_grouped(X, i32(0), 0, q_row=u8(64, 256), s_row=f32(64, 2)), ValueError, "groups"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, q_row=u8(64, 255), s_row=f32(64, 2)), ValueError, "q_row"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, row_index=i32(65), q_row=u8(64, 256), s_row=f32(64, 2)),
     ValueError, "q_row"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, q_col=u8(255, 384), s_col=f32(256, 3)), ValueError, "q_col"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, q_col=u8(256, 384), s_col=f32(256, 2)), ValueError, "s_col"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, q_col=u8(256, 384)), ValueError, "s_col is required"),
    (lambda: fq.fp8_grouped_gemm(u8(64, 256), 0, f32(64, 2), u8(3, 128, 256), 0, f32(3, 1, 2), i32(3), C),
     ValueError, "shape mismatch"),
    (lambda: fq.fp8_grouped_gemm(u8(64, 256), 0, f32(64, 1), u8(3, 128, 256), 0, f32(3, 1, 2), i32(4), C),
     ValueError, "sA must have"),
    (lambda: fq.fp8_grouped_gemm(u8(64, 256), 0, f32(64, 2), u8(3, 128, 256), 0, f32(3, 1, 1), i32(4), C),
     ValueError, "sB must have"),
    (lambda: fq.fp8_grouped_gemm(u8(64, 256), 0, f32(64, 2), u8(3, 128, 256), 0, f32(3, 1, 2), i32(4), C.float()),
     TypeError, "C must be"),
    (lambda: fq.fp8_grouped_gemm_wgrad(u8(128, 384), 1, f32(128, 3), u8(256, 384), 0, f32(256, 3), i32(4),
                                       f32(2, 128, 256)), ValueError, "C must be"),
    (lambda: fq.fp8_grouped_gemm_wgrad(u8(128, 384), 1, f32(128, 3), u8(256, 256), 0, f32(256, 2), i32(4),
                                       f32(3, 128, 256)), ValueError, "one col_stride"),
    (lambda: fq.fp8_grouped_gemm_wgrad(u8(127, 384), 1, f32(128, 3), u8(256, 384), 0, f32(256, 3), i32(4),
                                       f32(3, 128, 256)), ValueError, "A must be"),
    # right sizes and types, not on the GPU
    (lambda: fq.fp8_grouped_gemm(u8(64, 256), 0, f32(64, 2), u8(3, 128, 256), 0, f32(3, 1, 2), i32(4), C),
     ValueError, "GPU tensor"),
    (lambda: fq.fp8_quantize_grouped(X, i32(4), 0, q_row=u8(64, 256), s_row=f32(64, 2)), ValueError, "GPU tensor"),
]


@pytest.mark.parametrize("i", range(len(BAD_CALLS)))
def test_binding_refuses(i):
    call, exc, fragment = BAD_CALLS[i]
    with pytest.raises(exc, match=fragment):
        call()


def test_quantize_grouped_without_rows_does_nothing():
    """An expert rank that got no tokens: the buffers are empty, so their
    addresses are null."""
    for index, x_rows, qc in ((None, 0, None), (None, 64, None), (P[1], 64, None), (None, 64, P[5])):
        assert _q(x=P[0] if x_rows else None, x_rows=x_rows, index=index, rows=0, qr=None, sr=None, qc=qc,
                  sc=P[6] if qc else None) == fq.OK, fq.last_error()
    assert _q(cols=0, qr=None, sr=None, qc=None, sc=None) == fq.OK, fq.last_error()
    # what is wrong without rows too is still refused
    _expect(_q(rows=0, dt=2), fq.EINVAL, "dtype")
    _expect(_q(rows=0, off=None), fq.EINVAL, "offsets")
    _expect(_q(rows=0, stride=500), fq.EINVAL, "col_stride")


def test_more_tiles_than_one_launch_holds():
    """Refused on the host: a launch of 2^32 lanes or more would be cut off."""
    _expect(_g(rows=1 << 16, groups=1 << 16, N=1 << 15, K=128), fq.EUNSUPPORTED, "one launch")
    _expect(_g(rows=1 << 26, groups=1, N=1 << 13, K=128), fq.EUNSUPPORTED, "one launch")
    _expect(_w(groups=1, M=1 << 20, N=1 << 19), fq.EUNSUPPORTED, "one launch")
    _expect(_w(groups=1 << 16, M=1 << 12, N=1 << 10), fq.EUNSUPPORTED, "one launch")
