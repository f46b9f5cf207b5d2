"""Ragged groups: grouped 1x128 quantization against the oracle's block
quantizer, bit for bit, and the grouped GEMMs against products in 64 bits.

GEMM tolerances, with S = sum |weighted products| of an entry: the FP8 matrix
instruction's narrow adder is within 2^-11 S (the bound of the dense GEMM
tests), binary32 sums of n terms within n 2^-24 S, the store to bf16 half a
step, 2^-8."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_util import empty_codes, empty_f32, first_mismatches, host, same_f32, to_dev

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
E4, E5 = oracle.E4M3FN, oracle.E5M2
U = 2.0 ** -24


def decode64(q, fmt):
    return oracle.decode_table(fmt).astype(np.float64)[q]


def offsets_of(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def padded_of(sizes):
    return np.concatenate([[0], np.cumsum((np.asarray(sizes, np.int64) + 127) // 128 * 128)])


def gather(x, index):
    """Rows of x (float32 or bf16 bits) in group order; zero rows for indices outside."""
    out = np.zeros((len(index), x.shape[1]), x.dtype)
    ok = (index >= 0) & (index < x.shape[0])
    out[ok] = x[index[ok]]
    return out


def pad_rows(g, sizes):
    pad, off = padded_of(sizes), offsets_of(sizes)
    out = np.zeros((int(pad[-1]), g.shape[1]), g.dtype)
    for e, n in enumerate(sizes):
        out[pad[e]:pad[e] + n] = g[off[e]:off[e] + n]
    return out


def quantize(x, index, sizes, fmt, row=True, col=True, extra=0):
    rows = len(index) if index is not None else x.shape[0]
    cols, tp = x.shape[1], int(padded_of(sizes)[-1]) + extra
    o = dict(q_row=empty_codes((rows, cols)) if row else None, s_row=empty_f32((rows, cols // 128)) if row else None,
             q_col=empty_codes((cols, tp)) if col else None, s_col=empty_f32((cols, tp // 128)) if col else None)
    fq.fp8_quantize_grouped(to_dev(x), to_dev(offsets_of(sizes)), fmt,
                            row_index=None if index is None else to_dev(index.astype(np.int32)), **o)
    return {k: None if v is None else host(v) for k, v in o.items()}


def check_quantize(x, index, sizes, fmt, row=True, col=True, extra=0):
    got = quantize(x, index, sizes, fmt, row, col, extra)
    g = gather(x, index) if index is not None else x
    n = int(np.sum(sizes))
    if row and n:
        pad = np.zeros(((n + 127) // 128 * 128, g.shape[1]), g.dtype)
        pad[:n] = g[:n]
        q, s, _, _ = oracle.quantize_block(pad, fmt, 1)
        assert np.array_equal(got["q_row"][:n], q[:n]), first_mismatches(got["q_row"][:n], q[:n])
        assert same_f32(got["s_row"][:n], s[:n])
    if col:
        p = pad_rows(g, sizes)
        tp = p.shape[0]
        if tp:
            _, _, q, s = oracle.quantize_block(p, fmt, 1)
            assert np.array_equal(got["q_col"][:, :tp], q), first_mismatches(got["q_col"][:, :tp], q)
            assert same_f32(got["s_col"][:, :tp // 128], s)
        # columns past the last group stay as they were
        assert np.all(got["q_col"][:, tp:] == 0xA5) and np.all(got["s_col"][:, tp // 128:] == -7.25)


def routed(rows, groups, seed, empty=()):
    rng = np.random.default_rng(seed)
    p = rng.random(groups) + 0.05
    p[list(empty)] = 0
    return rng.multinomial(rows, p / p.sum())


GROUPS = [[1], [0, 1, 0], [128], [127, 129], [0, 0, 300, 0], [5, 0, 130, 1, 256], list(routed(700, 64, 1)),
          list(routed(200, 130, 2))]


@pytest.mark.parametrize("k", range(len(GROUPS)))
@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("bf16", [True, False])
def test_quantize(k, fmt, bf16):
    sizes = GROUPS[k]
    n = int(np.sum(sizes))
    rng = np.random.default_rng(k)
    x = rng.standard_normal((max(3, n // 2), 384)) * 3.0
    x = workloads.to_bf16_bits(x) if bf16 else x.astype(np.float32)
    index = rng.integers(0, x.shape[0], n)
    check_quantize(x, index, sizes, fmt)


@pytest.mark.parametrize("row,col", [(True, False), (False, True), (True, True)])
def test_quantize_copies_and_identity(row, col):
    sizes = [100, 0, 57, 300]
    x = workloads.to_bf16_bits(np.random.default_rng(3).standard_normal((457, 640)))
    check_quantize(x, None, sizes, E4, row, col)
    check_quantize(x, None, sizes, E4, row, col, extra=256)


def test_quantize_special_values_and_indices_outside():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 256)) * 2).astype(np.float32)
    sp = workloads.special_values_f32()
    x[3, :len(sp)] = sp
    x[7, 200], x[9, 5], x[11] = np.inf, np.nan, 0.0
    index = rng.integers(0, 40, 200)
    index[[0, 17, 130, 199]] = [-1, 40, 2 ** 31 - 1, -2 ** 31]
    index[[5, 6, 7, 8]] = [3, 7, 9, 11]
    check_quantize(x, index, [90, 0, 110], E4)
    check_quantize(x, index, [90, 0, 110], E5, col=False)


def test_quantize_short_stride_leaves_groups_out():
    """A columnwise buffer that ends before the groups do: what fits is right."""
    x = workloads.to_bf16_bits(np.random.default_rng(6).standard_normal((400, 128)))
    sizes = [100, 300]
    qr, sr = empty_codes((400, 128)), empty_f32((400, 1))
    qc, sc = empty_codes((128, 256)), empty_f32((128, 2))
    fq.fp8_quantize_grouped(to_dev(x), to_dev(offsets_of(sizes)), E4, q_row=qr, s_row=sr, q_col=qc, s_col=sc)
    _, _, q, s = oracle.quantize_block(pad_rows(x, sizes), E4, 1)
    assert np.array_equal(host(qc), q[:, :256]) and same_f32(host(sc), s[:, :2])
    pad = np.zeros((512, 128), x.dtype)
    pad[:400] = x
    assert np.array_equal(host(qr), oracle.quantize_block(pad, E4, 1)[0][:400])


def test_offsets_out_of_range_stay_inside():
    """Offsets that decrease or leave the buffer: nothing beside the outputs changes."""
    x = workloads.to_bf16_bits(np.random.default_rng(7).standard_normal((256, 256)))
    off = np.array([-5, 300, 20, 1000, -2 ** 31, 2 ** 31 - 1], np.int32)
    buf = empty_codes((256 * 256 + 512,))
    sr, qc, sc = empty_f32((256, 2)), empty_codes((256, 512)), empty_f32((256, 4))
    fq.fp8_quantize_grouped(to_dev(x), to_dev(off), E4, q_row=buf[256:-256].view(256, 256), s_row=sr, q_col=qc,
                            s_col=sc)
    got = host(buf)
    assert np.all(got[:256] == 0xA5) and np.all(got[-256:] == 0xA5)
    a = torch.zeros(256, 256, dtype=torch.uint8, device="cuda")
    b = torch.zeros(5, 128, 256, dtype=torch.uint8, device="cuda")
    cbuf = torch.full((256 * 128 + 256,), 5.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(a, E4, torch.ones(256, 2, device="cuda"), b, E4, torch.ones(5, 1, 2, device="cuda"),
                        to_dev(off), cbuf[128:-128].view(256, 128))
    dw = torch.full((5 * 256 * 256 + 256,), 5.0, device="cuda")
    fq.fp8_grouped_gemm_wgrad(qc, E4, sc, qc.clone(), E4, sc.clone(), to_dev(off), dw[128:-128].view(5, 256, 256))
    torch.cuda.synchronize()
    for t in (cbuf, dw):
        assert torch.all(t[:128] == 5.0) and torch.all(t[-128:] == 5.0)


def operands(rows, groups, n, k, fa, fb, seed):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal(((rows + 127) // 128 * 128, k)).astype(np.float32)
    qa, sa, _, _ = oracle.quantize_block(a, fa, 1)
    w = (rng.standard_normal((groups * n, k)) * 0.02).astype(np.float32)
    qb, sb, _, _ = oracle.quantize_block(w, fb, 128)
    return qa[:rows], sa[:rows], qb.reshape(groups, n, k), sb.reshape(groups, n // 128, k // 128)


def check_gemm(sizes, n, k, fa, fb, seed=0, first=0, extra=0):
    rows, groups = first + int(np.sum(sizes)) + extra, len(sizes)
    qa, sa, qb, sb = operands(rows, groups, n, k, fa, fb, seed)
    c = torch.full((rows, n), 777.0, dtype=torch.bfloat16, device="cuda")
    off = offsets_of(sizes, first)
    fq.fp8_grouped_gemm(to_dev(qa), fa, to_dev(sa), to_dev(qb), fb, to_dev(sb), to_dev(off), c)
    got = c.float().cpu().numpy().astype(np.float64)
    for e in range(groups):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        a = decode64(qa[lo:hi], fa) * np.repeat(sa[lo:hi].astype(np.float64), 128, 1)
        b = decode64(qb[e], fb) * np.repeat(np.repeat(sb[e].astype(np.float64), 128, 0), 128, 1)
        r, s = a @ b.T, np.abs(a) @ np.abs(b).T
        tol = (2.0 ** -11 + (k + k // 128 + 8) * U) * s
        assert np.all(np.abs(got[lo:hi] - r) <= tol + 2.0 ** -8 * (np.abs(r) + tol)), (e, np.abs(got[lo:hi] - r).max())
        # far inside the bound as a whole (a wrong scale or a swapped slice is not)
        assert np.linalg.norm(got[lo:hi] - r) <= 4e-3 * np.linalg.norm(r)


GEMM_SIZES = [[1], [0, 3, 0, 0], [16, 17], [64, 1, 63], [128, 0, 127, 129], [255, 257, 1], [40] * 9,
              list(routed(900, 33, 4)), [600, 0, 20], [1] * 70]


@pytest.mark.parametrize("k", range(len(GEMM_SIZES)))
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4)])
def test_gemm_groups(k, fa, fb):
    check_gemm(GEMM_SIZES[k], 256, 384, fa, fb, seed=k)


@pytest.mark.parametrize("n,kk", [(128, 128), (128, 1024), (640, 256), (384, 2176), (1024, 128)])
@pytest.mark.parametrize("sizes", [[2, 0, 5], [70, 300, 9]])
def test_gemm_shapes(n, kk, sizes):
    check_gemm(sizes, n, kk, E4, E4, seed=n + kk)


@pytest.mark.parametrize("fa,fb", [(E4, E5), (E5, E5)])
def test_gemm_other_formats(fa, fb):
    check_gemm([30, 200], 256, 256, fa, fb)


# one launch per tile that the rule on rows, groups and N picks (16 x 16 to
# 128 x 128 blocks, the large tiles with full, half and one-row remainders), with
# one, few, odd and even numbers of slices
TILE_CASES = [([9, 0, 3], 128, 384), ([8] * 40, 256, 128), ([33, 7], 4096, 128), ([128], 4096, 256),
              ([100, 141], 4096, 384), ([700, 130, 0, 1000, 170], 1152, 128), ([257, 1, 900, 384, 129], 1152, 384),
              ([1100, 256, 512, 128], 1024, 640), ([2300], 896, 1152), ([1] * 30 + [1500, 0, 700], 1024, 256)]


@pytest.mark.parametrize("k", range(len(TILE_CASES)))
def test_gemm_tiles(k):
    sizes, n, kk = TILE_CASES[k]
    check_gemm(sizes, n, kk, E5 if k % 2 else E4, E4, seed=50 + k)


def test_gemm_large_tiles_exact():
    """Small integers and unit scales through the large tiles: every entry exact."""
    rng = np.random.default_rng(18)
    sizes, n, k = [700, 0, 131, 1290, 18, 256], 1152, 640
    rows, groups = sum(sizes), len(sizes)
    ai, bi = rng.integers(-2, 3, (rows, k)), rng.integers(-2, 3, (groups, n, k))
    sa = 2.0 ** rng.integers(-1, 2, (rows, k // 128))
    sb = 2.0 ** rng.integers(-1, 2, (groups, n // 128, k // 128))
    c = torch.full((rows + 2, n), 777.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(to_dev(oracle.encode(E4, ai.astype(np.float32))), E4, to_dev(sa.astype(np.float32)),
                        to_dev(oracle.encode(E4, bi.astype(np.float32))), E4, to_dev(sb.astype(np.float32)),
                        to_dev(offsets_of(sizes)), c[1:-1])
    off = offsets_of(sizes)
    for e in range(groups):
        a = ai[off[e]:off[e + 1]] * np.repeat(sa[off[e]:off[e + 1]], 128, 1)
        b = bi[e] * np.repeat(np.repeat(sb[e], 128, 0), 128, 1)
        assert torch.equal(c[1 + off[e]:1 + off[e + 1]].cpu(), torch.from_numpy(a @ b.T).to(torch.bfloat16)), e
    assert torch.all(c[0] == 777.0) and torch.all(c[-1] == 777.0)


def test_gemm_rows_of_no_group():
    check_gemm([30, 0, 41], 128, 256, E4, E4, first=9, extra=13)


def test_gemm_exact_integers():
    """Small integers and unit scales: every entry exact, so a misplaced row,
    column, slice or scale shows."""
    rng = np.random.default_rng(8)
    sizes, n, k = [3, 0, 131, 290, 18], 384, 512
    rows, groups = sum(sizes), len(sizes)
    ai, bi = rng.integers(-2, 3, (rows, k)), rng.integers(-2, 3, (groups, n, k))
    sa = 2.0 ** rng.integers(-1, 2, (rows, k // 128))
    sb = 2.0 ** rng.integers(-1, 2, (groups, n // 128, k // 128))
    c = torch.full((rows, n), 777.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(to_dev(oracle.encode(E4, ai.astype(np.float32))), E4, to_dev(sa.astype(np.float32)),
                        to_dev(oracle.encode(E4, bi.astype(np.float32))), E4, to_dev(sb.astype(np.float32)),
                        to_dev(offsets_of(sizes)), c)
    off = offsets_of(sizes)
    for e in range(groups):
        a = ai[off[e]:off[e + 1]] * np.repeat(sa[off[e]:off[e + 1]], 128, 1)
        b = bi[e] * np.repeat(np.repeat(sb[e], 128, 0), 128, 1)
        want = torch.from_numpy(a @ b.T).to(torch.bfloat16)
        assert torch.equal(c[off[e]:off[e + 1]].cpu(), want), e


def test_gemm_no_rows_and_no_groups():
    b = torch.zeros(2, 128, 128, dtype=torch.uint8, device="cuda")
    fq.fp8_grouped_gemm(torch.empty(0, 128, dtype=torch.uint8, device="cuda"), E4, torch.empty(0, 1, device="cuda"), b,
                        E4, torch.ones(2, 1, 1, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                        torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))


def check_wgrad(sizes, m, n, fa, fb, dtype, seed=0, extra=0):
    rng = np.random.default_rng(seed)
    rows, groups = int(np.sum(sizes)), len(sizes)
    dy = (rng.standard_normal((max(rows, 1), m)) * 1e-3).astype(np.float32)
    x = rng.standard_normal((max(rows, 1), n)).astype(np.float32)
    tp = int(padded_of(sizes)[-1]) + extra
    qa, sa, qb, sb = empty_codes((m, tp)), empty_f32((m, tp // 128)), empty_codes((n, tp)), empty_f32((n, tp // 128))
    off = to_dev(offsets_of(sizes))
    fq.fp8_quantize_grouped(to_dev(dy), off, fa, q_col=qa, s_col=sa)
    fq.fp8_quantize_grouped(to_dev(x), off, fb, q_col=qb, s_col=sb)
    c = torch.full((groups, m, n), 777.0, dtype=dtype, device="cuda")
    fq.fp8_grouped_gemm_wgrad(qa, fa, sa, qb, fb, sb, off, c)
    got = c.double().cpu().numpy()
    A, SA, B, SB = host(qa), host(sa), host(qb), host(sb)
    pad = padded_of(sizes)
    for e in range(groups):
        lo, hi = int(pad[e]), int(pad[e + 1])
        if lo == hi:
            assert np.all(got[e] == 0)
            continue
        a = decode64(A[:, lo:hi], fa) * np.repeat(SA[:, lo // 128:hi // 128].astype(np.float64), 128, 1)
        b = decode64(B[:, lo:hi], fb) * np.repeat(SB[:, lo // 128:hi // 128].astype(np.float64), 128, 1)
        r, s = a @ b.T, np.abs(a) @ np.abs(b).T
        k = hi - lo
        if dtype == torch.float32:
            assert np.all(np.abs(got[e] - r) <= (k + k // 128 + 2) * U * s)
            assert np.linalg.norm(got[e] - r) <= 2e-6 * np.linalg.norm(r)
        else:
            tol = (2.0 ** -11 + (k + k // 128 + 2) * U) * s
            assert np.all(np.abs(got[e] - r) <= tol + 2.0 ** -8 * (np.abs(r) + tol))
            assert np.linalg.norm(got[e] - r) <= 4e-3 * np.linalg.norm(r)


@pytest.mark.parametrize("sizes", [[1], [0, 128, 0], [129, 1, 0, 300], list(routed(900, 17, 9)), [0, 0], [1500]])
@pytest.mark.parametrize("fa,fb", [(E5, E4), (E4, E4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_groups(sizes, fa, fb, dtype):
    check_wgrad(sizes, 256, 384, fa, fb, dtype, seed=len(sizes), extra=128)


@pytest.mark.parametrize("m,n", [(128, 128), (384, 128), (128, 640), (768, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_shapes(m, n, dtype):
    check_wgrad([200, 0, 77], m, n, E5, E4, dtype, seed=m + n)


@pytest.mark.parametrize("fa,fb", [(E4, E5), (E5, E5)])
def test_wgrad_other_formats(fa, fb):
    for dtype in (torch.float32, torch.bfloat16):
        check_wgrad([130, 40], 128, 256, fa, fb, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_exact_integers(dtype):
    """Small integers and unit scales over many slices: every entry exact."""
    rng = np.random.default_rng(19)
    sizes, m, n = [700, 0, 131, 1, 1290], 384, 640
    pad = padded_of(sizes)
    tp = int(pad[-1]) + 256
    ai, bi = np.zeros((m, tp), int), np.zeros((n, tp), int)
    for e, rows in enumerate(sizes):
        ai[:, pad[e]:pad[e] + rows] = rng.integers(-2, 3, (m, rows))
        bi[:, pad[e]:pad[e] + rows] = rng.integers(-2, 3, (n, rows))
    sa, sb = 2.0 ** rng.integers(-1, 2, (m, tp // 128)), 2.0 ** rng.integers(-1, 2, (n, tp // 128))
    c = torch.full((len(sizes), m, n), 777.0, dtype=dtype, device="cuda")
    fq.fp8_grouped_gemm_wgrad(to_dev(oracle.encode(E5, ai.astype(np.float32))), E5, to_dev(sa.astype(np.float32)),
                              to_dev(oracle.encode(E4, bi.astype(np.float32))), E4, to_dev(sb.astype(np.float32)),
                              to_dev(offsets_of(sizes)), c)
    for e in range(len(sizes)):
        s = slice(int(pad[e]), int(pad[e + 1]))
        sc = slice(int(pad[e]) // 128, int(pad[e + 1]) // 128)
        want = (ai[:, s] * np.repeat(sa[:, sc], 128, 1)) @ (bi[:, s] * np.repeat(sb[:, sc], 128, 1)).T
        assert torch.equal(c[e].cpu(), torch.from_numpy(want).to(dtype)), e


def test_wgrad_every_code_is_widened_exactly():
    """One token per code: dW = value(code) of both formats, bit for bit, in fp32."""
    for f in (E4, E5):
        codes = np.arange(256, dtype=np.uint8)
        fin = np.isfinite(oracle.decode_table(f)[codes])
        codes = codes[fin]
        m = 256
        a = np.zeros((m, 128), np.uint8)
        a[:len(codes), 5] = codes
        b = np.zeros((128, 128), np.uint8)
        b[:, 5] = oracle.encode(E4, np.ones(128, np.float32))
        c = torch.zeros(1, m, 128, device="cuda")
        fq.fp8_grouped_gemm_wgrad(to_dev(a), f, torch.ones(m, 1, device="cuda"), to_dev(b), E4,
                                  torch.ones(128, 1, device="cuda"), to_dev(offsets_of([100])), c)
        want = oracle.decode_table(f)[codes].astype(np.float32)
        assert np.array_equal(host(c)[0, :len(codes), 0], want)


def test_nonfinite_codes_stay_in_their_rows():
    """NaN codes of one token reach its row of C and no other."""
    qa, sa, qb, sb = operands(50, 2, 128, 256, E4, E4, 3)
    qa = qa.copy()
    qa[[4, 33], 9] = 0x7F
    c = torch.zeros(50, 128, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(to_dev(qa), E4, to_dev(sa), to_dev(qb), E4, to_dev(sb), to_dev(offsets_of([20, 30])), c)
    bad = torch.isnan(c.float()).all(1).cpu().numpy()
    assert np.array_equal(np.nonzero(bad)[0], [4, 33])
    assert not torch.isnan(c.float()).any(1).cpu().numpy()[~bad].any()


def test_streams_and_graph_replay():
    """Quantize, multiply and the weight gradient captured together, replayed
    with new routing on another stream's graph; every replay equals the eager run."""
    rng = np.random.default_rng(12)
    sizes = [[40, 0, 300], [100, 239, 1], [0, 340, 0]]
    rows, d, n, tp = 340, 256, 384, 340 // 128 * 128 + 3 * 128
    x = to_dev(workloads.to_bf16_bits(rng.standard_normal((rows, d))))
    _, _, qb, sb = operands(128, 3, n, d, E4, E4, 1)
    qb, sb = to_dev(qb), to_dev(sb)
    off = to_dev(offsets_of(sizes[0]))
    idx = to_dev(rng.permutation(rows).astype(np.int32))
    mk = lambda: dict(qr=empty_codes((rows, d)), sr=empty_f32((rows, 2)), qc=empty_codes((d, tp), 0),  # noqa: E731
                      sc=empty_f32((d, tp // 128)), c=torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"),
                      w=torch.zeros(3, d, d, device="cuda"))

    def step(o):
        fq.fp8_quantize_grouped(x, off, E4, row_index=idx, q_row=o["qr"], s_row=o["sr"], q_col=o["qc"], s_col=o["sc"])
        fq.fp8_grouped_gemm(o["qr"], E4, o["sr"], qb, E4, sb, off, o["c"])
        fq.fp8_grouped_gemm_wgrad(o["qc"], E4, o["sc"], o["qc2"], E4, o["sc2"], off, o["w"])

    outs = [mk(), mk()]
    for o in outs:  # X against itself
        o["qc2"], o["sc2"] = o["qc"], o["sc"]
    step(outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs[0])
    for s in sizes + sizes[:1]:
        off.copy_(to_dev(offsets_of(s)))
        idx.copy_(to_dev(rng.permutation(rows).astype(np.int32)))
        g.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(outs[1])
        torch.cuda.synchronize()
        used = int(padded_of(s)[-1])
        assert torch.equal(outs[0]["qr"], outs[1]["qr"])
        assert torch.equal(outs[0]["qc"][:, :used], outs[1]["qc"][:, :used])
        assert torch.equal(outs[0]["c"], outs[1]["c"]) and torch.equal(outs[0]["w"], outs[1]["w"])


def test_quantize_no_rows():
    """No token for any expert of this rank: every buffer is empty."""
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    for x, index in ((torch.empty(0, 256, device="cuda"), None),
                     (torch.ones(9, 256, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))):
        fq.fp8_quantize_grouped(x, off, E4, row_index=index, q_row=e(0, 256), s_row=f(0, 2))
        fq.fp8_quantize_grouped(x, off, E4, row_index=index, q_row=e(0, 256), s_row=f(0, 2), q_col=e(256, 0),
                                s_col=f(256, 0))
        qc, sc = empty_codes((256, 384)), empty_f32((256, 3))
        fq.fp8_quantize_grouped(x, off, E4, row_index=index, q_col=qc, s_col=sc)
        assert torch.all(qc == 0xA5) and torch.all(sc == -7.25)
    dw = torch.full((3, 256, 128), 5.0, device="cuda")
    fq.fp8_grouped_gemm_wgrad(e(256, 0), E5, f(256, 0), e(128, 0), E4, f(128, 0), off, dw)
    assert not dw.any()
