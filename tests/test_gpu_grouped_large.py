"""The expert-layer operators past 2^31 elements, where every offset must be
64-bit, and with more groups than a wave has lanes through the large tiles.
Samples across the whole range, the ends included, against 64 bits; tolerances
as in the small tests of the same operator."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
E4, E5 = oracle.E4M3FN, oracle.E5M2
U = 2.0 ** -24


def codes(gen, *shape):
    """Finite codes of both formats: bit 3 clear leaves out E4M3's NaN, bit 6 clear E5M2's top."""
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8) & 0xB7


def scales(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda") + 0.5


def offsets(sizes):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()


def value(q, fmt):
    return oracle.decode_table(fmt).astype(np.float64)[host(q)]


def close(got, a, b, k, bf16=True):
    """got against the weighted operands' product."""
    r, s = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (k + k // 128 + 8) * U * s
    if bf16:
        tol = tol + 2.0 ** -11 * s
        tol = tol + 2.0 ** -8 * (np.abs(r) + tol)
    g = got.double().cpu().numpy()
    assert np.all(np.abs(g - r) <= tol)
    assert np.linalg.norm(g - r) <= (4e-3 if bf16 else 2e-6) * np.linalg.norm(r)


def check_rows(sizes, n, k, sample, columns, fa=E4):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    rows, groups = int(np.sum(sizes)), len(sizes)
    a, sa = codes(gen, rows, k), scales(gen, rows, k // 128)
    b, sb = codes(gen, groups, n, k), scales(gen, groups, n // 128, k // 128)
    c = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    off = offsets(sizes)
    fq.fp8_grouped_gemm(a, fa, sa, b, E4, sb, off, c)
    group = np.repeat(np.arange(groups), sizes)
    for e in np.unique(group[sample]):
        t = torch.from_numpy(sample[group[sample] == e]).cuda()
        wa = value(a[t], fa) * np.repeat(host(sa[t]).astype(np.float64), 128, 1)
        col = torch.from_numpy(columns).cuda()
        wb = value(b[int(e)][col], E4) * np.repeat(host(sb[int(e)][col // 128]).astype(np.float64), 128, 1)
        close(c[t][:, col], wa, wb, k)


def test_gemm_output_past_2_31_elements():
    sizes = [40000, 0, 30001]
    rng = np.random.default_rng(1)
    sample = np.unique(np.concatenate([rng.integers(0, 70001, 40), np.arange(69990, 70001), [0, 39999, 40000]]))
    check_rows(sizes, 32896, 128, sample, np.arange(32896))


@pytest.mark.parametrize("per", [2, 300])  # small tiles and large ones
def test_gemm_weights_past_2_32_bytes(per):
    sizes = [per] * 33
    sample = np.array([0, 1, per * 16, per * 31 + 1, per * 33 - 1])
    columns = np.concatenate([np.arange(0, 8192, 61), np.arange(8128, 8192)])
    check_rows(sizes, 8192, 16384, sample, columns)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_output_past_2_31_elements(dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)
    sizes = np.random.default_rng(3).integers(0, 300, 33)
    sizes[[4, 32]] = 0, 130
    pad = np.concatenate([[0], np.cumsum((sizes + 127) // 128 * 128)])
    m, n, tp = 16512, 4096, int(pad[-1])
    a, sa, b, sb = codes(gen, m, tp), scales(gen, m, tp // 128), codes(gen, n, tp), scales(gen, n, tp // 128)
    c = torch.full((33, m, n), 7.0, dtype=dtype, device="cuda")
    fq.fp8_grouped_gemm_wgrad(a, E5, sa, b, E4, sb, offsets(sizes), c)
    row = torch.from_numpy(np.concatenate([np.arange(0, m, 1031), np.arange(m - 9, m)])).cuda()
    assert not c[4].any()
    for e in (0, 15, 31, 32):
        lo, hi = int(pad[e]), int(pad[e + 1])
        wa = value(a[row][:, lo:hi], E5) * np.repeat(host(sa[row][:, lo // 128:hi // 128]).astype(np.float64), 128, 1)
        wb = value(b[:, lo:hi], E4) * np.repeat(host(sb[:, lo // 128:hi // 128]).astype(np.float64), 128, 1)
        close(c[e][row], wa, wb, hi - lo, dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_more_groups_than_lanes(dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    sizes = np.random.default_rng(4).integers(0, 200, 150)
    pad = np.concatenate([[0], np.cumsum((sizes + 127) // 128 * 128)])
    m, n, tp = 384, 256, int(pad[-1])
    a, sa, b, sb = codes(gen, m, tp), scales(gen, m, tp // 128), codes(gen, n, tp), scales(gen, n, tp // 128)
    c = torch.full((150, m, n), 7.0, dtype=dtype, device="cuda")
    fq.fp8_grouped_gemm_wgrad(a, E5, sa, b, E4, sb, offsets(sizes), c)
    wa = value(a, E5) * np.repeat(host(sa).astype(np.float64), 128, 1)
    wb = value(b, E4) * np.repeat(host(sb).astype(np.float64), 128, 1)
    for e in range(150):
        lo, hi = int(pad[e]), int(pad[e + 1])
        if lo == hi:
            assert not c[e].any()
        else:
            close(c[e], wa[:, lo:hi], wb[:, lo:hi], hi - lo, dtype == torch.bfloat16)


def test_gemm_more_groups_than_lanes_in_large_tiles():
    sizes = np.random.default_rng(5).integers(100, 500, 80)
    sample = np.arange(0, int(sizes.sum()), 97)
    check_rows(list(sizes), 1024, 256, sample, np.arange(1024), fa=E5)


def test_gemm_without_a_contraction_is_zero():
    for rows, n in ((5, 256), (3000, 1024)):
        none = torch.empty(0, device="cuda")
        c = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
        fq.fp8_grouped_gemm(torch.empty(rows, 0, dtype=torch.uint8, device="cuda"), E4, none,
                            torch.empty(2, n, 0, dtype=torch.uint8, device="cuda"), E4, none,
                            offsets([rows // 3, rows - rows // 3]), c)
        assert not c.any()


def test_quantize_past_2_31_codes():
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5000, 4096, generator=gen, device="cuda").to(torch.bfloat16)
    rows, sizes = 540001, [300000, 0, 240001]
    index = torch.randint(0, 5000, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    stride = 300032 + 240128
    q, s = torch.empty(rows, 4096, dtype=torch.uint8, device="cuda"), torch.empty(rows, 32, device="cuda")
    qc, sc = torch.empty(4096, stride, dtype=torch.uint8, device="cuda"), torch.empty(4096, stride // 128, device="cuda")
    fq.fp8_quantize_grouped(x, offsets(sizes), E4, row_index=index, q_row=q, s_row=s, q_col=qc, s_col=sc)
    # the oracle's codes are those of the small tests; here the rows of x once
    q1, s1 = torch.empty(5000, 4096, dtype=torch.uint8, device="cuda"), torch.empty(5000, 32, device="cuda")
    fq.fp8_quantize_grouped(x, offsets([5000]), E4, q_row=q1, s_row=s1)
    for lo in range(0, rows, 60000):
        i = index[lo:lo + 60000].long()
        assert torch.equal(q[lo:lo + 60000], q1[i]) and torch.equal(s[lo:lo + 60000], s1[i])
    q.zero_()
    fq.fp8_quantize_grouped(x, offsets(sizes), E4, row_index=index, q_row=q, s_row=s)
    for lo in range(0, rows, 60000):
        assert torch.equal(q[lo:lo + 60000], q1[index[lo:lo + 60000].long()])
    for first, n in ((0, 128), (299904, 96), (300000, 128), (540000, 1)):
        c2, s2 = torch.empty(4096, 128, dtype=torch.uint8, device="cuda"), torch.empty(4096, 1, device="cuda")
        fq.fp8_quantize_grouped(x, offsets([n]), E4, row_index=index[first:first + n].contiguous(), q_col=c2, s_col=s2)
        at = first if first < 300000 else first + 32
        assert torch.equal(qc[:, at:at + 128], c2) and torch.equal(sc[:, at // 128:at // 128 + 1], s2)


def test_layernorm_past_2_31_elements():
    """A block of rows repeated: every repeat has the block's results, and the
    parameter gradients are those of the block times the repeats."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    block, reps, cols = 6000, 90, 4096
    x1 = torch.randn(block, cols, generator=gen, device="cuda").to(torch.bfloat16)
    d1 = torch.randn(block, cols, generator=gen, device="cuda").to(torch.bfloat16)
    gamma, beta = torch.rand(cols, generator=gen, device="cuda") + 0.5, torch.randn(cols, generator=gen, device="cuda")

    def run(x, dy):
        rows = x.shape[0]
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        ws = torch.empty(fq.fp8q_layernorm_backward_workspace(fq.BF16, rows, cols) // 4 + 1, device="cuda")
        fq.fp8q_layernorm(x, gamma, beta, 1e-5, y, mean, rstd)
        fq.fp8q_layernorm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws)
        return y, dx, mean, rstd, dg, db

    small, big = run(x1, d1), run(x1.repeat(reps, 1), d1.repeat(reps, 1))
    for a, b in zip(big[:4], small[:4]):
        assert all(torch.equal(a[i * block:(i + 1) * block], b) for i in range(reps))
    # a term is off by a few 2^-24, and a sum of 540000 of them in 1024 or more
    # partial sums by at most (540000 / 1024 + 1024 + 8) 2^-24 of their magnitudes
    x64, d64 = x1.double(), d1.double()
    xhat = (x64 - x64.mean(1, keepdim=True)) * torch.rsqrt(x64.var(1, unbiased=False, keepdim=True) + 1e-5)
    for got, terms in ((big[4], d64 * xhat), (big[5], d64)):
        err = (got.double() - reps * terms.sum(0)).abs()
        assert torch.all(err <= (540000 / 1024 + 1024 + 8) * U * reps * terms.abs().sum(0))


def test_clip_past_2_31_elements():
    n = (1 << 31) + 1029
    g = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    g[-1], g[(1 << 31) + 5] = 3.0, -5.0
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    want = np.sqrt((n - 2) * 2.0 ** -20 + 34.0)
    fq.fp8q_grad_norm_clip([g], 1.0, norm, coef)
    assert abs(float(norm) - want) <= 2 * U * want
    c = float(coef)
    assert abs(c - 1 / (want + 1e-6)) <= 4 * U * c
    for i, v in ((0, 2.0 ** -10), (n // 2, 2.0 ** -10), (n - 2, 2.0 ** -10), (n - 1, 3.0), ((1 << 31) + 5, -5.0)):
        assert abs(float(g[i]) - v * c) <= 2.0 ** -8 * abs(v * c) * (1 + 1e-3)
    assert int((g == g[0]).sum()) == n - 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[2000], [0, 1500, 130], [128 * 13], [700, 1, 900, 4000], [127 + 128 * 8]])
def test_wgrad_of_few_tiles(sizes, dtype):
    """Few tiles over many slices: quarters of the contraction of equal and of
    unequal length, empty ones among them."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    pad = np.concatenate([[0], np.cumsum((np.asarray(sizes) + 127) // 128 * 128)])
    for m, n in ((128, 128), (384, 256)):
        tp = int(pad[-1]) + 128
        a, sa, b, sb = codes(gen, m, tp), scales(gen, m, tp // 128), codes(gen, n, tp), scales(gen, n, tp // 128)
        buf = torch.full((len(sizes) * m * n + 256,), 7.0, dtype=dtype, device="cuda")
        c = buf[128:-128].view(len(sizes), m, n)
        fq.fp8_grouped_gemm_wgrad(a, E5, sa, b, E4, sb, offsets(sizes), c)
        wa = value(a, E5) * np.repeat(host(sa).astype(np.float64), 128, 1)
        wb = value(b, E4) * np.repeat(host(sb).astype(np.float64), 128, 1)
        for e in range(len(sizes)):
            lo, hi = int(pad[e]), int(pad[e + 1])
            if lo == hi:
                assert not c[e].any()
            else:
                close(c[e], wa[:, lo:hi], wb[:, lo:hi], hi - lo, dtype == torch.bfloat16)
        assert torch.all(buf[:128] == 7.0) and torch.all(buf[-128:] == 7.0)
        again = torch.empty_like(c)
        fq.fp8_grouped_gemm_wgrad(a, E5, sa, b, E4, sb, offsets(sizes), again)
        assert torch.equal(c, again)


@pytest.mark.parametrize("k", [128, 384, 1920, 2048, 3968, 4096, 4224])
def test_gemm_few_rows_over_long_contractions(k):
    """Fewer, as many and more slices than the waves that share a tile's contraction."""
    sizes = [1, 0, 9, 16, 17, 3] * 4
    check_rows(sizes, 2048, k, np.arange(sum(sizes)), np.arange(0, 2048, 3))


@pytest.mark.parametrize("k", [128, 256, 640, 1152, 2048, 2176])
@pytest.mark.parametrize("sizes,n", [([130, 0, 61, 128, 257, 100], 1024), ([900, 1100], 512), ([90, 120, 70], 4096)])
def test_gemm_of_few_tiles(sizes, n, k):
    """Few tiles whose slices two halves of a block share: one, odd and even numbers of slices."""
    check_rows(sizes, n, k, np.arange(sum(sizes)), np.arange(0, n, 5), fa=E5 if k % 512 else E4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_of_offsets_whose_blocks_pass_32_bits(dtype):
    """Offsets that fall back to 0 after every group, over many more rows than
    the copies have columns: the blocks before a group number up to 2^32.  The
    first group's block is in the copies, all others lie past them."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    groups, rows = 65536, 1 << 24
    a, sa, b, sb = codes(gen, 128, 128), scales(gen, 128, 1), codes(gen, 128, 128), scales(gen, 128, 1)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    buf = torch.full((groups * 128 * 128 + 256,), 7.0, dtype=dtype, device="cuda")
    c = buf[128:-128].view(groups, 128, 128)
    status = fq.lib.fp8_grouped_gemm_wgrad(a.data_ptr(), E5, sa.data_ptr(), b.data_ptr(), E4, sb.data_ptr(),
                                           off.data_ptr(), groups, rows, 128, 128, 128, c.data_ptr(),
                                           fq.F32 if dtype == torch.float32 else fq.BF16,
                                           torch.cuda.current_stream().cuda_stream)
    assert status == fq.OK, fq.last_error()
    wa = value(a, E5) * np.repeat(host(sa).astype(np.float64), 128, 1)
    wb = value(b, E4) * np.repeat(host(sb).astype(np.float64), 128, 1)
    close(c[0], wa, wb, 128, dtype == torch.bfloat16)
    assert not c[1:].any()
    assert torch.all(buf[:128] == 7.0) and torch.all(buf[-128:] == 7.0)


def test_quantize_more_tiles_than_one_launch_holds():
    """65536 groups, a few of them with rows: tiles for all that offsets could
    ask for, more than 2^32 lanes.  Codes and scales of both copies against the same
    rows quantized as the only group, which takes few tiles."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    rows, groups, cols = 65536, 65536, 32896
    x = torch.randn(64, cols, generator=gen, device="cuda").to(torch.bfloat16)
    index = torch.randint(0, 64, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    sizes = np.zeros(groups, np.int64)
    sizes[[0, 5, 40000, 65535]] = 20001, 1, 30000, 15534
    pad = np.concatenate([[0], np.cumsum((sizes + 127) // 128 * 128)])
    u8 = lambda *s: torch.full(s, 0xA5, dtype=torch.uint8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.full(s, -7.25, device="cuda")  # noqa: E731
    q, s, qc, sc = u8(rows, cols), f32(rows, cols // 128), u8(cols, int(pad[-1])), f32(cols, int(pad[-1]) // 128)
    fq.fp8_quantize_grouped(x, offsets(sizes), E4, row_index=index, q_row=q, s_row=s, q_col=qc, s_col=sc)
    first = np.concatenate([[0], np.cumsum(sizes)])
    for e in (0, 5, 40000, 65535):
        lo, hi, p0, p1 = int(first[e]), int(first[e + 1]), int(pad[e]), int(pad[e + 1])
        wq, ws = u8(hi - lo, cols), f32(hi - lo, cols // 128)
        wqc, wsc = u8(cols, p1 - p0), f32(cols, (p1 - p0) // 128)
        fq.fp8_quantize_grouped(x, offsets([hi - lo]), E4, row_index=index[lo:hi].clone(), q_row=wq, s_row=ws,
                                q_col=wqc, s_col=wsc)
        assert torch.equal(q[lo:hi], wq) and torch.equal(s[lo:hi], ws), e
        assert torch.equal(qc[:, p0:p1], wqc) and torch.equal(sc[:, p0 // 128:p1 // 128], wsc), e


def test_gemm_more_small_tiles_than_one_launch_holds():
    """One row a group on average over 65536 groups: the 16-row tiles that few
    rows take would be more than 2^32 lanes.  Only groups with rows have weights
    written; the others' are never read."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    rows, groups, n, k = 65536, 65536, 8320, 128
    sizes = np.zeros(groups, np.int64)
    live = [0, 5, 40000, 65535]
    sizes[live] = 20001, 1, 30000, 15534
    a, sa, sb = codes(gen, rows, k), scales(gen, rows, 1), scales(gen, groups, n // 128, 1)
    b = torch.empty(groups, n, k, dtype=torch.uint8, device="cuda")
    for e in live:
        b[e] = codes(gen, n, k)
    c = torch.full((rows, n), 777.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(a, E4, sa, b, E4, sb, offsets(sizes), c)
    col = np.concatenate([np.arange(0, n, 129), [n - 1]])
    first = np.concatenate([[0], np.cumsum(sizes)])
    for e in live:
        lo, hi = int(first[e]), int(first[e + 1])
        t = np.unique(np.concatenate([np.arange(lo, hi, 1009), [hi - 1]]))
        wa = value(a[torch.from_numpy(t).cuda()], E4) * host(sa)[t].astype(np.float64)
        wb = value(b[e][torch.from_numpy(col).cuda()], E4) * host(sb[e])[col // 128].astype(np.float64)
        close(c[torch.from_numpy(t).cuda()][:, torch.from_numpy(col).cuda()], wa, wb, k)
    del b, c
    torch.cuda.empty_cache()  # 70 GB that no other test takes
