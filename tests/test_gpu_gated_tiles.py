"""The gated product over long contractions, in each of its tiles: the 64-row
tiles hold all scales of a tile in LDS and end at 112 slices of 128.  Which tiles a
size runs in is asked of the workspace, which only the 16-row ones need.

g and u of the other tiles are fp8_scaled_gemm's binary32 results bit for bit, so
codes, scales and ReLU's h follow from those exactly; those, and the 16-row tiles'
sums, are within (2^-11 + (K + K / 128 + 18) 2^-24) S of the 64-bit ones, S the sum of
the products' magnitudes (the FP8 instruction's narrow adder, binary32 sums); a code
is within half a step, 2^-4 of its value (E4M3) or 2^-10 of the scale."""
import pytest
import torch

from gpu_util import host
from test_gpu_gated import check_rows

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
E4, RELU = fq.E4M3FN, fq.ACT_RELU
U = 2.0 ** -24

# rows of the groups, F, K, whether in 16-row tiles
CASES = [([64, 65], 1024, 14336, False),   # 64 rows, 112 slices: all that they hold
         ([64, 65], 1024, 14208, False),   # 111
         ([301], 1024, 4096, False),       # 64 rows, 32 slices
         ([150, 0, 80, 1], 1024, 4096, False),
         ([33, 33, 33], 2048, 8192, False),
         ([129], 2048, 14464, False),      # 113 slices: large tiles
         ([300, 1, 128], 1024, 16384, False),
         ([64, 65], 1024, 14464, True),    # 16 rows
         ([3, 0, 9], 256, 16384, True)]


def codes(gen, *shape):
    """Finite E4M3 codes of either sign, exponents around 1."""
    q = torch.randint(0x28, 0x48, shape, generator=gen, device="cuda", dtype=torch.uint8)
    return q | (torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.uint8) << 7)


def scales(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda") * 0.05 + 0.01


@pytest.mark.parametrize("k", range(len(CASES)))
def test_long_contractions(k):
    sizes, F, K, few = CASES[k]
    rows, groups, gen = sum(sizes), len(sizes), torch.Generator(device="cuda").manual_seed(k)
    assert (fq.fp8_gated_gemm_workspace(rows, groups, F, K) > 0) == few
    a, sa = codes(gen, rows, K), scales(gen, rows, K // 128)
    b, sb = codes(gen, groups, 2 * F, K), scales(gen, groups, 2 * F // 128, K // 128)
    off = torch.tensor([sum(sizes[:e]) for e in range(groups + 1)], dtype=torch.int32, device="cuda")
    size = fq.fp8_gated_gemm_workspace(rows, groups, F, K)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    H, q_gu = torch.empty(rows, F, device="cuda"), torch.empty(rows, 2 * F, dtype=torch.uint8, device="cuda")
    s_gu = torch.empty(rows, 2 * F // 128, device="cuda")
    fq.fp8_gated_gemm(a, E4, sa, b, E4, sb, RELU, offsets=off, H=H, q_gu=q_gu, s_gu=s_gu, workspace=ws)
    for e in range(groups):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        x = a[lo:hi].view(torch.float8_e4m3fn).float().double() * sa[lo:hi].double().repeat_interleave(128, 1)
        w = b[e].view(torch.float8_e4m3fn).float().double() * sb[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        want, most = x @ w.t(), x.abs() @ w.abs().t()
        tol = (2.0 ** -11 + (K + K // 128 + 18) * U) * most
        each = s_gu[lo:hi].double().repeat_interleave(128, 1)
        gu = q_gu[lo:hi].view(torch.float8_e4m3fn).float().double() * each
        half = (2.0 ** -4 + 4 * U) * (want.abs() + tol) + 2.0 ** -10 * each
        assert bool(((gu - want).abs() <= tol + half).all())
        h = want[:, :F].clamp_min(0) * want[:, F:]
        off_h = tol[:, :F] * (want[:, F:].abs() + tol[:, F:]) + want[:, :F].abs() * tol[:, F:] + U * h.abs()
        assert bool(((H[lo:hi].double() - h).abs() <= off_h).all())
        if few:
            continue
        n = (hi - lo + 127) // 128 * 128
        pa, ps = torch.zeros(n, K, dtype=torch.uint8, device="cuda"), torch.ones(n, K // 128, device="cuda")
        pa[:hi - lo], ps[:hi - lo] = a[lo:hi], sa[lo:hi]
        c = torch.empty(n, 2 * F, device="cuda")
        fq.fp8_scaled_gemm(pa, E4, ps, b[e], E4, sb[e], fq.BLOCK_1x128_128x128, c)
        c = c[:hi - lo].contiguous()
        assert bool(((c.double() - want).abs() <= tol).all())
        check_rows(host(q_gu[lo:hi]), host(s_gu[lo:hi]), host(c), E4)
        assert torch.equal(H[lo:hi], torch.where(c[:, :F] < 0, 0.0, c[:, :F]) * c[:, F:])


@pytest.mark.parametrize("rows", [3, 4100])  # 16-row tiles, and the large ones
def test_the_longest_contraction(rows):
    """K = 2^22, 32768 slices: rows at both ends against fp8_scaled_gemm, whose order of
    the slices' sums the large tiles have; the 16-row ones add 16 waves' instead, each
    order within 32768 2^-24 of the sum S of the slices' magnitudes."""
    F, K, gen = 128, 1 << 22, torch.Generator(device="cuda").manual_seed(rows)
    assert (fq.fp8_gated_gemm_workspace(rows, 1, F, K) > 0) == (rows == 3)
    a, sa, b, sb = codes(gen, rows, K), scales(gen, rows, K // 128), codes(gen, 2 * F, K), scales(gen, 2, K // 128)
    size = fq.fp8_gated_gemm_workspace(rows, 1, F, K)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    q_gu, s_gu = torch.empty(rows, 2 * F, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2, device="cuda")
    fq.fp8_gated_gemm(a, E4, sa, b, E4, sb, RELU, q_gu=q_gu, s_gu=s_gu, workspace=ws)
    for lo, hi in {(0, min(rows, 128)), (max(0, rows - 128), rows)}:
        pa, ps = torch.zeros(128, K, dtype=torch.uint8, device="cuda"), torch.ones(128, K // 128, device="cuda")
        pa[:hi - lo], ps[:hi - lo] = a[lo:hi], sa[lo:hi]
        c = torch.empty(128, 2 * F, device="cuda")
        fq.fp8_scaled_gemm(pa, E4, ps, b, E4, sb, fq.BLOCK_1x128_128x128, c)
        c = c[:hi - lo].contiguous()
        assert bool(torch.isfinite(c).all())
        if rows > 3:
            check_rows(host(q_gu[lo:hi]), host(s_gu[lo:hi]), host(c), E4)
            continue
        most = torch.zeros(hi - lo, 2 * F, dtype=torch.float64, device="cuda")  # a slice's part is at most its products'
        for k in range(0, K, 1 << 18):
            x = a[lo:hi, k:k + (1 << 18)].view(torch.float8_e4m3fn).float().double().abs()
            x *= sa[lo:hi, k // 128:k // 128 + 2048].double().repeat_interleave(128, 1)
            w = b[:, k:k + (1 << 18)].view(torch.float8_e4m3fn).float().double().abs()
            w *= sb[:, k // 128:k // 128 + 2048].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            most += x @ w.t()
        each = s_gu.double().repeat_interleave(128, 1)
        off = (q_gu.view(torch.float8_e4m3fn).float().double() * each - c.double()).abs()
        tol = 2 * 32768 * U * most
        assert bool((off <= tol + 2.0 ** -4 * (c.double().abs() + tol) + 2.0 ** -10 * each).all())
