"""Codes and scales of the gated backward pass and of the 8-bit columnwise copy,
bit for bit: in the calls that ask for no binary32 D, for every mantissa of a block's
largest value, past one launch's tiles and before rows of no group."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from test_gpu_gated import GELU, RELU, SILU, backward, check_backward, check_columns, check_rows, checkpoint
from test_gpu_grouped import offsets_of

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
E4, E5 = oracle.E4M3FN, oracle.E5M2


@pytest.mark.parametrize("D,col,hcol", [(None, True, True), (torch.bfloat16, True, True), (None, False, False),
                                        (torch.bfloat16, False, False), (None, True, False)])
@pytest.mark.parametrize("act", [RELU, GELU, SILU])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("sizes", [[1], [70, 0, 200], [128, 131]])
def test_codes_without_a_binary32_d(D, col, hcol, act, bf16, sizes):
    """They are those of the D that another call writes, which has the same values."""
    rows, F = sum(sizes), 384
    q, s = checkpoint(rows, F, E4, rows)
    dh = np.random.default_rng(rows + 1).standard_normal((rows, F)) * 1e-3
    dh = workloads.to_bf16_bits(dh) if bf16 else dh.astype(np.float32)
    off = offsets_of(sizes)
    got = backward(dh, q, s, E4, off, act, D=D, col=col, hcol=hcol, sizes=sizes)
    full = backward(dh, q, s, E4, off, act, row=False, col=False, hcol=False, sizes=sizes)["D"]
    check_rows(got["q_d"], got["s_d"], full, E5)
    if col:
        check_columns(got["qc_d"], got["sc_d"], full, sizes, E5)
    if D is not None:
        assert np.array_equal(got["D"], torch.from_numpy(full).to(D).float().numpy())
    if hcol:  # du is h where dh is u, and u's values are the checkpoint's
        u = (oracle.decode_table(E4)[q].astype(np.float32) * np.repeat(s, 128, 1))[:, F:].copy()
        h = backward(u, q, s, E4, off, act, row=False, col=False, hcol=False, sizes=sizes)["D"][:, F:]
        check_columns(got["qc_h"], got["sc_h"], h, sizes, E4)


@pytest.mark.parametrize("sizes", [[1], [2], [3], [129], [131], [5, 1]])
def test_rows_behind_a_short_tile_stay(sizes):
    """Tiles that end after one to three rows, with rows of no group behind them."""
    check_backward(sizes, 128, SILU, seed=sum(sizes), tail=130)
    check_backward(sizes, 256, SILU, D=torch.bfloat16, seed=sum(sizes), first=3, tail=5)


def test_more_tiles_than_one_launch_holds():
    """1100 groups of a row each and 8192 tiles of columns: 9e6 tiles."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rows, F = 1100, 1 << 20
    q = torch.randint(0x28, 0x48, (rows, 2 * F), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.rand(rows, 2 * F // 128, generator=gen, device="cuda") * 0.05 + 0.01
    dh = torch.randn(rows, F, generator=gen, device="cuda", dtype=torch.bfloat16)

    def run(lo, hi):
        off = torch.arange(hi - lo + 1, dtype=torch.int32, device="cuda")
        o = dict(q_d=torch.full((hi - lo, 2 * F), 0xA5, dtype=torch.uint8, device="cuda"),
                 s_d=torch.full((hi - lo, 2 * F // 128), -7.25, device="cuda"))
        fq.fp8_gated_backward(dh[lo:hi], q[lo:hi], s[lo:hi], E4, SILU, offsets=off, **o)
        return o
    whole = run(0, rows)
    for lo, hi in ((0, 8), (1016, 1032), (1092, 1100)):
        for k, v in run(lo, hi).items():
            assert torch.equal(whole[k][lo:hi], v), (k, lo)


# ------------------------------------------------- scales of every mantissa --
FP8 = {E4: torch.float8_e4m3fn, E5: torch.float8_e5m2}
FP8_MAX = {E4: 448.0, E5: 57344.0}


def check_scales(s, fmt, largest, other):
    """128 rows of a block of 128 columns, row r with scale s[r]: the value `largest`
    in column r, `other` elsewhere, so that column c's largest is that of row c.  The
    copy's scales are fl32(max(amax, 1e-12) / FP8_MAX) and its codes those of
    x fl32(1 / scale); quotients are rounded from binary64 ones, whose own rounding
    cannot change that of a quotient of two binary32 numbers."""
    rows = s.numel()
    code = torch.tensor([largest, other], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    eye = torch.eye(128, dtype=torch.bool, device="cuda")
    q = torch.where(eye, code[0], code[1]).repeat(rows // 128, 1).contiguous()
    qc, sc = torch.empty(128, rows, dtype=torch.uint8, device="cuda"), torch.empty(128, rows // 128, device="cuda")
    fq.fp8_requantize_grouped(q, s.view(rows, 1), E4, qc, sc, fmt)
    top = (s * largest).view(-1, 128).t()  # [column][block]
    scale = (top.clamp_min(1e-12).double() / FP8_MAX[fmt]).float()
    assert torch.equal(sc, scale)
    inverse = (1.0 / scale.double()).float()
    x = torch.where(eye, largest, other)[:, None, :] * s.view(-1, 128)[None]  # [column][block][row]
    want = (x * inverse[:, :, None]).to(FP8[fmt]).view(torch.uint8).view(128, rows)
    assert torch.equal(qc, want)


# 0.75 of the largest is 336 in E4M3, halfway between codes; 1.125 beside 1.75 is halfway
# in E5M2: with neighbouring mantissas in a block, a scale off by one in its last bit
# moves codes
@pytest.mark.parametrize("fmt,largest,other", [(E4, 1.0, 0.75), (E5, 1.0, 0.75), (E5, 1.75, 1.125)])
def test_scales_of_every_mantissa(fmt, largest, other):
    for chunk in range(8):
        bits = torch.arange(chunk << 20, (chunk + 1) << 20, dtype=torch.int32, device="cuda") | 0x3F800000
        check_scales(bits.view(torch.float32), fmt, largest, other)


@pytest.mark.parametrize("fmt", [E4, E5])
def test_scales_of_every_exponent(fmt):
    """From below the floor of 1e-12 (2^-40 < 1e-12 < 2^-39) to the largest binary32
    exponent, 4096 neighbouring mantissas at both ends and in three places between."""
    for exponent in range(127 - 45, 255):
        for start in (0, 0x2AA000, 0x3FF800, 0x555000, 0x7FF000):
            bits = torch.arange(start, start + 4096, dtype=torch.int32, device="cuda") + (exponent << 23)
            check_scales(bits.view(torch.float32), fmt, 1.0, 0.75)
    near = torch.tensor([1e-12], device="cuda").view(torch.int32)
    check_scales((near + torch.arange(-64, 64, dtype=torch.int32, device="cuda")).view(torch.float32), fmt, 1.0, 0.75)
