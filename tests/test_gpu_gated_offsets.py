"""The gated product's codes for offsets that decrease: whichever tiles the sizes
choose, a row of exactly one group has that group's results, a row of no group
stays as it was, and a row that groups share (whose values are unspecified) is
written, never from a workspace that no tile filled.  Values are compared with calls
whose offsets give a group its rows and the others none, bit for bit: a row's
result depends on no other row.  Groups that share rows may have more tiles than
rows in as many groups can have, which is what a launch covers (0 .. 419 and 140 ..
699 of 700 rows are 7 + 9 tiles of 64 rows, where 3 groups have at most 13): then some
of their tiles are left out, and only the rows of no group are as without them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
E4, SILU = fq.E4M3FN, fq.ACT_SILU
F, K = 256, 2048

# of 100 rows
OFFSETS = [[0, 100, 50], [50, 60, 0, 10], [0, 60, 20, 100], [-5, 40, 1000, 70, 100], [100, 100, 20, 40, 10, 30],
           list(range(0, 100, 2)) + [40] * 10 + [45] * 11]


def operands(rows, groups):
    gen = torch.Generator(device="cuda").manual_seed(rows + groups)

    def codes(*shape):
        q = torch.randint(0x28, 0x48, shape, generator=gen, device="cuda", dtype=torch.uint8)
        return q | (torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.uint8) << 7)

    def scales(*shape):
        return torch.rand(*shape, generator=gen, device="cuda") * 0.05 + 0.01
    return (codes(rows, K), E4, scales(rows, K // 128), codes(groups, 2 * F, K), E4,
            scales(groups, 2 * F // 128, K // 128))


def call(ops, offsets):
    rows, groups = ops[0].shape[0], ops[3].shape[0]
    o = dict(H=torch.full((rows, F), 768.0, device="cuda"),
             q_h=torch.full((rows, F), 0xA5, dtype=torch.uint8, device="cuda"),
             s_h=torch.full((rows, F // 128), -7.25, device="cuda"),
             q_gu=torch.full((rows, 2 * F), 0xA5, dtype=torch.uint8, device="cuda"),
             s_gu=torch.full((rows, 2 * F // 128), -7.25, device="cuda"))
    size = fq.fp8_gated_gemm_workspace(rows, groups, F, K)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None  # NaN bits
    fq.fp8_gated_gemm(*ops, SILU, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), workspace=ws, **o)
    return o, size


LEFT = dict(H=768.0, q_h=0xA5, s_h=-7.25, q_gu=0xA5, s_gu=-7.25)


@pytest.mark.parametrize("times", [1, 7, 200])  # tiles of 16 rows, and of 64 and more
@pytest.mark.parametrize("k", range(len(OFFSETS)))
def test_rows_of_decreasing_offsets(k, times):
    rows, off = 100 * times, [times * v for v in OFFSETS[k]]
    groups = len(off) - 1
    ops = operands(rows, groups)
    got, size = call(ops, off)
    assert (size > 0) == (times == 1)
    clamped = [min(max(v, 0), rows) for v in off]
    held = [0] * rows
    spans = [(e, clamped[e], clamped[e + 1]) for e in range(groups) if clamped[e] < clamped[e + 1]]
    for _, lo, hi in spans:
        for r in range(lo, hi):
            held[r] += 1
    held = torch.tensor(held, device="cuda")
    for name, v in got.items():
        assert bool((v[held == 0] == LEFT[name]).all()), name
    for name in ("H", "s_h", "s_gu"):
        assert bool(torch.isfinite(got[name]).all()), name
    if any(sum(-(-(hi - lo) // t) for _, lo, hi in spans) > (rows + min(rows, groups) * (t - 1)) // t
           for t in (16, 64, 256)):
        return
    for e, lo, hi in spans:
        want, _ = call(ops, [lo] * (e + 1) + [hi] * (groups - e))
        alone = torch.nonzero(held[lo:hi] == 1).flatten() + lo
        for name, v in got.items():
            assert torch.equal(v[alone], want[name][alone]), (name, e)
    for name in ("s_h", "s_gu"):
        assert bool((got[name][held > 1] > 0).all()), name


def test_more_tiles_than_one_buffer_can_have():
    """Groups that share rows over and over have more tiles than a launch covers: rows
    that no tile reaches stay as they were."""
    rows, off = 100, [0, 96, 0, 96, 0, 96, 0, 96, 0, 100]
    got, size = call(operands(rows, len(off) - 1), off)
    assert size > 0
    for name in ("s_h", "s_gu"):
        written = got[name] > 0
        assert bool((written | (got[name] == LEFT[name])).all()), name
        assert bool((written.all(1) | ~written.any(1)).all()), name
    assert bool(torch.isfinite(got["H"]).all())
