"""The global gradient norm and clipping against sums in 64 bits.

The squares are summed in binary64, so norm is off by its rounding to binary32
(2^-24), the coefficient by three more roundings, and an output by one product
and its own rounding (bf16: half a step, 2^-8)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def draw(sizes, seed, std=1e-2):
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.from_numpy((rng.standard_normal(n) * std).astype(np.float32))
        out.append(t.to(torch.bfloat16) if i % 2 else t)
    return out


def run(grads, max_norm, place="out"):
    g = [t.cuda() for t in grads]
    norm, coef = torch.full((1,), -7.0, device="cuda"), torch.full((1,), -7.0, device="cuda")
    out = [torch.full_like(t, 777.0) for t in g] if place == "out" else None
    fq.fp8q_grad_norm_clip(g, max_norm, norm, coef, out=out)
    torch.cuda.synchronize()
    if place == "out":
        assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(g, grads) if b.numel())
    return norm.item(), coef.item(), [t.cpu() for t in (out if place == "out" else g)]


def check(grads, max_norm, place="out"):
    norm, coef, out = run(grads, max_norm, place)
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert abs(norm - want) <= 2 * U * want
    c64 = min(1.0, max_norm / (want + 1e-6))
    assert abs(coef - c64) <= 6 * U * c64
    for a, b in zip(out, grads):
        w = b.double() * c64
        assert torch.all((a.double() - w).abs() <= (HALF[b.dtype] + 8 * U) * w.abs() + 1e-40)
    return norm, coef


SIZES = [[1], [7], [8191, 8192, 8193], [100003, 1, 0, 65536, 3], [257] * 48, [33] * 127, [40] * 128, [9] * 129,
         [1000 + i for i in range(300)], [3000017, 12]]


@pytest.mark.parametrize("k", range(len(SIZES)))
@pytest.mark.parametrize("place", ["out", "in place"])
def test_clips_by_the_global_norm(k, place):
    grads = draw(SIZES[k], 3 + k)
    norm, coef = check(grads, 0.01, place)
    assert coef <= 1.0


def test_small_norm_leaves_the_gradients():
    grads = draw([4000, 5001], 1)
    norm, coef, out = run(grads, 1e9, "in place")
    assert coef == 1.0 and all(torch.equal(a, b) for a, b in zip(out, grads))
    _, coef, out = run(grads, 1e9)
    assert coef == 1.0 and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_norm_alone():
    grads = draw([70000, 33, 12], 8)
    norm, coef, out = run(grads, math.inf, "in place")
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert abs(norm - want) <= 2 * U * want and coef == 1.0
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


def test_zero_and_empty():
    norm, coef, out = run([torch.zeros(100), torch.zeros(3, dtype=torch.bfloat16)], 1.0)
    assert norm == 0.0 and coef == 1.0 and all(torch.all(t == 0) for t in out)
    assert run([], 1.0)[:2] == (0.0, 1.0)
    assert run([torch.empty(0)], 0.5)[:2] == (0.0, 1.0)
    norm, coef, out = run([torch.ones(5)], 0.0)
    assert coef == 0.0 and torch.all(out[0] == 0)


def test_squares_beyond_binary32():
    """Gradients whose squares overflow or underflow binary32."""
    check([torch.tensor([3e30, -4e30]), torch.full((9000,), 1e25)], 1.0)
    check([torch.full((10000,), 1e-30), torch.full((77,), 1e-28)], 1e-31)


def test_nonfinite():
    norm, coef, out = run([torch.tensor([1.0, float("inf"), 2.0]), torch.ones(3)], 1.0)
    assert norm == math.inf and coef == 0.0
    assert torch.isnan(out[0][1]) and out[0][0] == 0 and torch.all(out[1] == 0)
    norm, coef, out = run([torch.tensor([1.0, float("nan")]), torch.ones(3, dtype=torch.bfloat16)], 1.0)
    assert math.isnan(norm) and math.isnan(coef) and all(torch.all(torch.isnan(t)) for t in out)


def test_unaligned_views_and_guards():
    """Slices of one flat buffer, as a bucket of gradients is: nothing beside them changes."""
    for dt in (torch.float32, torch.bfloat16):
        flat = (torch.randn(20011, generator=torch.Generator().manual_seed(1)) * 0.1).to(dt)
        cuts = [(1, 4), (5, 8200), (8201, 9001), (9003, 20010)]
        buf = flat.cuda()
        norm, coef = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        fq.fp8q_grad_norm_clip([buf[a:b] for a, b in cuts], 0.5, norm, coef)
        got = buf.cpu()
        want = math.sqrt(sum(float(flat[a:b].double().square().sum()) for a, b in cuts))
        assert abs(norm.item() - want) <= 2 * U * want
        beside = torch.ones(flat.numel(), dtype=torch.bool)
        for a, b in cuts:
            beside[a:b] = False
            w = flat[a:b].double() * (0.5 / (want + 1e-6))
            assert torch.all((got[a:b].double() - w).abs() <= (HALF[dt] + 8 * U) * w.abs())
        assert torch.equal(got[beside], flat[beside])


def test_equal_inputs_give_equal_bits_on_two_streams():
    grads = [t.cuda() for t in draw([500009, 70001], 4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [[torch.zeros(1, device="cuda") for _ in range(2)] for _ in streams]
    outs = [[torch.empty_like(t) for t in grads] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, r, o in zip(streams, res, outs):
            fq.fp8q_grad_norm_clip(grads, 0.25, r[0], r[1], out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_graph_replays():
    """Captured once, replayed with new gradients and eager work between."""
    grads = [t.cuda() for t in draw([300007, 4097, 12], 11)]
    out = [torch.empty_like(t) for t in grads]
    norm, coef = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    fq.fp8q_grad_norm_clip(grads, 0.1, norm, coef, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fq.fp8q_grad_norm_clip(grads, 0.1, norm, coef, out=out)
    for k in range(3):
        for t in grads:
            t.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        got = (norm.clone(), coef.clone(), [t.clone() for t in out])
        fq.fp8q_grad_norm_clip(grads, 0.1, norm, coef, out=out)
        torch.cuda.synchronize()
        assert torch.equal(got[0], norm) and torch.equal(got[1], coef)
        assert all(torch.equal(a, b) for a, b in zip(got[2], out))


def test_norm_alone_of_nonfinite_gradients():
    """Without a bound nothing is clipped, by an infinite norm neither; a NaN shows in both results."""
    big = [torch.full((5,), 3e38), torch.full((9000,), 3e38)]  # a norm past binary32
    for grads, nan in (([torch.tensor([1.0, math.inf, 2.0])], False), (big, False),
                       ([torch.tensor([1.0, math.nan]), torch.ones(3, dtype=torch.bfloat16)], True),
                       ([torch.tensor([math.inf, math.nan])], True)):
        norm, coef, out = run(grads, math.inf, "in place")
        assert math.isnan(norm) and math.isnan(coef) if nan else norm == math.inf and coef == 1.0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, grads))
