"""Layer norm and its backward pass against the definition in 64 bits.

Tolerances, with u = 2^-24 (half a binary32 step): a sum over a row is a chain
of at most `depth` additions per value (the vectors of one lane, six steps of
the wave, sixteen waves), so it is off by at most depth u sum |terms|; every
other step adds a few u; the store to bf16 adds half a step, 2^-8 relative
(fp32: 2^-24)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def depth(cols):
    """Additions a row's value can pass through (32 a lane in registers, the
    rest of a long row's, wave and block steps), with margin for the products
    and the division that follow."""
    return 32 + cols / 4096 + 6 + 16 + 16


def draw(rows, cols, dt, pt, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 + rng.standard_normal(cols) * 3.0 + 1.0
    mk = lambda a, t: torch.from_numpy(np.asarray(a, np.float32)).to(DT[t])  # noqa: E731
    return (mk(x, dt), mk(1.0 + 0.2 * rng.standard_normal(cols), pt), mk(0.3 * rng.standard_normal(cols), pt),
            mk(rng.standard_normal((rows, cols)), dt))


def forward64(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean) * rstd
    y = xh * (1.0 if gamma is None else gamma.double()) + (0.0 if beta is None else beta.double())
    return y, mean, rstd, xh


def run_forward(x, gamma, beta, eps):
    xd = x.cuda()
    y = torch.full_like(xd, 777.0)
    mean, rstd = torch.full((x.shape[0],), -7.0, device="cuda"), torch.full((x.shape[0],), -7.0, device="cuda")
    fq.fp8q_layernorm(xd, None if gamma is None else gamma.cuda(), None if beta is None else beta.cuda(), eps, y, mean,
                      rstd)
    torch.cuda.synchronize()
    return y.cpu(), mean.cpu(), rstd.cpu()


def check_forward(x, gamma, beta, eps, dt):
    y, mean, rstd = run_forward(x, gamma, beta, eps)
    y64, m64, r64, xh = forward64(x, gamma, beta, eps)
    d = depth(x.shape[1]) * U
    mabs = x.double().abs().mean(1, keepdim=True)
    # a wrong mean also moves the variance by its square
    var = 1.0 / r64.square() - eps
    r_rel = d + (d * mabs).square() / (2 * (var + eps)) + 4 * U
    assert torch.all((mean.double()[:, None] - m64).abs() <= d * mabs + 1e-45)
    assert torch.all((rstd.double()[:, None] - r64).abs() <= r_rel * r64)
    g = 1.0 if gamma is None else gamma.double().abs()
    b = 0.0 if beta is None else beta.double().abs()
    tol32 = (xh.abs() * (r_rel + 6 * U) + d * mabs * r64) * g + 2 * U * b + U * y64.abs()
    assert torch.all((y.double() - y64).abs() <= tol32 + HALF[dt] * (y64.abs() + tol32) + 1e-40)


SHAPES = [(1, 1), (3, 2), (1, 4096), (5, 7), (129, 64), (4, 511), (2, 512), (7, 513), (33, 1024), (9, 1111), (6, 2048),
          (3, 4097), (17, 5003), (2, 8192), (3, 16383), (2, 32768), (2, 40001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_forward(rows, cols, dt, pt):
    x, gamma, beta, _ = draw(rows, cols, dt, pt, rows * 131 + cols)
    check_forward(x, gamma, beta, 1e-5, dt)


def test_forward_many_rows_and_no_parameters():
    x, gamma, beta, _ = draw(4099, 257, "bf16", "f32", 5)
    check_forward(x, gamma, None, 1e-5, "bf16")
    check_forward(x, None, beta, 1e-5, "bf16")
    check_forward(x, None, None, 1e-3, "bf16")


def test_forward_far_mean_and_constant_rows():
    """A mean of 1000 deviations keeps its variance; a constant row gives beta."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy((1000.0 + rng.standard_normal((5, 3001))).astype(np.float32))
    check_forward(x, None, None, 1e-5, "f32")
    beta = torch.from_numpy(rng.standard_normal(640).astype(np.float32))
    y, mean, rstd = run_forward(torch.full((3, 640), 2.5), None, beta, 1e-5)
    assert torch.equal(y, beta.expand(3, 640)) and torch.all(mean == 2.5)
    y, _, _ = run_forward(torch.zeros(3, 640), None, None, 0.0)
    assert torch.all(torch.isnan(y))  # 0 * inf, as the formula


def test_forward_nonfinite_rows_stay_apart():
    x = torch.randn(6, 384, generator=torch.Generator().manual_seed(2))
    x[1, 5], x[3, 7] = float("nan"), float("inf")
    y, _, _ = run_forward(x, None, None, 1e-5)
    assert torch.all(torch.isnan(y[[1, 3]])) and torch.all(torch.isfinite(y[[0, 2, 4, 5]]))


def test_unaligned_rows_and_guards():
    """Views that start one element in: right values, nothing written beside y."""
    for dt, cols in (("bf16", 1001), ("f32", 515), ("bf16", 5000)):
        x, gamma, beta, _ = draw(4, cols, dt, dt, cols)
        buf = torch.zeros(4 * cols + 1, dtype=DT[dt], device="cuda")
        xv = buf[1:].view(4, cols)
        xv.copy_(x)
        out = torch.full((4 * cols + 2,), 777.0, dtype=DT[dt], device="cuda")
        yv = out[1:-1].view(4, cols)
        fq.fp8q_layernorm(xv, gamma.cuda(), beta.cuda(), 1e-5, yv)
        y, _, _ = run_forward(x, gamma, beta, 1e-5)
        assert torch.equal(yv.cpu(), y)
        assert out[0].item() == out[-1].item() == torch.tensor(777.0).to(DT[dt]).item()


def backward64(dy, x, gamma, mean, rstd):
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    h = dy * (1.0 if gamma is None else gamma.double())
    m1, m2 = h.mean(1, keepdim=True), (h * xh).mean(1, keepdim=True)
    dx = rstd * (h - m1 - xh * m2)
    scale = rstd * (h.abs() + h.abs().mean(1, keepdim=True) + xh.abs() * (h * xh).abs().mean(1, keepdim=True))
    return dx, scale, dy * xh, dy


def run_backward(dy, x, gamma, mean, rstd, pt, want=True):
    rows, cols = x.shape
    dx = torch.full_like(x, 777.0).cuda()
    dg = torch.full((cols,), 777.0, dtype=DT[pt], device="cuda") if want else None
    db = torch.full((cols,), 777.0, dtype=DT[pt], device="cuda") if want else None
    n = fq.fp8q_layernorm_backward_workspace(fq.F32 if x.dtype == torch.float32 else fq.BF16, rows, cols)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    fq.fp8q_layernorm_backward(dy.cuda(), x.cuda(), None if gamma is None else gamma.cuda(), mean.cuda(), rstd.cuda(),
                               dx, dg, db, ws[:n] if want else None)
    torch.cuda.synchronize()
    assert torch.all(ws[n:] == 0xFF)
    return dx.cpu(), None if dg is None else dg.cpu(), None if db is None else db.cpu()


def check_backward(x, dy, gamma, dt, pt):
    _, m64, r64, _ = forward64(x, None, None, 1e-5)
    mean, rstd = m64[:, 0].float(), r64[:, 0].float()
    dx, dg, db = run_backward(dy, x, gamma, mean, rstd, pt)
    dx64, scale, tg, tb = backward64(dy, x, gamma, mean, rstd)
    rows, cols = x.shape
    tol = depth(cols) * U * scale
    assert torch.all((dx.double() - dx64).abs() <= tol + HALF[dt] * (dx64.abs() + tol) + 1e-40)
    # each team's rows in turn, its partial among 512 taken by eight lanes
    d = (rows / 128 + 64 + 8 + 16) * U
    for got, terms in ((dg, tg), (db, tb)):
        want, tol = terms.sum(0), d * terms.abs().sum(0)
        assert torch.all((got.double() - want).abs() <= tol + HALF[pt] * (want.abs() + tol) + 1e-40)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_backward(rows, cols, dt, pt):
    x, gamma, _, dy = draw(rows, cols, dt, pt, rows * 17 + cols)
    check_backward(x, dy, gamma, dt, pt)


def test_backward_many_rows_no_gamma_and_no_parameter_gradients():
    x, gamma, _, dy = draw(4099, 300, "bf16", "f32", 9)
    check_backward(x, dy, gamma, "bf16", "f32")
    check_backward(x, dy, None, "bf16", "f32")
    _, m, r, _ = forward64(x, None, None, 1e-5)
    a = run_backward(dy, x, gamma, m[:, 0].float(), r[:, 0].float(), "f32")
    b = run_backward(dy, x, gamma, m[:, 0].float(), r[:, 0].float(), "f32", want=False)
    assert torch.equal(a[0], b[0])


def test_backward_of_no_rows_is_zero():
    e = torch.empty(0, 96, device="cuda")
    z = torch.empty(0, device="cuda")
    dg, db = torch.full((96,), 5.0, device="cuda"), torch.full((96,), 5.0, device="cuda")
    fq.fp8q_layernorm_backward(e, e, None, z, z, torch.empty_like(e), dg, db, None)
    assert torch.all(dg == 0) and torch.all(db == 0)
    fq.fp8q_layernorm(e, None, None, 1e-5, torch.empty_like(e))


def test_backward_against_differences():
    """dx, dgamma and dbeta against central differences of sum(dy y) in 64
    bits (step 2^-12: the differences are off by about step^2 times a third
    derivative of order one)."""
    x, gamma, beta, dy = draw(3, 40, "f32", "f32", 21)
    loss = lambda x, g, b: (forward64(x, g, b, 1e-5)[0] * dy.double()).sum()  # noqa: E731
    _, m, r, _ = forward64(x, None, None, 1e-5)
    dx, dg, db = run_backward(dy, x, gamma, m[:, 0].float(), r[:, 0].float(), "f32")
    step = 2.0 ** -12
    for which, got in ((0, dx), (1, dg), (2, db)):
        args = [x.double(), gamma.double(), beta.double()]
        flat = got.reshape(-1)
        for i in range(0, flat.numel(), 7):
            both = []
            for sgn in (1, -1):
                moved = [a.clone() for a in args]
                moved[which].view(-1)[i] += sgn * step
                both.append(loss(*moved))
            diff = (both[0] - both[1]) / (2 * step)
            assert abs(float(flat[i]) - float(diff)) <= 1e-5 + 1e-5 * abs(float(diff)), (which, i)


def test_equal_inputs_give_equal_bits():
    x, gamma, _, dy = draw(2049, 1500, "bf16", "f32", 4)
    _, m, r, _ = forward64(x, None, None, 1e-5)
    a = run_backward(dy, x, gamma, m[:, 0].float(), r[:, 0].float(), "f32")
    b = run_backward(dy, x, gamma, m[:, 0].float(), r[:, 0].float(), "f32")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_another_stream():
    x, gamma, beta, _ = draw(300, 2048, "bf16", "f32", 6)
    want, _, _ = run_forward(x, gamma, beta, 1e-5)
    s = torch.cuda.Stream()
    xd, g, b = x.cuda(), gamma.cuda(), beta.cuda()
    y = torch.empty_like(xd)
    torch.cuda.synchronize()
    fq.fp8q_layernorm(xd, g, b, 1e-5, y, stream=s)
    s.synchronize()
    assert torch.equal(y.cpu(), want)


def test_backward_of_more_columns_than_one_launch_of_the_fold_has_lanes():
    """2^27 columns and a few: with one row, dgamma = dy xh and dbeta = dy."""
    cols = (1 << 27) + 77
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, cols, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(1, cols, generator=gen, device="cuda").to(torch.bfloat16)
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 1.5, device="cuda")
    dx = torch.empty_like(x)
    dg, db = (torch.full((cols + 64,), 777.0, device="cuda") for _ in range(2))
    ws = torch.empty(fq.fp8q_layernorm_backward_workspace(fq.BF16, 1, cols), dtype=torch.uint8, device="cuda")
    fq.fp8q_layernorm_backward(dy, x, None, mean, rstd, dx, dg[:cols], db[:cols], ws)
    assert torch.equal(db[:cols], dy[0].float())
    want = dy[0].double() * ((x[0].double() - 0.25) * 1.5)
    # x - mean, its product with rstd (exact here but for one rounding each) and with dy
    assert torch.all((dg[:cols].double() - want).abs() <= 4 * U * want.abs())
    assert torch.all(dg[cols:] == 777.0) and torch.all(db[cols:] == 777.0)


# the register shapes that SHAPES leaves out: whole rows of vectors (256, 6144,
# 12288, 16384 columns) and rows that end inside one
@pytest.mark.parametrize("cols", [256, 2500, 3500, 6144, 7001, 10007, 12288, 16384, 20001])
@pytest.mark.parametrize("dt,pt", [("bf16", "f32"), ("f32", "bf16")])
def test_remaining_register_shapes(cols, dt, pt):
    # more rows than the backward pass has blocks, so that a row ahead is fetched
    rows = 1100
    x, gamma, beta, dy = draw(rows, cols, dt, pt, cols)
    check_forward(x, gamma, beta, 1e-5, dt)
    check_backward(x, dy, gamma, dt, pt)
