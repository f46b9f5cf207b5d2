"""The expert-layer example against automatic differentiation of the same layer
in 64 bits on the CPU, from the fp32 masters and without FP8.

Tolerances, on the relative 2-norm of an error: a cast to E4M3 is off by at
most 2^-4 of a value and by about 2^-4 / sqrt(6) = 0.026 in the mean (uniform
within the half step, the step's size relative to the value uniform in octaves),
E5M2 by twice that.  The longest chain holds the casts of x and w1, h and w2
(E4M3), and of two gradients and the two transposed weights; independent errors
add in squares: sqrt(6 0.026^2 + 2 0.052^2) = 0.098.  Twice that, 0.2, is
allowed for gradients, and sqrt(4) 0.026 = 0.05 doubled, 0.1, for the experts'
share of the output."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp8_scaled_quantization_reduce_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402


def setup(tokens, cols, hidden, experts, topk, idle):
    layer = expert_layer.ExpertLayer(cols, hidden, experts, topk, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(tokens + 1)
    if idle:
        # the mean of a normalised row is zero: this logit is -0.1 cols for every token
        layer.params["beta"].fill_(0.1)
        layer.params["router"][0] = -1.0
    x = torch.randn(tokens, cols, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, cols, generator=gen, device="cuda")
    return layer, x, dy


def reference(layer, x, dy, expert):
    """Output and gradients in 64 bits, with the experts that were chosen."""
    p = {k: v.double().cpu().requires_grad_() for k, v in layer.params.items()}
    x = x.double().cpu().requires_grad_()
    expert = expert.cpu()
    mean = x.mean(1, keepdim=True)
    xn = (x - mean) * torch.rsqrt((x - mean).square().mean(1, keepdim=True) + layer.eps) * p["gamma"] + p["beta"]
    prob = (xn @ p["router"].t()).gather(1, expert).softmax(1)
    y = x
    for e in range(layer.experts):
        o = torch.nn.functional.silu(xn @ p["w1"][e].t()) @ p["w2"][e].t()
        y = y + o * ((expert == e) * prob).sum(1, keepdim=True)
    y.backward(dy.double().cpu())
    return y.detach() - x.detach(), dict({k: v.grad for k, v in p.items()}, x=x.grad - dy.double().cpu())


def off(got, want):
    want = want.cuda()
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,cols,hidden,experts,topk,idle", [(301, 256, 384, 5, 2, True), (1, 128, 256, 4, 1, False),
                                                                  (1024, 512, 256, 8, 2, False),
                                                                  (77, 384, 128, 3, 3, False)])
def test_gradients(tokens, cols, hidden, experts, topk, idle):
    layer, x, dy = setup(tokens, cols, hidden, experts, topk, idle)
    y, saved = layer.forward(x)
    grads, dx = layer.backward(dy, saved)
    want_y, want = reference(layer, x, dy, saved[5])
    assert off(y - x.float(), want_y) < 0.1
    for name, g in dict(grads, x=dx - dy).items():
        if want[name].norm() == 0:  # one expert a token: its probability is 1, no gradient reaches the router
            assert float(g.abs().max()) == 0, name
            continue
        assert off(g, want[name]) < 0.2, name
    if idle:
        assert int(saved[9][1]) == 0
        assert not grads["w1"][0].any() and not grads["w2"][0].any()
    # the same bits again: no sum depends on an order of arrival
    again, dx2 = layer.backward(dy, layer.forward(x)[1])
    assert torch.equal(dx, dx2) and all(torch.equal(again[k], grads[k]) for k in grads)


def test_serving_form_equals_the_training_forward():
    layer, x, _ = setup(9, 256, 256, 4, 2, False)
    assert torch.equal(layer.forward(x, train=False)[0], layer.forward(x)[0])


def test_steps_lower_the_loss():
    layer, x, _ = setup(512, 256, 512, 4, 2, False)
    target = x.float() + torch.roll(x.float(), 1, 1)
    got = [layer.step(x, target, 0.5, max_norm=1.0) for _ in range(8)]
    loss = [float(v) for v, _ in got]
    norm = [float(v) for _, v in got]
    assert all(b < a for a, b in zip(loss, loss[1:])), loss
    assert all(n > 0 and n < float("inf") for n in norm), norm


def test_a_step_is_clipped():
    """The parameters move by rate max_norm: the weights' rounding is at most
    2^-24 of their 2-norm (about 45) in a move of 0.005, 6e-4."""
    layer, x, dy = setup(512, 256, 512, 4, 2, False)
    before = {k: v.clone() for k, v in layer.params.items()}
    _, norm = layer.step(x, x.float() + dy, 0.5, max_norm=0.01)
    assert float(norm) > 0.01
    moved = sum(float((layer.params[k].double() - before[k].double()).square().sum()) for k in before) ** 0.5
    assert abs(moved - 0.005) < 0.005 * 1e-3
