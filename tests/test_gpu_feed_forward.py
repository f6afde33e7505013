"""The operators together: the feed-forward example's pass against the same
block in 64 bits, and its training.

Tolerances (2-norm of the difference over 2-norm of the value).  A rounding to
e4m3 moves a value by at most 2^-4 of it, one to e5m2 by at most 2^-3, one to
bf16 by 2^-8; the errors of a product's terms are independent, so the product is
off by no more than the root of the sum of the squares of its operands' largest
relative errors, a function with a slope of at most 1.13 passes an error on as
1.13 times itself, and errors from successive steps add up.
"""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
E4, E5, BF = 2.0 ** -4, 2.0 ** -3, 2.0 ** -8


def plain(model, x, dout):
    """Output and gradients of the block in 64 bits, by autograd on the CPU."""
    p = {k: v.double().cpu().requires_grad_() for k, v in model.params.items()}
    x = x.double().cpu().requires_grad_()
    d = x - x.mean(1, keepdim=True)
    n = d / ((d * d).mean(1, keepdim=True) + model.eps).sqrt() * p["norm_w"] + p["norm_b"]
    z = n @ p["w1"].t() + p["b1"]
    h = z * 0.5 * torch.special.erfc(-z / 2 ** 0.5)
    branch = h @ p["w2"].t() + p["b2"]
    (x + branch).backward(dout.double().cpu())
    return branch.detach(), x.grad, {k: v.grad for k, v in p.items()}


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (96, 512, 1024), (250, 1040, 272)])
def test_one_pass_against_64_bits(tokens, width, hidden):
    from feed_forward import FeedForward
    model = FeedForward(width, hidden)
    g = torch.Generator(device="cuda").manual_seed(5)
    for name in ("norm_b", "b1", "b2"):
        model.params[name].normal_(std=0.2, generator=g)
    model.params["norm_w"].add_(torch.randn(width, generator=g, device="cuda") * 0.2)
    model.lay_out()
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    dout = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    out, saved = model.forward(x)
    dx, grads = model.backward(dout, saved)
    branch, want_dx, want = plain(model, x, dout)

    two = math.hypot(E4, E4)                       # a forward product
    up = 1.13 * two + BF                           # the hidden layer
    down = math.hypot(up + E4, E4) + BF
    assert rel(out.double() - x.double(), branch) <= down + BF * float(out.double().norm()) / float(branch.norm())
    back2 = math.hypot(E5, E4) + BF                # dh
    dz = back2 + 1.13 * two                        # its activation's slope from the pre-activation
    tol = {"w2": math.hypot(E5, E4 + up) + BF, "b2": BF, "w1": math.hypot(E5 + dz, E4) + BF, "b1": dz,
           "norm_w": dz + math.hypot(E5, E4) + BF, "norm_b": dz + math.hypot(E5, E4) + BF}
    for name, t in tol.items():
        assert grads[name].shape == model.params[name].shape
        assert rel(grads[name], want[name]) <= t, name
    assert rel(dx, want_dx) <= dz + math.hypot(E5, E4) + 2 * BF


def test_training_learns():
    from feed_forward import main
    losses = main(["--width", "256", "--hidden", "1024", "--tokens", "512", "--steps", "30"])
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]
