"""The operators of a training step together: the next-token example's gradients against
the same model in 64 bits, its steps, and the losses of a step captured into a graph.

Tolerances as in test_gpu_feed_forward: 2-norm of the difference over 2-norm of the
value; a rounding to e4m3 moves a value by at most 2^-4 of it, one to e5m2 by 2^-3,
one to bf16 by 2^-8, and errors from successive steps add up.  A logit's error d moves the
elements of p - onehot by at most 2 d of themselves.
"""
import math
import os
import sys

import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
E4, E5, BF = 2.0 ** -4, 2.0 ** -3, 2.0 ** -8


def plain(model, tokens, targets, weights):
    """(losses, logits, the block's branch and output, gradients) in 64 bits, by autograd on the CPU."""
    p = {k: v.double().cpu().requires_grad_() for k, v in model.params.items()}

    def norm(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return d / ((d * d).mean(1, keepdim=True) + model.eps).sqrt() * w + b

    x = p["embedding"][tokens.cpu()]
    z = norm(x, p["norm_w"], p["norm_b"]) @ p["w1"].t() + p["b1"]
    branch = (z * 0.5 * torch.special.erfc(-z / 2 ** 0.5)) @ p["w2"].t() + p["b2"]
    out = x + branch
    logits = norm(out, p["out_w"], p["out_b"]) @ p["head"].t()
    losses = torch.nn.functional.cross_entropy(logits, targets.cpu(), reduction="none")
    (losses * weights.double().cpu()).sum().backward()
    return losses.detach(), logits.detach(), branch.detach(), out.detach(), {k: v.grad for k, v in p.items()}


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,width,hidden,vocabulary", [(1, 256, 512, 300), (100, 512, 1024, 2005), (300, 1040, 272, 999)])
def test_one_pass_against_64_bits(tokens, width, hidden, vocabulary):
    from next_token import NextToken
    model = NextToken(width, hidden, vocabulary)
    g = torch.Generator(device="cuda").manual_seed(5)
    for name in ("norm_b", "b1", "b2", "out_b"):
        model.params[name].normal_(std=0.2, generator=g)
    model.lay_out()
    t = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    y = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    if tokens > 1:
        y[::7] = -100
    dloss = torch.rand(tokens, generator=g, device="cuda") + 0.5
    losses, saved = model.forward(t, y)
    grads = model.backward(dloss, saved)
    want, logits, branch, out, want_grads = plain(model, t, y, dloss)

    two = math.hypot(E4, E4)                       # a forward product
    up = 1.13 * two + BF                           # the hidden layer
    down = math.hypot(up + E4, E4) + BF
    eo = (down + BF) * float(branch.norm() / out.norm()) + 2 * BF           # out
    en = 2 * eo + BF                               # its norm (the deviation from the mean, over its own size)
    d = (math.hypot(two, en)) * float(logits.square().mean().sqrt())        # logits
    assert float((losses.double().cpu() - want).square().mean().sqrt()) <= 2 * d
    head = E5 + 2 * d                              # p - onehot, its codes
    back = math.hypot(head, E4) + BF               # dn
    eb = back + 2 * en + BF                        # through the norm
    back2 = eb + math.hypot(E5, E4) + BF           # dh
    dz = back2 + 1.13 * two
    tol = {"head": math.hypot(head, E4 + en) + BF, "out_w": back + en, "out_b": back, "w2": eb + math.hypot(E5, E4 + up) + BF,
           "b2": eb, "w1": math.hypot(E5 + dz, E4) + BF, "b1": dz, "norm_w": dz + math.hypot(E5, E4) + BF,
           "norm_b": dz + math.hypot(E5, E4) + BF, "embedding": dz + math.hypot(E5, E4) + 2 * BF}
    assert set(tol) == set(grads) == set(model.params)
    for name, most in tol.items():
        assert grads[name].shape == model.params[name].shape
        assert rel(grads[name], want_grads[name]) <= most, name


def test_ignored_tokens_leave_no_gradient():
    from next_token import NextToken
    model = NextToken(64, 128, 100)
    t = torch.arange(20, device="cuda")
    loss, saved = model.forward(t, torch.full_like(t, -100))
    assert (loss == 0).all()
    assert all((g == 0).all() for g in model.backward(torch.ones(1, device="cuda"), saved).values())


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_are_the_operators(bits):
    """A step moves every parameter as adamw_step does with its gradient, and the codes are the
    new weights'."""
    from next_token import AdamW, NextToken
    model = NextToken(128, 256, 333)
    optimizer = AdamW(model.params, bits)
    t = torch.randint(0, 333, (64,), device="cuda")
    for step in (1, 2):
        _, saved = model.forward(t, t.roll(1))
        grads = model.backward(torch.full((1,), 1 / 64, device="cuda"), saved)
        old = {k: v.clone() for k, v in model.params.items()}
        optimizer.step(grads, 1e-2)
        if step == 1:      # sign(g) lr, but for eps
            for k, g in grads.items():
                moved = (old[k] - model.params[k]).double()
                g = g.double()
                want = 1e-2 * g / (g.abs() + 1e-8)
                assert (moved - want).abs().max() <= 1e-2 * 2.0 ** -20 + 2.0 ** -22 * float(old[k].abs().max()), k
        model.lay_out()
        q = binding.fp8_quantize_weight(model.params["head"])
        assert torch.equal(q.q, model.head.q) and torch.equal(q.qt, model.head.qt)
        w1 = model.params["w1"].bfloat16()
        assert torch.equal(binding.fp8_quantize(w1)[0], model.block.codes["w1"][0])
        assert torch.equal(binding.fp8_quantize(w1.t().contiguous())[0], model.block.codes["w1t"][0])


@pytest.mark.parametrize("bits", ["8", "32"])
def test_training_runs(bits):
    from next_token import main
    losses = main(["--width", "128", "--hidden", "256", "--vocabulary", "211", "--tokens", "512", "--steps", "5", "--bits", bits])
    assert len(losses) == 5 and all(math.isfinite(v) for v in losses)


def test_a_whole_step_captured():
    """Loss, gradients, AdamW and codes in one graph, replayed beside the program's own work: the
    bits of eager steps."""
    M, V, K = 300, 2011, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, s = binding.fp8_quantize(x)
    y = torch.randint(0, V, (M,), generator=g, device="cuda")
    start = torch.randn(V, K, generator=g, device="cuda") * K ** -0.5
    dloss = torch.full((1,), 1 / M, device="cuda")

    def fresh():
        w = start.clone()
        return w, binding.adamw_state([w], 8), torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(w, state, count, seed):
        c = binding.fp8_quantize_weight(w)
        loss, lse = binding.fp8_linear_cross_entropy(q, c.q, s, c.scale, y)
        dx, dw = binding.fp8_linear_cross_entropy_backward(dloss, q, c.q, s, c.scale, y, loss, lse, x, c.qt, c.scale_t)
        binding.adamw_step([w], [dw], **state._asdict(), step=count, lr=1e-2, seed=seed)
        count.add_(1)
        seed.add_(1)
        return loss, dx

    eager, captured = fresh(), fresh()
    step(*fresh())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = step(*captured)
    for rep in range(4):
        want = step(*eager)
        graph.replay()
        step(*fresh())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep
        assert torch.equal(eager[0], captured[0]) and torch.equal(eager[2], captured[2])
