"""A next-token model on the package's FP8 operators, trained with AdamW:

    x = E[token],  out = x + W2 gelu(W1 norm(x) + b1) + b2        (feed_forward.py)
    loss = cross entropy of (H norm(out)) over the vocabulary

    python examples/next_token.py --width 1024 --hidden 4096 --vocabulary 50255 --tokens 4096 --steps 20 --bits 8

The logits are never written: the loss and its gradient make them tile by tile.  A
step is, forward: embedding, block, norm with its codes, loss; backward: the head's
gradients from the loss, then norm, block and embedding; then one AdamW step over all
tensors with gradients of one type, with moments of 8 or 32 bits, and the codes of the
new weights in both layouts.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from feed_forward import FeedForward  # noqa: E402

from precision_linear_amd import binding  # noqa: E402


class NextToken:
    def __init__(self, width, hidden, vocabulary, eps=1e-5, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.eps = eps
        self.block = FeedForward(width, hidden, eps, device, seed + 1)
        self.params = dict(self.block.params)      # the block's own tensors, updated in place
        self.params["embedding"] = torch.randn(vocabulary, width, generator=g, device=device)
        self.params["out_w"] = torch.ones(width, device=device)
        self.params["out_b"] = torch.zeros(width, device=device)
        self.params["head"] = torch.randn(vocabulary, width, generator=g, device=device) * width ** -0.5
        self.lay_out()

    def lay_out(self):
        self.block.lay_out()
        self.head = binding.fp8_quantize_weight(self.params["head"])

    def forward(self, tokens, targets):
        """(loss of each token, what backward() needs); targets of -100 are ignored."""
        x = self.params["embedding"][tokens].bfloat16()
        out, inner = self.block.forward(x)
        n = binding.fp8_layer_norm(out, self.params["out_w"], self.params["out_b"], self.eps, fmt="e4m3fn", stats=True)
        loss, lse = binding.fp8_linear_cross_entropy(n.q, self.head.q, n.scale, self.head.scale, targets)
        return loss, (tokens, targets, inner, out, n, loss, lse)

    def backward(self, dloss, saved):
        """Gradients of the parameters from dloss, the gradient of the losses (one for each
        token, or one number for all)."""
        tokens, targets, inner, out, n, loss, lse = saved
        dn, dhead = binding.fp8_linear_cross_entropy_backward(dloss, n.q, self.head.q, n.scale, self.head.scale, targets,
                                                              loss, lse, n.y, self.head.qt, self.head.scale_t)
        dout, dw, db = binding.fp8_layer_norm_backward(dn, out, n.mean, n.rstd, self.params["out_w"])
        dx, grads = self.block.backward(dout, inner)
        demb = torch.zeros_like(self.params["embedding"]).index_add_(0, tokens, dx.float())
        return grads | {"head": dhead, "out_w": dw, "out_b": db, "embedding": demb}


class AdamW:
    """The parameters' states, and a step over them: one call for each type of gradient."""

    def __init__(self, params, bits=32):
        self.params, self.bits, self.count, self.groups = params, bits, 0, {}

    def step(self, grads, rate, decay=0.0):
        self.count += 1
        for dtype in sorted({g.dtype for g in grads.values()}, key=str):
            names = [k for k, g in grads.items() if g.dtype == dtype]
            params = [self.params[k] for k in names]
            key = (dtype, tuple(names))
            if key not in self.groups:
                self.groups[key] = binding.adamw_state(params, self.bits)
            binding.adamw_step(params, [grads[k] for k in names], **self.groups[key]._asdict(), step=self.count, lr=rate,
                               weight_decay=decay, seed=self.count)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocabulary", type=int, default=50255)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32), help="of the moments")
    ap.add_argument("--rate", type=float, default=1e-3)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    model = NextToken(a.width, a.hidden, a.vocabulary)
    optimizer = AdamW(model.params, a.bits)
    # What it learns: each token is followed by one other.
    after = torch.randperm(a.vocabulary, generator=g, device="cuda")
    losses = []
    began = time.perf_counter()
    for _ in range(a.steps):
        tokens = torch.randint(0, a.vocabulary, (a.tokens,), generator=g, device="cuda")
        loss, saved = model.forward(tokens, after[tokens])
        losses.append(loss.mean())
        grads = model.backward(torch.full((1,), 1.0 / a.tokens, device="cuda"), saved)
        optimizer.step(grads, a.rate)
        model.lay_out()
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    losses = [float(v) for v in losses]
    print(f"{a.tokens} tokens of {a.vocabulary}, width {a.width}: loss {losses[0]:.4f} -> {losses[-1]:.4f} (chance "
          f"{math.log(a.vocabulary):.4f}) in {a.steps} steps, {took / a.steps * 1e3:.2f} ms a step")
    return losses


if __name__ == "__main__":
    main()
