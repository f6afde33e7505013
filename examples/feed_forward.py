"""A pre-norm feed-forward block on the package's FP8 operators, forward and
backward, trained for a few steps:

    out = x + W2 gelu(W1 norm(x) + b1) + b2

    python examples/feed_forward.py --width 2048 --hidden 8192 --tokens 1024 --steps 20

One pass is, forward: layer norm with the codes of its result, the up projection
with bias and gelu in its epilogue (and its pre-activation kept), the
quantisation of the hidden layer, the down projection with bias and the residual
in its epilogue; backward: the gradients of the two projections and of the norm,
which also adds the gradient along the residual path.  Weights are fp32 masters;
their codes, and those of their transposes for the backward pass, are laid out
once for each update.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from precision_linear_amd import binding  # noqa: E402


class FeedForward:
    def __init__(self, width, hidden, eps=1e-5, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        self.eps = eps
        self.params = {
            "norm_w": torch.ones(width, device=device), "norm_b": torch.zeros(width, device=device),
            "w1": normal(hidden, width, std=width ** -0.5), "b1": torch.zeros(hidden, device=device),
            "w2": normal(width, hidden, std=hidden ** -0.5), "b2": torch.zeros(width, device=device),
        }
        self.lay_out()

    def lay_out(self):
        """The weights' codes: N x K for the forward pass, K x N for the backward one."""
        self.codes = {}
        for name in ("w1", "w2"):
            q, scale, qt, scale_t = binding.fp8_quantize_weight(self.params[name].bfloat16())
            self.codes[name] = q, scale
            self.codes[name + "t"] = qt, scale_t
        self.bias = {name: self.params[name].bfloat16() for name in ("b1", "b2")}

    def forward(self, x, train=True):
        """(out, what backward() needs); x is tokens x width bf16."""
        p = self.params
        n = binding.fp8_layer_norm(x, p["norm_w"], p["norm_b"], self.eps, y=train, fmt="e4m3fn", stats=train)
        w1, s1 = self.codes["w1"]
        z = torch.empty((x.shape[0], w1.shape[0]), dtype=torch.bfloat16, device=x.device) if train else None
        h = binding.fp8_linear(n.q, w1, n.scale, s1, self.bias["b1"], activation="gelu", preact=z)
        qh, sh = binding.fp8_quantize(h, "rowwise")
        w2, s2 = self.codes["w2"]
        out = binding.fp8_linear(qh, w2, sh, s2, self.bias["b2"], x)
        return out, (x, n, z, h)

    def backward(self, dout, saved):
        """(dx, gradients of the parameters) from the gradient of out."""
        x, n, z, h = saved
        w2t, s2t = self.codes["w2t"]
        dh, dw2, db2 = binding.fp8_linear_backward(dout, h, w2t, s2t)
        w1t, s1t = self.codes["w1t"]
        dn, dw1, db1 = binding.fp8_linear_backward(dh, n.y, w1t, s1t, z, activation="gelu")
        dx, dnw, dnb = binding.fp8_layer_norm_backward(dn, x, n.mean, n.rstd, self.params["norm_w"],
                                                       residual_grad=dout)
        return dx, {"norm_w": dnw, "norm_b": dnb, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}

    def step(self, grads, rate):
        for name, g in grads.items():
            self.params[name].sub_(g.float(), alpha=rate)
        self.lay_out()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=None, help="default: 10 / hidden (the hidden layer's mean sets the "
                                                             "largest curvature, about 0.16 hidden)")
    a = ap.parse_args(argv)
    rate = 10 / a.hidden if a.rate is None else a.rate
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    # What it learns: another block of the same form.
    target, _ = FeedForward(a.width, a.hidden, seed=2).forward(x, train=False)
    model = FeedForward(a.width, a.hidden, seed=3)
    losses = []
    began = time.perf_counter()
    for _ in range(a.steps):
        out, saved = model.forward(x)
        diff = out.float() - target.float()
        losses.append((diff * diff).mean())
        dout = (diff * (2.0 / a.tokens)).bfloat16()      # of the mean over tokens of the squared distance
        _, grads = model.backward(dout, saved)
        model.step(grads, rate)
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    losses = [float(v) for v in losses]
    print(f"{a.tokens} tokens, {a.width} -> {a.hidden} -> {a.width}: loss {losses[0]:.4f} -> {losses[-1]:.4f} in "
          f"{a.steps} steps, {took / a.steps * 1e3:.2f} ms a step")
    return losses


if __name__ == "__main__":
    main()
