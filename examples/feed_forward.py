"""A pre-norm feed-forward block on the layer operators, as a model would run it.

    s = x + r;  y = rmsnorm(s) * g;  h = gelu(y W1^T + b1);  out = h W2^T + s

Training: bf16 (or float16; float32 trains too, but the 8-bit products give 16-bit
results) forward and backward and a gradient step.
Serving: the weights brought to 8 bits once; every step the norm writes 8-bit
rows with scales, both products read 8-bit operands, and the second adds the
residual stream in its epilogue.

    python examples/feed_forward.py [--tokens 512] [--width 1024] [--hidden 4096] [--steps 20] [--max-norm 1]

prints the loss of a few training steps on a fixed regression target and how far
the 8-bit block's output is from the trained 16-bit one's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402


class FeedForward:
    def __init__(self, width, hidden, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
        self.g = torch.ones(width, device="cuda", dtype=dtype)
        self.w1, self.b1 = new(hidden, width, std=width ** -0.5), new(hidden, std=0.02)
        self.w2 = new(width, hidden, std=hidden ** -0.5)
        self.q = None

    def forward(self, x, r):
        """Output and what the backward pass needs."""
        y, s, rstd = sg.add_rmsnorm(x, self.g, r)
        h, z = sg.linear(y, self.w1, self.b1, activation="gelu", save_preact=True)
        return sg.linear(h, self.w2, residual=s), (y, s, rstd, h, z)

    def backward(self, dout, saved):
        """Gradients of x (and r alike) and of the parameters."""
        y, s, rstd, h, z = saved
        dh, dw2, _ = sg.linear_backward(dout, h, self.w2, need_db=False)
        dy, dw1, db1 = sg.linear_backward(dh, y, self.w1, z, activation="gelu")
        dx, dg = sg.add_rmsnorm_backward(dy, s, rstd, self.g, dout)   # the residual's gradient joins
        return dx, {"g": dg, "w1": dw1, "b1": db1, "w2": dw2}

    def step(self, grads, rate, max_norm=None):
        """One step; with ``max_norm`` along the gradients clipped by their common norm."""
        if max_norm is not None:
            sg.clip_grad_norm(grads.values(), max_norm)
        for name, d in grads.items():
            p = getattr(self, name)
            p.add_(d, alpha=-rate)
        self.q = None

    def quantize(self):
        """8-bit weights with a scale per output feature, made once."""
        self.q = (*sg.quantize_rows(self.w1), *sg.quantize_rows(self.w2))

    def serve(self, x, r):
        q1, s1, q2, s2 = self.q
        y, ys, s, _ = sg.add_rmsnorm(x, self.g, r, quantize=True)
        h = sg.linear(y, q1, self.b1, activation="gelu", x_scale=ys, w_scale=s1,
                      out_dtype=x.dtype)
        hq, hs = sg.quantize_rows(h)
        return sg.linear(hq, q2, residual=s, x_scale=hs, w_scale=s2, out_dtype=x.dtype)


def run(tokens=512, width=1024, hidden=4096, steps=20, dtype=torch.bfloat16, max_norm=None):
    """(losses of the training steps, relative difference of the served output)"""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, target = ((torch.randn(tokens, width, generator=g, device="cuda") * 0.5).to(dtype)
                    for _ in range(3))
    block = FeedForward(width, hidden, dtype)
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, r)
        diff = out - target
        losses.append(float(diff.float().square().mean()))
        _, grads = block.backward(diff * (2.0 / tokens), saved)
        # the second product's curvature grows with the hidden width (h has a mean)
        block.step(grads, 1.0 / hidden, max_norm)
    out = block.forward(x, r)[0].float()
    block.quantize()
    served = block.serve(x, r).float()
    return losses, float((served - out).norm() / out.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 1024), ("hidden", 4096), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--max-norm", type=float, help="clip the gradients to this norm")
    a = ap.parse_args()
    losses, off = run(a.tokens, a.width, a.hidden, a.steps, max_norm=a.max_norm)
    print("loss:", " ".join("%.4f" % v for v in losses))
    print("8-bit against 16-bit output: %.2f %% in the 2-norm" % (100 * off))
