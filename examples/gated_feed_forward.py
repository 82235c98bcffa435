"""A pre-norm gated feed-forward block, trained with clipped gradients and served in 8 bits.

    s = x + r;  y = layernorm(s) * g + c;  h = silu(y Wg^T) * (y Wu^T);  out = h Wd^T + s

Training: forward and backward in bf16 (float16 or float32 as well), the gradients of all
parameters clipped by their common norm, and a step.  Nothing in a step waits for the
GPU on the host.
Serving: the weights brought to 8 bits once; every step the norm writes 8-bit rows with
scales, the gated product reads 8-bit operands, and the last product adds the residual
stream in its epilogue.

    python examples/gated_feed_forward.py [--tokens 512] [--width 1024] [--hidden 2816] [--steps 20]

prints the loss and the gradients' norm of a few training steps on a fixed regression target,
and how far the 8-bit block's output is from the trained 16-bit one's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402


class GatedFeedForward:
    PARAMETERS = ("g", "c", "wg", "wu", "wd")

    def __init__(self, width, hidden, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda n, k: (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(dtype)  # noqa: E731
        self.g = torch.ones(width, device="cuda", dtype=dtype)
        self.c = torch.zeros(width, device="cuda", dtype=dtype)
        self.wg, self.wu, self.wd = new(hidden, width), new(hidden, width), new(width, hidden)
        self.q = None

    def forward(self, x, r):
        """Output and what the backward pass needs."""
        y, s, mean, rstd = sg.add_layernorm(x, self.g, self.c, r)
        h, zg, zu = sg.gated_linear(y, self.wg, self.wu, save_preact=True)
        return sg.linear(h, self.wd, residual=s), (y, s, mean, rstd, h, zg, zu)

    def backward(self, dout, saved):
        """Gradients of x (and r alike) and of the parameters, in their order."""
        y, s, mean, rstd, h, zg, zu = saved
        dh, dwd, _ = sg.linear_backward(dout, h, self.wd, need_db=False)
        dy, dwg, dwu, _, _ = sg.gated_linear_backward(dh, y, self.wg, self.wu, zg, zu, need_db=False)
        dx, dg, dc = sg.add_layernorm_backward(dy, s, mean, rstd, self.g, dout)   # the residual's joins
        return dx, [dg, dc, dwg, dwu, dwd]

    def step(self, grads, rate, max_norm):
        """One step along the clipped gradients; returns their norm before clipping."""
        norm = sg.clip_grad_norm(grads, max_norm)
        for name, d in zip(self.PARAMETERS, grads):
            getattr(self, name).add_(d, alpha=-rate)
        self.q = None
        return norm

    def quantize(self):
        """8-bit weights with a scale per output feature, made once."""
        self.q = [sg.quantize_rows(w) for w in (self.wg, self.wu, self.wd)]

    def serve(self, x, r):
        (qg, sgate), (qu, sup), (qd, sdown) = self.q
        y, ys, s, _, _ = sg.add_layernorm(x, self.g, self.c, r, quantize=True)
        h = sg.gated_linear(y, qg, qu, x_scale=ys, gate_scale=sgate, up_scale=sup, out_dtype=x.dtype)
        hq, hs = sg.quantize_rows(h)
        return sg.linear(hq, qd, residual=s, x_scale=hs, w_scale=sdown, out_dtype=x.dtype)


def run(tokens=512, width=1024, hidden=2816, steps=20, dtype=torch.bfloat16, max_norm=1.0):
    """(losses, gradient norms of the training steps, relative difference of the served output)"""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, target = ((torch.randn(tokens, width, generator=gen, device="cuda") * 0.5).to(dtype)
                    for _ in range(3))
    block = GatedFeedForward(width, hidden, dtype)
    losses, norms = [], []
    for _ in range(steps):
        out, saved = block.forward(x, r)
        diff = out - target
        losses.append(diff.float().square().mean())
        _, grads = block.backward(diff * (2.0 / tokens), saved)
        norms.append(block.step(grads, 0.1, max_norm))
    out = block.forward(x, r)[0].float()
    block.quantize()
    served = block.serve(x, r).float()
    return ([float(v) for v in losses], [float(v) for v in norms],
            float((served - out).norm() / out.norm()))


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 1024), ("hidden", 2816), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    losses, norms, off = run(a.tokens, a.width, a.hidden, a.steps)
    print("loss:", " ".join("%.4f" % v for v in losses))
    print("norm:", " ".join("%.4f" % v for v in norms))
    print("8-bit against 16-bit output: %.2f %% in the 2-norm" % (100 * off))
