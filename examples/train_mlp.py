"""A two-layer perceptron trained with the library's own operators.

    y = relu2(x W1^T + b1) W2^T + b2 + x

Every product runs in dion.linear_forward / linear_backward (bias, activation
and residual in the product's epilogue); the weight matrices' gradients go
straight into dion.muon_step_batched, which orthogonalizes their momentum by
Newton-Schulz products, or into dion.step_batched (Orth-Dion).  The biases
take plain gradient steps.  Data: a fixed random teacher of the same shape.

    python examples/train_mlp.py [--optimizer muon|dion] [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import rank_orthonormalized_optimizer_dion_amd as dion  # noqa: E402


class Mlp:
    """bfloat16 compute copies of float32 master weights."""

    def __init__(self, width, hidden, gen):
        def matrix(n, k):
            return torch.randn(n, k, generator=gen, device="cuda").mul_(k ** -0.5)
        self.w = [matrix(hidden, width), matrix(width, hidden).mul_(0.1)]
        self.b = [torch.zeros(hidden, device="cuda"), torch.zeros(width, device="cuda")]

    def forward(self, x):
        t, width = x.shape
        hidden = self.w[0].shape[0]
        self.x, self.wb = x, [w.bfloat16() for w in self.w]
        self.z, self.h, y = x.new_empty(t, hidden), x.new_empty(t, hidden), x.new_empty(t, width)
        dion.linear_forward(x, self.wb[0], self.h, bias=self.b[0], act="relu2", preact=self.z)
        dion.linear_forward(self.h, self.wb[1], y, bias=self.b[1], residual=x)
        return y

    def backward(self, dy):
        """Gradients of the two weights (bfloat16) and biases (float32)."""
        dw = [torch.empty_like(w) for w in self.wb]
        db = [torch.empty_like(b) for b in self.b]
        dh = torch.empty_like(self.h)
        dion.linear_backward(dy, self.h, self.wb[1], dx=dh, dw=dw[1], db=db[1])
        dion.linear_backward(dh, self.x, dw=dw[0], db=db[0], act="relu2", preact=self.z)
        return dw, db


def train(optimizer="muon", steps=60, tokens=512, width=256, hidden=768, seed=0):
    """Returns the loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, model = Mlp(width, hidden, gen), Mlp(width, hidden, gen)
    if optimizer == "muon":
        state = [torch.zeros_like(w) for w in model.w]
    else:
        rank = width // 4
        state = [(torch.zeros_like(w),
                  torch.linalg.qr(torch.randn(w.shape[1], rank, generator=gen, device="cuda"))[0].contiguous())
                 for w in model.w]
    ws, losses = None, []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
        diff = model.forward(x).float() - teacher.forward(x).float()
        losses.append(float(diff.square().mean()))
        dw, db = model.backward((diff * (2.0 / diff.numel())).bfloat16())
        if optimizer == "muon":
            ws = dion.muon_step_batched(list(zip(model.w, dw, state)), lr=0.02, momentum=0.9,
                                        scale="spectral", math="f16", workspace=ws)
        else:
            ws = dion.step_batched([(w, g, r, v) for w, g, (r, v) in zip(model.w, dw, state)],
                                   0.02, 0.9, "orth", workspace=ws)
        dion.check_status(ws, len(model.w))
        for b, g in zip(model.b, db):
            b.sub_(g, alpha=0.1)
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--optimizer", choices=("muon", "dion"), default="muon")
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args(argv)
    losses = train(args.optimizer, args.steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
