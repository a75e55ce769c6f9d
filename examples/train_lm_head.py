"""Trains the end of a language model, from its last residual add to the loss, on
data that a teacher head labels: every step runs

  layer_norm             of the residual stream and the last block's output
  fused_linear_cross_entropy  of the normalised states with the head
  layer_norm_backward    of its gradient, down to the residual stream
  grad_norm              of all gradients, and the factor that clips them
  AdamW.step             with that factor, on the head's and the norm's weights

The head's master weight is fp32; the step also writes the bf16 copy that the
next projection reads.  Nothing waits for the host between the calls.

    python examples/train_lm_head.py [--steps N] [--moments fp32|8bit] [--norm rms|layer]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_cross_entropy_03_gb300 as flce  # noqa: E402


class Head:
    """The last norm and the head of a model, and their optimiser."""

    def __init__(self, hidden: int, vocabulary: int, *, norm="rms", moments="8bit", lr=1e-2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.norm = norm
        self.gain = torch.ones(hidden, device="cuda")
        self.shift = torch.zeros(hidden, device="cuda") if norm == "layer" else None
        self.master = torch.randn(vocabulary, hidden, generator=gen, device="cuda") * hidden ** -0.5
        self.weight = self.master.to(torch.bfloat16)
        norms = [self.gain] + ([self.shift] if self.shift is not None else [])
        self.optimizer = flce.AdamW(
            [self.master] + norms, lr=lr, betas=(0.9, 0.99), weight_decay=[0.01] + [0.0] * len(norms), moments=moments,
            copies=[self.weight] + [None] * len(norms), seed=seed if moments == "8bit" else None)

    def step(self, block_output, residual, target, *, max_norm=1.0):
        """One training step; returns the loss and the gradient of both inputs."""
        normed = flce.layer_norm(block_output, self.gain, self.shift, kind=self.norm, residual=residual)
        out = flce.fused_linear_cross_entropy(normed["y"], self.weight, target)
        back = flce.layer_norm_backward(out["grad_hidden"], normed["sum"], self.gain, mean=normed["mean"],
                                        rstd=normed["rstd"], kind=self.norm, grad_bias=self.shift is not None)
        grads = [out["grad_weight"], back["grad_weight"]] + ([back["grad_bias"]] if self.shift is not None else [])
        clip = flce.grad_norm(grads, max_norm=max_norm)
        self.optimizer.step(grads, grad_scale=clip["scale"], skip_nonfinite=True)
        return out["loss"], back["grad_x"]


def batches(tokens: int, hidden: int, vocabulary: int, seed=1):
    """Endless batches of (block output, residual stream, target) that a fixed teacher head labels."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn(vocabulary, hidden, generator=gen, device="cuda") * 3 * hidden ** -0.5
    while True:
        parts = torch.randn(2, tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
        states = parts.float().sum(0)
        states = states * torch.rsqrt(states.square().mean(1, keepdim=True))
        yield parts[0], parts[1], (states @ teacher.T).argmax(1)


def train(steps=60, *, tokens=2048, hidden=256, vocabulary=1000, norm="rms", moments="8bit", report=None):
    """Losses of `steps` training steps."""
    head = Head(hidden, vocabulary, norm=norm, moments=moments)
    losses = []
    for step, (block_output, residual, target) in zip(range(steps), batches(tokens, hidden, vocabulary)):
        loss, _ = head.step(block_output, residual, target)
        losses.append(loss)
        if report and step % report == 0:
            print(f"step {step}: loss {float(loss):.4f}")
    return [float(x) for x in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=200)
    parser.add_argument("--moments", choices=("fp32", "8bit"), default="8bit")
    parser.add_argument("--norm", choices=("rms", "layer"), default="rms")
    args = parser.parse_args()
    got = train(args.steps, norm=args.norm, moments=args.moments, report=20)
    print(f"loss {got[0]:.4f} -> {got[-1]:.4f}")
