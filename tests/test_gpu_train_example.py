"""The example's training step: its parts against the definitions in 64 bits, and
that it learns."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import training_oracle as T

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_one_step_end_to_end(norm):
    import train_lm_head as example
    head = example.Head(64, 300, norm=norm, moments="fp32", lr=1e-3)
    x, r, target = next(example.batches(96, 64, 300))
    master, gain = head.master.double().cpu().numpy(), np.ones(64)
    weight = head.weight.double().cpu().numpy()
    loss, grad_x = head.step(x, r, target)
    s = (x.float() + r.float()).to(torch.bfloat16).double().cpu().numpy()
    y, mean, rstd = T.norm_forward(s, gain, None, 1e-5, norm == "rms")
    z = y @ weight.T
    z -= z.max(1, keepdims=True)
    p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
    t = target.cpu().numpy()
    want = -np.log(p[np.arange(96), t]).mean()
    assert abs(float(loss) / want - 1) < 1e-2      # the hidden states are rounded to bf16 in between
    p[np.arange(96), t] -= 1
    p /= 96
    gx, gw, gb = T.norm_backward(p @ weight, s, gain, mean, rstd, None, norm == "rms")
    assert np.abs(grad_x.double().cpu().numpy() - gx).max() <= 3e-2 * np.abs(gx).max()
    grads = [p.T @ y, gw] + ([gb] if norm == "layer" else [])
    scale = min(1.0, 1.0 / (np.sqrt(sum((g * g).sum() for g in grads)) + 1e-6))
    new, _, _ = T.adamw(master, grads[0] * scale, 0.0, 0.0, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, decay=0.01, step=1)
    got = head.master.double().cpu().numpy()
    # the first step moves each weight by lr * sign of its gradient: where that is clear of the bf16 noise, the same way
    clear = np.abs(grads[0]) > 3e-2 * np.abs(grads[0]).max()
    assert clear.sum() > 200 and np.abs(got - new)[clear].max() < 1e-6
    assert torch.equal(head.weight, head.master.to(torch.bfloat16))


@pytest.mark.parametrize("norm,moments", [("rms", "8bit"), ("layer", "fp32"), ("rms", "fp32")])
def test_learns(norm, moments):
    import train_lm_head as example
    losses = example.train(60, norm=norm, moments=moments)
    assert all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0], (losses[0], losses[-1])


def test_8bit_moments_train_like_fp32_ones():
    import train_lm_head as example
    ends = [np.mean(example.train(80, moments=m)[-10:]) for m in ("fp32", "8bit")]
    assert abs(ends[1] / ends[0] - 1) < 0.05, ends
