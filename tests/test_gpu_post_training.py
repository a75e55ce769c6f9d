"""A step of post-training as a program runs it, on a table that the embedding and
the head share: lookup, norm, head, a loss with its gradient on the logits, and
back down to the table, whose gradient is the head's and the embedding's; then the
clip and AdamW.  Against the same in 64 bits, and captured in a graph."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import close, cuda, f32, wide
from oracle import losses_oracle as L
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu

N, H, V = 96, 64, 520
SCALE = 8.0


class Model:
    """A table, a gain, and what a step needs of a batch."""

    def __init__(self, loss, seed=3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.loss = loss
        self.master = torch.randn(V, H, generator=gen, device="cuda") * H ** -0.5
        self.gain = torch.rand(H, generator=gen, device="cuda") + 0.5
        self.optimizer = flce.AdamW([self.master, self.gain], lr=1e-3, weight_decay=0.0, capturable=True)
        self.tokens = cuda(rng.integers(0, 40, N))
        self.target = cuda(np.where(rng.random(N) < 0.2, -100, rng.integers(0, V, N)))
        self.advantage = cuda(f32(rng.normal(size=N)), torch.float32)
        self.old = cuda(f32(-rng.random(N) - 6.0), torch.float32)
        self.ids = cuda(np.stack([rng.choice(V, 9, replace=False) for _ in range(N)]))
        self.values = cuda(f32(rng.normal(size=(N, 9)) * 2), torch.float32)
        self.offsets = cuda(np.array([0, 30, 50, 75, 96]))

    def run_loss(self, z):
        if self.loss == "policy":
            return flce.policy_loss(z, self.target, self.advantage, old_logp=self.old, clip=0.5)
        if self.loss == "preference":
            return flce.preference_loss(z, self.target, offsets=self.offsets, beta=0.5)
        return flce.distillation_loss(z, self.ids, self.values, temperature=2.0)

    def want_loss(self, z):
        if self.loss == "policy":
            return L.policy(z, wide(self.target).astype(np.int64), wide(self.advantage), old_logp=wide(self.old), clip=0.5)
        if self.loss == "preference":
            return L.preference(z, wide(self.target).astype(np.int64), offsets=wide(self.offsets).astype(np.int64), beta=0.5)
        return L.distill(z, wide(self.ids).astype(np.int64), wide(self.values), temperature=2.0)

    def gradients(self):
        x = flce.embedding(self.master, self.tokens, scale=SCALE)["y"]
        normed = flce.layer_norm(x, self.gain, kind="rms")
        z = normed["y"] @ self.master.T
        out = self.run_loss(z)
        table = out["grad_logits"].T @ normed["y"]
        back = flce.layer_norm_backward(out["grad_logits"] @ self.master, x, self.gain, rstd=normed["rstd"], kind="rms",
                                        grad_bias=False)
        flce.embedding_backward(back["grad_x"], self.tokens, scale=SCALE, grad_weight_out=table, accumulate=True)
        return out["loss"], [table, back["grad_weight"]]

    def step(self):
        loss, grads = self.gradients()
        clip = flce.grad_norm(grads, max_norm=1.0)
        self.optimizer.step(grads, grad_scale=clip["scale"], skip_nonfinite=True)
        return loss

    def loss_at(self, master, gain):
        x = master[wide(self.tokens).astype(np.int64)] * SCALE
        y, _, rstd = T.norm_forward(x, gain, None, 1e-5, True)
        out = self.want_loss(y @ master.T)
        return out, x, y, rstd


LOSSES = ["policy", "preference", "distill"]


@pytest.mark.parametrize("loss", LOSSES)
def test_gradients_end_to_end(loss):
    model = Model(loss)
    master, gain = wide(model.master), wide(model.gain)
    got, grads = model.gradients()
    want, x, y, rstd = model.loss_at(master, gain)
    table = want["grad"].T @ y
    gx, gw, _ = T.norm_backward(want["grad"] @ master, x, gain, None, rstd, None, True)
    below, size = L.embedding_gradient(gx, wide(model.tokens).astype(np.int64), V, scale=SCALE)
    # fp32 products of 64 to 520 terms with torch's own order: 520 * 2^-24 of the terms' sizes, and the losses' 2e-5
    tol = 1e-4 * (np.abs(want["grad"]).T @ np.abs(y) + size)
    assert abs(float(got) - want["loss"]) <= 1e-4 * max(1.0, abs(want["loss"]))
    close(wide(grads[0]), table + below, tol, "table")
    close(wide(grads[1]), gw, 1e-4 * (np.abs(want["grad"] @ master) * np.abs(x) * rstd[:, None]).sum(0), "gain")
    # and the formulas against differences of the loss, along one direction
    rng = np.random.default_rng(1)
    d, e, h = rng.normal(size=master.shape), rng.normal(size=gain.shape), 1e-6
    up, down = (model.loss_at(master + s * h * d, gain + s * h * e)[0]["loss"] for s in (1, -1))
    slope = ((table + below) * d).sum() + (gw * e).sum()
    # a ratio that crosses the clip's border within h would show here: none of these does
    assert abs((up - down) / (2 * h) - slope) <= 1e-5 * (np.abs((table + below) * d).sum() + np.abs(gw * e).sum())


@pytest.mark.parametrize("loss", LOSSES)
def test_steps_captured_in_a_graph(loss):
    eager, model = Model(loss), Model(loss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = model.step()
    torch.cuda.synchronize()
    assert torch.equal(first, eager.step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss_of_step = model.step()
    for _ in range(5):
        graph.replay()
        want = eager.step()
        torch.cuda.synchronize()
        assert torch.equal(loss_of_step, want) and torch.equal(model.master, eager.master)
        assert torch.equal(model.gain, eager.gain)
