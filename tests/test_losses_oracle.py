"""The 64-bit definitions of the post-training losses against differences of
their own losses, against torch's autograd, and at values that are known."""
import math

import numpy as np
import pytest
import torch

from oracle import losses_oracle as L


def numbers(seed=0, n=7, v=11):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(n, v)) * 2
    t = rng.integers(0, v, n)
    t[2] = -100
    return rng, z, t


def by_differences(loss, z, h=1e-6):
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        g[i] = (loss(up) - loss(down)) / (2 * h)
    return g


# a central difference of step h is off by h^2 / 6 of the third derivative and 2^-53 / h of the value
TOL = 1e-8


@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("kl,temperature,clip_high", [(0.0, 1.0, None), (0.3, 1.0, 0.4), (0.1, 1.7, math.inf)])
def test_policy_gradient_by_differences(kl, temperature, clip_high, reduction):
    rng, z, t = numbers(1)
    a, w = rng.normal(size=7), rng.uniform(0.5, 2, 7)
    logp = L.policy(z, t, a, temperature=temperature)["logp"]
    old, ref = logp + rng.normal(size=7) * 0.3, logp + rng.normal(size=7)
    kw = dict(old_logp=old, ref_logp=ref, kl_weight=kl, temperature=temperature, clip_high=clip_high, row_weight=w,
              reduction=reduction)
    out = L.policy(z, t, a, **kw)
    assert (out["grad"][2] == 0).all() and out["rows"][2] == 0
    assert np.abs(out["grad"] - by_differences(lambda x: L.policy(x, t, a, **kw)["loss"], z)).max() < TOL


def test_policy_without_old_logp_is_the_plain_gradient():
    rng, z, t = numbers(2)
    a = rng.normal(size=7)
    x = torch.tensor(z, requires_grad=True)
    live = torch.tensor(t) >= 0
    logp = torch.log_softmax(x, 1)[torch.arange(7), torch.tensor(t).clamp(min=0)]
    (-(torch.tensor(a) * logp)[live].sum()).backward()
    out = L.policy(z, t, a, reduction="sum")
    assert np.abs(out["grad"] - x.grad.numpy()).max() < 1e-12
    assert np.allclose(out["rows"], np.where(t >= 0, -a, 0))


@pytest.mark.parametrize("temperature", [1.0, 2.5])
@pytest.mark.parametrize("weighted", [False, True])
def test_distill_gradient_by_differences_and_torch(temperature, weighted):
    rng, z, _ = numbers(3)
    ids = np.stack([rng.permutation(11)[:4] for _ in range(7)])
    ids[1, 2:] = -1
    ids[3] = -1
    ids[4, 1] = ids[4, 0]                        # a column that is named twice
    values = rng.normal(size=(7, 4)) * 2
    values[5, 3] = -np.inf
    w = rng.uniform(0.5, 2, 7) if weighted else None
    kw = dict(temperature=temperature, row_weight=w)
    out = L.distill(z, ids, values, **kw)
    assert np.abs(out["grad"] - by_differences(lambda x: L.distill(x, ids, values, **kw)["loss"], z)).max() < TOL
    # a full list is torch's divergence
    full, teacher = np.tile(np.arange(11), (7, 1)), rng.normal(size=(7, 11))
    want = torch.nn.functional.kl_div(torch.log_softmax(torch.tensor(z) / temperature, 1),
                                      torch.softmax(torch.tensor(teacher) / temperature, 1), reduction="sum")
    got = L.distill(z, full, teacher, temperature=temperature, reduction="sum")["loss"]
    assert abs(got - float(want) * temperature ** 2) < 1e-10
    same = L.distill(z, full, z, temperature=temperature, reduction="sum")
    assert abs(same["loss"]) < 1e-12 and np.abs(same["grad"]).max() < 1e-12


@pytest.mark.parametrize("kind,smoothing,margin", [("sigmoid", 0.0, 0.0), ("sigmoid", 0.2, 0.5), ("hinge", 0.0, 0.3),
                                                   ("ipo", 0.0, 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_by_differences(kind, smoothing, margin, average):
    rng, z, t = numbers(4, n=13)
    offsets = np.array([0, 4, 4, 9, 12])          # an empty sequence, and a row behind the last one
    kw = dict(offsets=offsets, ref_logp=rng.normal(size=4), kind=kind, beta=0.3, label_smoothing=smoothing,
              margin=margin, average=average)
    out = L.preference(z, t, **kw)
    assert (out["grad"][12] == 0).all() and out["logp"][1] == 0
    # a loss is off by a few times 2^-53 of its size (ipo's are in the hundreds), its difference by that over the step
    tol = TOL + 8 * 2.0 ** -53 * abs(out["loss"]) / 1e-6
    assert np.abs(out["grad"] - by_differences(lambda x: L.preference(x, t, **kw)["loss"], z)).max() < tol


def test_preference_at_known_values():
    z, t = np.zeros((4, 8)), np.array([1, 2, 3, 4])
    out = L.preference(z, t, offsets=np.array([0, 2, 4]))
    assert abs(out["loss"] - math.log(2)) < 1e-12 and np.allclose(out["logp"], -2 * math.log(8))
    assert abs(out["grad"][0, 1] - (-0.1 * 0.5 * (1 - 1 / 8))) < 1e-12   # the chosen token's logit has to rise
    assert abs(out["grad"][2, 3] - 0.1 * 0.5 * (1 - 1 / 8)) < 1e-12


def test_embedding_gradient_is_torch_s():
    rng = np.random.default_rng(5)
    ids, gy = rng.integers(0, 6, 20), rng.normal(size=(20, 3))
    w = torch.zeros(6, 3, dtype=torch.float64, requires_grad=True)
    (torch.nn.functional.embedding(torch.tensor(ids), w, padding_idx=2) * torch.tensor(gy) * 1.5).sum().backward()
    got, _ = L.embedding_gradient(gy, ids, 6, scale=1.5, padding_index=2)
    assert np.abs(got - w.grad.numpy()).max() < 1e-12
