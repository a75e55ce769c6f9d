"""A teacher's list that names columns which the student's mask rules out, wherever in the list
they stand.

The distance is sum q (ln q - ln p).  With zt the largest logit that a list names, its terms are
q_k (v_k - ln sum e^v) and q_k (z_k - zt) / T, each off by 2^-21 of itself, and ln p of zt: the
tolerance that the lists without a mask have, with logits of the size of those that the mask
leaves.  A masked column's term is q_k |z_k - zt| / T; its share is an exponential of up to -88,
off by 90 * 2^-22 of itself."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import LNS, close, close_grad, cuda, f32, make_logits, wide
from oracle import losses_oracle as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mask", [-3e4, -1e10, -1e30])
@pytest.mark.parametrize("k", [33, 64, 65, 100, 1000])
@pytest.mark.parametrize("v", [1500, 20000, 66000, 280000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_columns_of_small_shares(dtype, v, k, mask):
    n, temperature = 8, 2.0
    z = make_logits(n, v, dtype, k)
    rng = np.random.default_rng(k)
    ids = np.stack([rng.choice(v, k, replace=False) for _ in range(n)])
    values = rng.normal(size=(n, k))
    low = float(torch.tensor(mask, dtype=z.dtype))
    masked = np.zeros((n, k), bool)
    for i, at in enumerate([0, 1, 31, 32, k - 1, k // 2, 0, 0]):
        masked[i, at] = True
    masked[6, :k // 2] = True                      # half of the list
    masked[7, ::2] = True                          # a lane's all
    # shares so that a masked column's term is 1e-3 to 10
    size = -np.log(abs(low) / temperature) + np.log(10.0) * rng.uniform(-3, 1, size=(n, k))
    values = f32(np.where(masked, temperature * size, values))
    for i in range(n):
        z[i, cuda(ids[i][masked[i]])] = low
    out = flce.distillation_loss(z, cuda(ids), cuda(values, torch.float32), temperature=temperature, reduction="none")
    want = L.distill(wide(z), ids, values, temperature=temperature, reduction="none")
    zw = wide(z)
    named = np.take_along_axis(zw, ids, 1)
    q = np.exp(values / temperature - (values / temperature).max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    top = np.where(masked, -np.inf, named).max(1, keepdims=True)
    terms = np.where(masked, q * (top - named), 0).sum(1) / temperature
    plain = np.abs(np.where(zw == low, 0, zw)).max(1) / temperature
    spread = np.abs(want["loss"]) / temperature ** 2
    tol = temperature ** 2 * (LNS + (spread + 2 * plain + 16) * 2.0 ** -20 + terms * 90 * 2.0 ** -22)
    close(wide(out["loss"]), want["loss"], tol, "loss")
    close_grad(out["grad_logits"], want, np.abs(want["f"]) * 90 * 2.0 ** -22, dtype)
