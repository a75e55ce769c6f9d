"""Rows that a policy loss holds one by one: ratios beyond fp32, and rows of no number."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import cuda, f32, make_logits, wide
from test_gpu_losses import DTYPES, check_policy, policy_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v", [700, 9000, 70001, 290000])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reference", [False, True])
def test_an_advantage_of_zero_takes_no_ratio(dtype, v, reference):
    """exp(logp - old_logp) leaves fp32 at 88, and 0 times it is 0 all the same."""
    z = make_logits(8, v, dtype, v)
    t, a, kw = policy_inputs(z, 3, reference=reference)
    t[:5] = np.arange(5)
    a[:3] = 0.0
    a[3] = abs(a[3])                               # cut
    if reference:
        kw["ref_logp"][:5] = -9.0
    kw["old_logp"][:5] = [-150.0, -400.0, -3.0, -200.0, -5.0]
    for reduction in ("none", "mean"):
        got, _ = check_policy(z, t, a, dict(kw, reduction=reduction), dtype)
    assert got["loss"].isfinite() and got["grad_logits"].isfinite().all()
    if not reference:
        assert (got["grad_logits"][:4] == 0).all()


@pytest.mark.parametrize("v", [700, 9000, 70001, 290000])
@pytest.mark.parametrize("clip", [0.2, math.inf])
def test_rows_of_no_number_on_fresh_samples(v, clip):
    """Without old log-probabilities a row with NaN or infinity has a loss of NaN as well, and no other has."""
    z = make_logits(8, v, "bf16", v)
    t = np.arange(8)
    z[1, 300], z[2, 301], z[3] = float("nan"), float("inf"), float("-inf")
    z[4, 4] = float("-inf")                        # a target of no probability: the ratio is 1
    z[5, 5] = float("nan")                         # the target itself
    t[7], z[7] = -100, float("nan")
    a = torch.tensor([1.0, 2, -1, 1, 1.5, 0, 2, 1], device="cuda")
    out = flce.policy_loss(z, cuda(t), a, clip=clip, reduction="none")
    bad, good = [1, 2, 3, 5], [0, 4, 6, 7]
    assert out["loss"][bad].isnan().all() and out["grad_logits"][bad].isnan().all()
    assert torch.equal(out["loss"][good], -a[good] * torch.tensor([1.0, 1, 1, 0], device="cuda"))
    assert out["grad_logits"][good].isfinite().all() and (out["grad_logits"][7] == 0).all()
    mean = flce.policy_loss(z, cuda(t), a, clip=clip)
    assert mean["loss"].isnan()


@pytest.mark.parametrize("v", [2, 700, 9000, 70001, 290000])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
def test_a_difference_of_log_probabilities_keeps_its_digits(temperature, v):
    """A target far below the one column that has a share: logp is a number of -60 to -120, where fp32 has steps
    of 2^-18 and 2^-17, and logp - old_logp of at most 0.5.  The ratio is off by expf's two units, and three roundings
    of numbers of at most its size: below 2^-21 of it."""
    n, rng = 64, np.random.default_rng(v)
    t32 = float(np.float32(temperature))
    z = torch.full((n, v), -4000.0, device="cuda")
    z[:, 0] = torch.linspace(-9, 9, n, device="cuda")
    t = rng.integers(1, v, n)
    z[torch.arange(n), cuda(t)] = cuda(rng.uniform(-120, -60, n) * temperature, torch.float32)
    zw = z.double().cpu().numpy()
    logp = (zw[np.arange(n), t] - zw[:, 0]) / t32
    old, a = f32(logp - rng.uniform(-0.5, 0.5, n)), f32(rng.normal(size=n))
    out = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), old_logp=cuda(old, torch.float32), clip=math.inf,
                           temperature=temperature, reduction="none")
    want = a * np.exp(logp - old)
    assert (np.abs(-wide(out["loss"]) - want) <= np.abs(want) * 2.0 ** -21).all()
    assert (np.abs(wide(out["logp"]) - logp) <= np.abs(logp) * 2.0 ** -24 + 2.0 ** -30).all()    # half a step of fp32
    slope = wide(out["grad_logits"])[np.arange(n), t] * t32
    assert (np.abs(slope + want) <= np.abs(want) * 2.0 ** -20).all()                             # two products more
