"""Rows that a policy loss holds one by one: ratios beyond fp32, and rows of no number."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import cuda, f32, make_logits
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
