"""The losses without their gradients, as log-probabilities of samples are made: rows by
parts then have several parts on their way at once."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import cuda, f32, make_logits
from test_gpu_losses import DTYPES, check_distill, check_policy, check_preference, on_gpu, policy_inputs, sequences, teacher

pytestmark = pytest.mark.gpu

COLUMNS = [9000, 16384, 33001, 40001, 70001, 128256, 151936, 262144]


@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("place", [(0, 0), (3, 1)])
def test_against_the_definitions(dtype, v, place):
    z = make_logits(6, v, dtype, v, ld=v + place[0], offset=place[1])
    keep = z._base.clone()
    t, a, kw = policy_inputs(z, v)
    out = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), clip=0.2, kl_weight=0.1, want_grad=False)
    assert out["grad_logits"] is None
    check_policy(z, t, a, kw, dtype, out=out)
    for k in (24, 200):
        ids, values = teacher(6, v, k, v)
        check_distill(z, ids, values, dtype, place=dict(want_grad=False), temperature=2.0)
    z, t, offsets = sequences([2, 1, 2, 1], 0, v, dtype, v)
    check_preference(z, t, offsets, dtype, out=flce.preference_loss(z, cuda(t), offsets=cuda(offsets), want_grad=False))
    assert torch.equal(keep.view(torch.uint8), make_logits(6, v, dtype, v, ld=v + place[0], offset=place[1])._base.view(torch.uint8))


@pytest.mark.parametrize("n,v", [(4000, 9000), (2500, 16384), (1500, 40001), (700, 128256), (400, 262144)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("entries", [8, 64, 65, 300])
def test_many_rows_are_those_with_a_gradient(n, v, dtype, entries):
    """Every CTA takes row after row through all of its places in shared memory."""
    z = make_logits(n, v, dtype, n)
    rng = np.random.default_rng(n)
    t, a = cuda(rng.integers(0, v, n)), cuda(f32(rng.normal(size=n)), torch.float32)
    ids, values = cuda(rng.integers(0, v, (n, entries))), cuda(rng.normal(size=(n, entries)), torch.float32)
    for call in (lambda **k: flce.policy_loss(z, t, a, old_logp=a - 9, reduction="none", **k),
                 lambda **k: flce.distillation_loss(z, ids, values, reduction="none", **k)):
        want, got = call(), call(want_grad=False)
        assert torch.equal(got["loss"], want["loss"]) and want["loss"].isfinite().all()
        if "logp" in want:
            assert torch.equal(got["logp"], want["logp"])
