"""What stands beside logits [..., V] has an element for each row in the rows' order: a
tensor of another shape is refused, as its elements would go to other rows."""
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import make_logits

pytestmark = pytest.mark.gpu

B, T, V = 6, 4, 900


@pytest.fixture(scope="module")
def made():
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = make_logits(B * T, V, "bf16", 3).view(B, T, V)
    f = torch.randn(B, T, generator=gen, device="cuda")
    return z, torch.randint(0, V, (B, T), generator=gen, device="cuda"), f


def calls(z, t, f, r=None):
    """Each loss with `t` and `f` in every place that wants an element a row."""
    ids = torch.arange(B * T * 3, device="cuda").view(B, T, 3)
    ref = torch.zeros(B, device="cuda") if r is None else r
    return {
        "target": lambda: flce.policy_loss(z, t, torch.zeros(B, T, device="cuda")),
        "advantage": lambda: flce.policy_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"), f),
        "old_logp": lambda: flce.policy_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"),
                                             torch.zeros(B, T, device="cuda"), old_logp=f),
        "ref_logp": lambda: flce.policy_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"),
                                             torch.zeros(B, T, device="cuda"), ref_logp=f, kl_weight=0.1),
        "row_weight": lambda: flce.policy_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"),
                                               torch.zeros(B, T, device="cuda"), row_weight=f),
        "grad_out": lambda: flce.policy_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"),
                                             torch.zeros(B, T, device="cuda"), reduction="none", grad_out=f),
        "row_weight of a teacher": lambda: flce.distillation_loss(z, ids, torch.zeros(B, T, 3, device="cuda"),
                                                                  row_weight=f),
        "target of pairs": lambda: flce.preference_loss(z, t),
        "reference of pairs": lambda: flce.preference_loss(z, torch.zeros(B, T, dtype=torch.int64, device="cuda"),
                                                           ref_logp=ref),
    }


PLACES = ["target", "advantage", "old_logp", "ref_logp", "row_weight", "grad_out", "row_weight of a teacher",
          "target of pairs", "reference of pairs"]


@pytest.mark.parametrize("place", PLACES)
def test_another_shape_is_refused(made, place):
    z, t, f = made
    for other_t, other_f, other_r in ((t.t().contiguous(), f.t().contiguous(), torch.zeros(B // 2, 2, device="cuda")),
                                      (t.view(2, B // 2, T), f.view(2, B // 2, T), torch.zeros(B // 2, 1, 2, device="cuda"))):
        with pytest.raises(flce.FlceError) as e:
            calls(z, other_t, other_f, other_r)[place]()
        assert e.value.status == 1


@pytest.mark.parametrize("place", PLACES)
def test_the_rows_shape_and_a_flat_one_are_taken(made, place):
    """Also with dimensions of one element, which change no order."""
    z, t, f = made
    r = torch.arange(float(B), device="cuda")
    want = calls(z, t, f, r)[place]()
    for other_t, other_f, other_r in ((t.view(-1), f.view(-1), r.view(B, 1)), (t.view(-1, 1), f.view(-1, 1), r.view(1, B)),
                                      (t.view(B, 1, T), f.view(1, B, T, 1), r.view(2, B // 2))):
        got = calls(z, other_t, other_f, other_r)[place]()
        assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["grad_logits"], want["grad_logits"])


def test_flat_logits_take_what_has_their_rows(made):
    z, t, f = made
    want = flce.policy_loss(z, t, f, row_weight=f)
    got = flce.policy_loss(z.view(B * T, V), t, f, row_weight=f)
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["grad_logits"].view_as(z), want["grad_logits"])


def test_a_term_without_its_reference_is_refused_by_name(made):
    z, t, f = made
    with pytest.raises(flce.FlceError, match="policy_loss: ref_logp"):
        flce.policy_loss(z, t, f, old_logp=f, kl_weight=0.1)
