"""The post-training losses and the embedding on the CPU: what their entry points
refuse, before anything touches a GPU, and their workspace sizes."""
import math

import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from linear_cross_entropy_03_gb300 import _build

FAKE, FAR = 0x10000, 1 << 40   # never dereferenced by the refused calls
INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = 1, 2, 3, 7
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return flce.lib()


ROWS = dict(logits=FAKE, dtype="bf16", ld=100, grad_logits=FAR, ld_grad=100, N=16, V=100, reduction="mean",
            grad_scale=1.0, grad_out_none=None, loss=FAKE, workspace=FAKE, workspace_bytes=1 << 40, status_dev=None,
            stream=0)

# what all three refuse alike
ALIKE = [
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(N=-1), INVALID), (dict(N=1 << 31), INVALID),
    (dict(V=0), INVALID), (dict(V=1 << 31, ld=1 << 31, ld_grad=1 << 31), INVALID), (dict(ld=99), INVALID),
    (dict(ld_grad=99), INVALID), (dict(ld=1 << 57), INVALID), (dict(reduction=3), INVALID),
    (dict(reduction=-1), INVALID), (dict(grad_out_none=FAKE), INVALID), (dict(loss=None), INVALID),
    (dict(logits=None), INVALID), (dict(logits=FAKE + 1), MISALIGNED), (dict(grad_logits=FAR + 1), MISALIGNED),
    (dict(loss=FAKE + 2), MISALIGNED), (dict(status_dev=FAKE + 2), MISALIGNED), (dict(workspace=None), WORKSPACE),
    (dict(workspace=FAKE + 128), WORKSPACE), (dict(workspace_bytes=1000), WORKSPACE),
    (dict(grad_logits=FAKE + 32), INVALID), (dict(grad_logits=FAKE, ld_grad=104), INVALID),  # overlap, another pitch
    (dict(dtype="fp32", logits=FAKE + 2), MISALIGNED), (dict(grad_out_none=FAKE + 2, reduction="none"), MISALIGNED),
]


def _policy(numbers=None, **kw):
    args = dict(ROWS, target=FAKE, advantage=FAKE, old_logp=FAKE, ref_logp=FAKE, row_weight=FAKE, ignore_index=-100,
                logp=FAKE, numbers=flce.PolicyNumbers(0.2, 0.2, 0.1, 1.0) if numbers is None else
                flce.PolicyNumbers(*numbers))
    args.update(kw)
    return flce.policy_fwd_bwd(**args)


@pytest.mark.parametrize("kw,code", ALIKE + [
    (dict(target=None), INVALID), (dict(advantage=None), INVALID), (dict(ref_logp=None), INVALID),
    (dict(numbers=(-0.1, 0.2, 0.0, 1.0)), INVALID), (dict(numbers=(0.2, -0.1, 0.0, 1.0)), INVALID),
    (dict(numbers=(NAN, 0.2, 0.0, 1.0)), INVALID), (dict(numbers=(0.2, NAN, 0.0, 1.0)), INVALID),
    (dict(numbers=(0.2, 0.2, -1.0, 1.0)), INVALID), (dict(numbers=(0.2, 0.2, INF, 1.0)), INVALID),
    (dict(numbers=(0.2, 0.2, NAN, 1.0)), INVALID), (dict(numbers=(0.2, 0.2, 0.0, 0.0)), INVALID),
    (dict(numbers=(0.2, 0.2, 0.0, -1.0)), INVALID), (dict(numbers=(0.2, 0.2, 0.0, INF)), INVALID),
    (dict(numbers=(0.2, 0.2, 0.0, NAN)), INVALID), (dict(numbers=(0.2, 0.2, 0.0, 9e-5)), INVALID),
    (dict(numbers=(0.2, 0.2, 0.0, 1.1e4)), INVALID), (dict(target=FAKE + 4), MISALIGNED),
    (dict(advantage=FAKE + 2), MISALIGNED), (dict(old_logp=FAKE + 1), MISALIGNED), (dict(logp=FAKE + 2), MISALIGNED),
    (dict(row_weight=FAKE + 2), MISALIGNED), (dict(ref_logp=FAKE + 2), MISALIGNED),
])
def test_policy_refuses(kw, code):
    assert _policy(**kw) == code


def test_policy_refuses_no_numbers():
    args = dict(ROWS, target=FAKE, advantage=FAKE, old_logp=None, ref_logp=None, row_weight=None, ignore_index=-100,
                logp=None, numbers=None)
    assert flce.policy_fwd_bwd(**args) == INVALID


def _distill(**kw):
    args = dict(ROWS, ids=FAKE, index_type="int64", values=FAKE, value_dtype="bf16", top=8, row_weight=None,
                temperature=1.0)
    args.update(kw)
    return flce.distill_fwd_bwd(**args)


@pytest.mark.parametrize("kw,code", ALIKE + [
    (dict(ids=None), INVALID), (dict(values=None), INVALID), (dict(index_type=2), INVALID),
    (dict(index_type="int16"), INVALID), (dict(value_dtype=3), UNSUPPORTED), (dict(top=0), INVALID),
    (dict(top=1025), UNSUPPORTED), (dict(temperature=0.0), INVALID), (dict(temperature=NAN), INVALID),
    (dict(temperature=INF), INVALID), (dict(temperature=1e-5), INVALID), (dict(temperature=1e5), INVALID),
    (dict(ids=FAKE + 4), MISALIGNED), (dict(values=FAKE + 1), MISALIGNED),
    (dict(index_type="int32", ids=FAKE + 2), MISALIGNED), (dict(row_weight=FAKE + 2), MISALIGNED),
])
def test_distill_refuses(kw, code):
    assert _distill(**kw) == code


def _preference(numbers=(0, 0, 0.1, 0.0, 0.0), **kw):
    args = dict(ROWS, target=FAKE, offsets=FAKE, ref_logp=FAKE, pairs=4, ignore_index=-100, logp=FAKE,
                numbers=flce.PreferenceNumbers(*numbers))
    args.update(kw)
    return flce.preference_fwd_bwd(**args)


@pytest.mark.parametrize("kw,code", ALIKE + [
    (dict(target=None), INVALID), (dict(pairs=-1), INVALID), (dict(pairs=1 << 30), INVALID),
    (dict(numbers=(3, 0, 0.1, 0.0, 0.0)), INVALID), (dict(numbers=(-1, 0, 0.1, 0.0, 0.0)), INVALID),
    (dict(numbers=(0, 2, 0.1, 0.0, 0.0)), INVALID), (dict(numbers=(0, 0, 0.0, 0.0, 0.0)), INVALID),
    (dict(numbers=(0, 0, NAN, 0.0, 0.0)), INVALID), (dict(numbers=(0, 0, 0.1, 1.0, 0.0)), INVALID),
    (dict(numbers=(0, 0, 0.1, -0.1, 0.0)), INVALID), (dict(numbers=(1, 0, 0.1, 0.1, 0.0)), INVALID),
    (dict(numbers=(2, 0, 0.1, 0.0, 0.5)), INVALID), (dict(numbers=(0, 0, 0.1, 0.0, INF)), INVALID),
    (dict(offsets=None, N=15), INVALID), (dict(offsets=None, pairs=0), INVALID), (dict(offsets=FAKE + 4), MISALIGNED),
    (dict(ref_logp=FAKE + 2), MISALIGNED), (dict(logp=FAKE + 2), MISALIGNED), (dict(target=FAKE + 4), MISALIGNED),
    (dict(N=(1 << 31) - 1, V=1 << 20, ld=1 << 20, ld_grad=1 << 20, grad_logits=1 << 62), UNSUPPORTED),
])
def test_preference_refuses(kw, code):
    assert _preference(**kw) == code


def test_loss_workspace_sizes():
    assert flce.row_loss_workspace_size(-1) == 0 and flce.row_loss_workspace_size(1 << 31) == 0
    assert 0 < flce.row_loss_workspace_size(0) <= flce.row_loss_workspace_size(1 << 20) < 1 << 17
    assert flce.preference_workspace_size(-1, 2) == 0 and flce.preference_workspace_size(5, -1) == 0
    small, large = flce.preference_workspace_size(1 << 10, 4), flce.preference_workspace_size(1 << 20, 4)
    assert large - small == ((1 << 20) - (1 << 10)) * 16     # logp, factor and two statistics a row


def _lookup(**kw):
    args = dict(dtype="bf16", table=FAR, ld_table=64, ids=FAKE, index_type="int64", N=16, V=100, H=64, scale=1.0,
                y=2 * FAR, ld_y=64, status_dev=None, stream=0)
    args.update(kw)
    return flce.embedding_fwd(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNSUPPORTED), (dict(index_type=5), INVALID), (dict(N=-1), INVALID), (dict(V=0), INVALID),
    (dict(H=0), INVALID), (dict(H=1 << 24, ld_table=1 << 24, ld_y=1 << 24), INVALID), (dict(ld_table=63), INVALID),
    (dict(ld_y=63), INVALID), (dict(ld_y=1 << 57), INVALID), (dict(table=None), INVALID), (dict(ids=None), INVALID),
    (dict(y=None), INVALID), (dict(table=FAR + 1), MISALIGNED), (dict(y=2 * FAR + 1), MISALIGNED),
    (dict(ids=FAKE + 4), MISALIGNED), (dict(index_type="int32", ids=FAKE + 2), MISALIGNED),
    (dict(status_dev=FAKE + 2), MISALIGNED), (dict(y=FAR + 64), INVALID), (dict(y=FAR), INVALID),
])
def test_embedding_fwd_refuses(kw, code):
    assert _lookup(**kw) == code


def _gradient(**kw):
    args = dict(dtype="bf16", grad_y=FAR, ld_grad_y=64, ids=FAKE, index_type="int64", N=16, V=100, H=64, scale=1.0,
                padding_index=-1, grad_table=2 * FAR, accumulate=0, workspace=FAKE, workspace_bytes=1 << 40,
                status_dev=None, stream=0)
    args.update(kw)
    return flce.embedding_bwd(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), UNSUPPORTED), (dict(index_type=2), INVALID), (dict(N=-1), INVALID), (dict(N=1 << 31), INVALID),
    (dict(V=0), INVALID), (dict(H=0), INVALID), (dict(H=1 << 24), INVALID), (dict(ld_grad_y=-1), INVALID),
    (dict(ld_grad_y=1 << 57), INVALID), (dict(padding_index=-2), INVALID), (dict(padding_index=100), INVALID),
    (dict(accumulate=2), INVALID), (dict(grad_y=None), INVALID), (dict(ids=None), INVALID),
    (dict(grad_table=None), INVALID), (dict(grad_y=FAR + 1), MISALIGNED), (dict(grad_table=2 * FAR + 2), MISALIGNED),
    (dict(ids=FAKE + 4), MISALIGNED), (dict(workspace=None), WORKSPACE), (dict(workspace=FAKE + 16), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE), (dict(grad_table=FAR + 64), INVALID), (dict(status_dev=FAKE + 2), MISALIGNED),
    (dict(N=(1 << 31) - 64, H=1 << 20, ld_grad_y=0, workspace_bytes=1 << 62), UNSUPPORTED),
])
def test_embedding_bwd_refuses(kw, code):
    assert _gradient(**kw) == code


def test_embedding_workspace_sizes():
    assert flce.embedding_workspace_size(-1, 5, 5) == 0 and flce.embedding_workspace_size(5, 0, 5) == 0
    assert flce.embedding_workspace_size(0, 5, 5) > 0
    # partial rows are far fewer than the rows of grad_y
    assert flce.embedding_workspace_size(1 << 14, 128256, 4096) < (1 << 14) * 4096 * 2 / 4


def test_tensors_that_are_not_on_the_gpu_are_refused():
    z, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call in (lambda: flce.policy_loss(z, t, f), lambda: flce.preference_loss(z, t, offsets=t[:3]),
                 lambda: flce.distillation_loss(z, t[:, None], f[:, None]), lambda: flce.embedding(z, t),
                 lambda: flce.embedding_backward(z, t, 5), lambda: flce.policy_loss(None, t, f)):
        with pytest.raises(flce.FlceError) as e:
            call()
        assert e.value.status == INVALID
