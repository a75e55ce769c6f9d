"""The norm and optimiser entry points on the CPU: what they refuse, before
anything touches a GPU, and their workspace sizes."""
import ctypes
import math

import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from linear_cross_entropy_03_gb300 import _build

FAKE = 0x10000   # never dereferenced by the refused calls
FAR = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = 1, 2, 3, 7


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return flce.lib()


def _fwd(**kw):
    args = dict(kind="layer", dtype="bf16", x=FAKE, ld_x=64, residual=None, ld_residual=0, weight=FAKE, bias=FAKE,
                param_dtype="bf16", N=16, H=64, eps=1e-5, y=FAR, ld_y=64, sum=None, ld_sum=0, mean=FAKE, rstd=FAKE,
                stream=0)
    args.update(kw)
    return flce.ln_fwd(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=2), INVALID), (dict(kind="other"), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(param_dtype=9), UNSUPPORTED), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(H=1 << 24), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(ld_x=-1), INVALID), (dict(ld_y=63), INVALID),
    (dict(ld_x=1 << 30), INVALID), (dict(ld_y=1 << 30), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(sum=3 * FAR, ld_sum=64), INVALID),
    (dict(residual=2 * FAR, ld_residual=64, sum=3 * FAR, ld_sum=32), INVALID),
    (dict(residual=2 * FAR, ld_residual=-5), INVALID),
    (dict(kind="rms"), INVALID),                                     # a mean is asked for
    (dict(x=FAKE + 1), MISALIGNED), (dict(y=FAR + 1), MISALIGNED), (dict(dtype="fp32", x=FAKE + 2), MISALIGNED),
    (dict(rstd=FAKE + 2), MISALIGNED), (dict(param_dtype="fp32", weight=FAKE + 2), MISALIGNED),
    (dict(y=FAKE + 16), INVALID), (dict(y=FAKE, ld_y=128), INVALID),  # partial overlap, another pitch
    (dict(residual=FAR, ld_residual=64, sum=FAR, ld_sum=64), INVALID),  # y and sum the same
    (dict(ld_x=0, y=FAKE), INVALID),                                  # one row read N times and written over
])
def test_ln_fwd_refuses(kw, code):
    assert _fwd(**kw) == code


def _bwd(**kw):
    args = dict(kind="layer", dtype="bf16", grad_y=FAKE, ld_grad_y=64, x=FAR, ld_x=64, weight=FAKE, param_dtype="bf16",
                mean=FAKE, rstd=FAKE, grad_sum=None, ld_grad_sum=0, N=16, H=64, grad_x=2 * FAR, ld_grad_x=64,
                grad_weight=FAKE, grad_bias=FAKE, accumulate=0, workspace=FAKE, workspace_bytes=1 << 30, stream=0)
    args.update(kw)
    return flce.ln_bwd(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=-1), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(param_dtype=5), UNSUPPORTED), (dict(N=-1), INVALID),
    (dict(H=0), INVALID), (dict(accumulate=2), INVALID), (dict(ld_grad_y=-1), INVALID), (dict(ld_x=-1), INVALID),
    (dict(ld_grad_x=63), INVALID), (dict(grad_sum=3 * FAR, ld_grad_sum=-1), INVALID),
    (dict(grad_sum=3 * FAR, ld_grad_sum=64, grad_x=None), INVALID), (dict(kind="rms"), INVALID),
    (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(x=None), INVALID), (dict(grad_y=None), INVALID),
    (dict(x=FAR + 1), MISALIGNED), (dict(grad_weight=FAKE + 2), MISALIGNED), (dict(grad_x=FAR + 32), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=FAKE + 16), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE),
])
def test_ln_bwd_refuses(kw, code):
    assert _bwd(**kw) == code


def test_ln_workspace_sizes():
    assert flce.ln_workspace_size(-1, 8) == 0 and flce.ln_workspace_size(4, 0) == 0
    assert flce.ln_workspace_size(0, 8) > 0
    small, large = flce.ln_workspace_size(16384, 4096), flce.ln_workspace_size(1 << 20, 4096)
    assert large - small == ((1 << 20) - 16384) * 8      # grows with the rows by their two means alone
    assert small < 16384 * 4096 * 2 / 8


def _norm(entries, **kw):
    table = (flce.TensorEntry * max(1, len(entries)))(*[flce.TensorEntry(*e) for e in entries])
    args = dict(tensors=table, count=len(entries), grad_scale=1.0, max_norm=1.0, eps=1e-6, out=FAKE, workspace=FAKE,
                workspace_bytes=1 << 30, stream=0)
    args.update(kw)
    return flce.grad_norm_raw(**args)


@pytest.mark.parametrize("entries,kw,code", [
    ([], dict(count=-1), INVALID), ([], dict(count=2, tensors=None), INVALID), ([], dict(out=None), INVALID),
    ([], dict(out=FAKE + 2), MISALIGNED), ([], dict(max_norm=-1.0), INVALID), ([], dict(max_norm=math.nan), INVALID),
    ([], dict(grad_scale=math.inf), INVALID), ([], dict(eps=-1.0), INVALID), ([], dict(workspace=None), WORKSPACE),
    ([], dict(workspace_bytes=64), WORKSPACE), ([(FAKE, -1, 1, 0)], {}, INVALID), ([(None, 5, 1, 0)], {}, INVALID),
    ([(FAKE, 5, 3, 0)], {}, UNSUPPORTED), ([(FAKE + 2, 5, 1, 0)], {}, MISALIGNED), ([(FAKE + 1, 5, 0, 0)], {}, MISALIGNED),
])
def test_grad_norm_refuses(entries, kw, code):
    assert _norm(entries, **kw) == code


def test_grad_norm_workspace_sizes():
    assert flce.grad_norm_workspace_size(-1) == 0
    assert 0 < flce.grad_norm_workspace_size(0) <= flce.grad_norm_workspace_size(100000)


def _entry(**kw):
    e = dict(param=FAKE, grad=FAR, exp_avg=2 * FAR, exp_avg_sq=3 * FAR, exp_avg_scale=None, exp_avg_sq_scale=None,
             copy=None, n=100, lr_scale=1.0, weight_decay=0.1, param_dtype=1, grad_dtype=1, copy_dtype=0,
             moment_bits=32)
    e.update(kw)
    return flce.AdamWEntry(**e)


def _numbers(**kw):
    n = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=1.0)
    n.update(kw)
    return flce.AdamWNumbers(**n)


@pytest.mark.parametrize("entry,numbers,code", [
    (dict(n=-1), {}, INVALID), (dict(param=None), {}, INVALID), (dict(grad=None), {}, INVALID),
    (dict(exp_avg=None), {}, INVALID), (dict(exp_avg_sq=None), {}, INVALID), (dict(param_dtype=3), {}, UNSUPPORTED),
    (dict(grad_dtype=-1), {}, UNSUPPORTED), (dict(copy=FAKE, copy_dtype=4), {}, UNSUPPORTED),
    (dict(moment_bits=16), {}, UNSUPPORTED), (dict(moment_bits=8), {}, INVALID),
    (dict(moment_bits=8, exp_avg_scale=FAKE), {}, INVALID), (dict(exp_avg_scale=FAKE), {}, INVALID),
    (dict(moment_bits=8, exp_avg_scale=FAKE, exp_avg_sq_scale=FAKE + 2), {}, MISALIGNED),
    (dict(param=FAKE + 2), {}, MISALIGNED), (dict(grad=FAR + 1, grad_dtype=0), {}, MISALIGNED),
    (dict(exp_avg=FAR + 2), {}, MISALIGNED), (dict(copy=FAKE + 1), {}, MISALIGNED),
    (dict(lr_scale=math.nan), {}, INVALID), (dict(weight_decay=math.inf), {}, INVALID),
    ({}, dict(beta1=1.0), INVALID), ({}, dict(beta2=-0.1), INVALID), ({}, dict(beta1=math.nan), INVALID),
    ({}, dict(eps=-1e-8), INVALID), ({}, dict(lr=math.inf), INVALID), ({}, dict(step=0), INVALID),
    ({}, dict(skip_nonfinite=2), INVALID), ({}, dict(stochastic=-1), INVALID),
    ({}, dict(step_dev=FAKE + 4), MISALIGNED), ({}, dict(lr_dev=FAKE + 2), MISALIGNED),
    ({}, dict(grad_scale_dev=FAKE + 2), MISALIGNED),
])
def test_adamw_refuses(entry, numbers, code):
    table = (flce.AdamWEntry * 1)(_entry(**entry))
    assert flce.adamw_step(table, 1, _numbers(**numbers), 0) == code


def test_adamw_refuses_tables():
    assert flce.adamw_step(None, 1, _numbers(), 0) == INVALID
    assert flce.adamw_step(None, -1, _numbers(), 0) == INVALID
    assert flce.adamw_step(None, 0, None, 0) == INVALID
    assert flce.adamw_step(None, 0, _numbers(), 0) == 0          # nothing to do


def test_structures_match_the_header():
    assert ctypes.sizeof(flce.TensorEntry) == 24
    assert ctypes.sizeof(flce.AdamWEntry) == 88
    assert ctypes.sizeof(flce.AdamWNumbers) == 88
    assert flce.flce_kernel_name(14) == "adamw" and flce.KERNEL_NAMES[14] == "adamw"
    assert all(flce.flce_kernel_name(i) == name for i, name in enumerate(flce.KERNEL_NAMES))


def test_tensors_that_are_not_on_the_gpu_are_refused():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: flce.layer_norm(x), lambda: flce.layer_norm_backward(x, x, rstd=torch.ones(4)),
                 lambda: flce.grad_norm([x]), lambda: flce.AdamW([x], lr=1e-3)):
        with pytest.raises(flce.FlceError):
            call()
    with pytest.raises(flce.FlceError):
        flce.layer_norm(x.double())
