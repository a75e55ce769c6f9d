"""The sizes that the embedding's gradient and the preference loss take: a workspace has a
size where, and only where, the call that it is for is not refused for its sizes."""
import pytest

import linear_cross_entropy_03_gb300 as flce
from test_losses_cpu import FAKE, FAR, INVALID, UNSUPPORTED, WORKSPACE, _gradient, _preference, lib  # noqa: F401


@pytest.mark.parametrize("n,v,h,code", [
    (16, 100, 2097120, WORKSPACE), (16, 100, 2097121, UNSUPPORTED), (16, 100, 1 << 23, UNSUPPORTED),
    (16, 100, 1 << 24, INVALID), ((1 << 31) - 64, 100, 1 << 20, UNSUPPORTED), ((1 << 31) - 64, 100, 128, WORKSPACE),
    ((1 << 31) - 32, 100, 128, INVALID), (16, (1 << 31) - 2, 64, WORKSPACE), (16, (1 << 31) - 1, 64, INVALID)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_embedding_sizes(dtype, n, v, h, code):
    size = flce.embedding_workspace_size(n, v, h)
    assert (size > 0) == (code == WORKSPACE)
    far = dict(dtype=dtype, N=n, V=v, H=h, ld_grad_y=0, grad_y=FAKE, grad_table=FAR)
    assert _gradient(**far, workspace_bytes=max(size, 1) - 1) == code


@pytest.mark.parametrize("n,v,grad,code", [
    ((1 << 31) - 1, 1024, True, WORKSPACE), ((1 << 30) - 1, 2048, True, WORKSPACE), (1 << 30, 2048, True, UNSUPPORTED),
    (1 << 30, 1025, True, UNSUPPORTED), (1 << 30, 2048, False, WORKSPACE), ((1 << 31) - 1, 1 << 20, False, WORKSPACE)])
def test_preference_sizes(n, v, grad, code):
    """Rows times pieces of 1024 columns below 2^31 where a gradient is wanted, as the header has it."""
    size = flce.preference_workspace_size(n, 4)
    assert size > 0
    got = _preference(N=n, V=v, ld=v, ld_grad=v, grad_logits=1 << 62 if grad else None,
                      workspace_bytes=size - (code == WORKSPACE))       # (what has room would be launched)
    assert got == code
