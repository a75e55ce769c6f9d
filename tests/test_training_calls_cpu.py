"""What the norm and optimiser calls do with their tensors on the host: no GPU is needed."""
import gc
import weakref

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import linear_cross_entropy_03_gb300 as flce
from linear_cross_entropy_03_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return flce.lib()


def test_a_failing_call_lets_go_of_its_gradients():
    """A tensor without memory makes torch throw inside the extension: what an iterator yielded goes all the same."""
    with FakeTensorMode():
        held = [torch.empty(4, device="cuda")]
    seen = weakref.ref(held[0])

    def yields():
        yield held.pop()

    with pytest.raises(RuntimeError):
        flce.grad_norm(yields())
    gc.collect()
    assert seen() is None
