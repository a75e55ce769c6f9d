"""How a program holds the tensors that it hands to the norm and optimiser calls:
in iterators, and in places that it gives up."""
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce

pytestmark = pytest.mark.gpu


def normal(n, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------ gradients of an iterator

@pytest.mark.parametrize("count,n", [(1, 1000), (3, 300), (20, 1000), (20, 100000), (300, 4001), (1500, 130)])
def test_norm_of_gradients_that_nobody_else_holds(count, n):
    """The memory of temporaries is theirs until the call's kernels are on the stream."""
    grads = [normal(n, k, dtype=torch.bfloat16) for k in range(count)]
    wide = [g.float() for g in grads]
    want = flce.grad_norm(wide, max_norm=1.0)
    for make in (lambda: (g.float() for g in grads), lambda: map(torch.Tensor.float, grads),
                 lambda: [g.float() for g in grads]):
        for _ in range(10):
            got = flce.grad_norm(make(), max_norm=1.0)
            assert torch.equal(got["norm"], want["norm"]) and torch.equal(got["scale"], want["scale"])


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_step_with_gradients_that_nobody_else_holds(moments):
    sizes = [5000, 3, 70001]
    grads = [normal(n, k, 1e-2, torch.bfloat16) for k, n in enumerate(sizes)]
    params = [[normal(n, 10 + k) for k, n in enumerate(sizes)] for _ in range(2)]
    for p, make in zip(params, (list, iter)):
        opt = flce.AdamW(p, lr=1e-2, moments=moments)
        for _ in range(5):
            opt.step(make([g.float() for g in grads]))
    assert all(torch.equal(a, b) for a, b in zip(*params))
    for wrong in (2, 4):
        with pytest.raises(flce.FlceError):
            opt.step(g for g in (grads * 2)[:wrong])
