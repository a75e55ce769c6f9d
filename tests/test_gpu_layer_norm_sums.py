"""Long fp32 sums of the layer norm: their error follows from the sizes, not from the
luck of the roundings.

A sum of terms of one sign whose longest chain has k additions is off by at most
k 2^-24 of it (one rounding each).  The terms here are the same in every row or
column, so that the roundings of a chain go one way for long stretches; the rows
of a matrix are one row at a distance of 0, which costs no memory.
"""
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def positive(n, seed, dtype="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (0.1 + 1.9 * torch.rand(n, generator=g, device="cuda")).to(TYPES[dtype])


def check_column_sums(n, h, dtype, chain):
    """n times one row: the sums over the rows are n times its elements."""
    x, gy = positive(h, 1, dtype), positive(h, 2, dtype)
    ones, zeros = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    out = flce.layer_norm_backward(gy.expand(n, h), x.expand(n, h), mean=zeros, rstd=ones, grad_x=False)
    for got, term in ((out["grad_weight"], gy.double() * x.double()), (out["grad_bias"], gy.double())):
        off = (got.double() / (n * term) - 1).abs().max()
        assert float(off) <= (chain + 1) * UNIT, float(off)   # and the product's own rounding


@pytest.mark.parametrize("n,h,dtype", [(1 << 18, 20001, "fp32"), (100003, 16385, "bf16"), (1 << 20, 63, "bf16")])
def test_column_sums_by_elements(n, h, dtype):
    ranges = max(1, min(304, 8 * 152 // -(-h // 64)))
    rows = -(-n // (4 * ranges))                          # of a thread: batches of 64, then the batches
    chain = 64 + -(-rows // 64) + 4 + -(-304 // 32) + 10  # and four threads' sums, and the ranges'
    check_column_sums(n, h, dtype, chain)


@pytest.mark.parametrize("h", [100001, (1 << 20) + 1, (1 << 24) - 1])
def test_row_sums_of_very_long_rows(h):
    """Rows of one number each: their means, mean squares and, backward, the means of u and u xhat."""
    values = torch.tensor([0.1, 0.7, 1.1, 1.7], device="cuda")
    x = values[:, None].expand(4, h).contiguous()
    exact = values.double()
    chain = 64 + -(-h // (64 * 256)) + 13                 # batches of 64, then the batches, then 256 threads
    tol = (chain + 4) * UNIT                              # and a division, a root, two products
    out = flce.layer_norm(x)
    assert float((out["mean"].double() / exact - 1).abs().max()) <= tol
    out = flce.layer_norm(x, kind="rms", eps=0.0)
    assert float((out["rstd"].double() * exact - 1).abs().max()) <= tol
    assert float((out["y"].double() - 1).abs().max()) <= tol
    # xhat = 0: grad_x = grad_y - mean(grad_y) = 0;  rms with xhat = 1: grad_x = grad_y - mean(grad_y) = 0
    ones, gy = torch.ones(4, device="cuda"), x
    back = flce.layer_norm_backward(gy, x, mean=values, rstd=ones, grad_weight=False, grad_bias=False)
    assert float((back["grad_x"].double().abs().amax(1) / exact).max()) <= tol
    back = flce.layer_norm_backward(gy, torch.ones_like(x), rstd=ones, kind="rms", grad_weight=False, grad_bias=False)
    assert float((back["grad_x"].double().abs().amax(1) / exact).max()) <= tol
