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


ROWS = 1024   # of a group in one launch


@pytest.mark.parametrize("n,h,dtype,groups", [(1 << 21, 4096, "fp32", 1), (1 << 23, 4096, "bf16", 2),
                                              (3 << 20, 8194, "bf16", 1)])
def test_column_sums_of_very_many_rows(n, h, dtype, groups):
    at_once = ROWS * min(304, torch.cuda.get_device_properties(0).multi_processor_count) * groups
    chain = ROWS + groups + -(-n // at_once) + -(-304 // 32) + 10   # a thread's, the groups', the launches', the CTAs'
    check_column_sums(n, h, dtype, chain)


@pytest.mark.parametrize("h,first,kind", [(8200, 0, "layer"), (8201, 3, "layer"), (8208, 0, "rms")])
def test_rows_of_several_launches(h, first, kind):
    """A call of more rows than one launch takes is the calls of its parts, bit for bit."""
    at_once = ROWS * min(304, torch.cuda.get_device_properties(0).multi_processor_count)
    n = at_once + 1003
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, gy, gx, gx2 = (torch.empty(n * h + 8, dtype=torch.bfloat16, device="cuda")[first:first + n * h].view(n, h)
                      for _ in range(4))
    x.normal_(generator=gen), gy.normal_(generator=gen)
    weight = positive(h, 5, "bf16")
    mean = 0.1 * positive(n, 6) if kind == "layer" else None
    rstd = positive(n, 7)
    sums = [torch.ones(h, device="cuda") for _ in range(4)]

    def backward(rows, out, at):
        flce.layer_norm_backward(gy[rows], x[rows], weight, mean=None if mean is None else mean[rows], rstd=rstd[rows],
                                 kind=kind, grad_sum=x[rows], grad_bias=mean is not None, out=out[rows],
                                 grad_weight_out=sums[at], grad_bias_out=None if mean is None else sums[at + 1],
                                 accumulate=True)

    backward(slice(0, n), gx, 0)
    backward(slice(0, at_once), gx2, 2)
    backward(slice(at_once, n), gx2, 2)
    assert torch.equal(gx, gx2) and torch.equal(sums[0], sums[2]) and torch.equal(sums[1], sums[3])
    # and the rows of the second launch against the definition
    some = slice(n - 200, n)
    xhat = (x[some].double() - (0 if mean is None else mean[some].double()[:, None])) * rstd[some].double()[:, None]
    u = gy[some].double() * weight.double()
    want = u - xhat * (u * xhat).mean(1, keepdim=True) - (0 if mean is None else u.mean(1, keepdim=True))
    want = want * rstd[some].double()[:, None] + x[some].double()
    assert ((gx[some].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all()
