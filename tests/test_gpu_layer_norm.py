"""Layer norm and its rms form on the GPU against the definition in 64 bits.

Tolerances, fixed by the arithmetic: u is half a unit in the last place of the
stored type (2^-8, 2^-11, 2^-24).  The row sums run in fp32 over chains of at
most H / 256 + 10 additions, so with H <= 20000 a mean is off by less than 2^-17
of the mean magnitude of its terms; everything after is a handful of roundings.
"""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}
SUM = 2.0 ** -17


def host(t):
    return None if t is None else t.double().cpu().numpy()


def rows(n, h, dtype, seed, scale=1.0, mean=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    channel = torch.exp(0.5 * torch.randn(h, generator=g, device="cuda"))
    return ((torch.randn(n, h, generator=g, device="cuda") * channel + mean) * scale).to(TYPES[dtype])


def vector(h, dtype, seed, mean):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + 0.2 * torch.randn(h, generator=g, device="cuda")).to(TYPES[dtype])


def check_forward(out, x, residual, weight, bias, eps, rms, dtype):
    """`out` against the definition on the sum that the call stored (which is checked too)."""
    u, s = UNIT[dtype], host(x)
    if residual is not None:
        exact, s = s + host(residual), host(out["sum"])
        assert (np.abs(s - exact) <= (u + 2.0 ** -23) * np.abs(exact) + TINY[dtype]).all()
    y, mean, rstd = T.norm_forward(s, host(weight), host(bias), eps, rms)
    w = np.abs(host(weight)) if weight is not None else 1.0
    b = np.abs(host(bias)) if bias is not None else 0.0
    xhat = np.abs(s - mean[:, None]) * rstd[:, None]
    reach = np.abs(s).max(1, keepdims=True) * rstd[:, None]
    tol = u * np.abs(y) + TINY[dtype] + SUM * (w * (reach + xhat) + b)
    got = host(out["y"]).reshape(y.shape)
    assert (np.abs(got - y) <= tol).all(), np.max(np.abs(got - y) / tol)
    if rms:
        assert out["mean"] is None
    else:
        assert (np.abs(host(out["mean"]).reshape(-1) - mean) <= SUM * np.abs(s).mean(1) + 1e-30).all()
    off = np.abs(host(out["rstd"]).reshape(-1) / rstd - 1)
    assert (off <= SUM * (1 + (reach[:, 0] if not rms else 0))).all()


def backward_reference(gy, x, weight, mean, rstd, grad_sum, rms):
    ref = T.norm_backward(host(gy), host(x), host(weight), host(mean), host(rstd), host(grad_sum), rms)
    inv = host(rstd)[:, None]
    xhat = np.abs(host(x) - (0 if rms else host(mean)[:, None])) * inv
    g = np.abs(host(gy))
    size = g if weight is None else g * np.abs(host(weight))
    # |u| + mean |u| + |xhat| mean |u xhat|, each to the sums' precision
    loose = inv * (size + (0 if rms else size.mean(1, keepdims=True)) + 2 * xhat * (size * xhat).mean(1, keepdims=True))
    return ref, SUM * loose, (g * xhat).sum(0), g.sum(0)


def check_backward(out, gy, x, weight, mean, rstd, grad_sum, rms, dtype):
    (gx, gw, gb), loose, size_w, size_b = backward_reference(gy, x, weight, mean, rstd, grad_sum, rms)
    if out["grad_x"] is not None:
        tol = UNIT[dtype] * np.abs(gx) + TINY[dtype] + loose
        if grad_sum is not None:
            tol += 2.0 ** -23 * np.abs(host(grad_sum))
        got = host(out["grad_x"]).reshape(gx.shape)
        assert (np.abs(got - gx) <= tol).all(), np.max(np.abs(got - gx) / tol)
    # sums over the rows: chains of at most N / 4 / parts + 20 additions
    if out["grad_weight"] is not None:
        assert (np.abs(host(out["grad_weight"]) - gw) <= 2 * SUM * size_w + 1e-30).all()
    if out["grad_bias"] is not None:
        assert (np.abs(host(out["grad_bias"]) - gb) <= 2 * SUM * size_b + 1e-30).all()


SIZES = [(1, 1), (1, 8), (3, 1), (2, 33), (5, 64), (4, 127), (7, 128), (64, 256), (9, 1000), (33, 1024), (31, 2047),
         (130, 2048), (1, 4096), (301, 4096), (17, 5120), (20, 8192), (9, 12289), (3, 16384), (700, 768), (1, 20000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,h", SIZES)
def test_forward_and_backward(n, h, dtype):
    for k, (kind, residual, affine) in enumerate([("layer", False, True), ("rms", True, True), ("layer", True, False),
                                                 ("rms", False, False)]):
        x = rows(n, h, dtype, 1)
        r = rows(n, h, dtype, 2) if residual else None
        w = vector(h, dtype, 3, 1.0) if affine else None
        b = vector(h, dtype, 4, 0.0) if affine and kind == "layer" else None
        out = flce.layer_norm(x, w, b, kind=kind, eps=1e-5, residual=r)
        check_forward(out, x, r, w, b, 1e-5, kind == "rms", dtype)
        gy = rows(n, h, dtype, 5, 1e-2, 0.0)
        gs = rows(n, h, dtype, 6, 1e-2, 0.0) if residual else None
        s = out["sum"] if residual else x
        grads = flce.layer_norm_backward(gy, s, w, mean=out["mean"], rstd=out["rstd"], kind=kind, grad_sum=gs)
        check_backward(grads, gy, s, w, out["mean"], out["rstd"], gs, kind == "rms", dtype)


@pytest.mark.parametrize("n,h", [(5000, 384), (2500, 2050), (4999, 1536)])
def test_many_rows(n, h):
    x, gy = rows(n, h, "bf16", 1), rows(n, h, "bf16", 2, 1e-2, 0.0)
    w = vector(h, "bf16", 3, 1.0)
    out = flce.layer_norm(x, w, kind="layer")
    check_forward(out, x, None, w, None, 1e-5, False, "bf16")
    grads = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"])
    check_backward(grads, gy, x, w, out["mean"], out["rstd"], None, False, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h", [1, 8, 63, 64, 65, 100, 129, 200, 256, 261, 512, 515, 1027])
def test_many_short_rows(h, dtype):
    """More rows than the SMs hold warps: several a warp, and many a group of the backward pass."""
    n = 12001
    x, gy = rows(n, h, dtype, 1), rows(n, h, dtype, 2, 1e-2, 0.0)
    r, w, b = rows(n, h, dtype, 5), vector(h, dtype, 3, 1.0), vector(h, dtype, 4, 0.0)
    out = flce.layer_norm(x, w, b, residual=r)
    check_forward(out, x, r, w, b, 1e-5, False, dtype)
    grads = flce.layer_norm_backward(gy, out["sum"], w, mean=out["mean"], rstd=out["rstd"], grad_sum=x)
    check_backward(grads, gy, out["sum"], w, out["mean"], out["rstd"], x, False, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h,first", [(500, 1), (1000, 7), (2047, 3), (2048, 5), (4099, 2), (8200, 6)])
def test_rows_that_start_inside_a_vector(h, first, dtype):
    """Contiguous matrices whose first element lies anywhere in 16 bytes, with weights at another such place."""
    n = 37
    def shifted(k, scale=1.0):
        flat = rows(1, n * h + 16, dtype, k, scale)[0]
        return flat[first:first + n * h].view(n, h)
    x, r, gy, gs = shifted(1), shifted(2), shifted(3, 1e-2), shifted(4, 1e-2)
    out_y, out_s, out_g = shifted(5), shifted(6), shifted(7)
    for at in (0, 1, 3):
        w, b = vector(h + 8, dtype, 8, 1.0)[at:at + h], vector(h + 8, "fp32", 9, 0.0)[at:at + h].to(TYPES[dtype])
        out = flce.layer_norm(x, w, b, residual=r, out=out_y, sum_out=out_s)
        check_forward(out, x, r, w, b, 1e-5, False, dtype)
        grads = flce.layer_norm_backward(gy, out_s, w, mean=out["mean"], rstd=out["rstd"], grad_sum=gs, out=out_g)
        check_backward(grads, gy, out_s, w, out["mean"], out["rstd"], gs, False, dtype)
        grads = flce.layer_norm_backward(gy, out_s, w.float(), mean=out["mean"], rstd=out["rstd"])
        check_backward(grads, gy, out_s, w.float(), out["mean"], out["rstd"], None, False, dtype)


@pytest.mark.parametrize("n,h,dtype", [(1, 64, "bf16"), (3, 2047, "bf16"), (9, 1001, "fp16"), (29, 2048, "fp32"), (7, 77, "fp32"),
                                       (500, 4096, "bf16"), (400, 513, "bf16"), (5, 30, "bf16"), (700, 20001, "bf16")])
def test_workspace_of_the_stated_size_is_enough(n, h, dtype):
    """Nothing behind the workspace or the column sums is written."""
    x, gy = rows(n, h, dtype, 1), rows(n, h, dtype, 2)
    out = flce.layer_norm(x)
    stats = dict(mean=out["mean"], rstd=out["rstd"])
    want = flce.layer_norm_backward(gy, x, **stats)
    size = flce.ln_workspace_size(n, h)
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    sums = torch.full((2, h + 64), 9.0, device="cuda")
    got = flce.layer_norm_backward(gy, x, **stats, workspace=room[:size], grad_weight_out=sums[0, :h],
                                   grad_bias_out=sums[1, :h])
    assert (room[size:] == 77).all() and (sums[:, h:] == 9).all()
    assert torch.equal(got["grad_weight"], want["grad_weight"]) and torch.equal(got["grad_x"], want["grad_x"])


@pytest.mark.parametrize("n,h,dtype", [(2, 40000, "bf16"), (3, 70001, "bf16"), (2, 33000, "fp32"), (5, 65536, "fp16")])
def test_long_rows(n, h, dtype):
    x, gy = rows(n, h, dtype, 1), rows(n, h, dtype, 2, 1e-2, 0.0)
    w, b = vector(h, dtype, 3, 1.0), vector(h, dtype, 4, 0.0)
    out = flce.layer_norm(x, w, b)
    # chains of up to 300 additions here: SUM holds four times over for 70001 / 256
    y, mean, rstd = T.norm_forward(host(x), host(w), host(b), 1e-5, False)
    reach = np.abs(host(x)).max(1, keepdims=True) * rstd[:, None]
    tol = UNIT[dtype] * np.abs(y) + TINY[dtype] + 4 * SUM * (np.abs(host(w)) * 2 * reach + np.abs(host(b)))
    assert (np.abs(host(out["y"]) - y) <= tol).all()
    grads = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"])
    (gx, gw, gb), loose, size_w, size_b = backward_reference(gy, x, w, out["mean"], out["rstd"], None, False)
    assert (np.abs(host(grads["grad_x"]) - gx) <= UNIT[dtype] * np.abs(gx) + TINY[dtype] + 4 * loose).all()
    assert (np.abs(host(grads["grad_weight"]) - gw) <= 2 * SUM * size_w + 1e-30).all()
    assert (np.abs(host(grads["grad_bias"]) - gb) <= 2 * SUM * size_b + 1e-30).all()


@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("fp16", "fp32"), ("fp32", "bf16"), ("bf16", "fp16")])
@pytest.mark.parametrize("h", [96, 1024, 2047, 4096])
def test_weights_of_another_type(h, dtype, param):
    x, w, b = rows(37, h, dtype, 1), vector(h, param, 2, 1.0), vector(h, param, 3, 0.0)
    out = flce.layer_norm(x, w, b)
    check_forward(out, x, None, w, b, 1e-5, False, dtype)
    gy = rows(37, h, dtype, 4, 1e-2, 0.0)
    grads = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"])
    check_backward(grads, gy, x, w, out["mean"], out["rstd"], None, False, dtype)


def test_bias_without_weight():
    x, b = rows(9, 640, "bf16", 1), vector(640, "bf16", 3, 0.0)
    out = flce.layer_norm(x, None, b)
    check_forward(out, x, None, None, b, 1e-5, False, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h,pitch,first", [(256, 264, 0), (256, 300, 3), (1000, 1003, 1), (4096, 8192, 4096), (33, 64, 31),
                                           (2048, 2056, 8)])
def test_pitches_and_offsets(h, pitch, first, dtype):
    """Rows that are part of a wider matrix, from any column; what lies around the outputs stays."""
    n = 29
    wide = [rows(n, pitch, dtype, k) for k in range(4)]
    x, r, gy, gs = (m[:, first:first + h] for m in wide)
    w = vector(h + 1, dtype, 7, 1.0)[1:]                    # not 16-byte aligned
    y, s, gx = (torch.full((n, pitch), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(3))
    part = slice(first, first + h)
    out = flce.layer_norm(x, w, kind="rms", residual=r, out=y[:, part], sum_out=s[:, part])
    check_forward(out, x, r, w, None, 1e-5, True, dtype)
    grads = flce.layer_norm_backward(gy, s[:, part], w, rstd=out["rstd"], kind="rms", grad_sum=gs, out=gx[:, part])
    check_backward(grads, gy, s[:, part], w, None, out["rstd"], gs, True, dtype)
    for m in (y, s, gx):
        assert (m[:, :first] == 7).all() and (m[:, first + h:] == 7).all()


def test_repeated_row():
    """A broadcast input (rows 0 elements apart): its gradient is the sum of the rows', which is the caller's."""
    one = rows(1, 512, "bf16", 1)
    out = flce.layer_norm(one.expand(40, 512))
    check_forward(out, one.expand(40, 512), None, None, None, 1e-5, False, "bf16")
    gy = rows(1, 512, "bf16", 2).expand(40, 512)
    grads = flce.layer_norm_backward(gy, one.expand(40, 512), mean=out["mean"], rstd=out["rstd"])
    check_backward(grads, gy, one.expand(40, 512), None, out["mean"], out["rstd"], None, False, "bf16")


@pytest.mark.parametrize("h", [768, 777, 4096])
def test_outputs_in_the_inputs_place(h):
    check_in_place(h)


@pytest.mark.parametrize("h", [33, 20001, 66001])
def test_outputs_in_the_inputs_place_by_elements(h):
    check_in_place(h)


def check_in_place(h):
    x, r, w = rows(50, h, "bf16", 1), rows(50, h, "bf16", 2), vector(h, "bf16", 3, 1.0)
    want = flce.layer_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    got = flce.layer_norm(a, w, residual=b, out=a, sum_out=b)
    assert torch.equal(a, want["y"]) and torch.equal(b, want["sum"]) and torch.equal(got["rstd"], want["rstd"])
    a, b = x.clone(), r.clone()
    flce.layer_norm(a, w, residual=b, out=b, sum_out=a)
    assert torch.equal(b, want["y"]) and torch.equal(a, want["sum"])
    a = x.clone()
    flce.layer_norm(a, w, out=a)
    assert torch.equal(a, flce.layer_norm(x, w)["y"])
    gy, gs, s = rows(50, h, "bf16", 4), rows(50, h, "bf16", 5), want["sum"]
    stats = dict(mean=want["mean"], rstd=want["rstd"])
    grads = flce.layer_norm_backward(gy, s, w, **stats, grad_sum=gs)
    for k in range(3):
        t = [gy.clone(), s.clone(), gs.clone()]
        g = flce.layer_norm_backward(t[0], t[1], w, **stats, grad_sum=t[2], out=t[k])
        for name in ("grad_x", "grad_weight", "grad_bias"):
            assert torch.equal(g[name], grads[name])


@pytest.mark.parametrize("h", [64, 65, 4096])
def test_rows_that_are_not_finite_stay_to_themselves(h):
    x = rows(6, h, "bf16", 1)
    x[1, 3], x[4, 0] = float("inf"), float("nan")
    out = flce.layer_norm(x)
    bad = torch.tensor([False, True, False, False, True, False], device="cuda")
    assert out["y"][bad].isnan().all() and out["y"][~bad].isfinite().all()
    good = flce.layer_norm(x[~bad].contiguous())
    assert torch.equal(out["y"][~bad], good["y"])
    gy = rows(6, h, "bf16", 2)
    grads = flce.layer_norm_backward(gy, x, mean=out["mean"], rstd=out["rstd"])
    again = flce.layer_norm_backward(gy[~bad].contiguous(), x[~bad].contiguous(), mean=out["mean"][~bad],
                                     rstd=out["rstd"][~bad])
    assert torch.equal(grads["grad_x"][~bad], again["grad_x"]) and grads["grad_x"][bad].isnan().all()


def test_constant_rows_and_large_offsets():
    x = torch.full((4, 1024), 3.0, device="cuda")
    b = vector(1024, "fp32", 1, 0.5)
    out = flce.layer_norm(x, None, b)
    assert torch.equal(out["y"], b.expand(4, 1024)) and (out["mean"] == 3).all()
    # the variance is taken about the mean: 1e4 + noise of 1 keeps its digits
    x = 1e4 + rows(8, 4096, "fp32", 2, 1.0, 0.0)
    check_forward(flce.layer_norm(x), x, None, None, None, 1e-5, False, "fp32")


def test_no_rows():
    x, w = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda"), vector(96, "bf16", 1, 1.0)
    out = flce.layer_norm(x, w)
    assert out["y"].shape == (0, 96) and out["rstd"].shape == (0,)
    gw, gb = torch.full((96,), 5.0, device="cuda"), torch.full((96,), 6.0, device="cuda")
    flce.layer_norm_backward(x, x, w, mean=out["mean"], rstd=out["rstd"], grad_weight_out=gw, grad_bias_out=gb,
                             accumulate=True)
    assert (gw == 5).all() and (gb == 6).all()
    flce.layer_norm_backward(x, x, w, mean=out["mean"], rstd=out["rstd"], grad_weight_out=gw, grad_bias_out=gb)
    assert (gw == 0).all() and (gb == 0).all()


def test_leading_dimensions_and_parts_left_out():
    x, w = rows(24, 320, "bf16", 1).view(2, 3, 4, 320), vector(320, "bf16", 2, 1.0)
    out = flce.layer_norm(x, w)
    assert out["y"].shape == x.shape and out["rstd"].shape == (2, 3, 4)
    flat = flce.layer_norm(x.view(24, 320), w, row_stats=False)
    assert flat["rstd"] is None and flat["mean"] is None and torch.equal(flat["y"], out["y"].view(24, 320))
    gy = rows(24, 320, "bf16", 3).view_as(x)
    both = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"])
    for off in ("grad_x", "grad_weight", "grad_bias"):
        got = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"], **{off: False})
        for name in both:
            assert (got[name] is None) if name == off else torch.equal(got[name], both[name])


@pytest.mark.parametrize("h", [512, 513])
def test_accumulates(h):
    x, gy = rows(70, h, "bf16", 1), rows(70, h, "bf16", 2)
    out = flce.layer_norm(x)
    stats = dict(mean=out["mean"], rstd=out["rstd"])
    once = flce.layer_norm_backward(gy, x, **stats)
    gw, gb = torch.full((h,), 0.5, device="cuda"), torch.full((h,), -2.0, device="cuda")
    flce.layer_norm_backward(gy, x, **stats, grad_weight_out=gw, grad_bias_out=gb, accumulate=True)
    assert torch.equal(gw, once["grad_weight"] + 0.5) and torch.equal(gb, once["grad_bias"] - 2.0)
    with pytest.raises(flce.FlceError):
        flce.layer_norm_backward(gy, x, **stats, accumulate=True)


@pytest.mark.parametrize("n,h", [(16384, 256), (3000, 4096), (999, 1001)])
def test_same_bits_every_run(n, h):
    x, gy = rows(n, h, "bf16", 1), rows(n, h, "bf16", 2)
    out = flce.layer_norm(x)
    first = flce.layer_norm_backward(gy, x, mean=out["mean"], rstd=out["rstd"])
    for _ in range(5):
        got = flce.layer_norm_backward(gy, x, mean=out["mean"], rstd=out["rstd"])
        assert all(torch.equal(got[k], first[k]) for k in got)


def test_offsets_past_32_bits():
    """Rows so far apart that the last starts past 2^31 elements."""
    pitch, n, h = 1 << 29, 6, 1024
    buffer = torch.empty((n - 1) * pitch + h, dtype=torch.bfloat16, device="cuda")
    x = buffer.as_strided((n, h), (pitch, 1))
    x.copy_(rows(n, h, "bf16", 1))
    out = flce.layer_norm(x)
    assert torch.equal(out["y"], flce.layer_norm(x.contiguous())["y"])
    gy = rows(n, h, "bf16", 2)
    stats = dict(mean=out["mean"], rstd=out["rstd"])
    want = flce.layer_norm_backward(gy, x.contiguous(), **stats)
    got = flce.layer_norm_backward(gy, x, **stats, out=x)
    assert torch.equal(x.contiguous(), want["grad_x"]) and torch.equal(got["grad_weight"], want["grad_weight"])


def test_on_another_stream_and_in_a_graph():
    x, w = rows(300, 1024, "bf16", 1), vector(1024, "bf16", 2, 1.0)
    gy = rows(300, 1024, "bf16", 3)
    want = flce.layer_norm(x, w)
    grads = flce.layer_norm_backward(gy, x, w, mean=want["mean"], rstd=want["rstd"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        out = flce.layer_norm(x, w, stream=stream)
        got = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"], stream=stream)
        side.synchronize()
        assert torch.equal(out["y"], want["y"]) and torch.equal(got["grad_weight"], grads["grad_weight"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.layer_norm(x, w)
        got = flce.layer_norm_backward(gy, x, w, mean=out["mean"], rstd=out["rstd"])
    for _ in range(3):
        got["grad_weight"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["y"], want["y"])
        assert all(torch.equal(got[k], grads[k]) for k in grads)


@pytest.mark.parametrize("n,h", [(1, 4096), (5, 64), (40, 200), (33, 777), (256, 128), (512, 65), (2000, 512), (9, 4098)])
def test_backward_with_any_workspace_and_in_a_graph(n, h):
    """What the workspace held does not matter, and a replayed call finds its last CTA again."""
    x, gy = rows(n, h, "bf16", 1), rows(n, h, "bf16", 2, 1e-2, 0.0)
    w = vector(h, "bf16", 3, 1.0)
    out = flce.layer_norm(x, w)
    stats = dict(mean=out["mean"], rstd=out["rstd"])
    work = torch.empty(flce.ln_workspace_size(n, h), dtype=torch.uint8, device="cuda")
    want = None
    for fill in (0, 0xFF, 0x5A, None):
        if fill is None:
            work.random_(0, 256)
        else:
            work.fill_(fill)
        for _ in range(3):
            got = flce.layer_norm_backward(gy, x, w, **stats, workspace=work)
            want = want or got
            assert all(torch.equal(got[k], want[k]) for k in got)
    check_backward(want, gy, x, w, out["mean"], out["rstd"], None, False, "bf16")
    sums = torch.full((2, h), 0.25, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        flce.layer_norm_backward(gy, x, w, **stats, workspace=work, grad_weight_out=sums[0], grad_bias_out=sums[1],
                                 accumulate=True)
    for k in range(3):
        sums.fill_(0.25)
        graph.replay()
        assert torch.equal(sums[0], want["grad_weight"] + 0.25) and torch.equal(sums[1], want["grad_bias"] + 0.25)


def test_refusals():
    x, w = rows(4, 64, "bf16", 1), vector(64, "bf16", 2, 1.0)
    st = torch.ones(4, device="cuda")
    calls = [
        lambda: flce.layer_norm(x.t()),                                   # columns apart
        lambda: flce.layer_norm(rows(4, 64, "bf16", 1).view(2, 2, 64).transpose(0, 1), w[:63]),
        lambda: flce.layer_norm(torch.empty(6, 4, 64, dtype=torch.bfloat16, device="cuda")[:, ::3]),   # rows of two strides
        lambda: flce.layer_norm(x, w[:32]), lambda: flce.layer_norm(x, w[::2]), lambda: flce.layer_norm(x.int()),
        lambda: flce.layer_norm(x, w, w.float()), lambda: flce.layer_norm(x, residual=x[:2]),
        lambda: flce.layer_norm(x, residual=x.float()), lambda: flce.layer_norm(x, kind="batch"),
        lambda: flce.layer_norm(x, eps=-1.0), lambda: flce.layer_norm(x, out=x.float()),
        lambda: flce.layer_norm(x, out=x[:1].expand(4, 64)), lambda: flce.layer_norm(x, sum_out=x),
        lambda: flce.layer_norm(x, w.cpu()), lambda: flce.layer_norm(torch.empty(3, 0, device="cuda")),
        lambda: flce.layer_norm_backward(x, x, rstd=st), lambda: flce.layer_norm_backward(x, x, mean=st, rstd=st[:3]),
        lambda: flce.layer_norm_backward(x[:3], x, mean=st, rstd=st),
        lambda: flce.layer_norm_backward(x, x, mean=st, rstd=st.double()),
        lambda: flce.layer_norm_backward(x, x, mean=st, rstd=st, kind="rms"),
        lambda: flce.layer_norm_backward(x, x, mean=st, rstd=st, grad_x=False, grad_sum=x),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(flce.FlceError):
            call()
            pytest.fail(f"call {k} was not refused")
