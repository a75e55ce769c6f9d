"""Losses on logits far from zero: masks of large finite values, rows about one large
level, and maxima beside the size from which exponents are formed another way.

A softmax knows differences alone, so each call is compared with the oracle's on
logits that give the same differences near zero: columns under a mask as -inf (what
lies 1e9 / T below the others has no share in 64 bits either), a row about a level
as that row less its largest logit, which is exact for what has a share.  The
tolerances are those of logits near zero: a difference z - M costs the same roundings
wherever M is, if it is formed before anything is rounded.
"""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import LNS, close, close_grad, cuda, f32, make_logits
from oracle import losses_oracle as L
from test_gpu_losses import check_distill, check_policy, check_preference, wide

pytestmark = pytest.mark.gpu

# rows by warps, by one CTA's parts, by clusters with odd places and of whole vectors, and read twice
COLUMNS = [700, 5000, 40001, 128256, 280003]


def filled(out, want):
    """`out` with the oracle's gradient where the call gave 0 for a share of at most 2^-62 of the largest.

    By parts an exponent is x = z c - r with r = M c rounded, c = log2(e) / T.  Its offset M c - r is at most
    half a unit in the last place of r: 64 for |M c| < 2^31.  2^x is held down to 2^-126, so what may vanish
    are shares p of log2(p) - 64 < -126 (of 2^-62 times a gradient's factor, below any rounding of the rest)."""
    g = torch.from_numpy(np.where((wide(out["grad_logits"]) == 0) & (want["p"] <= 2.0 ** -62) & (want["named"] == 0),
                                  want["grad"], wide(out["grad_logits"])))
    return dict(out, grad_logits=g)


def check_losses(given, near, t, dtype, temperature, columns, vanish=False):
    """All three losses on `given`, whose differences are those of `near`; teachers name `columns` [n, k]."""
    rng = np.random.default_rng(len(t) + columns.size)
    a = f32(rng.normal(size=len(t)))
    logp = L.policy(wide(near), t, a, temperature=temperature)["logp"]
    old = f32(logp - 0.05)
    for want_grad in (True, False):
        out = flce.policy_loss(given, cuda(t), cuda(a, torch.float32), old_logp=cuda(old, torch.float32), clip=0.2,
                               temperature=temperature, want_grad=want_grad)
        kw = dict(old_logp=old, temperature=temperature)
        if vanish and want_grad:
            out = filled(out, L.policy(wide(near), t, a, clip=0.2, **kw))
        check_policy(near, t, a, kw, dtype, out=out)
    for k in (columns.shape[1], 70):               # short lists, and long ones
        ids = np.concatenate([columns, np.full((len(t), k - columns.shape[1]), -1)], 1)
        values = rng.normal(size=ids.shape) * min(1.0, temperature)
        out = flce.distillation_loss(given, cuda(ids), cuda(values, torch.float32), temperature=temperature)
        if vanish:
            out = filled(out, L.distill(wide(near), ids, f32(values), temperature=temperature))
        want = L.distill(wide(near), ids, f32(values), temperature=temperature)
        if want["rows"].all():
            check_distill(near, ids, f32(values), dtype, temperature=temperature, out=out)
        else:
            # a list of the one column that has a share is no distance: the loss is T^2 ln S, and ln S off by LNS
            close(wide(out["loss"]), want["loss"], temperature ** 2 * LNS + 2.0 ** -20 * abs(want["loss"]), "loss")
            close_grad(out["grad_logits"], want, np.abs(want["f"]) * 2.0 ** -21, dtype)
    if temperature == 1:
        offsets = np.array([0, 1, len(t) // 2, len(t) - 1, len(t)])
        out = flce.preference_loss(given, cuda(t), offsets=cuda(offsets))
        check_preference(near, t, offsets, dtype, out=out)


@pytest.mark.parametrize("fill", [-1e9, -3e9, -1e10, -1e12, -1e15, -1e20, -1e25, -1e30])
@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks_of_finite_values(dtype, v, fill):
    """A few columns of a row are allowed; whole warps meet the mask alone."""
    z = make_logits(6, v, dtype, v)
    allowed = np.array([0, 1, v // 3, v // 2, v // 2 + 9, v - 1])
    near = torch.full_like(z, float("-inf"))
    near[:, allowed] = z[:, allowed]
    z[:] = torch.where(near.isinf(), fill, near)
    t = allowed[np.arange(6) % 6]
    columns = np.stack([np.roll(allowed, i) for i in range(6)])
    for temperature in (0.1, 0.3, 1.0, 2.0):
        check_losses(z, near, t, dtype, temperature, columns)


@pytest.mark.parametrize("v", COLUMNS)
def test_masks_of_fp16(v):
    """The largest value of fp16 over the smallest temperature."""
    z = make_logits(6, v, "fp16", v)
    allowed = np.array([0, 1, v // 3, v // 2, v // 2 + 9, v - 1])
    near = torch.full_like(z, float("-inf"))
    near[:, allowed] = (z[:, allowed].float() * 2.0 ** -12).half()
    z[:] = torch.where(near.isinf(), -65504.0, near)
    check_losses(z, near, allowed.copy(), "fp16", 1e-4, np.stack([allowed] * 6))


@pytest.mark.parametrize("level", [3e4, 1e9, 1.4e9, 1.6e9, 1e10, 1e12, 1e20, 1e25, 1e30])
@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_at_one_level(dtype, v, level):
    """Every column at the same far value, or but for a few two units in the last place below: shares are equal."""
    z = make_logits(6, v, dtype, v)
    high = torch.tensor(level, dtype=z.dtype, device="cuda")
    low = high * (1 - 4 * torch.finfo(z.dtype).eps)
    z[:4] = torch.tensor([1.0, -1.0, 1.0, 1.0], dtype=z.dtype, device="cuda")[:, None] * high
    z[4:] = low
    z[3, ::7] = low
    z[4, v // 2:v // 2 + 5] = high
    z[5, v - 3:] = high
    near = (z - z.amax(1, keepdim=True)).contiguous()
    t = np.array([0, v - 1, v // 2, 1, v // 2 + 1, v - 1])
    columns = np.array([[5, v - 2], [0, 1], [v // 3, 2], [1, 2], [v // 2, v // 2 + 2], [v - 1, v - 2]])
    for temperature in (0.3, 1.0, 2.0):
        check_losses(z, near, t, dtype, temperature, columns)


@pytest.mark.parametrize("v", [5000, 40001, 128256])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [19, 22, 26, 28, 30, 31, 32])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1e-4])
def test_maxima_beside_a_border(temperature, power, sign, v):
    """fp32 maxima a few units in the last place around 2^power of the scaled exponent, other warps' maxima beside them."""
    at = np.float32(sign * 2.0 ** power * np.log(2.0) * temperature)
    steps = np.zeros(13, np.float32)
    steps[6] = at
    for i in range(6):
        steps[5 - i] = np.nextafter(steps[6 - i], np.float32(-np.inf))
        steps[7 + i] = np.nextafter(steps[6 + i], np.float32(np.inf))
    n = 8
    z = torch.empty(n, v, device="cuda")
    t, columns = np.zeros(n, np.int64), np.zeros((n, 2), np.int64)
    for i in range(n):                             # the row's largest is steps[3 + i], in one stretch; others go below it
        lower = torch.from_numpy(steps[np.maximum(3 + i - 1 - np.arange(v) // 517 % 4, 0)]).cuda()
        z[i] = lower
        at0 = (i * v // n) // 2
        z[i, at0:at0 + 300] = float(steps[3 + i])
        t[i], columns[i] = at0 + 7, (at0 + 1, at0 + 299)
    near = z - z.amax(1, keepdim=True)
    check_losses(z, near, t, "fp32", temperature, columns, vanish=power > 26)


@pytest.mark.parametrize("v", [5000, 70001])
def test_large_logits_at_the_smallest_temperature(v):
    """Logits of 1e5 to 1e6 over 1e-4: the largest alone has a share."""
    z = make_logits(8, v, "fp32", v)
    z += torch.linspace(1e5, 1e6, 8, device="cuda")[:, None]
    z -= 3e5 * (torch.arange(8, device="cuda") % 2)[:, None]
    t = z.argmax(1).cpu().numpy()
    z[torch.arange(8), t] += 1.0
    near = z - z.amax(1, keepdim=True)
    check_losses(z, near, t, "fp32", 1e-4, t[:, None])
