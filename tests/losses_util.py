"""What the tests of the losses on logits share: inputs, and how far fp32 may be
from the definitions in 64 bits.

A row's ln S: an exponent x = (z - M) / T has two roundings, off by 2^-23 |x|,
and exp itself 2^-22, so a term e^x is off by (|x| + 2) 2^-22 of itself; |x| is
weighted by e^x, which leaves at most ln V + 1 on average.  Adding up V terms by
threads, lanes, warps and CTAs is a chain of at most 200 additions, each off by
2^-24.  Together below (ln V + 3) 2^-22 + 200 * 2^-24 < 1.6e-5 for V up to 2^20:
LNS.  logp has that and two roundings of (z_t - M) / T.

A gradient f (p - named) is off by f's own error, by p's (the exponent's, and
LNS), and by one rounding to its type.
"""
import numpy as np
import torch

LNS = 1.6e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SMALLEST = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}   # half a subnormal step, or flushed


def wide(t):
    return t.detach().double().cpu().numpy()


def make_logits(n, v, dtype, seed, scale=2.0, ld=None, offset=0):
    """[n, v] logits, their rows ld apart, the first `offset` elements into a 16-byte vector."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = v if ld is None else ld
    buffer = torch.full((offset + n * ld + 8,), 77.0, dtype=TYPES[dtype], device="cuda")
    z = buffer[offset:offset + n * ld].view(n, ld)[:, :v] if n else buffer[:0].view(0, v)
    z.copy_((torch.randn(n, v, generator=gen, device="cuda") * scale).to(TYPES[dtype]))
    return z


def targets(z, seed, ignored=0.2):
    """Likely and unlikely columns, some rows ignored but not the first."""
    n, v = z.shape
    rng = np.random.default_rng(seed)
    t = rng.integers(0, v, n)
    likely = rng.random(n) < 0.5
    t = np.where(likely, wide(z).argmax(1), t)
    t[rng.random(n) < ignored] = -100
    if n and t[0] < 0:
        t[0] = rng.integers(0, v)
    return t


def cuda(a, dtype=None):
    return None if a is None else torch.as_tensor(a, device="cuda", dtype=dtype)


def f32(a):
    """What the package is given of an array of the tests, and what the oracle has to see."""
    return None if a is None else np.asarray(a, np.float32).astype(np.float64)


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = np.isnan(want) & np.isnan(got) | (got == want)
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.flatnonzero(bad)[0], bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, the first at {i}: {got[i]} for {want[i]}, "
                             f"allowed {np.broadcast_to(tol, bad.shape)[i]}")


def close_grad(got, want, f_error, dtype, temperature=1.0):
    """`want` the oracle's dict, f_error how far each row's factor may be off."""
    f, p, named = np.abs(want["f"])[:, None], want["p"], want["named"]
    with np.errstate(divide="ignore"):
        x = np.minimum(-np.log(np.maximum(p, 1e-60)), 120.0)      # |z - M| / T is at most this
    # p: its exponent, ln S, the exponential and three multiplications; q: the same of the list
    tol = f * (p * (LNS + (x + 12) * 2.0 ** -22) + named * (LNS + 40 * 2.0 ** -22)) + \
        np.asarray(f_error)[:, None] * np.abs(p - named)
    g = np.abs(want["grad"])
    eps = torch.finfo(TYPES[dtype]).eps / 2
    with np.errstate(invalid="ignore"):
        close(wide(got), want["grad"], tol + eps * (g + tol) + SMALLEST[dtype] + f * 2.0 ** -125, "grad")
    zero = (want["f"] == 0)
    assert (wide(got)[zero] == 0).all(), "rows without a gradient hold zeros"


def logp_error(logp):
    return LNS + np.abs(np.where(np.isfinite(logp), logp, 0)) * 2.0 ** -22
