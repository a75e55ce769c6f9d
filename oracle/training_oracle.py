"""Plain definitions, in 64 bits, of the operators around the head: layer norm
and its form without the mean with their gradients, the gradients' norm, and
AdamW with fp32 or 8-bit moments.  Used by the tests only; numpy, and no code
of the package.
"""
from __future__ import annotations

import numpy as np


def norm_forward(s, weight, bias, eps, rms):
    """(y, mean, rstd) of rows s [N, H]; weight and bias [H] or None."""
    s = np.asarray(s, np.float64)
    mean = np.zeros(s.shape[0]) if rms else s.sum(1) / s.shape[1]
    d = s - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(1) / s.shape[1] + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def norm_backward(grad_y, s, weight, mean, rstd, grad_sum, rms):
    """(grad_s + grad_sum, grad_weight, grad_bias), at given row statistics."""
    s, grad_y = np.asarray(s, np.float64), np.asarray(grad_y, np.float64)
    xhat = (s - (0.0 if rms else mean[:, None])) * rstd[:, None]
    u = grad_y if weight is None else grad_y * weight
    g = u - xhat * (u * xhat).sum(1, keepdims=True) / s.shape[1]
    if not rms:
        g = g - u.sum(1, keepdims=True) / s.shape[1]
    g = g * rstd[:, None]
    if grad_sum is not None:
        g = g + grad_sum
    return g, (grad_y * xhat).sum(0), grad_y.sum(0)


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, decay, step):
    """(p, m, v) after one step."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(v / (1 - beta2 ** step))
    return p * (1 - lr * decay) - lr * (m / (1 - beta1 ** step)) / (root + eps), m, v


# ------------------------------------------------------------ 8-bit moments

BLOCK, LARGEST = 256, 448.0


def e4m3_values():
    """The value of each code 0..255 (NaN for 0x7F and 0xFF)."""
    code = np.arange(256)
    e, f = (code >> 3) & 15, code & 7
    value = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    value = np.where((code & 0x7F) == 0x7F, np.nan, value)
    return np.where(code & 0x80, -value, value)


def e4m3_spacing(x):
    """The distance of e4m3 numbers around |x|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)


def mix(x):
    x = np.asarray(x, np.uint64)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0xA54D2F6B)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xD1B54A33)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def rounding_bits(seed, step, tensor, n):
    """The 32 random bits of each of a tensor's n elements."""
    key = mix(seed & 0xFFFFFFFF)
    for word in (seed >> 32, step & 0xFFFFFFFF, tensor):
        key = mix(key ^ np.uint64(word))
    place = np.arange(n, dtype=np.uint64)
    return mix((place & np.uint64(0xFFFFFFFF)) ^ mix(key ^ (place >> np.uint64(32))))


def encode(x, bits16, keep):
    """(codes, scales) of fp32 moments x, in the arithmetic the format states: fp32, each operation
    rounded by itself.  bits16: random bits for each element, or None for rounding to nearest; keep: what
    is above 0 is held as at least the smallest number."""
    x = np.asarray(x, np.float32)
    blocks = -(-x.size // BLOCK)
    full = np.zeros(blocks * BLOCK, np.float32)
    full[:x.size] = x
    finite = np.where(np.isfinite(full), np.abs(full), np.float32(0)).reshape(blocks, BLOCK).max(1)
    scale = finite * np.float32(1 / LARGEST)
    scale = np.where(finite > 0, np.maximum(scale, np.float32(2.0 ** -126)), np.float32(0))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inverse = np.where(scale > 0, np.float32(1) / scale, np.float32(0)).astype(np.float32)
        y = (full.reshape(blocks, BLOCK) * inverse[:, None]).reshape(-1)[:x.size]
    a = np.minimum(np.abs(y).astype(np.float64), LARGEST)
    a = np.where(np.isfinite(a), a, 0.0)
    spacing = e4m3_spacing(a)
    if bits16 is None:
        a = np.rint(a / spacing) * spacing          # ties to even
    else:
        # below the normal numbers 2^-6 is added first, in fp32
        low = np.float32(2.0 ** -6)
        a = np.where(a < low, (a.astype(np.float32) + low).astype(np.float64) - low, a)
        a = np.floor(a / spacing + bits16.astype(np.float64) / 65536) * spacing
    a = np.minimum(a, LARGEST)
    if keep:
        a = np.where((a == 0) & (x > 0), 2.0 ** -9, a)
    code = np.searchsorted(e4m3_values()[:127], a).astype(np.uint8)
    code = np.where(np.signbit(y) & ~np.isnan(y), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8), scale
