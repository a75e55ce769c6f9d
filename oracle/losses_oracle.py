"""Plain definitions, in 64 bits, of the losses of post-training on logits and of
the embedding with its gradient.  Used by the tests only; numpy, and no code of
the package.

Each loss returns a dict with ``loss``, ``grad`` [N, V] and what a comparison
needs to know how far rounding may carry: ``p`` the row's probabilities, ``f`` the
factor of each row, so that grad = f * (p - what the row names).
"""
from __future__ import annotations

import numpy as np


def log_softmax(z, temperature=1.0):
    z = np.asarray(z, np.float64) / temperature
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = z - top
        return d - np.log(np.exp(d).sum(1, keepdims=True))


def _reduce(loss, count, reduction):
    if reduction == "none":
        return loss
    return loss.sum() / count if reduction == "mean" and count else np.nan if reduction == "mean" else loss.sum()


def _scale(n, count, reduction, grad_scale, grad_out):
    s = np.full(n, float(grad_scale))
    if reduction == "mean":
        s /= max(count, 1)
    return s if grad_out is None else s * grad_out


def policy(z, target, advantage, *, old_logp=None, ref_logp=None, clip=0.2, clip_high=None, kl_weight=0.0,
           temperature=1.0, row_weight=None, ignore_index=-100, reduction="mean", grad_scale=1.0, grad_out=None):
    n, v = z.shape
    clip_high = clip if clip_high is None else clip_high
    live = (target != ignore_index) & (target >= 0) & (target < v)
    at = np.where(live, target, 0)
    log_p = log_softmax(z, temperature)
    logp = np.where(live, log_p[np.arange(n), at], 0.0)
    a = np.asarray(advantage, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        ratio = np.exp(logp - (logp if old_logp is None else old_logp))
        cut = ((a > 0) & (ratio > 1 + clip_high)) | ((a < 0) & (ratio < 1 - clip))
        loss = -np.minimum(ratio * a, np.clip(ratio, 1 - clip, 1 + clip_high) * a)
        slope = np.where(cut, 0.0, -ratio * a)
        if kl_weight:
            d = ref_logp - logp
            loss = loss + kl_weight * (np.expm1(d) - d)
            slope = slope - kl_weight * np.expm1(d)
    w = np.ones(n) if row_weight is None else np.asarray(row_weight, np.float64)
    used = live & (w != 0)
    loss, slope = np.where(used, loss * w, 0.0), np.where(used, slope * w, 0.0)
    count = int(live.sum())
    f = -slope * _scale(n, count, reduction, grad_scale, grad_out) / temperature
    p = np.exp(log_p)
    onehot = np.zeros((n, v))
    onehot[np.arange(n)[live], target[live]] = 1.0
    with np.errstate(invalid="ignore"):
        grad = np.where((f == 0)[:, None], 0.0, f[:, None] * (p - onehot))
    return dict(loss=_reduce(loss, count, reduction), rows=loss, logp=logp, grad=grad, f=f, p=p, named=onehot, ratio=ratio)


def distill(z, ids, values, *, temperature=1.0, row_weight=None, reduction="mean", grad_scale=1.0, grad_out=None):
    n, v = z.shape
    log_p = log_softmax(z, temperature)
    q = np.zeros((n, v))
    loss = np.zeros(n)
    live = ids[:, 0] >= 0
    for i in range(n):
        ends = np.flatnonzero(ids[i] < 0)
        k = np.arange(ends[0] if len(ends) else ids.shape[1])
        k = k[(ids[i, k] < v)]
        t = np.asarray(values[i, k], np.float64) / temperature
        if len(k) == 0 or t.max() == -np.inf:
            continue
        share = np.exp(t - t.max())
        log_share = t - t.max() - np.log(share.sum())
        share /= share.sum()
        np.add.at(q[i], ids[i, k], share)
        held = share > 0
        loss[i] = (share[held] * (log_share[held] - log_p[i, ids[i, k][held]])).sum() * temperature ** 2
    w = np.ones(n) if row_weight is None else np.asarray(row_weight, np.float64)
    taught = (q.sum(1) > 0) & (w != 0)
    loss = np.where(taught, loss * w, 0.0)
    count = int(live.sum())
    f = np.where(taught, temperature * w * _scale(n, count, reduction, grad_scale, grad_out), 0.0)
    p = np.exp(log_p)
    with np.errstate(invalid="ignore"):
        grad = np.where((f == 0)[:, None], 0.0, f[:, None] * (p - q))
    return dict(loss=_reduce(loss, count, reduction), rows=loss, grad=grad, f=f, p=p, named=q)


def preference(z, target, *, offsets, ref_logp=None, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0,
               average=False, ignore_index=-100, reduction="mean", grad_scale=1.0, grad_out=None):
    n, v = z.shape
    pairs = (len(offsets) - 1) // 2
    live = (target != ignore_index) & (target >= 0) & (target < v)
    log_p = log_softmax(z)
    logp = np.where(live, log_p[np.arange(n), np.where(live, target, 0)], 0.0)
    count = np.array([max(1, live[a:b].sum()) if average else 1 for a, b in zip(offsets[:-1], offsets[1:])])
    s = np.array([logp[a:b].sum() for a, b in zip(offsets[:-1], offsets[1:])]) / count
    ratio = s - (0.0 if ref_logp is None else np.asarray(ref_logp, np.float64))
    x = ratio[:pairs] - ratio[pairs:]
    u = beta * x - margin
    if kind == "sigmoid":
        loss = np.logaddexp(0, -u) * (1 - label_smoothing) + (np.logaddexp(0, u) * label_smoothing if label_smoothing else 0)
        slope = beta * (np.exp(-np.logaddexp(0, -u)) - (1 - label_smoothing))
    elif kind == "hinge":
        loss, slope = np.maximum(0, 1 - u), np.where(u < 1, -beta, 0.0)
    else:
        loss, slope = (x - 0.5 / beta) ** 2, 2 * (x - 0.5 / beta)
    slope = slope * _scale(pairs, pairs, reduction, grad_scale, grad_out)
    f = np.zeros(n)
    for q in range(2 * pairs):
        f[offsets[q]:offsets[q + 1]] = slope[q % pairs] / count[q] * (-1 if q < pairs else 1)
    f = np.where(live, f, 0.0)
    p = np.exp(log_p)
    onehot = np.zeros((n, v))
    onehot[np.arange(n)[live], target[live]] = 1.0
    with np.errstate(invalid="ignore"):
        grad = np.where((f == 0)[:, None], 0.0, f[:, None] * (p - onehot))
    return dict(loss=_reduce(loss, pairs, reduction), pairs=loss, x=x, logp=s, grad=grad, f=f, p=p, named=onehot,
                count=count)


def embedding_gradient(grad_y, ids, v, *, scale=1.0, padding_index=None, start=None):
    """(the table's gradient, the sum of sizes that each element adds up)."""
    g = np.asarray(grad_y, np.float64) * scale
    keep = (ids >= 0) & (ids < v) & (ids != (-1 if padding_index is None else padding_index))
    out, size = np.zeros((v, g.shape[1])), np.zeros((v, g.shape[1]))
    np.add.at(out, ids[keep], g[keep])
    np.add.at(size, ids[keep], np.abs(g[keep]))
    if start is not None:
        out, size = out + start, size + np.abs(start)
    return out, size
