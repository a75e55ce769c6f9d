"""The losses of post-training on a language model's logits, and the embedding
whose table the head may share.

``policy_fwd_bwd``, ``preference_fwd_bwd``, ``distill_fwd_bwd``,
``embedding_fwd`` and ``embedding_bwd`` marshal their arguments for the C entry
points; ``policy_loss``, ``preference_loss``, ``distillation_loss``,
``embedding`` and ``embedding_backward`` take tensors, check them, allocate what
is not given and raise on an error status (in csrc/binding_losses.cpp).

Each loss gives its gradient on the logits in the same call, as ``cross_entropy``
does; nothing is recorded for autograd.  What a call writes (``in_place`` logits,
``grad_out_buffer``, ``out``, ``grad_weight_out``, ``status``) counts as changed
in place.  Memory that a call allocates belongs to the stream that the call runs
on; a tensor that was written on another stream has to be waited for by the
caller.
"""
from __future__ import annotations

import ctypes

from . import _dt, _ptr, _red, _stream, lib
from ._training import _native, _on

PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
INDEX_TYPES = {"int64": 0, "int32": 1}


class PolicyNumbers(ctypes.Structure):
    """flce_policy_t"""
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_weight", ctypes.c_float),
                ("temperature", ctypes.c_float)]


class PreferenceNumbers(ctypes.Structure):
    """flce_preference_t"""
    _fields_ = [("kind", ctypes.c_int32), ("average", ctypes.c_int32), ("beta", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("margin", ctypes.c_float)]


# ------------------------------------------------------------------ raw ABI

def _index(index_type) -> int:
    return INDEX_TYPES.get(index_type, -1) if isinstance(index_type, str) else int(index_type)


def row_loss_workspace_size(N: int) -> int:
    return lib().row_loss_workspace_size(N)


def preference_workspace_size(N: int, pairs: int) -> int:
    return lib().preference_workspace_size(N, pairs)


def embedding_workspace_size(N: int, V: int, H: int) -> int:
    return lib().embedding_workspace_size(N, V, H)


def policy_fwd_bwd(logits, dtype, ld, grad_logits, ld_grad, target, advantage, old_logp, ref_logp, row_weight, N, V,
                   numbers, ignore_index, reduction, grad_scale, grad_out_none, loss, logp, workspace, workspace_bytes,
                   status_dev, stream=None) -> int:
    """`numbers` is a PolicyNumbers."""
    return lib().policy_fwd_bwd(
        _ptr(logits), _dt(dtype), ld, _ptr(grad_logits), ld_grad, _ptr(target), _ptr(advantage), _ptr(old_logp),
        _ptr(ref_logp), _ptr(row_weight), N, V, None if numbers is None else ctypes.byref(numbers), ignore_index,
        _red(reduction), float(grad_scale), _ptr(grad_out_none), _ptr(loss), _ptr(logp), _ptr(workspace),
        int(workspace_bytes), _ptr(status_dev), _stream(stream))


def preference_fwd_bwd(logits, dtype, ld, grad_logits, ld_grad, target, offsets, ref_logp, pairs, N, V, numbers,
                       ignore_index, reduction, grad_scale, grad_out_none, loss, logp, workspace, workspace_bytes,
                       status_dev, stream=None) -> int:
    """`numbers` is a PreferenceNumbers."""
    return lib().preference_fwd_bwd(
        _ptr(logits), _dt(dtype), ld, _ptr(grad_logits), ld_grad, _ptr(target), _ptr(offsets), _ptr(ref_logp), pairs,
        N, V, None if numbers is None else ctypes.byref(numbers), ignore_index, _red(reduction), float(grad_scale),
        _ptr(grad_out_none), _ptr(loss), _ptr(logp), _ptr(workspace), int(workspace_bytes), _ptr(status_dev),
        _stream(stream))


def distill_fwd_bwd(logits, dtype, ld, grad_logits, ld_grad, ids, index_type, values, value_dtype, top, row_weight, N,
                    V, temperature, reduction, grad_scale, grad_out_none, loss, workspace, workspace_bytes, status_dev,
                    stream=None) -> int:
    return lib().distill_fwd_bwd(
        _ptr(logits), _dt(dtype), ld, _ptr(grad_logits), ld_grad, _ptr(ids), _index(index_type), _ptr(values),
        _dt(value_dtype), top, _ptr(row_weight), N, V, float(temperature), _red(reduction), float(grad_scale),
        _ptr(grad_out_none), _ptr(loss), _ptr(workspace), int(workspace_bytes), _ptr(status_dev), _stream(stream))


def embedding_fwd(dtype, table, ld_table, ids, index_type, N, V, H, scale, y, ld_y, status_dev, stream=None) -> int:
    return lib().embedding_fwd(_dt(dtype), _ptr(table), ld_table, _ptr(ids), _index(index_type), N, V, H, float(scale),
                               _ptr(y), ld_y, _ptr(status_dev), _stream(stream))


def embedding_bwd(dtype, grad_y, ld_grad_y, ids, index_type, N, V, H, scale, padding_index, grad_table, accumulate,
                  workspace, workspace_bytes, status_dev, stream=None) -> int:
    return lib().embedding_bwd(_dt(dtype), _ptr(grad_y), ld_grad_y, _ptr(ids), _index(index_type), N, V, H,
                               float(scale), padding_index, _ptr(grad_table), int(accumulate), _ptr(workspace),
                               int(workspace_bytes), _ptr(status_dev), _stream(stream))


# ------------------------------------------------------------------ losses

def policy_loss(logits, target, advantage, *, old_logp=None, ref_logp=None, clip: float = 0.2, clip_high=None,
                kl_weight: float = 0.0, temperature: float = 1.0, row_weight=None, ignore_index: int = -100,
                reduction="mean", grad_scale: float = 1.0, grad_out=None, in_place: bool = False,
                want_grad: bool = True, grad_out_buffer=None, workspace=None, status=None, stream=None) -> dict:
    """The clipped policy loss of sampled tokens with a KL term, and its gradient on the logits.

    With logp the log-probability of a row's target under softmax(logits /
    temperature), ratio = exp(logp - old_logp) and d = ref_logp - logp:

        loss = -min(ratio * advantage, clamp(ratio, 1 - clip, 1 + clip_high) * advantage)
               + kl_weight * (exp(d) - 1 - d)

    logits [..., V] bf16, fp16 or fp32, rows contiguous and one stride apart;
    target [...] int64; advantage, old_logp, ref_logp and row_weight [...] fp32,
    contiguous, of the logits' leading dimensions (or either of them flat).
    Without old_logp the ratio is 1 and its gradient that of logp; a kl_weight
    other than 0 wants ref_logp; without clip_high it is clip; infinity does not
    cut; temperature lies in [1e-4, 1e4].  row_weight multiplies a row's loss;
    "mean" divides by the rows that take part, whatever their weights.
    Returns a dict with ``loss``, ``grad_logits`` (or None), ``logp`` (fp32, 0 for
    ignored rows: the next update's old_logp) and ``status``: the one that was
    given, which bits are added to, or the workspace's own, which is this call's
    until another call uses that workspace.
    """
    if stream is not None:
        with _on(stream):
            return policy_loss(logits, target, advantage, old_logp=old_logp, ref_logp=ref_logp, clip=clip,
                               clip_high=clip_high, kl_weight=kl_weight, temperature=temperature,
                               row_weight=row_weight, ignore_index=ignore_index, reduction=reduction,
                               grad_scale=grad_scale, grad_out=grad_out, in_place=in_place, want_grad=want_grad,
                               grad_out_buffer=grad_out_buffer, workspace=workspace, status=status)
    loss, grad, logp, word = _native().policy_loss(
        logits, _red(reduction), grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status, target,
        advantage, old_logp, ref_logp, row_weight, clip, clip if clip_high is None else clip_high, kl_weight,
        temperature, ignore_index)
    return {"loss": loss, "grad_logits": grad, "logp": logp, "status": word}


def preference_loss(logits, target, *, offsets=None, ref_logp=None, kind="sigmoid", beta: float = 0.1,
                    label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                    ignore_index: int = -100, reduction="mean", grad_scale: float = 1.0, grad_out=None,
                    in_place: bool = False, want_grad: bool = True, grad_out_buffer=None, workspace=None, status=None,
                    stream=None) -> dict:
    """A loss over pairs of sequences by their log-probability ratios, and its gradient on the logits.

    The first half of the sequences are the chosen ones, the second half the
    rejected ones in the same order.  A sequence's log-probability is the sum of
    its tokens' (their mean with ``average``); with x the chosen one's, less the
    reference model's (``ref_logp``, fp32 [2 * pairs], or None), less the same of
    the rejected one, and u = beta * x - margin:

        "sigmoid"  -(1 - label_smoothing) * log sigmoid(u) - label_smoothing * log sigmoid(-u)
        "hinge"    max(0, 1 - u)
        "ipo"      (x - 1 / (2 * beta)) ** 2

    logits [2 * pairs, tokens, V], or sequences packed one after another as
    [tokens of all, V] with ``offsets`` (int64 [2 * pairs + 1]); target of the
    logits' shape without V, int64.  Returns a dict with ``loss`` (fp32 [pairs] or
    []), ``grad_logits`` (or None), ``logp`` (fp32 [2 * pairs]) and ``status``.
    """
    if stream is not None:
        with _on(stream):
            return preference_loss(logits, target, offsets=offsets, ref_logp=ref_logp, kind=kind, beta=beta,
                                   label_smoothing=label_smoothing, margin=margin, average=average,
                                   ignore_index=ignore_index, reduction=reduction, grad_scale=grad_scale,
                                   grad_out=grad_out, in_place=in_place, want_grad=want_grad,
                                   grad_out_buffer=grad_out_buffer, workspace=workspace, status=status)
    kind = PREFERENCE_KINDS.get(kind, -1) if isinstance(kind, str) else int(kind)
    loss, grad, logp, word = _native().preference_loss(
        logits, _red(reduction), grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status, target,
        offsets, ref_logp, kind, beta, label_smoothing, margin, average, ignore_index)
    return {"loss": loss, "grad_logits": grad, "logp": logp, "status": word}


def distillation_loss(logits, teacher_ids, teacher_logits, *, temperature: float = 1.0, row_weight=None,
                      reduction="mean", grad_scale: float = 1.0, grad_out=None, in_place: bool = False,
                      want_grad: bool = True, grad_out_buffer=None, workspace=None, status=None, stream=None) -> dict:
    """The distance of a student's logits from a teacher of which each row has the top logits, and its gradient.

    With q = softmax(teacher_logits / temperature) over a row's list and p =
    softmax(logits / temperature) over all columns, loss = temperature ** 2 *
    sum of q * (log q - log p).

    logits [..., V] as in ``policy_loss``; teacher_ids [..., top] int64 or int32,
    up to a row's first negative one (a row that starts with one takes no part);
    teacher_logits [..., top] of any of the three types, logits or
    log-probabilities; both contiguous, top at most 1024.  row_weight (fp32
    [...]) multiplies a row's loss; "mean" divides by the rows that take part.
    Returns a dict with ``loss``, ``grad_logits`` (or None) and ``status``.
    """
    if stream is not None:
        with _on(stream):
            return distillation_loss(logits, teacher_ids, teacher_logits, temperature=temperature,
                                     row_weight=row_weight, reduction=reduction, grad_scale=grad_scale,
                                     grad_out=grad_out, in_place=in_place, want_grad=want_grad,
                                     grad_out_buffer=grad_out_buffer, workspace=workspace, status=status)
    loss, grad, word = _native().distillation_loss(
        logits, _red(reduction), grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status,
        teacher_ids, teacher_logits, row_weight, temperature)
    return {"loss": loss, "grad_logits": grad, "status": word}


# ------------------------------------------------------------------ embedding

def embedding(weight, ids, *, scale: float = 1.0, out=None, status=None, stream=None) -> dict:
    """Rows of ``weight`` by token, times ``scale``, rounded once.

    weight [V, H] bf16, fp16 or fp32, rows contiguous and one stride apart; ids
    [...] int64 or int32, contiguous.  Returns a dict with ``y`` [..., H].  An id
    outside [0, V) gives a row of zeros and sets a bit of ``status`` (an int32
    element on the device) where that is given.
    """
    if stream is not None:
        with _on(stream):
            return embedding(weight, ids, scale=scale, out=out, status=status)
    return {"y": _native().embedding(weight, ids, scale, out, status)}


def embedding_backward(grad_y, ids, vocabulary=None, *, scale: float = 1.0, padding_index=None, grad_weight_out=None,
                       accumulate: bool = False, workspace=None, status=None, stream=None) -> dict:
    """The gradient of ``embedding``'s weight: sums of grad_y, times ``scale``, over the tokens of each id.

    grad_y [..., H] bf16, fp16 or fp32; ids as in ``embedding``; ``vocabulary``
    rows, or those of ``grad_weight_out`` (fp32 [V, H]).  ``accumulate`` adds to
    grad_weight_out and leaves rows of no token alone: the gradient of a weight
    that the head shares, as ``fused_linear_cross_entropy`` left it.  Tokens of
    ``padding_index`` add nothing.  Sums run in an order that ids and sizes fix.
    Returns a dict with ``grad_weight``.
    """
    if stream is not None:
        with _on(stream):
            return embedding_backward(grad_y, ids, vocabulary, scale=scale, padding_index=padding_index,
                                      grad_weight_out=grad_weight_out, accumulate=accumulate, workspace=workspace,
                                      status=status)
    return {"grad_weight": _native().embedding_backward(
        grad_y, ids, -1 if vocabulary is None else vocabulary, scale, -1 if padding_index is None else padding_index,
        grad_weight_out, accumulate, workspace, status)}
