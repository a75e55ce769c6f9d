"""The losses of post-training on logits against their definitions in 64 bits:
types, row lengths around every border between the kernels, rows that start
anywhere in a vector, masks, lists, packed and padded sequences."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import LNS, TYPES, close, close_grad, cuda, f32, logp_error, make_logits, targets, wide
from oracle import losses_oracle as L

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "fp16", "fp32"]
# rows of single elements, of less than a vector, of warps, of parts by one CTA and by clusters of 2, 4 and 8, at the
# borders between them, and longer than any of these
COLUMNS = [1, 3, 7, 8, 9, 31, 257, 1000, 2047, 2048, 2056, 4099, 8200, 16384, 16392, 16401, 32768, 33001, 50257, 65536,
           65600, 131072, 131081, 128256, 151936, 256000, 270337, 300007]


def rows_for(v):
    return 5 if v > 40000 else 37


# ------------------------------------------------------------ policy

def policy_inputs(z, seed, reference=True, weighted=True, temperature=1.0):
    rng = np.random.default_rng(seed)
    n = z.shape[0]
    t = targets(z, seed)
    logp = L.policy(wide(z), t, np.zeros(n), temperature=temperature)["logp"]
    change = rng.normal(size=n) * 0.2
    for border in (0.8, 1.2):                     # a ratio at a border of the clip may fall on either side
        change = np.where(np.abs(np.exp(change) - border) < 1e-3, change + 4e-3, change)
    old = f32(np.where(t < 0, 0, logp - change))
    ref = f32(logp + rng.normal(size=n) * 0.5) if reference else None
    w = f32(rng.uniform(0.2, 2, n)) if weighted else None
    return t, f32(rng.normal(size=n)), dict(old_logp=old, ref_logp=ref, row_weight=w)


def on_gpu(kw):
    return {k: cuda(v, torch.float32) if isinstance(v, np.ndarray) else v for k, v in kw.items()}


def check_policy(z, t, a, kw, dtype, *, out=None, **call):
    numbers = dict(clip=0.2, kl_weight=0.1 if kw.get("ref_logp") is not None else 0.0)
    numbers.update({k: v for k, v in kw.items() if not isinstance(v, np.ndarray) and k != "ref_logp"})
    arrays = {k: v for k, v in kw.items() if isinstance(v, np.ndarray)}
    want = L.policy(wide(z), t, a, **{k: v for k, v in {**numbers, **arrays}.items()})
    got = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(arrays), **numbers, **call) if out is None else out
    temperature, kl = numbers.get("temperature", 1.0), numbers["kl_weight"]
    dl = logp_error(want["logp"]) / min(1.0, temperature)
    n = len(t)
    w = np.abs(arrays.get("row_weight", np.ones(n)))
    r = want["ratio"]
    size = np.abs(a) * np.maximum(r, 1.2) * w
    x = 0.0
    if kl:
        d = arrays["ref_logp"] - want["logp"]
        x = kl * w * np.exp(np.abs(d))
    used = (want["rows"] != 0) | (want["f"] != 0)
    # loss: its slope by logp times logp's error, and a few roundings of its terms
    d_loss = np.where(used, (size + x) * dl + 2.0 ** -20 * (size + 2 * x), 0.0)
    close(wide(got["logp"]), want["logp"], np.where(t < 0, 0.0, dl), "logp")
    red = numbers.get("reduction", "mean")
    scale = {"none": 1.0, "sum": 1.0, "mean": 1 / max(1, (t >= 0).sum())}[red]
    tol = d_loss if red == "none" else d_loss.sum() * scale + 2.0 ** -23 * abs(np.nan_to_num(want["loss"]))
    close(wide(got["loss"]), want["loss"], tol, "loss")
    if got["grad_logits"] is not None:
        slope = np.where(used, (size + 2 * x) * (dl + 2.0 ** -20), 0.0)
        g = np.abs(numbers.get("grad_scale", 1.0)) * np.abs(arrays.get("grad_out", np.ones(n)))
        close_grad(got["grad_logits"], want, slope * scale * g / temperature, dtype)
    assert int(got["status"]) == 0
    return got, want


@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_columns(v, dtype):
    z = make_logits(rows_for(v), v, dtype, v)
    t, a, kw = policy_inputs(z, v + 1)
    check_policy(z, t, a, kw, dtype)


@pytest.mark.parametrize("v,ld,offset", [(1000, 1003, 1), (2049, 2051, 3), (8190, 8200, 5), (33001, 33003, 1), (5, 6, 1),
                                         (70001, 70007, 7), (270337, 270339, 3), (4096, 4104, 0), (1999, 1999, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("place", ["in_place", "same", "other"])
def test_policy_rows_that_start_anywhere(v, ld, offset, dtype, place):
    """Rows inside padded buffers, the gradient over the logits, equally and otherwise aligned: what lies between stays."""
    z = make_logits(9, v, dtype, v, ld=ld, offset=offset)
    keep = z.clone()
    t, a, kw = policy_inputs(z, v)
    call = {}
    base = z._base if z._base is not None else z
    if place == "in_place":
        call["in_place"] = True
    else:
        call["grad_out_buffer"] = make_logits(9, v, dtype, 1, ld=ld + (0 if place == "same" else 1),
                                              offset=offset + (0 if place == "same" else 1))
    numbers = dict(clip=0.2, kl_weight=0.1)
    out = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), **numbers, **call)
    check_policy(keep, t, a, kw, dtype, out=out)
    if place != "in_place":
        assert torch.equal(z, keep) and out["grad_logits"].data_ptr() == call["grad_out_buffer"].data_ptr()
        base = call["grad_out_buffer"]._base
    step = out["grad_logits"].stride(0)
    gaps = base[out["grad_logits"].storage_offset():][:8 * step].view(8, step)[:, v:]
    assert (gaps == 77).all() and (base[:out["grad_logits"].storage_offset()] == 77).all()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("n,v", [(1, 500), (33, 3000), (700, 520), (5000, 64), (20000, 17), (300, 33000), (2500, 9000)])
def test_policy_reductions_and_rows(reduction, n, v):
    z = make_logits(n, v, "bf16", n)
    t, a, kw = policy_inputs(z, n)
    if reduction == "none":
        kw["grad_out"] = f32(np.random.default_rng(n).normal(size=n))
    check_policy(z, t, a, dict(kw, reduction=reduction, grad_scale=0.7), "bf16")


@pytest.mark.parametrize("numbers", [dict(temperature=0.6), dict(temperature=3.0), dict(clip=math.inf), dict(clip=0.0),
                                     dict(clip=0.1, clip_high=0.4), dict(clip=2.5), dict(kl_weight=0.0)])
@pytest.mark.parametrize("v", [700, 40000])
def test_policy_numbers(numbers, v):
    z = make_logits(40, v, "fp32", 3)
    t, a, kw = policy_inputs(z, 4, temperature=numbers.get("temperature", 1.0))
    if numbers.get("clip") == 0.0 or "clip_high" in numbers:   # other borders: keep clear of them as well
        logp = L.policy(wide(z), t, a, temperature=1.0)["logp"]
        kw["old_logp"] = f32(np.where(t < 0, 0, logp - np.random.default_rng(9).choice([-0.3, -0.05, 0.05, 0.2, 0.6], 40)))
    check_policy(z, t, a, dict(kw, **numbers), "fp32")


@pytest.mark.parametrize("v", [300, 5000, 70000])
def test_policy_on_fresh_samples(v):
    """Without old log-probabilities the ratio is 1; without a reference there is no KL term."""
    z = make_logits(20, v, "bf16", 3)
    t, a, _ = policy_inputs(z, 4)
    got, want = check_policy(z, t, a, {}, "bf16")
    rows = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), reduction="none")["loss"]
    assert torch.equal(rows, torch.where(cuda(t) < 0, 0.0, -cuda(a, torch.float32)))


@pytest.mark.parametrize("v", [300, 5000, 40001, 280000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_masked_columns_and_bad_rows(v, dtype):
    """-inf and the type's lowest value are columns of no probability; NaN and infinity stay in their rows."""
    z = make_logits(12, v, dtype, v)
    t, a, kw = policy_inputs(z, 5)
    t[:] = np.random.default_rng(1).integers(0, v // 2, 12)
    t[11] = -100
    z[:, v // 2:] = float("-inf")
    z[1, v // 2:] = torch.finfo(TYPES[dtype]).min
    t[2] = v // 2 + 1                                           # a target of no probability
    logp = L.policy(wide(z), t, a)["logp"]
    kw = dict(old_logp=f32(np.where(t < 0, 0, logp - 0.05)))
    kw["old_logp"][2] = -3.0
    a = np.abs(a)
    check_policy(z, t, a, kw, dtype)
    z[3, 1] = float("nan")
    z[4, 2] = float("inf")
    z[5] = float("-inf")
    z[11] = float("nan")                                        # an ignored row
    out = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), reduction="none")
    bad = [3, 4, 5]
    good = [i for i in range(12) if i not in bad]
    assert out["loss"][bad].isnan().all() and out["loss"][good].isfinite().all()
    assert out["grad_logits"][bad].isnan().all() and out["grad_logits"][good].isfinite().all()
    assert (out["grad_logits"][11] == 0).all() and out["loss"][11] == 0 and out["logp"][11] == 0


@pytest.mark.parametrize("v", [1000, 9000])
def test_policy_rows_of_weight_zero(v):
    z = make_logits(8, v, "bf16", 2)
    t, a, kw = policy_inputs(z, 3)
    kw["row_weight"][1:3] = 0
    z[1] = float("nan")
    kw["old_logp"][2] = -1e6                                    # an infinite ratio
    out = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), reduction="none")
    assert (out["grad_logits"][1:3] == 0).all() and (out["loss"][1:3] == 0).all() and out["loss"].isfinite().all()


def test_policy_far_logits_keep_their_digits():
    """A common level of 3e4 takes nothing from the differences (fp32 logits there are 2^-9 apart)."""
    z = make_logits(10, 3000, "fp32", 1)
    z += 3e4
    t, a, kw = policy_inputs(z, 2)
    check_policy(z, t, a, kw, "fp32")


@pytest.mark.parametrize("n,v", [(30, 600), (3000, 600), (30, 30000), (4, 290000)])
def test_policy_without_any_row_and_targets_outside(n, v):
    z = make_logits(n, v, "bf16", 2)
    a = torch.ones(n, device="cuda")
    t = torch.full((n,), -100, device="cuda")
    for reduction, value in (("mean", math.nan), ("sum", 0.0)):
        out = flce.policy_loss(z, t, a, reduction=reduction)
        assert (math.isnan(value) and math.isnan(float(out["loss"]))) or float(out["loss"]) == value
        assert (out["grad_logits"] == 0).all() and int(out["status"]) == 0
    t[0], t[1], t[2] = 1, v, -7
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for status in (None, word):
        out = flce.policy_loss(z, t, a, status=status, reduction="mean")
        assert int(out["status"]) == flce.STATUS_BIT_TARGET_RANGE and float(out["loss"]) == -1.0
        assert (out["grad_logits"][1:] == 0).all() and (out["grad_logits"][0] != 0).any()
    flce.policy_loss(z, t.clamp(max=0), a, status=word)
    assert int(word) == flce.STATUS_BIT_TARGET_RANGE            # never cleared


def test_policy_empty_batches():
    z = torch.empty(0, 50, dtype=torch.bfloat16, device="cuda")
    t, a = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    assert float(flce.policy_loss(z, t, a, reduction="sum")["loss"]) == 0
    assert math.isnan(float(flce.policy_loss(z, t, a)["loss"]))
    out = flce.policy_loss(z, t, a, reduction="none")
    assert out["loss"].shape == (0,) and out["grad_logits"].shape == (0, 50)


def test_policy_leading_dimensions_and_no_gradient():
    z = make_logits(24, 900, "fp16", 2)
    t, a, kw = policy_inputs(z, 3)
    want = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), reduction="none")
    shaped = {k: v.view(4, 6) for k, v in on_gpu(kw).items() if v is not None}
    got = flce.policy_loss(z.view(4, 6, 900), cuda(t).view(4, 6), cuda(a, torch.float32).view(4, 6), **shaped,
                           reduction="none")
    assert got["loss"].shape == got["logp"].shape == (4, 6) and got["grad_logits"].shape == (4, 6, 900)
    assert torch.equal(got["loss"].view(-1), want["loss"]) and torch.equal(got["grad_logits"].view(24, 900), want["grad_logits"])
    none = flce.policy_loss(z, cuda(t), cuda(a, torch.float32), **on_gpu(kw), reduction="none", want_grad=False)
    assert none["grad_logits"] is None and torch.equal(none["loss"], want["loss"])


@pytest.mark.parametrize("rest", [-0.3, -0.1])
def test_policy_sum_over_a_row_of_millions(rest):
    """One column of 0 and 2^26 - 1 equal ones.  A thread adds 16 terms, 64 steps of those, 128
    batches, and 512 threads are joined; ln S is off by these roundings and the exponent's 2^-21."""
    v = 2 ** 26
    z = torch.full((1, v), rest, dtype=torch.float32, device="cuda")
    z[0, 12345] = 0
    out = flce.policy_loss(z, torch.tensor([12345], device="cuda"), torch.ones(1, device="cuda"), want_grad=False,
                           reduction="none")
    want = -math.log((v - 1) * math.exp(float(np.float32(rest))) + 1)
    tol = (16 + 64 + 128 + 16 + 8) * 2.0 ** -24 + 2.0 ** -21 + abs(want) * 2.0 ** -23
    assert abs(float(out["logp"][0]) - want) <= tol


# ------------------------------------------------------------ distillation

def teacher(n, v, k, seed, id_type=np.int64):
    rng = np.random.default_rng(seed)
    k = min(k, v)
    ids = np.stack([rng.choice(v, k, replace=False) for _ in range(n)]).astype(id_type)
    values = rng.normal(size=(n, k)) * 3
    length = rng.integers(1, k + 1, n)
    length[n // 2:] = k
    if n > 4:
        length[2] = 0
    ids[np.arange(k)[None] >= length[:, None]] = -1
    return ids, values


def check_distill(z, ids, values, dtype, *, value_dtype="fp32", status=0, out=None, place=None, **kw):
    held = cuda(values, TYPES[value_dtype])
    arrays = {k: v for k, v in kw.items() if isinstance(v, np.ndarray)}
    want = L.distill(wide(z), ids, wide(held), **kw)
    rest = {k: v for k, v in kw.items() if k not in arrays}
    if out is None:
        out = flce.distillation_loss(z, cuda(ids), held, **on_gpu(arrays), **rest, **(place or {}))
    temperature, n = kw.get("temperature", 1.0), len(ids)
    w = np.abs(arrays.get("row_weight", np.ones(n)))
    # each row: ln S, and the list's sum q (ln q - z / T), whose terms q ln q and q z / T are off by 2^-21 of their size
    spread = np.abs(np.where(np.isfinite(want["rows"]), want["rows"], 0)) / temperature ** 2 / np.maximum(w, 1e-30)
    zs = np.abs(np.where(np.isfinite(wide(z)), wide(z), 0)).max(1) / temperature
    d = np.where(want["rows"] != 0, temperature ** 2 * w * (LNS + (spread + 2 * zs + 16) * 2.0 ** -20), 0)
    red = kw.get("reduction", "mean")
    scale = {"none": 1.0, "sum": 1.0, "mean": 1 / max(1, (ids[:, 0] >= 0).sum())}[red]
    tol = d if red == "none" else d.sum() * scale + 2.0 ** -23 * abs(np.nan_to_num(want["loss"]))
    close(wide(out["loss"]), want["loss"], tol, "loss")
    if out["grad_logits"] is not None:
        close_grad(out["grad_logits"], want, np.abs(want["f"]) * 2.0 ** -21, dtype)
    assert int(out["status"]) == status
    return out


@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_distill_columns(v, dtype):
    n = rows_for(v)
    z = make_logits(n, v, dtype, v)
    ids, values = teacher(n, v, 20, v)
    check_distill(z, ids, values, dtype, temperature=1.5)


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 100, 256, 1000, 1024])
@pytest.mark.parametrize("v", [1500, 20000, 66000, 280000])
@pytest.mark.parametrize("id_type", [np.int64, np.int32])
def test_distill_lists(k, v, id_type):
    n = 6
    z = make_logits(n, v, "bf16", k)
    ids, values = teacher(n, v, k, k, id_type)
    check_distill(z, ids, values, "bf16", value_dtype="bf16", temperature=2.0)


@pytest.mark.parametrize("v,ld,offset", [(1000, 1003, 1), (8190, 8200, 5), (33001, 33003, 1), (70001, 70007, 7)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("place", ["in_place", "other"])
def test_distill_rows_that_start_anywhere(v, ld, offset, dtype, place):
    z = make_logits(9, v, dtype, v, ld=ld, offset=offset)
    keep = z.clone()
    ids, values = teacher(9, v, 40, v)
    ids[4, :3] = [0, v - 1, 1]                     # the ends of a row
    at = dict(in_place=True) if place == "in_place" else \
        dict(grad_out_buffer=make_logits(9, v, dtype, 1, ld=ld + 1, offset=offset + 1))
    out = flce.distillation_loss(z, cuda(ids), cuda(values, torch.float32), **at)
    check_distill(keep, ids, values, dtype, out=out)


@pytest.mark.parametrize("v", [64, 1500, 20000, 66000, 280000])
@pytest.mark.parametrize("k", [4, 48, 500])
def test_distill_columns_that_are_named_twice(v, k):
    """All shares of a column add up, wherever in the list they stand."""
    z = make_logits(8, v, "fp32", v)
    rng = np.random.default_rng(k)
    ids = rng.integers(0, min(v, k), (8, k))
    ids[1] = ids[1, 0]                             # one column alone
    ids[2, -1] = ids[2, 0]
    check_distill(z, ids, rng.normal(size=(8, k)), "fp32")


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("n,v", [(1, 700), (50, 3000), (700, 520), (3000, 64), (300, 33000)])
def test_distill_reductions_weights_and_rows(reduction, n, v):
    z = make_logits(n, v, "fp16", n)
    ids, values = teacher(n, v, 12, n)
    rng = np.random.default_rng(n)
    kw = dict(row_weight=f32(rng.uniform(0.2, 2, n)), reduction=reduction, grad_scale=0.7)
    if n > 3:
        kw["row_weight"][3] = 0
    if reduction == "none":
        kw["grad_out"] = f32(rng.normal(size=n))
    check_distill(z, ids, values, "fp16", value_dtype="fp16", **kw)


@pytest.mark.parametrize("v", [300, 5000, 40001, 280000])
def test_distill_masks_and_ids_outside(v):
    z = make_logits(10, v, "bf16", v)
    ids, values = teacher(10, v, 16, v)
    ids[:, :8] = np.arange(8)
    values[3, 2:] = -np.inf                        # two of the list have a share
    values[4] = -np.inf                            # none has
    values[5, 0] = -60000.0                        # nor has this one
    z[6, 100:] = float("-inf")
    ids[6, 8:] = -1
    out = check_distill(z, ids, values, "bf16")
    assert (out["grad_logits"][4] == 0).all()
    ids[7, 3], ids[8, 0] = v, v + 5                # left out, and flagged
    check_distill(z, ids, values, "bf16", status=flce.STATUS_BIT_TARGET_RANGE, reduction="none")
    ids[6, 0] = 200                                # a place without probability: an infinite distance, a finite gradient
    out = check_distill(z, ids, values, "bf16", status=flce.STATUS_BIT_TARGET_RANGE, reduction="none")
    assert out["loss"][6] == math.inf and out["grad_logits"][6].isfinite().all()
    z[9, 3] = float("nan")
    out = flce.distillation_loss(z, cuda(ids), cuda(values, torch.float32), reduction="none")
    assert out["grad_logits"][9].isnan().all() and out["loss"][9].isnan() and out["loss"][:6].isfinite().all()


def test_distill_from_itself_is_nothing():
    """A teacher with the student's own logits, all of them: loss and gradient vanish but for rounding."""
    z = make_logits(4, 1000, "fp32", 1)
    ids = torch.arange(1000, device="cuda").expand(4, 1000).contiguous()
    out = flce.distillation_loss(z, ids, z, reduction="none", temperature=2.0)
    assert out["loss"].abs().max() < 4 * 2 * (LNS + 30 * 2.0 ** -20) and out["grad_logits"].abs().max() < 2 * 2 * LNS


# ------------------------------------------------------------ preference

def sequences(lengths, behind, v, dtype, seed, ld=None, offset=0):
    n = sum(lengths) + behind
    z = make_logits(n, v, dtype, seed, ld=ld, offset=offset)
    t = targets(z, seed) if n else np.zeros(0, np.int64)
    return z, t, np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def check_preference(z, t, offsets, dtype, *, out=None, packed=True, status=0, **kw):
    arrays = {k: v for k, v in kw.items() if isinstance(v, np.ndarray)}
    want = L.preference(wide(z), t, offsets=offsets, **kw)
    if out is None:
        out = flce.preference_loss(z, cuda(t), offsets=cuda(offsets) if packed else None, **on_gpu(arrays),
                                   **{k: v for k, v in kw.items() if k not in arrays})
    pairs = (len(offsets) - 1) // 2
    beta, kind = kw.get("beta", 0.1), kw.get("kind", "sigmoid")
    live = (t >= 0) & (t < z.shape[1])
    rows = np.where(live, logp_error(L.policy(wide(z), t, np.zeros(len(t)))["logp"]), 0.0)
    d_seq = np.array([rows[a:b].sum() for a, b in zip(offsets[:-1], offsets[1:])]) / want["count"]
    close(wide(out["logp"]), want["logp"], d_seq + 2.0 ** -23 * np.abs(want["logp"]), "logp")
    ref = arrays.get("ref_logp", np.zeros(2 * pairs))
    dx = d_seq[:pairs] + d_seq[pairs:] + 2.0 ** -50 * (np.abs(want["logp"]) + np.abs(ref)).sum()
    slope = 2 * np.abs(want["x"] - 0.5 / beta) + dx if kind == "ipo" else beta
    d_pair = slope * dx + 2.0 ** -23 * np.abs(want["pairs"])
    red = kw.get("reduction", "mean")
    scale = 1 / max(1, pairs) if red == "mean" else 1.0
    tol = d_pair if red == "none" else d_pair.sum() * scale + 2.0 ** -23 * abs(np.nan_to_num(want["loss"]))
    close(wide(out["loss"]), want["loss"], tol, "loss")
    if out["grad_logits"] is not None:
        # the slope's own slope by x is at most 2 (ipo) or beta^2 / 4 (sigmoid), and it is rounded once
        curve = {"ipo": 2.0, "sigmoid": beta * beta / 4, "hinge": 0.0}[kind]
        g = np.abs(kw.get("grad_scale", 1.0)) * np.abs(arrays.get("grad_out", np.ones(pairs))) * scale
        f_error = np.zeros(len(t))
        for q in range(2 * pairs):
            f_error[offsets[q]:offsets[q + 1]] = curve * dx[q % pairs] * g[q % pairs if np.ndim(g) else ...] / want["count"][q]
        close_grad(out["grad_logits"], want, f_error + np.abs(want["f"]) * 2.0 ** -22, dtype)
    assert int(out["status"]) == status
    return out


@pytest.mark.parametrize("v", COLUMNS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_preference_columns(v, dtype):
    z, t, offsets = sequences([3, 1, 2, 4], 1, v, dtype, v)
    check_preference(z, t, offsets, dtype, ref_logp=f32(np.random.default_rng(v).normal(size=4) * 5 - 20), beta=0.2)


@pytest.mark.parametrize("kind,numbers", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.2, margin=0.4)),
                                          ("hinge", {}), ("hinge", dict(margin=-0.3)), ("ipo", {})])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_preference_kinds(kind, numbers, average, reduction):
    """Empty sequences, one whose tokens are all ignored, rows behind the last one."""
    z, t, offsets = sequences([7, 0, 30, 1, 12, 5], 3, 700, "bf16", 4)
    t[offsets[5]:offsets[6]] = -100
    rng = np.random.default_rng(5)
    kw = dict(ref_logp=f32(rng.normal(size=6) * 4 - 30), kind=kind, average=average, reduction=reduction, beta=0.3,
              grad_scale=1.3, **numbers)
    if reduction == "none":
        kw["grad_out"] = f32(rng.normal(size=3))
    out = check_preference(z, t, offsets, "bf16", **kw)
    assert (out["grad_logits"][-3:] == 0).all()


@pytest.mark.parametrize("pairs,tokens,v", [(1, 1, 40), (2, 9, 2100), (5, 31, 300), (3, 4, 33000)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_preference_padded_batches(pairs, tokens, v, dtype):
    n = 2 * pairs * tokens
    z = make_logits(n, v, dtype, n)
    t = targets(z, 3, ignored=0.4)
    shaped = z.view(2 * pairs, tokens, v)
    out = flce.preference_loss(shaped, cuda(t).view(2 * pairs, tokens))
    assert out["grad_logits"].shape == shaped.shape
    flat = dict(out, grad_logits=out["grad_logits"].view(n, v))
    check_preference(z, t, np.arange(2 * pairs + 1) * tokens, dtype, out=flat)


@pytest.mark.parametrize("v,ld,offset", [(1000, 1003, 1), (8190, 8200, 5), (33001, 33003, 1), (70001, 70007, 7), (5, 6, 1)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("place", ["in_place", "same", "other"])
def test_preference_rows_that_start_anywhere(v, ld, offset, dtype, place):
    z, t, offsets = sequences([3, 2, 1, 2], 0, v, dtype, v, ld=ld, offset=offset)
    keep = z.clone()
    shift = 0 if place == "same" else 1
    at = dict(in_place=True) if place == "in_place" else \
        dict(grad_out_buffer=make_logits(8, v, dtype, 1, ld=ld + shift, offset=offset + shift))
    out = flce.preference_loss(z, cuda(t), offsets=cuda(offsets), beta=0.5, **at)
    check_preference(keep, t, offsets, dtype, out=out, beta=0.5)
    g = out["grad_logits"]
    gaps = g._base[g.storage_offset():][:7 * g.stride(0)].view(7, g.stride(0))[:, v:]
    assert (gaps == 77).all()


@pytest.mark.parametrize("bad", [[0, 5, 3, 9, 12], [0, 3, 6, 9, 1 << 40], [-4, 3, 6, 9, 12], [1 << 62, 3, -(1 << 62), 9, 12]])
def test_preference_offsets_outside_are_cut_and_flagged(bad):
    z, t, _ = sequences([3, 3, 3, 3], 0, 500, "bf16", 1)
    out = flce.preference_loss(z, cuda(t), offsets=cuda(np.array(bad)))
    assert int(out["status"]) == flce.STATUS_BIT_SEQUENCE_RANGE
    assert out["logp"].isfinite().all() and out["grad_logits"].isfinite().all()


def test_preference_without_pairs_rows_or_gradient():
    z, t, offsets = sequences([3, 2], 2, 500, "bf16", 1)
    none = flce.preference_loss(z, cuda(t), offsets=cuda(offsets[:1]), reduction="sum")
    assert float(none["loss"]) == 0 and (none["grad_logits"] == 0).all() and none["logp"].shape == (0,)
    assert math.isnan(float(flce.preference_loss(z, cuda(t), offsets=cuda(offsets[:1]))["loss"]))
    empty = flce.preference_loss(z[:0], cuda(t[:0]), offsets=cuda(np.zeros(3, np.int64)))
    assert abs(float(empty["loss"]) - math.log(2)) < 1e-6
    loss = flce.preference_loss(z, cuda(t), offsets=cuda(offsets), want_grad=False)
    assert loss["grad_logits"] is None
    check_preference(z, t, offsets, "bf16", out=loss)


@pytest.mark.parametrize("v", [300, 40001])
def test_preference_masks_and_bad_rows_stay_in_their_pair(v):
    z, t, offsets = sequences([3, 3, 3, 3], 0, v, "bf16", 2)
    t[:] = np.random.default_rng(0).integers(0, v // 2, 12)
    z[:, v // 2:] = float("-inf")
    check_preference(z, t, offsets, "bf16")
    t[1] = v - 1                                   # a chosen token of no probability
    out = flce.preference_loss(z, cuda(t), offsets=cuda(offsets), reduction="none")
    assert out["loss"][0] == math.inf and out["logp"][0] == -math.inf and out["grad_logits"].isfinite().all()
    t[1] = 5
    z[0, 3] = float("nan")
    out = flce.preference_loss(z, cuda(t), offsets=cuda(offsets), reduction="none")
    assert out["loss"][0].isnan() and out["loss"][1].isfinite()
    rows = [0, 1, 2, 6, 7, 8]
    assert out["grad_logits"][rows].isnan().any(1).all()
    assert out["grad_logits"][[3, 4, 5, 9, 10, 11]].isfinite().all()


def test_preference_long_sequences():
    """Sums over thousands of tokens, and more pairs than one launch has CTAs."""
    z, t, offsets = sequences([6000, 5000], 0, 70, "bf16", 3)
    check_preference(z, t, offsets, "bf16")
    lengths = list(np.random.default_rng(1).integers(0, 4, 6000))
    z, t, offsets = sequences(lengths, 1, 40, "fp32", 3)
    check_preference(z, t, offsets, "fp32", kind="ipo", beta=0.4)


def test_preference_many_target_errors():
    z, t, offsets = sequences([5, 5], 0, 90, "bf16", 3)
    t[3], t[7] = 90, -5
    check_preference(z, np.where((t < 0) | (t >= 90), -100, t), offsets, "bf16",
                     out=flce.preference_loss(z, cuda(t), offsets=cuda(offsets)), status=flce.STATUS_BIT_TARGET_RANGE)


@pytest.mark.parametrize("temperature", [1e-4, 1e4])
@pytest.mark.parametrize("v", [700, 40000])
def test_the_ends_of_the_temperature(temperature, v):
    """Where all but the largest have no share, and where all have the same."""
    z = make_logits(12, v, "fp32", 5, scale=3.0)
    t = np.array([int(x) for x in wide(z).argmax(1)])
    t[3] = (t[3] + 1) % v
    a = f32(np.random.default_rng(1).normal(size=12))
    check_policy(z, t, a, dict(temperature=temperature), "fp32")
    ids, values = teacher(12, v, 20, v)
    # the teacher's and the student's differences over 1e-4 reach 1e5: fp32 leaves 2^-23 of that in the exponents
    out = flce.distillation_loss(z, cuda(ids), cuda(values, torch.float32), temperature=temperature, reduction="none")
    want = L.distill(wide(z), ids, f32(values), temperature=temperature, reduction="none")
    tol = temperature ** 2 * (LNS + 2.0 ** -19 * (60 / temperature + 16))
    close(wide(out["loss"]), want["loss"], tol, "loss")


@pytest.mark.parametrize("v", [500, 9000, 70001, 290000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_the_lowest_value(v, dtype):
    """Where a mask of the type's lowest value leaves nothing, all columns are alike; beside others they have no share."""
    z = make_logits(4, v, dtype, 3)
    low = torch.finfo(TYPES[dtype]).min
    z[0] = low
    z[1, : v // 2] = low
    z[2] = torch.finfo(TYPES[dtype]).max
    z[3, 1:] = low
    t = np.array([3, v - 1, 5, 0])
    check_policy(z, t, f32(np.ones(4)), {}, dtype)
    ids = np.array([[0, 2], [v - 1, v - 2], [1, 3], [0, 0]])
    check_distill(z, ids, np.zeros((4, 2)), dtype, reduction="none")
    check_preference(z, t, np.array([0, 2, 4]), dtype)
