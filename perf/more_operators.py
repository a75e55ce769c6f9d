"""Cases for the losses of post-training on a language model's logits, and for
the embedding whose table the head may share, in plain torch and through this
package.

  policy       clipped policy loss with a KL term over the tokens that a policy
               sampled, and its gradient on the logits
  preference   loss over pairs of sequences by their log-probability ratios to a
               reference model, and its gradient on the logits
  distill      divergence from a teacher of which each row holds the top logits,
               and its gradient on the logits
  embed        rows of a table by token, times a factor
  embed_bwd    the table's gradient: sums over the tokens that share a row

``own`` chooses between the plain form (elementary torch operations in 32 bits)
and the package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
IDS = {"int32": torch.int32, "int64": torch.int64}
IGNORE = -100
MOST_LOGITS = 4096 * 128256      # of the largest listed case
MOST_TABLE = 128256 * 4096


# ---------------------------------------------------------------- cases

def _policy(name, n, v, dtype, clip, kl, temperature, reference, weighted, reduction):
    return dict(name=name, op="policy", n=n, v=v, dtype=dtype, clip=clip, kl=kl, temperature=temperature,
                reference=reference, weighted=weighted, reduction=reduction)


def _preference(name, pairs, longest, v, dtype, kind, beta, smoothing, average, reduction, mix):
    return dict(name=name, op="preference", pairs=pairs, longest=longest, v=v, dtype=dtype, kind=kind, beta=beta,
                smoothing=smoothing, average=average, reduction=reduction, mix=mix)


def _distill(name, n, v, k, dtype, ids, temperature, weighted, reduction):
    return dict(name=name, op="distill", n=n, v=v, k=k, dtype=dtype, ids=ids, temperature=temperature,
                weighted=weighted, reduction=reduction)


def _embed(name, op, n, v, h, dtype, ids, scale, accumulate=False, padding=0.0):
    return dict(name=name, op=op, n=n, v=v, h=h, dtype=dtype, ids=ids, scale=scale, accumulate=accumulate,
                padding=padding)


def listed():
    return [
        # the tiny workload's logits: one small update, bound by latency
        _policy("policy 256x1024", 256, 1024, "bf16", 0.2, 0.05, 1.0, True, False, "mean"),
        # a minibatch of sampled tokens at the Llama-3 vocabulary, with a reference model's term
        _policy("policy 4096x128256", 4096, 128256, "bf16", 0.2, 0.05, 1.0, True, False, "mean"),
        # fp32 logits of an odd vocabulary, sampled at a temperature, tokens weighted by 1 / length of their answer
        _policy("policy 1000x50257", 1000, 50257, "fp32", 0.2, 0.0, 0.7, False, True, "sum"),
        # two short pairs, packed one after another
        _preference("preference 2 pairs", 2, 41, 32768, "bf16", "sigmoid", 0.1, 0.0, False, "mean", 3),
        # a step's pairs of answers of up to 512 tokens at the Llama-3 vocabulary
        _preference("preference 4 pairs", 4, 512, 128256, "bf16", "sigmoid", 0.1, 0.1, False, "mean", 5),
        # a few rows with a teacher's eight best
        _distill("distill 64x32768 top 8", 64, 32768, 8, "fp16", "int64", 1.0, False, "mean"),
        # a minibatch at the Llama-3 vocabulary with 64 stored logits a token
        _distill("distill 4096x128256 top 64", 4096, 128256, 64, "bf16", "int32", 2.0, False, "mean"),
        # fp32, odd vocabulary and batch, weighted rows
        _distill("distill 1999x32001 top 33", 1999, 32001, 33, "fp32", "int64", 1.5, True, "none"),
        # one token when serving: latency
        _embed("embed 1x4096", "embed", 1, 128256, 4096, "bf16", "int64", 1.0),
        # a training step's tokens, hidden states scaled by the root of their width
        _embed("embed 16384x4096", "embed", 16384, 128256, 4096, "bf16", "int64", 64.0),
        # the tiny workload's batch, its table's gradient from zero
        _embed("embed_bwd 256x128", "embed_bwd", 256, 1024, 128, "fp32", "int64", 1.0),
        # added to the gradient that the fused head left for the weight it shares; a fifth of the tokens are padding
        _embed("embed_bwd 16384x4096", "embed_bwd", 16384, 128256, 4096, "bf16", "int64", 1.0, True, 0.2),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("policy", "preference", "distill", "embed", "embed_bwd"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    reduction = rng.choice(("none", "sum", "mean"))
    if op in ("embed", "embed_bwd"):
        h = _log(rng, 64, 16384)
        h = h if rng.random() < 0.4 else -(-h // 64) * 64
        v = _log(rng, 256, min(256000, MOST_TABLE // h))
        n = _log(rng, 1, max(1, min(65536, (1 << 26) // h)))
        return dict(op=op, n=n, v=v, h=h, dtype=dtype, ids=rng.choice(("int64", "int32")),
                    scale=rng.choice((1.0, h ** 0.5)), accumulate=op == "embed_bwd" and rng.random() < 0.5,
                    padding=rng.choice((0.0, 0.2, 0.5)) if op == "embed_bwd" else 0.0)
    v = _log(rng, 512, 256000)
    v = v if rng.random() < 0.4 else -(-v // 64) * 64
    most = MOST_LOGITS // v // (2 if dtype == "fp32" else 1)
    if op == "preference":
        pairs = _log(rng, 1, 64)
        return dict(op=op, pairs=pairs, longest=_log(rng, 1, max(1, min(2048, most // (2 * pairs)))), v=v, dtype=dtype,
                    kind=rng.choice(("sigmoid", "hinge", "ipo")), beta=rng.choice((0.05, 0.1, 0.5)),
                    smoothing=rng.choice((0.0, 0.1)), average=rng.random() < 0.3, reduction=reduction,
                    mix=rng.randrange(1 << 20))
    n = _log(rng, 1, min(16384, most))
    if op == "policy":
        return dict(op=op, n=n, v=v, dtype=dtype, clip=rng.choice((0.1, 0.2)), kl=rng.choice((0.0, 0.04, 0.1)),
                    temperature=rng.choice((1.0, 0.7, 1.3)), reference=rng.random() < 0.6, weighted=rng.random() < 0.4,
                    reduction=reduction)
    return dict(op=op, n=n, v=v, k=_log(rng, 1, 256), dtype=dtype, ids=rng.choice(("int64", "int32")),
                temperature=rng.choice((1.0, 2.0, 4.0)), weighted=rng.random() < 0.4, reduction=reduction)


def _lengths(case):
    """Tokens of each of the 2 * pairs sequences: the longest first, the others between one and that."""
    rng = random.Random(case["mix"])
    return [case["longest"]] + [_log(rng, max(1, case["longest"] // 4), case["longest"])
                                for _ in range(2 * case["pairs"] - 1)]


def _zipf(v):
    """Probabilities of the ids, most frequent first."""
    p = np.arange(1, v + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op in ("embed", "embed_bwd"):
        n, v, h = case["n"], case["v"], case["h"]
        live = n * (1 - case["padding"])
        rows = float((1 - np.exp(live * np.log1p(-_zipf(v)))).sum())      # different ids that are expected
        size = 8 if case["ids"] == "int64" else 4
        if op == "embed":
            return {"bytes": n * size + (rows + n) * h * b, "flops": n * h}
        table = 2 * rows * h * 4 if case["accumulate"] else v * h * 4
        return {"bytes": n * size + live * h * b + table, "flops": 2 * live * h}
    n, v = sum(_lengths(case)) if op == "preference" else case["n"], case["v"]
    rest = dict(policy=n * (8 + 4 * 2 + 4 * case.get("reference", 0) + 4 * case.get("weighted", 0) + 4),
                preference=n * 8 + 16 * case.get("pairs", 0),
                distill=n * (case.get("k", 0) * (b + (8 if case.get("ids") == "int64" else 4)) + 4))[op]
    return {"bytes": 2 * n * v * b + rest, "flops": 8 * n * v}


# ---------------------------------------------------------------- inputs

def _logits(normal, n, v, dtype):
    """A model's logits: noise about a common level for each id, as unigram frequencies give it."""
    z = normal(n, v)
    z += 1.5 * normal(v)
    return z, z.to(TYPES[dtype])


def _sampled(gen, z, logits, dtype):
    """Targets that a model would sample: mostly likely ids, some of them rare, and prompt tokens that are ignored."""
    n, v = z.shape
    target = torch.randint(0, v, (n,), generator=gen, device=DEV)
    lift = torch.rand(n, generator=gen, device=DEV) * 14
    at = torch.arange(n, device=DEV)
    logits[at, target] = (z[at, target] + lift).to(TYPES[dtype])
    ignored = torch.rand(n, generator=gen, device=DEV) < 0.1
    ignored[0] = False                       # a batch with no token at all is not a step
    target[ignored] = IGNORE
    return target


def _logp(logits, target, temperature):
    """Log-probabilities of the targets, 0 for ignored ones: what the models that sampled them left behind."""
    z = logits.float() / temperature
    picked = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    return torch.where(target == IGNORE, 0.0, picked - torch.logsumexp(z, 1))


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(scale)

    op = case["op"]
    if op in ("embed", "embed_bwd"):
        n, v, h = case["n"], case["v"], case["h"]
        share = torch.from_numpy(np.cumsum(_zipf(v))).to(DEV)
        rank = torch.searchsorted(share, torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)).clamp_(max=v - 1)
        ids = torch.randperm(v, generator=gen, device=DEV)[rank]
        if case["padding"]:
            ids[torch.rand(n, generator=gen, device=DEV) < case["padding"]] = 0
        s = dict(ids=ids.to(IDS[case["ids"]]))
        if op == "embed":
            s["weight"] = normal(v, h, scale=0.02).to(TYPES[case["dtype"]])
            return s
        s["grad_y"] = normal(n, h, scale=1e-2).to(TYPES[case["dtype"]])
        if case["accumulate"]:
            s["grad"] = normal(v, h, scale=1e-3)
        return s
    n = sum(_lengths(case)) if op == "preference" else case["n"]
    z, logits = _logits(normal, n, case["v"], case["dtype"])
    s = dict(logits=logits)
    if op == "distill":
        k = min(case["k"], case["v"])
        values, ids = (z.mul_(0.8) + 0.6 * normal(n, case["v"])).topk(k, dim=1)
        # lists cut where the teacher's probability is used up, and prompt tokens that have none
        length = torch.randint(1, k + 1, (n, 1), generator=gen, device=DEV)
        length[1:][torch.rand(n - 1, generator=gen, device=DEV) < 0.05] = 0
        ids[torch.arange(k, device=DEV)[None] >= length] = -1
        s.update(ids=ids.to(IDS[case["ids"]]), values=values.to(TYPES[case["dtype"]]))
        s["weight"] = torch.rand(n, generator=gen, device=DEV) + 0.5 if case["weighted"] else None
        return s
    s["target"] = _sampled(gen, z, logits, case["dtype"])
    if op == "policy":
        logp = _logp(logits, s["target"], case["temperature"])
        change = normal(n, scale=0.15)
        # a ratio that rounding could put on either side of the clip's border says nothing about a kernel
        for border in (1 - case["clip"], 1 + case["clip"]):
            change = torch.where((change - math.log(border)).abs() < 1e-4, change + 4e-4, change)
        s["advantage"] = normal(n)
        s["old_logp"] = torch.where(s["target"] == IGNORE, 0.0, logp - change)
        s["ref_logp"] = logp + normal(n, scale=0.3) if case["reference"] else None
        s["weight"] = 1 / torch.randint(16, 512, (n,), generator=gen, device=DEV).float() if case["weighted"] else None
        return s
    ends = torch.tensor(_lengths(case), device=DEV).cumsum(0)
    s["offsets"] = torch.cat([torch.zeros_like(ends[:1]), ends])
    sums = _sums(_logp(logits, s["target"], 1.0), s["target"], s["offsets"], case["average"])
    s["ref_logp"] = (sums + normal(2 * case["pairs"], scale=0.2 if case["average"] else 5.0)).float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _softmax(logits, temperature):
    """(exp(z - largest), largest, sum of the first) of z = logits / temperature, in 32 bits."""
    z = logits.float()
    if temperature != 1:
        z = z / temperature
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    return e, z, top, e.sum(1, keepdim=True)


def _gradient(e, total, factor, target, live, dtype):
    """factor * (softmax - onehot), by rows."""
    g = e * (factor / total[:, 0])[:, None]
    at = torch.arange(len(target), device=DEV)
    g[at, target] -= torch.where(live, factor, 0.0)
    return g.to(dtype)


def _policy_own(s):
    import linear_cross_entropy_03_gb300 as flce
    c = s["case"]
    out = flce.policy_loss(s["logits"], s["target"], s["advantage"], old_logp=s["old_logp"], ref_logp=s["ref_logp"],
                           clip=c["clip"], kl_weight=c["kl"] if c["reference"] else 0.0, temperature=c["temperature"],
                           row_weight=s["weight"], ignore_index=IGNORE, reduction=c["reduction"])
    return [out["loss"], out["logp"], out["grad_logits"]]


def _policy_plain(s):
    c = s["case"]
    live = s["target"] != IGNORE
    target = s["target"].clamp(min=0)
    e, z, top, total = _softmax(s["logits"], c["temperature"])
    logp = (z.gather(1, target[:, None]) - top - total.log())[:, 0]
    a, low, high = s["advantage"], 1 - c["clip"], 1 + c["clip"]
    ratio = torch.exp(logp - s["old_logp"])
    loss = -torch.minimum(ratio * a, ratio.clamp(low, high) * a)
    cut = ((a > 0) & (ratio > high)) | ((a < 0) & (ratio < low))
    slope = torch.where(cut, 0.0, -a * ratio)                     # of the loss by logp
    if s["ref_logp"] is not None and c["kl"]:
        d = s["ref_logp"] - logp
        loss = loss + c["kl"] * (torch.expm1(d) - d)
        slope = slope - c["kl"] * torch.expm1(d)
    if s["weight"] is not None:
        loss, slope = loss * s["weight"], slope * s["weight"]
    loss, slope = torch.where(live, loss, 0.0), torch.where(live, slope, 0.0)
    if c["reduction"] == "mean":
        slope = slope / live.sum()
    if c["reduction"] != "none":
        total_loss = loss.double().sum()
        loss = (total_loss / live.sum() if c["reduction"] == "mean" else total_loss).float()
    grad = _gradient(e, total, -slope / c["temperature"], target, live, s["logits"].dtype)
    return [loss, torch.where(live, logp, 0.0), grad]


def _sums(logp, target, offsets, average):
    """Each sequence's log-probability, in 64 bits."""
    run = torch.cat([torch.zeros(1, dtype=torch.float64, device=DEV), logp.double().cumsum(0)])
    total = run[offsets[1:]] - run[offsets[:-1]]
    return total / _counts(target, offsets).clamp(min=1) if average else total


def _counts(target, offsets):
    seen = torch.cat([torch.zeros_like(target[:1]), (target != IGNORE).cumsum(0)])
    return seen[offsets[1:]] - seen[offsets[:-1]]


def _pair_loss(x, kind, beta, smoothing):
    """A pair's loss and its slope by x, the chosen sequence's log ratio less the other's."""
    u = beta * x
    if kind == "sigmoid":
        def softplus(w):
            return torch.clamp(w, min=0) + torch.log1p(torch.exp(-w.abs()))
        loss = (1 - smoothing) * softplus(-u) + smoothing * softplus(u)
        return loss, beta * (torch.sigmoid(u) - (1 - smoothing))
    if kind == "hinge":
        return torch.clamp(1 - u, min=0), torch.where(u < 1, -beta, 0.0)
    far = x - 1 / (2 * beta)
    return far * far, 2 * far


def _preference_own(s):
    import linear_cross_entropy_03_gb300 as flce
    c = s["case"]
    out = flce.preference_loss(s["logits"], s["target"], offsets=s["offsets"], ref_logp=s["ref_logp"], kind=c["kind"],
                               beta=c["beta"], label_smoothing=c["smoothing"] if c["kind"] == "sigmoid" else 0.0,
                               average=c["average"], ignore_index=IGNORE, reduction=c["reduction"])
    return [out["loss"], out["logp"], out["grad_logits"]]


def _preference_plain(s):
    c, target, offsets = s["case"], s["target"], s["offsets"]
    live = target != IGNORE
    at = target.clamp(min=0)
    e, z, top, total = _softmax(s["logits"], 1.0)
    logp = torch.where(live, (z.gather(1, at[:, None]) - top - total.log())[:, 0], 0.0)
    sums = _sums(logp, target, offsets, c["average"])
    ratio = sums - s["ref_logp"].double()
    p = c["pairs"]
    loss, slope = _pair_loss(ratio[:p] - ratio[p:], c["kind"], c["beta"], c["smoothing"] if c["kind"] == "sigmoid" else 0.0)
    if c["reduction"] == "mean":
        slope = slope / p
    if c["reduction"] != "none":
        loss = loss.mean() if c["reduction"] == "mean" else loss.sum()
    slope = torch.cat([slope, -slope])
    if c["average"]:
        slope = slope / _counts(target, offsets).clamp(min=1)
    slope = slope.float().repeat_interleave(offsets[1:] - offsets[:-1], output_size=len(target))
    grad = _gradient(e, total, torch.where(live, -slope, 0.0), at, live, s["logits"].dtype)
    return [loss.float(), sums.float(), grad]


def _distill_own(s):
    import linear_cross_entropy_03_gb300 as flce
    c = s["case"]
    out = flce.distillation_loss(s["logits"], s["ids"], s["values"], temperature=c["temperature"],
                                 row_weight=s["weight"], reduction=c["reduction"])
    return [out["loss"], out["grad_logits"]]


def _distill_plain(s):
    c, t = s["case"], s["case"]["temperature"]
    ids, held = s["ids"].long().clamp(min=0), s["ids"] >= 0
    live = held[:, 0]
    best = torch.where(held, s["values"].float() / t, float("-inf"))
    best = best - torch.where(live, best.amax(1), 0.0)[:, None]
    q = torch.exp(best)
    norm = torch.where(live, q.sum(1), 1.0)[:, None]
    q, log_q = q / norm, best - norm.log()
    e, z, top, total = _softmax(s["logits"], t)
    log_p = z.gather(1, ids) - top - total.log()
    loss = t * t * torch.where(q > 0, q * (log_q - log_p), 0.0).sum(1)
    factor = torch.where(live, float(t), 0.0)
    if s["weight"] is not None:
        loss, factor = loss * s["weight"], factor * s["weight"]
    if c["reduction"] == "mean":
        factor = factor / live.sum()
    if c["reduction"] != "none":
        all_rows = loss.double().sum()
        loss = (all_rows / live.sum() if c["reduction"] == "mean" else all_rows).float()
    grad = e * (factor / total[:, 0])[:, None]
    grad.scatter_add_(1, ids, -factor[:, None] * q)
    return [loss, grad.to(s["logits"].dtype)]


def _embed_own(s):
    import linear_cross_entropy_03_gb300 as flce
    return [flce.embedding(s["weight"], s["ids"], scale=s["case"]["scale"])["y"]]


def _embed_plain(s):
    return [(s["weight"][s["ids"]].float() * s["case"]["scale"]).to(s["weight"].dtype)]


def _embed_bwd_own(s):
    import linear_cross_entropy_03_gb300 as flce
    c = s["case"]
    out = flce.embedding_backward(s["grad_y"], s["ids"], c["v"], scale=c["scale"],
                                  padding_index=0 if c["padding"] else None, grad_weight_out=s.get("grad"),
                                  accumulate=c["accumulate"])
    return [out["grad_weight"]]


def _embed_bwd_plain(s):
    c = s["case"]
    g = s["grad_y"].float() * c["scale"]
    if c["padding"]:
        g = g * (s["ids"] != 0)[:, None]
    table = s["grad"] if c["accumulate"] else torch.zeros(c["v"], c["h"], device=DEV)
    return [table.index_add_(0, s["ids"], g)]


_own = dict(policy=_policy_own, preference=_preference_own, distill=_distill_own, embed=_embed_own,
            embed_bwd=_embed_bwd_own)
_plain = dict(policy=_policy_plain, preference=_preference_plain, distill=_distill_plain, embed=_embed_plain,
              embed_bwd=_embed_bwd_plain)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    s, c, op = _inputs(case, seed), case, case["op"]
    if op == "embed":
        return [torch.index_select(s["weight"], 0, s["ids"].long()).double() * c["scale"]]
    if op == "embed_bwd":
        keep = (s["ids"] != 0) if c["padding"] else torch.ones_like(s["ids"], dtype=torch.bool)
        table = s["grad"].double() if c["accumulate"] else torch.zeros(c["v"], c["h"], device=DEV, dtype=torch.float64)
        return [table.index_put_((s["ids"][keep].long(),), c["scale"] * s["grad_y"][keep].double(), accumulate=True)]
    t = c.get("temperature", 1.0)
    z = s["logits"].double().div_(t)
    log_p = z.sub_(torch.logsumexp(z, 1, keepdim=True))
    if op == "distill":
        k = s["ids"].shape[1]
        held = s["ids"] >= 0
        rows = held.any(1)
        at = torch.where(held, s["ids"].long(), 0)
        log_q = torch.log_softmax(torch.where(held, s["values"].double() / t, -torch.inf), 1)
        log_q[~rows] = -torch.inf
        q = log_q.exp()
        terms = torch.where(q > 0, q * (torch.where(q > 0, log_q, 0.0) - log_p.gather(1, at)), 0.0)
        w = s["weight"].double() if s["weight"] is not None else torch.ones(len(rows), device=DEV, dtype=torch.float64)
        w = w * rows
        div = float(rows.sum()) if c["reduction"] == "mean" else 1.0
        loss = t * t * w * terms.sum(1)
        grad = log_p.exp_().mul_((w * t / div)[:, None])
        for j in range(k):
            grad[torch.arange(len(rows), device=DEV), at[:, j]] -= w * t / div * q[:, j]
        return [loss if c["reduction"] == "none" else loss.sum() / div, grad]
    live = s["target"] != IGNORE
    at = torch.where(live, s["target"], 0)
    rows = torch.arange(len(at), device=DEV)
    logp = log_p[rows, at] * live
    if op == "policy":
        a, r = s["advantage"].double(), torch.exp(logp - s["old_logp"].double())
        inside = ~torch.where(a >= 0, r > 1 + c["clip"], r < 1 - c["clip"])
        loss = -a * torch.where(inside, r, torch.where(a >= 0, 1 + c["clip"], 1 - c["clip"]))
        by_logp = -a * r * inside
        if s["ref_logp"] is not None:
            x = s["ref_logp"].double() - logp
            loss = loss + c["kl"] * (x.exp() - x - 1)
            by_logp = by_logp + c["kl"] * (1 - x.exp())
        w = live * (s["weight"].double() if s["weight"] is not None else 1.0)
        loss, by_logp = loss * w, by_logp * w
        div = float(live.sum()) if c["reduction"] == "mean" else 1.0
        out = loss if c["reduction"] == "none" else loss.sum() / div
        by_logp = by_logp / div
    else:
        bounds = s["offsets"].tolist()
        p = c["pairs"]
        parts = [slice(x, y) for x, y in zip(bounds[:-1], bounds[1:])]
        count = [max(1, int(live[x].sum())) if c["average"] else 1 for x in parts]
        seq = torch.stack([logp[x].sum() / n for x, n in zip(parts, count)])
        x = (seq - s["ref_logp"].double()).requires_grad_(True)
        d = x[:p] - x[p:]
        if c["kind"] == "sigmoid":
            up, down = torch.nn.functional.logsigmoid(c["beta"] * d), torch.nn.functional.logsigmoid(-c["beta"] * d)
            loss = -(1 - c["smoothing"]) * up - c["smoothing"] * down
        else:
            loss = torch.relu(1 - c["beta"] * d) if c["kind"] == "hinge" else (d - 0.5 / c["beta"]) ** 2
        out = dict(none=loss, sum=loss.sum(), mean=loss.sum() / p)[c["reduction"]]
        by_seq, = torch.autograd.grad(out.sum(), x)
        out, by_logp = out.detach(), torch.zeros_like(logp)
        for k, part in enumerate(parts):
            by_logp[part] = by_seq[k] / count[k]
        by_logp, logp = by_logp * live, seq
    by_logit = by_logp / t
    grad = log_p.exp_().mul_(-by_logit[:, None])
    grad[rows, at] += by_logit
    return [out, logp, grad]
