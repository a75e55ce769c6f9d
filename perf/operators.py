"""Cases for the operators around the language-model head, in plain torch and
through this package.

The operators are what a training step runs beside the fused linear cross
entropy, and what a serving step runs before the head:

  ln_fwd     y = norm(x [+ residual]) * weight + bias: layer norm, or its form
             without the mean ("rms"); also the sum and the row statistics
  ln_bwd     grad_x, grad_weight and grad_bias of the same
  grad_norm  the 2-norm of many gradients together and the factor that clips it
  adamw      one AdamW step over many tensors with fp32 moments, and the 16-bit
             copies of the parameters that the products read
  adamw8     the same with moments in 8 bits: e4m3 numbers, one fp32 scale for
             each block of 256 (the second moment is held as its root)

``own`` chooses between the plain form (elementary torch operations in 32 bits)
and the package's calls.  The tensors of an optimiser case lie one after another
in flat buffers, so that the plain form is one expression over a buffer.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 256          # moments that share a scale in adamw8
E4M3 = 448.0         # the largest e4m3 number
EPS = 1e-5
LR, BETAS, ADAM_EPS, DECAY = 1e-4, (0.9, 0.95), 1e-8, 0.1
STEP0 = 100          # steps already taken when a case starts
MAX_NORM = 1.0


# ---------------------------------------------------------------- cases

def _ln(name, op, n, h, dtype, kind, residual, bias):
    return dict(name=name, op=op, n=n, h=h, dtype=dtype, kind=kind, residual=residual, bias=bias)


def _opt(name, op, tensors, smallest, largest, mix, grad, copy="none", seed=-1):
    return dict(name=name, op=op, tensors=tensors, smallest=smallest, largest=largest, mix=mix, grad=grad,
                copy=copy, seed=seed)


def listed():
    return [
        # one token of a decoder before its head, when serving: latency
        _ln("ln_fwd 1x4096 rms", "ln_fwd", 1, 4096, "bf16", "rms", True, False),
        # the norm before the Llama-3-8B head in a training step, with its residual add
        _ln("ln_fwd 16384x4096 rms", "ln_fwd", 16384, 4096, "bf16", "rms", True, False),
        # rows that are no whole number of vectors, on a batch that is none of tiles
        _ln("ln_fwd 8191x2047 layer", "ln_fwd", 8191, 2047, "fp16", "layer", False, True),
        # the tiny workload's batch: a backward pass bound by latency
        _ln("ln_bwd 256x128 layer", "ln_bwd", 256, 128, "fp32", "layer", False, True),
        # the same norms' backward passes in training
        _ln("ln_bwd 16384x4096 rms", "ln_bwd", 16384, 4096, "bf16", "rms", True, False),
        _ln("ln_bwd 8191x2048 layer", "ln_bwd", 8191, 2048, "fp32", "layer", False, True),
        # the head's fp32 gradient, as the fused linear cross entropy leaves it (Llama-3.2-1B), and a norm's weight
        _opt("grad_norm 1B head", "grad_norm", 2, 2048, 128256 * 2048, 0, "fp32"),
        # a model's many 16-bit gradients, packed one after another, from single numbers up
        _opt("grad_norm 300 packed", "grad_norm", 300, 1, 2000003, 7, "bf16"),
        # the head's weight and a norm's, fp32 with the bf16 copy that the products read
        _opt("adamw 1B head", "adamw", 2, 2048, 128256 * 2048, 0, "fp32", "bf16"),
        # a model's many tensors, packed one after another, with 16-bit gradients
        _opt("adamw 200 packed", "adamw", 200, 1, 1000003, 11, "bf16", "bf16"),
        # the Llama-3-8B head with moments in 8 bits, rounded stochastically so that small changes are kept
        _opt("adamw8 8B head", "adamw8", 2, 4096, 128256 * 4096, 0, "fp32", "bf16", 1234),
        # many ragged tensors with moments in 8 bits, rounded to nearest
        _opt("adamw8 120 ragged", "adamw8", 120, 1, 500009, 13, "bf16", "none", -1),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "grad_norm", "adamw", "adamw8"))
    if op in ("ln_fwd", "ln_bwd"):
        h = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            h = -(-h // 64) * 64          # widths that models have; the others are odd ones among them
        n = _log(rng, 1, max(1, min(65536, (1 << 26) // h)))
        return dict(op=op, n=n, h=h, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")), kind=rng.choice(("layer", "rms")),
                    residual=rng.random() < 0.5, bias=rng.random() < 0.5)
    tensors = _log(rng, 1, 300)
    largest = _log(rng, 1000, min(1 << 26, (1 << 28) // tensors))
    return dict(op=op, tensors=tensors, smallest=_log(rng, 1, largest), largest=largest, mix=rng.randrange(1 << 20),
                grad=rng.choice(("fp32", "bf16", "fp16")), copy=rng.choice(("none", "bf16", "fp16")),
                seed=rng.choice((-1, rng.randrange(1 << 30))))


def _sizes(case):
    """Elements of each tensor: the smallest and the largest, and others between them."""
    rng, t = random.Random(case["mix"]), case["tensors"]
    return [case["largest"], case["smallest"]][:t] + [_log(rng, case["smallest"], case["largest"]) for _ in range(t - 2)]


def _starts(case):
    """Where each tensor starts in the flat buffers, and their length.  Packed, but for 8-bit moments, whose
    tensors start a block (the gaps stay zero)."""
    step, at, starts = BLOCK if case["op"] == "adamw8" else 1, 0, []
    for n in _sizes(case):
        starts.append(at)
        at += -(-n // step) * step
    return starts, at


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        n, h, b = case["n"], case["h"], SIZE[case["dtype"]]
        stats = 4 * n * (1 if case["kind"] == "rms" else 2)
        params = h * b * (2 if case["bias"] else 1)
        if op == "ln_fwd":
            return {"bytes": (4 if case["residual"] else 2) * n * h * b + params + stats, "flops": 8 * n * h}
        grads = 4 * h * (2 if case["bias"] else 1)
        return {"bytes": (4 if case["residual"] else 3) * n * h * b + h * b + grads + stats, "flops": 15 * n * h}
    n, g = sum(_sizes(case)), SIZE[case["grad"]]
    if op == "grad_norm":
        return {"bytes": n * g + 8, "flops": 2 * n}
    copy = SIZE.get(case["copy"], 0)
    if op == "adamw":
        return {"bytes": n * (24 + g + copy), "flops": 16 * n}
    blocks = sum(-(-k // BLOCK) for k in _sizes(case))
    return {"bytes": n * (12 + g + copy) + 16 * blocks, "flops": 30 * n}


# ---------------------------------------------------------------- inputs

def _views(buffer, starts, sizes):
    """Each tensor, as a view of the flat buffer it lies in."""
    return [buffer[a:a + n] for a, n in zip(starts, sizes)]


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).to(dtype)

    if case["op"] in ("ln_fwd", "ln_bwd"):
        n, h, dt = case["n"], case["h"], TYPES[case["dtype"]]
        channels = torch.exp(0.5 * normal(h))            # hidden states differ in scale from channel to channel
        s = dict(x=(normal(n, h) * channels + 0.3).to(dt), weight=(1 + 0.2 * normal(h)).to(dt),
                 bias=normal(h, dtype=dt, scale=0.1) if case["bias"] else None)
        if case["op"] == "ln_fwd":
            s["residual"] = normal(n, h, dtype=dt) if case["residual"] else None
            return s
        x = s["x"].float()
        s["mean"] = x.mean(1) if case["kind"] == "layer" else None
        centred = x - s["mean"][:, None] if case["kind"] == "layer" else x
        s["rstd"] = torch.rsqrt((centred * centred).mean(1) + EPS)
        s["grad_y"] = normal(n, h, dtype=dt, scale=1e-2)
        s["grad_sum"] = normal(n, h, dtype=dt, scale=1e-2) if case["residual"] else None
        return s
    starts, length = _starts(case)
    sizes = _sizes(case)
    live = None
    if case["op"] == "adamw8":
        live = torch.zeros(length, dtype=torch.bool, device=DEV)
        for v in _views(live, starts, sizes):
            v.fill_(True)

    def buffer(scale):
        t = normal(length, scale=scale)
        return t if live is None else t.mul_(live)

    s = dict(sizes=sizes, starts=starts, grad=buffer(2e-3).to(TYPES[case["grad"]]))
    if case["op"] == "grad_norm":
        return s
    s["param"] = buffer(0.02)
    s["exp_avg"] = buffer(5e-4)
    s["exp_avg_sq"] = buffer(2e-3).square_()
    if case["copy"] != "none":
        s["copy"] = s["param"].to(TYPES[case["copy"]])
    if case["op"] == "adamw8":
        for name in ("exp_avg", "exp_avg_sq"):
            old = s[name].view(-1, BLOCK)
            old = old.sqrt() if name == "exp_avg_sq" else old
            scale = old.abs().amax(1) / E4M3
            inv = torch.where(scale > 0, 1 / scale, 0)
            s[name] = (old * inv[:, None]).clamp_(-E4M3, E4M3).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] in ("ln_fwd", "ln_bwd"):
        return s

    def view(buffer):
        return _views(buffer, s["starts"], s["sizes"])

    s["grads"] = view(s["grad"])
    s["step"] = STEP0
    # a gradient clip's factor, as grad_norm leaves it on the device
    s["clip"] = torch.full((1,), 0.75, device=DEV)
    if own and case["op"] in ("adamw", "adamw8"):
        import linear_cross_entropy_03_gb300 as flce
        state = dict(exp_avg=view(s["exp_avg"]), exp_avg_sq=view(s["exp_avg_sq"]))
        if case["op"] == "adamw8":
            first = [a // BLOCK for a in s["starts"]]
            blocks = [-(-n // BLOCK) for n in s["sizes"]]
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                state[name] = _views(s[name], first, blocks)
        s["optimizer"] = flce.AdamW(
            view(s["param"]), lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, step=STEP0, state=state,
            copies=view(s["copy"]) if "copy" in s else None, seed=case["seed"] if case["seed"] >= 0 else None)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _ln_fwd_own(s):
    import linear_cross_entropy_03_gb300 as flce
    out = flce.layer_norm(s["x"], s["weight"], s["bias"], kind=s["case"]["kind"], eps=EPS, residual=s["residual"])
    return [out["y"], out["sum"], out["mean"], out["rstd"]]


def _ln_fwd_plain(s):
    layer, dt = s["case"]["kind"] == "layer", s["x"].dtype
    total = s["x"].float()
    if s["residual"] is not None:
        total = (total + s["residual"].float()).to(dt)
    h = total.float()
    mean = h.mean(1) if layer else None
    centred = h - mean[:, None] if layer else h
    rstd = torch.rsqrt((centred * centred).mean(1) + EPS)
    y = centred * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return [y.to(dt), total if s["residual"] is not None else None, mean, rstd]


def _ln_bwd_own(s):
    import linear_cross_entropy_03_gb300 as flce
    out = flce.layer_norm_backward(s["grad_y"], s["x"], s["weight"], mean=s["mean"], rstd=s["rstd"],
                                   kind=s["case"]["kind"], grad_sum=s["grad_sum"], grad_bias=s["bias"] is not None)
    return [out["grad_x"], out["grad_weight"], out["grad_bias"]]


def _ln_bwd_plain(s):
    layer, dt = s["case"]["kind"] == "layer", s["x"].dtype
    x, gy, rstd = s["x"].float(), s["grad_y"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd if layer else x * rstd
    wgy = gy * s["weight"].float()
    gx = wgy - xhat * (wgy * xhat).mean(1, keepdim=True)
    if layer:
        gx = gx - wgy.mean(1, keepdim=True)
    gx = gx * rstd
    if s["grad_sum"] is not None:
        gx = gx + s["grad_sum"].float()
    return [gx.to(dt), (gy * xhat).sum(0), gy.sum(0) if s["bias"] is not None else None]


def _grad_norm_own(s):
    import linear_cross_entropy_03_gb300 as flce
    out = flce.grad_norm(s["grads"], max_norm=MAX_NORM)
    return [out["norm"], out["scale"]]


def _grad_norm_plain(s):
    g = s["grad"].float()
    norm = (g * g).sum().sqrt()
    return [norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]


def _adamw_outputs(s):
    names = ("param", "exp_avg", "exp_avg_sq", "copy", "exp_avg_scale", "exp_avg_sq_scale")
    return [s[k] for k in names if k in s]


def _adamw_own(s):
    s["optimizer"].step(s["grads"], grad_scale=s["clip"])
    return _adamw_outputs(s)


def _factors(step):
    return LR / (1 - BETAS[0] ** step), 1 / math.sqrt(1 - BETAS[1] ** step)


def _update(s, m, v, root):
    """The parameters' update from the new moments (`root` is the second's root)."""
    rate, correction = _factors(s["step"])
    p = s["param"].mul_(1 - LR * DECAY)
    p.sub_(m / (root * correction + ADAM_EPS) * rate)
    if "copy" in s:
        s["copy"].copy_(p)


def _moments(s, m, v):
    b1, b2 = BETAS
    g = s["grad"].float() * s["clip"]
    return m * b1 + g * (1 - b1), v * b2 + g * g * (1 - b2)


def _adamw_plain(s):
    s["step"] += 1
    m, v = _moments(s, s["exp_avg"], s["exp_avg_sq"])
    s["exp_avg"].copy_(m)
    s["exp_avg_sq"].copy_(v)
    _update(s, m, v, v.sqrt())
    return _adamw_outputs(s)


def _mix(x):
    """32 bits to 32 bits (held in int64): two multiplications between shifted exclusive ors."""
    x = ((x ^ (x >> 16)) * 0xA54D2F6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xD1B54A33) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _bits(s):
    """32 bits for each element of the flat buffer, from the seed, the step, the tensor and its place in it."""
    seed, starts = s["case"]["seed"], torch.tensor(s["starts"], device=DEV)
    key = _mix(torch.full_like(starts, seed & 0xFFFFFFFF))
    key = _mix(key ^ (seed >> 32))
    key = _mix(key ^ s["step"])
    key = _mix(key ^ torch.arange(len(starts), device=DEV))
    key = _mix(key)                                       # the high half of the place, 0 here
    which = torch.zeros_like(s["param"], dtype=torch.int64)
    which[starts[1:]] = 1
    which = which.cumsum(0)                               # the tensor of each element
    place = torch.arange(len(which), device=DEV) - starts[which]
    return _mix(place ^ key[which])


def _e4m3(x, bits):
    """x (up to 448 in size) as e4m3 numbers; `bits` (16 of them) round stochastically, None to nearest."""
    if bits is None:
        return x.clamp(-E4M3, E4M3).to(torch.float8_e4m3fn)
    a = x.abs().clamp(max=E4M3)
    lift = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)     # below the normal numbers the spacing stays 2^-9
    a = ((a + lift).view(torch.int32) + (bits << 4).to(torch.int32)) & ~0xFFFFF
    a = (a.view(torch.float32) - lift).clamp(max=E4M3)
    return torch.copysign(a, x).to(torch.float8_e4m3fn)


def _encode(x, bits, keep):
    """Blocks of x as e4m3 numbers and scales; `keep`: what is not zero stays at least the smallest number."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1) / E4M3
    scale = torch.where((scale > 0) & (scale < 2.0 ** -126), 2.0 ** -126, scale)
    inv = torch.where(scale > 0, 1 / scale, 0.0)
    y = x * inv[:, None]
    code = _e4m3(y, None if bits is None else bits.view(-1, BLOCK))
    if keep:
        code = torch.where((x > 0) & (code.float() == 0), 2.0 ** -9, code.float()).to(torch.float8_e4m3fn)
    return code.view(-1), scale


def _adamw8_plain(s):
    s["step"] += 1
    m = s["exp_avg"].float().view(-1, BLOCK) * s["exp_avg_scale"][:, None]
    r = s["exp_avg_sq"].float().view(-1, BLOCK) * s["exp_avg_sq_scale"][:, None]
    m, v = _moments(s, m.view(-1), (r * r).view(-1))
    root = v.sqrt()
    bits = _bits(s) if s["case"]["seed"] >= 0 else None
    for name, x, b in (("exp_avg", m, None if bits is None else bits >> 16),
                       ("exp_avg_sq", root, None if bits is None else bits & 0xFFFF)):
        code, scale = _encode(x, b, name == "exp_avg_sq")
        s[name].copy_(code)
        s[name + "_scale"].copy_(scale)
    _update(s, m, v, root)
    return _adamw_outputs(s)


_own = dict(ln_fwd=_ln_fwd_own, ln_bwd=_ln_bwd_own, grad_norm=_grad_norm_own, adamw=_adamw_own, adamw8=_adamw_own)
_plain = dict(ln_fwd=_ln_fwd_plain, ln_bwd=_ln_bwd_plain, grad_norm=_grad_norm_plain, adamw=_adamw_plain,
              adamw8=_adamw8_plain)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "ln_fwd":
        h = d["x"]
        if case["residual"]:
            h = (h + d["residual"]).to(TYPES[case["dtype"]]).double()   # the sum is held in the inputs' type
        mu = h.sum(1) / case["h"] if case["kind"] == "layer" else torch.zeros_like(h[:, 0])
        second = (h - mu[:, None]).square().sum(1) / case["h"]
        inv = 1.0 / (second + EPS).sqrt()
        y = (h - mu[:, None]) * inv[:, None] * d["weight"] + (d["bias"] if case["bias"] else 0.0)
        return [y, h if case["residual"] else None, mu if case["kind"] == "layer" else None, inv]
    if case["op"] == "ln_bwd":
        # grad_x = J^T (weight * grad_y), J the derivative of xhat(x) at the saved statistics
        xhat = (d["x"] - (d["mean"][:, None] if case["kind"] == "layer" else 0.0)) * d["rstd"][:, None]
        u = d["grad_y"] * d["weight"]
        dot = torch.einsum("nh,nh->n", u, xhat) / case["h"]
        gx = u - dot[:, None] * xhat - (u.sum(1, keepdim=True) / case["h"] if case["kind"] == "layer" else 0.0)
        gx = gx * d["rstd"][:, None] + (d["grad_sum"] if case["residual"] else 0.0)
        return [gx, torch.einsum("nh,nh->h", d["grad_y"], xhat), d["grad_y"].sum(0) if case["bias"] else None]
    if case["op"] == "grad_norm":
        norm = float(torch.linalg.vector_norm(d["grad"]))
        return [torch.tensor(norm, dtype=torch.float64), torch.tensor(min(1.0, MAX_NORM / (norm + 1e-6)), dtype=torch.float64)]
    # the inputs are the moments as held; lr, betas and the clip factor are the user's numbers
    t, (b1, b2) = STEP0 + 1, BETAS
    g = d["grad"].mul_(0.75)
    if case["op"] == "adamw8":
        m = d["exp_avg"].view(-1, BLOCK).mul_(d["exp_avg_scale"][:, None]).view(-1)
        v = d["exp_avg_sq"].view(-1, BLOCK).mul_(d["exp_avg_sq_scale"][:, None]).square_().view(-1)
    else:
        m, v = d["exp_avg"], d["exp_avg_sq"]
    m.mul_(b1).add_(g, alpha=1 - b1)
    v.mul_(b2).addcmul_(g, g, value=1 - b2)
    p = d["param"]
    p.mul_(1 - LR * DECAY).sub_(LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + ADAM_EPS))
    copy = [p] if case["copy"] != "none" else []
    if case["op"] == "adamw":
        return [p, m, v] + copy
    coded, scales = [], []
    for x in (m, v.sqrt()):
        x = x.view(-1, BLOCK)
        scale = x.abs().amax(1) / E4M3
        x = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0)
        # the spacing of e4m3 numbers around x; rounding to nearest is one value of what either rounding gives
        spacing = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        coded.append(((x / spacing).round() * spacing).view(-1) if case["seed"] < 0 else x.reshape(-1))
        scales.append(scale)
    return [p] + coded + copy + scales
