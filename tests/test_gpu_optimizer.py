"""The gradients' norm and AdamW on the GPU against the definitions in 64 bits.

Tolerances, fixed by the arithmetic (fp32, unit 2^-24): the moments are two
products and a sum of constants rounded to fp32, 4 units of the terms' sizes;
the update is those, a root, a division and two products, 2^-18 of its size; the
parameter adds three roundings of its own and one to its type.
"""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}
SIZES = [1, 3, 4, 7, 8, 255, 256, 257, 1000, 4095, 4096, 4097, 5000, 20011, 70000]


def host(t):
    return t.double().cpu().numpy().reshape(-1)


def normal(n, seed, scale=1.0, dtype="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(TYPES[dtype])


# ------------------------------------------------------------ gradients' norm

def norm_of(tensors):
    return math.sqrt(sum(float((host(t) ** 2).sum()) for t in tensors))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_norm(dtype):
    grads = [normal(n, k, 0.1, dtype) for k, n in enumerate(SIZES)]
    want = norm_of(grads)
    for max_norm in (None, 0.5, 1e9):
        out = flce.grad_norm(grads, max_norm=max_norm)
        assert abs(float(out["norm"]) / want - 1) < 2.0 ** -16
        clip = 1.0 if max_norm is None else min(1.0, max_norm / (want + 1e-6))
        assert abs(float(out["scale"]) / clip - 1) < 2.0 ** -16
    out = flce.grad_norm(grads, max_norm=0.5, grad_scale=0.125)
    assert abs(float(out["norm"]) / (want / 8) - 1) < 2.0 ** -16
    assert abs(float(out["scale"]) / (0.125 * min(1, 0.5 / (want / 8 + 1e-6))) - 1) < 2.0 ** -16


def test_norm_of_mixed_types_offsets_and_empty_tensors():
    base = {d: normal(100003, 9, 1.0, d) for d in TYPES}
    grads = [base[d][o:o + n] for d in TYPES for o in range(9) for n in (0, 1, 5, 1000 + o, 40000)]
    out = flce.grad_norm(grads + [None])
    assert abs(float(out["norm"]) / norm_of(grads) - 1) < 2.0 ** -16


@pytest.mark.parametrize("count", [1, 500, 1280, 1281, 3000])
def test_norm_of_many_tensors(count):
    flat = normal(count * 37, 2)
    grads = list(flat.view(count, 37))
    assert abs(float(flce.grad_norm(grads)["norm"]) / norm_of([flat]) - 1) < 2.0 ** -16


def test_norm_edges():
    zero = torch.zeros(10, device="cuda")
    for grads in ([], [None], [zero[:0]], [zero]):
        out = flce.grad_norm(grads, max_norm=1.0)
        assert float(out["norm"]) == 0 and float(out["scale"]) == 1
    out = flce.grad_norm([zero + 2], max_norm=0.0)
    assert float(out["scale"]) == 0
    for bad in (math.inf, -math.inf, math.nan):
        g = normal(100000, 1)
        g[77777] = bad
        out = flce.grad_norm([zero, g], max_norm=1.0)
        assert not math.isfinite(float(out["norm"])) and math.isnan(float(out["scale"]))


def test_norm_is_the_same_every_run_and_clips_a_large_tensor():
    g = normal((1 << 27) + 5, 3)
    first = flce.grad_norm([g], max_norm=1.0)
    want = math.sqrt(float(g.double().square().sum()))
    assert abs(float(first["norm"]) / want - 1) < 2.0 ** -16
    for _ in range(4):
        again = flce.grad_norm([g], max_norm=1.0)
        assert torch.equal(again["norm"], first["norm"]) and torch.equal(again["scale"], first["scale"])


@pytest.mark.parametrize("count", [1, 3, 700, 3000])
def test_norm_with_any_workspace_and_in_a_graph(count):
    """What the workspace held does not matter, and a replayed call finds its last CTA again."""
    grads = list(normal(count * 5003, 4).view(count, 5003))
    want = flce.grad_norm(grads, max_norm=1.0)
    work = torch.empty(flce.grad_norm_workspace_size(count), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, device="cuda")
    for fill in (0, 0xFF, 0x5A, None):
        if fill is None:
            work.random_(0, 256)
        else:
            work.fill_(fill)
        for _ in range(3):
            out.zero_()
            got = flce.grad_norm(grads, max_norm=1.0, workspace=work, out=out)
            assert torch.equal(got["norm"], want["norm"]) and torch.equal(got["scale"], want["scale"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = flce.grad_norm(grads, max_norm=1.0, workspace=work, out=out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        assert torch.equal(got["norm"], want["norm"])
    work.fill_(0xFF)
    graph.replay()
    assert torch.equal(got["norm"], want["norm"])


# ------------------------------------------------------------ AdamW, fp32 moments

class Reference:
    """The step in 64 bits on copies of an optimiser's tensors."""

    def __init__(self, opt, **numbers):
        self.opt, self.numbers = opt, numbers

    def check(self, before, grads, *, lr, step, factor=1.0, decay=0.01, lr_scale=1.0):
        for i, (p0, m0, v0) in enumerate(before):
            if grads[i] is None:
                continue
            d = decay[i] if isinstance(decay, list) else decay
            rate = lr * (lr_scale[i] if isinstance(lr_scale, list) else lr_scale)
            g = host(grads[i]) * factor
            p, m, v = T.adamw(p0, g, m0, v0, lr=rate, decay=d, step=step, **self.numbers)
            b1, b2 = self.numbers["beta1"], self.numbers["beta2"]
            t = self.opt.params[i].dtype
            size_m = b1 * np.abs(m0) + (1 - b1) * np.abs(g)
            assert (np.abs(host(self.opt.exp_avg[i]) - m) <= 2.0 ** -21 * size_m + 1e-37).all(), i
            assert (np.abs(host(self.opt.exp_avg_sq[i]) - v) <= 2.0 ** -21 * v + 1e-37).all(), i
            step_size = rate * size_m / (1 - b1 ** step) / (np.sqrt(v / (1 - b2 ** step)) + self.numbers["eps"])
            tol = 2.0 ** -22 * np.abs(p0) + 2.0 ** -18 * step_size + UNIT[t] * np.abs(p) + TINY[t]
            assert (np.abs(host(self.opt.params[i]) - p) <= tol).all(), i
            c = self.opt.copies[i]
            if c is not None:
                tol += UNIT[c.dtype] * np.abs(p) + TINY[c.dtype]
                assert (np.abs(host(c) - p) <= tol).all(), i

    def before(self):
        return [(host(p), host(m), host(v)) for p, m, v in zip(self.opt.params, self.opt.exp_avg, self.opt.exp_avg_sq)]


NUMBERS = dict(beta1=0.9, beta2=0.95, eps=1e-8)


def make(sizes, param="fp32", copy=None, offset=0, **kw):
    params = [normal(n + offset, k, 0.05, param)[offset:] for k, n in enumerate(sizes)]
    copies = None
    if copy is not None:
        copies = [torch.zeros(n + offset, dtype=TYPES[copy], device="cuda")[offset:] for n in sizes]
    return flce.AdamW(params, lr=1e-2, betas=(0.9, 0.95), copies=copies, **kw)


@pytest.mark.parametrize("param,grad,copy", [("fp32", "fp32", None), ("fp32", "fp32", "bf16"), ("fp32", "bf16", "bf16"),
                                             ("fp32", "fp16", "fp16"), ("bf16", "bf16", None), ("fp16", "fp32", None),
                                             ("bf16", "fp32", "fp32")])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_adamw(param, grad, copy, offset):
    opt = make(SIZES, param, copy, offset)
    ref = Reference(opt, **NUMBERS)
    for step in range(1, 4):
        grads = [normal(n + offset, 100 * step + k, 1e-2, grad)[offset:] for k, n in enumerate(SIZES)]
        before = ref.before()
        opt.step(grads)
        ref.check(before, grads, lr=1e-2, step=step)
    assert opt.steps == 3


def test_adamw_numbers_of_each_tensor_and_gradients_left_out():
    sizes = [5000, 64, 300]
    decay, scale = [0.1, 0.0, 0.3], [1.0, 0.5, 0.0]
    opt = make(sizes, weight_decay=decay, lr_scale=scale)
    ref = Reference(opt, **NUMBERS)
    grads = [normal(n, k, 1e-2) for k, n in enumerate(sizes)]
    before = ref.before()
    opt.step(grads, lr=3e-3, grad_scale=0.25)
    ref.check(before, grads, lr=3e-3, step=1, factor=0.25, decay=decay, lr_scale=scale)
    before, p = ref.before(), opt.params[1].clone()
    grads[1] = None
    opt.step(grads, grad_scale=torch.tensor([0.5], device="cuda"))
    ref.check(before, grads, lr=1e-2, step=2, factor=0.5, decay=decay, lr_scale=scale)
    assert torch.equal(p, opt.params[1])
    grads[1] = normal(64, 5, 1e-2)
    before = ref.before()
    opt.step(grads)
    ref.check(before, grads, lr=1e-2, step=3, decay=decay, lr_scale=scale)


@pytest.mark.parametrize("count", [4, 5, 40, 41, 360, 361, 800])
def test_adamw_over_many_tensors(count):
    rng = np.random.default_rng(count)
    sizes = [int(n) for n in rng.integers(1, 900, count)]
    sizes[-1] = 9001
    opt = make(sizes)
    ref = Reference(opt, **NUMBERS)
    grads = [normal(n, 7 + k, 1e-2) for k, n in enumerate(sizes)]
    before = ref.before()
    opt.step(grads)
    ref.check(before, grads, lr=1e-2, step=1)


def test_adamw_alignments_that_differ():
    """Parameter, gradient, moments and copy at offsets of their own."""
    n = 3001
    for shift in range(1, 5):
        at = [(k * shift) % 5 for k in range(5)]
        p, g, m, v, c = (normal(n + 8, k, 1e-2)[a:a + n] for k, a in enumerate(at))
        v.square_()
        opt = flce.AdamW([p], lr=1e-2, betas=(0.9, 0.95), copies=[c], state=dict(exp_avg=[m], exp_avg_sq=[v]), step=9)
        ref = Reference(opt, **NUMBERS)
        before = ref.before()
        opt.step([g])
        ref.check(before, [g], lr=1e-2, step=10)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_what_lies_around_the_tensors_stays(moments):
    n, room = 5003, 16
    flat = torch.full((n + 2 * room,), 9.0, device="cuda")
    copy = torch.full((n + 2 * room,), 9.0, dtype=torch.bfloat16, device="cuda")
    for first in (room, room + 1, room + 3):
        flat.fill_(9.0), copy.fill_(9.0)
        opt = flce.AdamW([flat[first:first + n]], lr=1e-2, copies=[copy[first:first + n]], moments=moments)
        opt.step([normal(n, 1)])
        for t in (flat, copy):
            assert (t[:first] == 9).all() and (t[first + n:] == 9).all()
        inner = slice(first, first + n)
        assert (flat[inner] != 9).all() and torch.equal(copy[inner], flat[inner].to(torch.bfloat16))


def test_adamw_step_edges():
    # beta 0: the moments are the gradient and its square; the first step is lr * sign
    p = torch.zeros(100, device="cuda")
    opt = flce.AdamW([p], lr=0.5, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0)
    g = normal(100, 1)
    opt.step([g])
    assert torch.allclose(p, -0.5 * g.sign(), rtol=2.0 ** -20, atol=0)
    # a gradient of zeros moves nothing but the decay
    p = torch.ones(100, device="cuda")
    flce.AdamW([p], lr=0.5, weight_decay=0.1).step([torch.zeros(100, device="cuda")])
    assert torch.allclose(p, torch.full_like(p, 0.95), rtol=2.0 ** -22, atol=0)
    opt = flce.AdamW([], lr=0.1)
    opt.step([])
    assert opt.steps == 1
    opt = flce.AdamW([p[:0], p], lr=0.1)
    opt.step([p[:0], torch.zeros_like(p)])


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_skips_a_step_that_is_not_finite(moments):
    opt = make([5000, 300], copy="bf16", moments=moments)
    grads = [normal(5000, 1), normal(300, 2)]
    opt.step(grads)
    tensors = opt.params + opt.exp_avg + opt.exp_avg_sq + opt.copies
    tensors += [t for t in opt.exp_avg_scale + opt.exp_avg_sq_scale if t is not None]
    kept = [t.clone() for t in tensors]
    grads[0][17] = math.inf
    clip = flce.grad_norm(grads, max_norm=1.0)["scale"]
    opt.step(grads, grad_scale=clip, skip_nonfinite=True)
    opt.step(grads, grad_scale=math.nan, skip_nonfinite=True)
    for t, k in zip(tensors, kept):
        assert torch.equal(t.view(torch.uint8), k.view(torch.uint8))
    assert opt.steps == 2          # the host knew of the second only
    opt.step(grads)                # without the switch the step is taken, and only what is not finite spoils
    assert not opt.params[0][17].isfinite() and opt.params[0].isfinite().sum() == 4999


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_captured_step(moments):
    seed = 5 if moments == "8bit" else None
    opt, other = (make([9000, 700], copy="bf16", moments=moments, seed=seed, capturable=c) for c in (True, False))
    grads = [normal(9000, 1, 1e-2), normal(700, 2, 1e-2)]
    lr, factor = torch.tensor([1e-2], device="cuda"), torch.ones(1, device="cuda")
    opt.step(grads, lr=lr, grad_scale=factor, skip_nonfinite=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads, lr=lr, grad_scale=factor, skip_nonfinite=True)
    factor.fill_(math.nan)
    graph.replay()
    assert opt.steps == 1
    factor.fill_(1.0)
    for _ in range(3):
        graph.replay()
    assert opt.steps == 4
    for _ in range(4):
        other.step(grads)
    for a, b in zip(opt.params, other.params):
        # the device forms the bias corrections itself, in fp32: a few units of the update
        assert (a - b).abs().max() <= 1e-2 * 4 * (2.0 ** -18 if moments == "fp32" else 0.1)
    if moments == "fp32":
        assert all(torch.equal(a, b) for a, b in zip(opt.exp_avg, other.exp_avg))


def test_refused_step_does_not_count():
    for capturable in (False, True):
        opt = make([100], capturable=capturable)
        g, two = normal(100, 1), torch.ones(2, device="cuda")
        for bad in (dict(grads=[g[:50]]), dict(grads=[g], grad_scale=two), dict(grads=[g], grad_scale=two, skip_nonfinite=True),
                    dict(grads=[g], lr=two), dict(grads=[g], lr="fast"), dict(grads=[])):
            with pytest.raises((flce.FlceError, TypeError)):
                opt.step(**bad)
        assert opt.steps == 0
        opt.step([g])
        assert opt.steps == 1


def test_on_another_stream():
    opt, other = make([9000]), make([9000])
    g = normal(9000, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        clip = flce.grad_norm([g], max_norm=1.0, stream=stream)
        opt.step([g], grad_scale=clip["scale"], stream=stream)
        side.synchronize()
        other.step([g], grad_scale=flce.grad_norm([g], max_norm=1.0)["scale"])
    assert torch.equal(opt.params[0], other.params[0])


def test_state_goes_on():
    for moments in ("fp32", "8bit"):
        a = make([6000, 10], moments=moments)
        g = [normal(6000, 1, 1e-2), normal(10, 2, 1e-2)]
        a.step(g)
        saved = {k: [t if t is None else t.clone() for t in v] if isinstance(v, list) else v
                 for k, v in a.state_dict().items()}
        b = flce.AdamW([p.clone() for p in a.params], lr=1e-2, betas=(0.9, 0.95), state=saved)
        assert b.steps == 1
        a.step(g), b.step(g)
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


# ------------------------------------------------------------ 8-bit moments

def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("seed", [None, 0, 0x123456789ABCDEF])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
def test_8bit_moments_bit_for_bit(grad, seed, offset):
    """The codes and scales follow from fp32 operations that each round by themselves: numpy's give the same bits."""
    sizes = [n for n in SIZES if n < 30000]
    params = [normal(n + offset, k, 0.05)[offset:] for k, n in enumerate(sizes)]
    opt = flce.AdamW(params, lr=1e-2, betas=(0.9, 0.95), moments="8bit", min_8bit_size=0, seed=seed,
                     weight_decay=0.1)
    b1, b2, c1, c2 = (np.float32(x) for x in (0.9, 0.95, 1 - 0.9, 1 - 0.95))
    values = T.e4m3_values().astype(np.float32)
    state = [[np.zeros(n, np.uint8), np.zeros(-(-n // 256), np.float32)] * 2 for n in sizes]
    for step in range(1, 5):
        grads = [normal(n + offset, 50 * step + k, 1e-2, grad)[offset:] for k, n in enumerate(sizes)]
        factor = 0.75
        before = [host(p) for p in params]
        opt.step(grads, grad_scale=factor)
        for i, n in enumerate(sizes):
            mc, ms, vc, vs = state[i]
            g = grads[i].float().cpu().numpy() * np.float32(factor)
            m0 = values[mc] * np.repeat(ms, 256)[:n]
            r0 = values[vc] * np.repeat(vs, 256)[:n]
            m = m0 * b1 + g * c1
            v = (r0 * r0) * b2 + (g * g) * c2
            bits = T.rounding_bits(seed, step, i, n) if seed is not None else None
            root = np.sqrt(v)
            mc, ms = T.encode(m, None if bits is None else bits >> np.uint64(16), False)
            vc, vs = T.encode(root, None if bits is None else bits & np.uint64(0xFFFF), True)
            assert np.array_equal(bytes_of(opt.exp_avg[i]), mc) and np.array_equal(bytes_of(opt.exp_avg_sq[i]), vc)
            assert np.array_equal(opt.exp_avg_scale[i].cpu().numpy(), ms)
            assert np.array_equal(opt.exp_avg_sq_scale[i].cpu().numpy(), vs)
            state[i] = [mc, ms, vc, vs]
            up = 1e-2 / (1 - 0.9 ** step) * m.astype(np.float64) / (root / np.sqrt(1 - 0.95 ** step) + 1e-8)
            want = before[i] * (1 - 1e-3) - up
            assert (np.abs(host(params[i]) - want) <= 2.0 ** -22 * np.abs(before[i]) + 2.0 ** -18 * np.abs(up)).all()


def test_8bit_moments_mixed_with_fp32_ones():
    opt = make([100, 5000, 4095, 4096], moments="8bit")
    assert [t.dtype for t in opt.exp_avg] == [torch.float32, torch.float8_e4m3fn, torch.float32, torch.float8_e4m3fn]
    grads = [normal(t.numel(), k, 1e-2) for k, t in enumerate(opt.params)]
    before = [host(p) for p in opt.params]
    opt.step(grads)
    for p, p0, g in zip(opt.params, before, grads):   # first step: both kinds of moments give lr * sign
        want = p0 * (1 - 1e-4) - 1e-2 * np.sign(host(g)) * (np.abs(host(g)) / (np.abs(host(g)) + 1e-8))
        assert np.abs(host(p) - want).max() < 1e-6


def test_8bit_moments_that_are_not_finite_leave_their_block_alone():
    p = normal(1000, 1)
    opt = flce.AdamW([p], lr=1e-2, moments="8bit", min_8bit_size=0)
    g = normal(1000, 2)
    g[300], g[301] = math.inf, math.nan
    opt.step([g])
    codes = bytes_of(opt.exp_avg[0]), bytes_of(opt.exp_avg_sq[0])
    for c in codes:
        assert c[300] == c[301] == 0x7F and (c[:300] & 0x7F != 0x7F).all() and (c[302:] & 0x7F != 0x7F).all()
    assert torch.isfinite(opt.exp_avg_scale[0]).all() and p.isfinite().sum() == 998


def test_stochastic_rounding_keeps_small_changes():
    """A second moment whose gradients fell tenfold: its mean has to follow, which rounding to nearest cannot do."""
    n, steps = 1 << 16, 300
    held = {}
    for seed in (None, 11):
        p = torch.zeros(n, device="cuda")
        opt = flce.AdamW([p], lr=0.0, betas=(0.9, 0.999), moments="8bit", seed=seed)
        one = torch.ones(n, device="cuda")
        one[::256] = 1000.0            # holds each block's scale
        opt.step([one])
        for _ in range(steps):
            one[1::2] = 3.0
            opt.step([one])
        root = opt.exp_avg_sq[0].float() * opt.exp_avg_sq_scale[0].repeat_interleave(256)
        held[seed] = float((root * root)[1::2].mean())
    v = 0.001
    for _ in range(steps):
        v = 0.999 * v + 0.001 * 9.0
    assert abs(held[11] / v - 1) < 0.02
    assert abs(held[None] / v - 1) > 0.2


def test_large_tensor_past_32_bits():
    """2^32 + 700 elements: places beyond 32 bits in fp8 states, bf16 parameters and gradients."""
    n = (1 << 32) + 700
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    ends = [0, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1]
    for i in ends:
        g[i] = 1.0
    opt = flce.AdamW([p], lr=0.5, weight_decay=0.0, moments="8bit", seed=3)
    out = flce.grad_norm([g], max_norm=1.0)
    assert abs(float(out["norm"]) / math.sqrt(5) - 1) < 1e-6
    opt.step([g])
    assert all(float(p[i]) == -0.5 for i in ends)
    assert int((p != 0).sum()) == 5
    blocks = sorted({i // 256 for i in ends})
    assert torch.nonzero(opt.exp_avg_scale[0]).view(-1).tolist() == blocks


def test_refusals():
    p, q = torch.zeros(10, 10, device="cuda"), torch.zeros(100, device="cuda")
    calls = [
        lambda: flce.AdamW([p.t()[1:]], lr=0.1), lambda: flce.AdamW([p.long()], lr=0.1), lambda: flce.AdamW([p.cpu()], lr=0.1),
        lambda: flce.AdamW([p, p], lr=0.1), lambda: flce.AdamW([q, q[50:]], lr=0.1),
        lambda: flce.AdamW([p], lr=0.1, copies=[q[:99]]), lambda: flce.AdamW([p], lr=0.1, copies=[]),
        lambda: flce.AdamW([p], lr=0.1, copies=[p.view(-1)]), lambda: flce.AdamW([p], lr=0.1, betas=(1.0, 0.9)),
        lambda: flce.AdamW([p], lr=math.nan), lambda: flce.AdamW([p], lr=0.1, eps=-1.0),
        lambda: flce.AdamW([p], lr=0.1, weight_decay=[0.1, 0.2]), lambda: flce.AdamW([p], lr=0.1, moments="4bit"),
        lambda: flce.AdamW([p], lr=0.1, seed=-1), lambda: flce.AdamW([p], lr=0.1, step=-1),
        lambda: flce.AdamW([p], lr=0.1, state=dict(exp_avg=[q], exp_avg_sq=[q[:50]])),
        lambda: flce.AdamW([p], lr=0.1, state=dict(exp_avg=[q], exp_avg_sq=[q.double()])),
        lambda: flce.AdamW([p], lr=0.1, state=dict(exp_avg=[q.to(torch.float8_e4m3fn)], exp_avg_sq=[q.to(torch.float8_e4m3fn)])),
        lambda: flce.AdamW([p], lr=0.1).step([]), lambda: flce.AdamW([p], lr=0.1).step([q[:99]]),
        lambda: flce.AdamW([p], lr=0.1).step([p.t()]), lambda: flce.AdamW([p], lr=0.1).step([p.cpu()]),
        lambda: flce.AdamW([p], lr=0.1).step([p.double()]),
        lambda: flce.AdamW([p], lr=0.1).step([q], grad_scale=torch.ones(2, device="cuda")),
        lambda: flce.AdamW([p], lr=0.1).step([q], lr=torch.ones(1, dtype=torch.float64, device="cuda")),
        lambda: flce.grad_norm([p.t()]), lambda: flce.grad_norm([p.long()]), lambda: flce.grad_norm([p], max_norm=-1.0),
        lambda: flce.grad_norm([p], out=q), lambda: flce.grad_norm([p], grad_scale=math.nan),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(flce.FlceError):
            call()
            pytest.fail(f"call {k} was not refused")
