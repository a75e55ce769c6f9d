"""How a program holds the tensors that it hands to the norm and optimiser calls:
in iterators, and in places that it gives up."""
import threading

import pytest
import torch

import linear_cross_entropy_03_gb300 as flce

pytestmark = pytest.mark.gpu


def normal(n, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------ gradients of an iterator

@pytest.mark.parametrize("count,n", [(1, 1000), (3, 300), (20, 1000), (20, 100000), (300, 4001), (1500, 130)])
def test_norm_of_gradients_that_nobody_else_holds(count, n):
    """The memory of temporaries is theirs until the call's kernels are on the stream."""
    grads = [normal(n, k, dtype=torch.bfloat16) for k in range(count)]
    wide = [g.float() for g in grads]
    want = flce.grad_norm(wide, max_norm=1.0)
    for make in (lambda: (g.float() for g in grads), lambda: map(torch.Tensor.float, grads),
                 lambda: [g.float() for g in grads]):
        for _ in range(10):
            got = flce.grad_norm(make(), max_norm=1.0)
            assert torch.equal(got["norm"], want["norm"]) and torch.equal(got["scale"], want["scale"])


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_step_with_gradients_that_nobody_else_holds(moments):
    sizes = [5000, 3, 70001]
    grads = [normal(n, k, 1e-2, torch.bfloat16) for k, n in enumerate(sizes)]
    params = [[normal(n, 10 + k) for k, n in enumerate(sizes)] for _ in range(2)]
    for p, make in zip(params, (list, iter)):
        opt = flce.AdamW(p, lr=1e-2, moments=moments)
        for _ in range(5):
            opt.step(make([g.float() for g in grads]))
    assert all(torch.equal(a, b) for a, b in zip(*params))
    for wrong in (2, 4):
        with pytest.raises(flce.FlceError):
            opt.step(g for g in (grads * 2)[:wrong])


# ------------------------------------------------------------ parameters that move

def two_alike(moments, **kw):
    """Two optimisers of equal tensors, and their gradients."""
    sizes = [5000, 300]
    made = []
    for _ in range(2):
        params = [normal(n, k, 0.05) for k, n in enumerate(sizes)]
        made.append(flce.AdamW(params, lr=1e-2, moments=moments, copies=[p.bfloat16() for p in params], **kw))
    return made, [normal(n, 50 + k, 1e-2) for k, n in enumerate(sizes)]


def tensors_of(opt):
    lists = (opt.params, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale, opt.copies)
    return [t for ts in lists for t in ts if t is not None]


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(tensors_of(a), tensors_of(b)))


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_step_follows_tensors_that_were_given_other_memory(moments):
    (opt, still), grads = two_alike(moments)
    opt.step(grads), still.step(grads)
    old = [t.detach() for t in tensors_of(opt)]      # aliases: they keep the memory, so that nothing else lies there
    kept = [t.clone() for t in old]
    for t in tensors_of(opt):
        t.data = t.data.clone()
    opt.step(grads), still.step(grads)
    assert equal(opt, still)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(old, kept))


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_step_follows_other_tensors_in_its_lists(moments):
    (opt, still), grads = two_alike(moments)
    opt.step(grads), still.step(grads)
    before = tensors_of(opt)
    kept = [t.clone() for t in before]
    for ts in (opt.params, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale, opt.copies):
        ts[:] = [t if t is None else t.clone() for t in ts]
    opt.step(grads), still.step(grads)
    assert equal(opt, still)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, kept))


def test_step_follows_tensors_that_the_gradients_iterator_moves():
    (opt, still), grads = two_alike("fp32")
    old = [t.detach() for t in tensors_of(opt)]
    kept = [t.clone() for t in old]

    def moves():
        for t in tensors_of(opt):
            t.data = t.data.clone()
        yield from grads

    opt.step(moves()), still.step(grads)
    assert equal(opt, still) and all(torch.equal(a, b) for a, b in zip(old, kept))


def test_step_follows_a_parameter_of_another_type():
    (opt, still), grads = two_alike("fp32")
    first = opt.params[0]
    first.data = first.data.half()
    want = flce.AdamW([first.clone()], lr=1e-2)
    opt.step(grads), still.step(grads), want.step(grads[:1])
    assert first.dtype == torch.float16 and torch.equal(first, want.params[0])
    assert torch.equal(opt.params[1], still.params[1])


def test_step_refuses_what_its_tensors_have_become():
    def longer(o):
        o.params[0].data = torch.zeros(5001, device="cuda")

    def elsewhere(o):
        o.params[0].data = o.params[0].data.cpu()

    def strided(o):
        o.params[0].data = torch.zeros(10000, device="cuda")[::2]

    def another_type(o):
        o.exp_avg[0].data = o.exp_avg[0].data.double()

    def shared(o):
        o.exp_avg[0] = o.exp_avg_sq[0]

    def one_more(o):
        o.params.append(torch.zeros(5, device="cuda"))

    def none(o):
        o.params[0] = None

    for change in (longer, elsewhere, strided, another_type, shared, one_more, none):
        (opt, _), grads = two_alike("fp32")
        change(opt)
        rest = opt.params[1].clone()
        for _ in range(2):                      # the second time too
            with pytest.raises(flce.FlceError):
                opt.step(grads)
        assert opt.steps == 0 and torch.equal(opt.params[1], rest)


def test_captured_step_number_on_another_gpu_is_refused(monkeypatch):
    opt = flce.AdamW([normal(10, 1)], lr=1e-2, capturable=True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(flce.FlceError):
        opt.step([normal(10, 2)])
    monkeypatch.undo()
    assert opt.steps == 0


# ------------------------------------------------------------ calls of several threads

def test_norm_backward_from_several_threads():
    """Calls of one kernel whose launches differ in shared memory do not take it from one another."""
    shapes = [(4000, 4096, True), (152, 4096, False), (400, 4096, True), (300, 4096, False)]
    made = []
    for n, h, residual in shapes:
        x, gy = normal(n * h, n, dtype=torch.bfloat16).view(n, h), normal(n * h, n + 1, dtype=torch.bfloat16).view(n, h)
        rstd = torch.ones(n, device="cuda")
        want = flce.layer_norm_backward(gy, x, rstd=rstd, kind="rms", grad_sum=x if residual else None, grad_bias=False)
        size = flce.ln_workspace_size(n, h)
        out = torch.empty_like(x), torch.empty(h, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
        made.append((n, h, residual, x, gy, rstd, want, out, size, torch.cuda.Stream()))
    torch.cuda.synchronize()
    codes, start = [[] for _ in made], threading.Barrier(len(made))

    def calls(k):
        n, h, residual, x, gy, rstd, _, (gx, gw, work), size, stream = made[k]
        at = [t.data_ptr() for t in (gy, x, rstd, gx, gw, work)]
        start.wait()
        for _ in range(1000):
            codes[k].append(flce.ln_bwd("rms", "bf16", at[0], h, at[1], h, None, "bf16", None, at[2],
                                        at[1] if residual else None, h, n, h, at[3], h, at[4], None, 0, at[5], size,
                                        stream.cuda_stream))

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [sum(c != 0 for c in one) for one in codes] == [0] * len(made) and all(len(c) == 1000 for c in codes)
    for *_, want, (gx, gw, _), _, _ in made:
        assert torch.equal(gx, want["grad_x"]) and torch.equal(gw, want["grad_weight"])


# ------------------------------------------------------------ the smallest eps

@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-38, 1e-40, 1e-46, 1e-300])
@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_a_parameter_without_gradients_stays_with_the_smallest_eps(moments, eps):
    """0 / (0 + eps) is 0 for every eps above 0, those below the normal numbers of fp32 among them."""
    p = normal(1000, 1)
    before, g = p.clone(), normal(1000, 2)
    g[::2] = 0
    opt = flce.AdamW([p], lr=0.25, eps=eps, weight_decay=0.0, moments=moments, min_8bit_size=0)
    opt.step([g])
    assert torch.equal(p[::2], before[::2])
    # the first step is lr * sign(gradient), off by 2^-18 of the update and a rounding of the parameter
    want = before[1::2].double() - 0.25 * g[1::2].sign().double()
    assert ((p[1::2].double() - want).abs() <= 0.25 * 2.0 ** -18 + 2.0 ** -23 * want.abs()).all()


# ------------------------------------------------------------ autograd

@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_autograd_sees_what_a_step_changes(moments):
    (opt, _), grads = two_alike(moments)
    for p in opt.params:
        p.requires_grad_(True)
    versions = [t._version for t in tensors_of(opt)]
    saved = [(p * p).sum() for p in opt.params]              # their backward passes need p as it is
    opt.step([grads[0], None])
    changed = {id(opt.params[0]), id(opt.copies[0])}         # and the moments, which are in no graph
    assert [t._version - v for t, v in zip(tensors_of(opt), versions)] == \
        [int(id(t) in changed) for t in tensors_of(opt)]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved[0].backward()
    saved[1].backward()                                      # this one had no gradient
    assert torch.equal(opt.params[1].grad, 2 * opt.params[1].detach())


def test_autograd_sees_what_a_call_is_given_to_write():
    n, h = 5, 64
    x, r = normal(n * h, 1).view(n, h), normal(n * h, 2).view(n, h)
    y, s, gx = (torch.zeros(n, h, device="cuda") for _ in range(3))
    gw, gb, out = (torch.zeros(k, device="cuda") for k in (h, h, 2))
    given = normal(n * h, 3).view(n, h)
    written, read = (y, s, gx, gw, gb, out), (x, r, given)
    before = [t._version for t in written + read]
    normed = flce.layer_norm(x, residual=r, out=y, sum_out=s)
    flce.layer_norm_backward(given, normed["sum"], mean=normed["mean"], rstd=normed["rstd"], out=gx,
                             grad_weight_out=gw, grad_bias_out=gb)
    flce.grad_norm([gx], out=out)
    assert [t._version - v for t, v in zip(written + read, before)] == [1] * 6 + [0] * 3
    # y in place of x, which a product had saved
    w = torch.ones(h, device="cuda", requires_grad=True)
    loss = (x * w).sum()
    flce.layer_norm(x, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_results_have_no_graph():
    x = normal(320, 1).view(5, 64).requires_grad_(True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    out = flce.layer_norm(x, w)
    assert not out["y"].requires_grad
    back = flce.layer_norm_backward(x, x, w, mean=out["mean"], rstd=out["rstd"])
    assert not any(t.requires_grad for t in back.values())


def test_tensors_of_inference_mode():
    with torch.inference_mode():
        p, g = normal(300, 1), normal(300, 2)
        x = normal(320, 3).view(5, 64)
    opt = flce.AdamW([p], lr=1e-2)
    opt.step([g])
    flce.layer_norm(x, out=x)
    with torch.inference_mode():
        opt.step([g])
        flce.layer_norm(x, out=x)
    assert opt.steps == 2 and p.isfinite().all()
