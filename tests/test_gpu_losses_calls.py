"""How a program calls the post-training losses and the embedding: in workspaces
that other calls used, on several streams and threads, captured in graphs, with
tensors that autograd knows, beyond 2^31 elements."""
import threading

import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import TYPES, cuda, make_logits, targets

pytestmark = pytest.mark.gpu

# short rows, rows of one CTA, of clusters, with odd places, and rows that are read twice
SHAPES = [(300, 700), (40, 9000), (60, 33001), (30, 128256), (6, 300007)]


def batch(n, v, dtype="bf16", seed=1, k=24):
    """Everything that the three losses and the embedding want for n rows of v logits."""
    rng = np.random.default_rng(seed)
    z = make_logits(n, v, dtype, seed)
    ids = cuda(np.stack([rng.choice(v, k, replace=False) for _ in range(n)]))
    return dict(
        z=z, t=cuda(targets(z, seed)), a=cuda(rng.normal(size=n), torch.float32),
        old=cuda(-rng.random(n) * 8 - 2, torch.float32), ref=cuda(-rng.random(n) * 8 - 2, torch.float32), ids=ids,
        values=cuda(rng.normal(size=(n, k)) * 2, torch.float32),
        offsets=cuda(np.array([0, n // 4, n // 2, n // 2 + 1, n - 1])), gy=make_logits(n, 256, dtype, seed + 1),
        tokens=cuda(rng.integers(0, 90, n)), table=make_logits(90, 256, dtype, seed + 2))


def policy(b, **kw):
    return flce.policy_loss(b["z"], b["t"], b["a"], old_logp=b["old"], ref_logp=b["ref"], kl_weight=0.1, **kw)


def preference(b, **kw):
    return flce.preference_loss(b["z"], b["t"], offsets=b["offsets"], **kw)


def distill(b, **kw):
    return flce.distillation_loss(b["z"], b["ids"], b["values"], temperature=2.0, **kw)


def lookup(b, **kw):
    return flce.embedding(b["table"], b["tokens"], scale=3.0, **kw)


def gradient(b, **kw):
    return flce.embedding_backward(b["gy"], b["tokens"], 90, scale=3.0, **kw)


LOSSES = [policy, preference, distill]
CALLS = LOSSES + [lookup, gradient]


def same(x, y):
    """Bit for bit, NaN included."""
    def bits(t):
        return None if t is None else t.reshape(-1).view(torch.uint8)
    return x.keys() == y.keys() and all(torch.equal(bits(x[k]), bits(y[k])) for k in x)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n,v", SHAPES)
def test_the_same_every_time(call, n, v):
    b = batch(n, v)
    first = call(b)
    for _ in range(4):
        assert same(call(b), first)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_one_dirty_workspace_for_all(reduction):
    """The word that finds the last CTA may hold anything, another call's tag among it."""
    size = max(flce.row_loss_workspace_size(300), flce.preference_workspace_size(300, 2),
               flce.embedding_workspace_size(300, 90, 256))
    for fill in (0, 0xFF, 0x5A):
        work = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for n, v in SHAPES:
            b = batch(n, v, seed=n)
            for call in LOSSES:
                assert same(call(b, workspace=work, reduction=reduction), call(b, reduction=reduction))
            assert same(gradient(b, workspace=work), gradient(b))


@pytest.mark.parametrize("call", CALLS)
def test_on_another_stream(call):
    b = batch(200, 9000)
    want = call(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = call(b, stream=stream)
        side.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("n,v", SHAPES)
def test_beside_kernels_that_hold_sms(n, v):
    """A row's CTAs run at the same time as one cluster whatever else runs; CTAs of other rows need not."""
    b = batch(n, v)
    want = [call(b) for call in CALLS]
    side = torch.cuda.Stream()
    m = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(4):
                m = (m @ m).clamp_(-1, 1)
        got = [call(b) for call in CALLS]
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, want))


def test_from_several_threads():
    shapes = [(300, 700), (40, 9000), (60, 33001), (30, 128256)]
    made = [(batch(n, v, seed=k), torch.cuda.Stream()) for k, (n, v) in enumerate(shapes)]
    want = [[call(b) for call in CALLS] for b, _ in made]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(made))

    def calls(k):
        b, stream = made[k]
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = [call(b) for call in CALLS]
                stream.synchronize()
                if not all(same(x, y) for x, y in zip(got, want[k])):
                    bad.append(k)

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


@pytest.mark.parametrize("n,v", SHAPES)
def test_captured_and_replayed(n, v):
    """Two graphs that share a workspace, replayed in turn, on inputs that change between."""
    size = max(flce.row_loss_workspace_size(n), flce.preference_workspace_size(n, 2),
               flce.embedding_workspace_size(n, 90, 256))
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    b, other = batch(n, v, seed=1), batch(n, v, seed=2)
    wanted = [[call(x) for call in CALLS] for x in (b, other)]
    buffers = {k: t.clone() for k, t in b.items()}

    def step():
        return [call(buffers, workspace=work) for call in LOSSES] + [lookup(buffers), gradient(buffers, workspace=work)]

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step()
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            got.append(step())
    for _ in range(3):
        for which, source in ((0, b), (1, other), (0, other), (1, b)):
            for k, t in source.items():
                buffers[k].copy_(t)
            graphs[which].replay()
            torch.cuda.synchronize()
            want = wanted[0] if source is b else wanted[1]
            skip = {"status"}                    # in the workspace, where the later calls write too
            for x, y in zip(got[which], want):
                for k in x:
                    assert k in skip or torch.equal(x[k].view(-1).view(torch.uint8), y[k].view(-1).view(torch.uint8)), k


def test_captured_beside_an_eager_graph_of_the_same_leaves():
    """The calls record nothing, so that a capture meets no graph that autograd holds."""
    b = batch(50, 9000)
    w = b["z"].float().requires_grad_(True)
    loss = torch.log_softmax(w, 1).sum()         # lives through the capture
    buffers = dict(b, z=w)
    want = [call(buffers) for call in LOSSES]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(buffers) for call in LOSSES]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x["grad_logits"], y["grad_logits"]) for x, y in zip(got, want))
    loss.backward()
    assert not any(x["loss"].requires_grad or x["grad_logits"].requires_grad for x in want)


def test_autograd_sees_what_a_call_writes():
    b = batch(20, 900)
    g, y, gw = torch.zeros_like(b["z"]), torch.zeros(20, 256, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(90, 256, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = [t._version for t in (g, y, gw, word, *b.values())]
    policy(b, grad_out_buffer=g, status=word)
    lookup(b, out=y)
    gradient(b, grad_weight_out=gw)
    after = [t._version for t in (g, y, gw, word, *b.values())]
    assert [x - z for x, z in zip(after, before)] == [1, 1, 1, 1] + [0] * len(b)
    for call in LOSSES:
        w = torch.ones(900, device="cuda", requires_grad=True)
        loss = (b["z"] * w.bfloat16()).sum()
        call(b, in_place=True)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_inference_mode(call):
    with torch.inference_mode():
        b = batch(20, 900)
        inside = call(b)
    assert same(call(b), {k: v for k, v in inside.items()})


@pytest.mark.parametrize("call", LOSSES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_in_place_is_the_same(call, dtype):
    for n, v in SHAPES:
        b = batch(n, v, dtype)
        want = call(b)
        got = call(b, in_place=True)
        assert got["grad_logits"].data_ptr() == b["z"].data_ptr() and same(got, want)


def test_rows_beyond_2_to_the_31_elements():
    """The last rows of 4.4 GB of logits are those of a call with them alone."""
    n, v = 17000, 128256
    z = torch.empty(n, v, dtype=torch.bfloat16, device="cuda")
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    rng = np.random.default_rng(1)
    t, a = cuda(rng.integers(0, v, n)), cuda(rng.normal(size=n), torch.float32)
    ids, values = cuda(rng.integers(0, v, (n, 8))), cuda(rng.normal(size=(n, 8)), torch.float32)
    last = slice(n - 20, n)
    tail = z[last].clone()
    small = [flce.policy_loss(tail, t[last], a[last], reduction="none"),
             flce.distillation_loss(tail, ids[last], values[last], reduction="none"),
             flce.preference_loss(tail.view(2, 10, v), t[last].view(2, 10))]
    g = torch.empty_like(z)
    large = [flce.policy_loss(z, t, a, reduction="none", grad_out_buffer=g)]
    assert torch.equal(large[0]["loss"][last], small[0]["loss"]) and torch.equal(g[last], small[0]["grad_logits"])
    large = flce.distillation_loss(z, ids, values, reduction="none", grad_out_buffer=g)
    assert torch.equal(large["loss"][last], small[1]["loss"]) and torch.equal(g[last], small[1]["grad_logits"])
    offsets = cuda(np.array([n - 20, n - 10, n]))
    large = flce.preference_loss(z, t, offsets=offsets, in_place=True)
    assert torch.equal(large["logp"], small[2]["logp"]) and torch.equal(z[last], small[2]["grad_logits"].view(20, v))
    assert (z[:n - 20:997] == 0).all()


def test_tables_beyond_2_to_the_31_elements():
    v, h = 530000, 4096
    ids = torch.tensor([v - 1, 5, v - 1, v - 2, 524288, 5], device="cuda")
    w = torch.empty(v, h, dtype=torch.bfloat16, device="cuda")
    w[ids] = torch.randn(6, h, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    assert torch.equal(flce.embedding(w, ids)["y"], w[ids])
    del w
    gy = torch.randn(6, h, device="cuda")
    got = flce.embedding_backward(gy, ids, v)["grad_weight"]
    assert torch.equal(got[v - 2], gy[3]) and torch.equal(got[524288], gy[4])
    assert torch.equal(got[v - 1], gy[0] + gy[2]) and torch.equal(got[5], gy[1] + gy[5])
    assert (got[6:v - 2:501] == 0).all()
    many = torch.cat([ids, torch.randint(0, v, (3000,), device="cuda")])    # by sorting
    gy = torch.randn(3006, h, device="cuda")
    flce.embedding_backward(gy, many, grad_weight_out=got)
    want = torch.zeros(h, dtype=torch.float64, device="cuda")
    for i in (many == v - 1).nonzero().flatten().tolist():
        want += gy[i].double()
    assert ((got[v - 1].double() - want).abs() <= 2.0 ** -20).all()         # a few numbers of size 4


def test_refusals_of_tensors():
    b = batch(8, 40)
    z, t, a, ids, values = b["z"], b["t"], b["a"], b["ids"], b["values"]
    o = torch.tensor([0, 4, 8], device="cuda")
    f = torch.zeros(8, device="cuda")
    refused = [
        lambda: flce.policy_loss(z.double(), t, a), lambda: flce.policy_loss(z[0], t, a),
        lambda: flce.policy_loss(z, t.int(), a), lambda: flce.policy_loss(z, t[:7], a),
        lambda: flce.policy_loss(z, t.repeat(2)[::2], a), lambda: flce.policy_loss(z, t, a.double()),
        lambda: flce.policy_loss(z, t, a[:7]), lambda: flce.policy_loss(z, t.cpu(), a),
        lambda: flce.policy_loss(z, t, a, kl_weight=0.1), lambda: flce.policy_loss(z, t, a, clip=-1.0),
        lambda: flce.policy_loss(z, t, a, temperature=0.0), lambda: flce.policy_loss(z, t, a, grad_out=f),
        lambda: flce.policy_loss(z, t, a, reduction="none", grad_out=f[:3]),
        lambda: flce.policy_loss(z, t, a, in_place=True, want_grad=False),
        lambda: flce.policy_loss(z, t, a, in_place=True, grad_out_buffer=z),
        lambda: flce.policy_loss(z, t, a, grad_out_buffer=z.float()),
        lambda: flce.policy_loss(z, t, a, grad_out_buffer=z[:7]), lambda: flce.policy_loss(z.t(), t, a),
        lambda: flce.policy_loss(z, t, a, want_grad=False, grad_out_buffer=torch.empty_like(z)),
        lambda: flce.policy_loss(z, t, a, status=t), lambda: flce.policy_loss(z, t, a, row_weight=f[:1]),
        lambda: flce.policy_loss(z[:1].expand(8, 40), t, a),
        lambda: flce.preference_loss(z, t), lambda: flce.preference_loss(z.view(1, 8, 40), t.view(1, 8)),
        lambda: flce.preference_loss(z, t, offsets=o.int()), lambda: flce.preference_loss(z, t, offsets=o[:2]),
        lambda: flce.preference_loss(z, t, offsets=o, kind="other"),
        lambda: flce.preference_loss(z, t, offsets=o, beta=0.0),
        lambda: flce.preference_loss(z, t, offsets=o, kind="ipo", margin=1.0),
        lambda: flce.preference_loss(z, t, offsets=o, kind="hinge", label_smoothing=0.1),
        lambda: flce.preference_loss(z, t, offsets=o, ref_logp=f),
        lambda: flce.preference_loss(z, t, offsets=o, reduction="none", grad_out=f),
        lambda: flce.distillation_loss(z, ids.short(), values), lambda: flce.distillation_loss(z, ids, values[:, :3]),
        lambda: flce.distillation_loss(z, ids[:7], values[:7]), lambda: flce.distillation_loss(z, ids, values.double()),
        lambda: flce.distillation_loss(z, ids[:, :0], values[:, :0]),
        lambda: flce.distillation_loss(z, ids[:, ::2], values[:, ::2]),
        lambda: flce.distillation_loss(z, ids, values, temperature=-1.0),
        lambda: flce.distillation_loss(z, ids.repeat(1, 50), values.repeat(1, 50)),
    ]
    for k, call in enumerate(refused):
        with pytest.raises(flce.FlceError):
            call()
            pytest.fail(f"call {k} was not refused")


def test_workspaces_that_are_too_small_are_replaced():
    b = batch(300, 700)
    want = policy(b)
    assert same(policy(b, workspace=torch.empty(1000, dtype=torch.uint8, device="cuda")), want)


def test_kernels_are_named():
    b = batch(3000, 700)
    flce.flce_profile_enable(64)
    try:
        policy(b), preference(b), lookup(b), gradient(b)
        torch.cuda.synchronize()
        names = [name for name, _ in flce.flce_profile_read()]
    finally:
        flce.flce_profile_disable()
    assert names == ["row_count", "row_loss", "row_loss", "pair_loss", "row_grad", "embedding", "token_sort",
                     "embedding_bwd", "embedding_join"]
