"""The embedding and its gradient against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_03_gb300 as flce
from losses_util import TYPES, close, cuda, wide
from oracle import losses_oracle as L

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "fp16", "fp32"]
IDS = {"int64": torch.int64, "int32": torch.int32}


def table_of(v, h, dtype, seed, ld=None, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = h if ld is None else ld
    buffer = torch.full((offset + v * ld + 8,), 77.0, dtype=TYPES[dtype], device="cuda")
    t = buffer[offset:offset + v * ld].view(v, ld)[:, :h]
    t.copy_(torch.randn(v, h, generator=gen, device="cuda").to(TYPES[dtype]))
    return t


@pytest.mark.parametrize("n,h,ld,offset", [(1, 4096, 4096, 0), (1, 1, 1, 0), (7, 8, 8, 0), (300, 127, 130, 1), (1000, 64, 64, 0),
                                           (33, 2047, 2048, 0), (2, 16384, 16384, 0), (5, 1024, 1032, 4), (513, 640, 640, 0)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ids", ["int64", "int32"])
def test_lookup(n, h, ld, offset, dtype, ids):
    w = table_of(50, h, dtype, h, ld, offset)
    at = torch.randint(0, 50, (n,), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
    same = flce.embedding(w, at.to(IDS[ids]))["y"]
    assert same.shape == (n, h) and torch.equal(same, w[at])
    scaled = flce.embedding(w, at.to(IDS[ids]), scale=h ** 0.5)["y"]
    factor = float(np.float32(h ** 0.5))
    eps = torch.finfo(TYPES[dtype]).eps / 2
    want = wide(w[at]) * factor
    # the product is rounded to fp32 and then to the type
    close(wide(scaled), want, np.abs(want) * (eps + 2.0 ** -23), "y")
    out = table_of(n, h, dtype, 1, ld + 3, 2)
    got = flce.embedding(w, at.to(IDS[ids]), scale=h ** 0.5, out=out)["y"]
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, scaled)
    assert (out._base[2:2 + n * (ld + 3)].view(n, ld + 3)[:, h:] == 77).all() and (out._base[:2] == 77).all()


def test_lookup_shapes_and_ids_outside():
    w = table_of(20, 96, "bf16", 1)
    ids = torch.tensor([[0, 19, 3], [20, -1, 5]], device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = flce.embedding(w, ids, status=word)["y"]
    assert y.shape == (2, 3, 96) and int(word) == flce.STATUS_BIT_TARGET_RANGE
    assert (y[1, :2] == 0).all() and torch.equal(y[0], w[ids[0]]) and torch.equal(y[1, 2], w[5])
    assert flce.embedding(w, ids[:0])["y"].shape == (0, 3, 96)
    word.zero_()
    flce.embedding(w, ids[0], status=word)
    assert int(word) == 0
    w[3] = float("nan")
    assert flce.embedding(w, ids)["y"][1, :2].eq(0).all()


def ids_like(kind, n, v, seed):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        return rng.integers(0, v, n)
    if kind == "one":
        return np.full(n, v // 2)
    if kind == "half":                              # half of the tokens are padding
        return np.where(rng.random(n) < 0.5, 0, rng.integers(0, v, n))
    if kind == "few":                               # ids that go over many tiles
        return rng.integers(0, min(v, 5), n) * (v // min(v, 5))
    return np.minimum(rng.zipf(1.2, n) - 1, v - 1)


def check_gradient(gy, ids, v, *, id_type="int64", accumulate=False, padding=None, scale=1.0, offset=0):
    h = gy.shape[1]
    start = None
    call = {}
    if accumulate:
        buffer = torch.randn(offset + v * h, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
        call = dict(grad_weight_out=buffer[offset:].view(v, h), accumulate=True)
        start = wide(call["grad_weight_out"])
    got = flce.embedding_backward(gy, cuda(ids).to(IDS[id_type]), v, scale=scale, padding_index=padding, **call)
    factor = float(np.float32(scale))
    want, size = L.embedding_gradient(wide(gy), ids, v, scale=factor, padding_index=padding, start=start)
    # additions: 32 in a tile, those of the tiles of a frequent id over 8 warps, 8 of the warps; a product and a sum more
    chain = 32 + -(-len(ids) // (32 * 8)) + 8 + 2
    close(wide(got["grad_weight"]), want, size * chain * 2.0 ** -24, "grad_weight")
    if accumulate:
        still = np.ones(v, bool)
        still[ids[(ids >= 0) & (ids < v) & (ids != (-1 if padding is None else padding))]] = False
        assert (wide(got["grad_weight"])[still] == start[still]).all()
    return got["grad_weight"]


@pytest.mark.parametrize("kind", ["uniform", "one", "half", "few", "zipf"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 100, 1000, 4096, 4097, 9000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_ids(kind, n, accumulate):
    gy = table_of(n, 24, "fp32", n)
    check_gradient(gy, ids_like(kind, n, 1000, n), 1000, accumulate=accumulate, scale=0.75)


@pytest.mark.parametrize("h", [1, 3, 8, 31, 127, 128, 136, 520, 1000, 1024, 1032, 2047, 4096])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_columns(h, dtype, accumulate):
    gy = table_of(200, h, dtype, h)
    check_gradient(gy, ids_like("half", 200, 70, h), 70, accumulate=accumulate, scale=h ** 0.5)


@pytest.mark.parametrize("v", [1, 2, 31, 33, 511, 512, 513, 32000, 128256, 262143, 262144, 300000])
@pytest.mark.parametrize("id_type", ["int64", "int32"])
def test_gradient_vocabularies(v, id_type):
    gy = table_of(300, 16, "bf16", 1)
    check_gradient(gy, ids_like("uniform", 300, v, v), v, id_type=id_type)
    check_gradient(gy, ids_like("zipf", 300, v, v), v, id_type=id_type, accumulate=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_pitches_and_places(dtype, accumulate):
    for h, ld, offset in ((96, 104, 0), (96, 97, 1), (64, 64, 1), (100, 128, 4)):
        gy = table_of(150, h, dtype, 3, ld, offset)
        check_gradient(gy, ids_like("zipf", 150, 60, 4), 60, accumulate=accumulate, offset=offset)
    one = table_of(1, 64, dtype, 3).expand(40, 64)   # a broadcast row
    check_gradient(one, ids_like("half", 40, 9, 4), 9, accumulate=accumulate)


@pytest.mark.parametrize("n", [50, 5000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_padding_and_ids_outside(n, accumulate):
    gy = table_of(n, 40, "bf16", n)
    ids = ids_like("half", n, 300, n)
    check_gradient(gy, ids, 300, padding=0, accumulate=accumulate)
    ids[1], ids[7], ids[-1] = 300, -3, 1 << 40
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_gradient(gy, ids, 300, accumulate=accumulate)
    flce.embedding_backward(gy, cuda(ids), 300, status=word)
    assert int(word) == flce.STATUS_BIT_TARGET_RANGE
    word.zero_()
    flce.embedding_backward(gy, cuda(ids_like("half", n, 300, n)), 300, padding_index=0, status=word)
    assert int(word) == 0
    nothing = flce.embedding_backward(gy, cuda(np.zeros(n, np.int64)), 300, padding_index=0)["grad_weight"]
    assert (nothing == 0).all()


def test_gradient_of_padding_takes_no_values():
    """What the tokens left out hold does not matter, NaN among it."""
    gy = table_of(100, 40, "fp32", 1)
    ids = ids_like("half", 100, 30, 1)
    gy[ids == 0] = float("nan")
    check_gradient(torch.where(torch.tensor(ids, device="cuda")[:, None] == 0, 0, gy), ids, 30, padding=0)
    assert flce.embedding_backward(gy, cuda(ids), 30, padding_index=0)["grad_weight"].isfinite().all()


def test_gradient_shapes_and_empty_batches():
    gy = table_of(12, 40, "bf16", 1)
    ids = torch.randint(0, 9, (3, 4), device="cuda")
    got = flce.embedding_backward(gy.view(3, 4, 40), ids, 9)["grad_weight"]
    assert torch.equal(got, flce.embedding_backward(gy, ids.view(-1), 9)["grad_weight"])
    empty = flce.embedding_backward(gy[:0], ids.view(-1)[:0], 9)["grad_weight"]
    assert empty.shape == (9, 40) and (empty == 0).all()
    kept = torch.ones(9, 40, device="cuda")
    assert (flce.embedding_backward(gy[:0], ids.view(-1)[:0], grad_weight_out=kept, accumulate=True)["grad_weight"] == 1).all()


def test_gradient_is_the_same_every_time():
    gy = table_of(6000, 256, "bf16", 1)
    ids = cuda(ids_like("zipf", 6000, 400, 1))
    first = flce.embedding_backward(gy, ids, 400)["grad_weight"]
    for _ in range(5):
        assert torch.equal(flce.embedding_backward(gy, ids, 400)["grad_weight"], first)


@pytest.mark.parametrize("value", [0.1, 0.7, 3.14159])
def test_gradient_of_one_id_over_millions_of_tokens(value):
    """The longest chain: 32 tokens of a tile, 64 tiles of a batch, 192 batches of a warp, 8
    warps; each addition rounds by 2^-24 of a sum that is at most the whole."""
    n = 3 * 2 ** 20
    gy = torch.full((n, 4), value, dtype=torch.float32, device="cuda")
    out = flce.embedding_backward(gy, torch.full((n,), 2, device="cuda"), 5)["grad_weight"]
    want = n * float(np.float32(value))
    assert (out[2].double() / want - 1).abs().max() <= (32 + 64 + 192 + 8) * 2.0 ** -24
    assert (out[[0, 1, 3, 4]] == 0).all()


def test_gradient_in_a_dirty_workspace():
    gy = table_of(5000, 64, "bf16", 1)
    size = flce.embedding_workspace_size(5000, 2000, 64)
    work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    for seed in range(3):
        ids = cuda(ids_like("zipf", 5000, 2000, seed))
        got = flce.embedding_backward(gy, ids, 2000, workspace=work)["grad_weight"]
        assert torch.equal(got, flce.embedding_backward(gy, ids, 2000)["grad_weight"])


def test_refusals_of_tensors():
    w, ids = table_of(20, 16, "bf16", 1), torch.zeros(4, dtype=torch.int64, device="cuda")
    gy, grad = table_of(4, 16, "bf16", 2), torch.zeros(20, 16, device="cuda")
    for call in (lambda: flce.embedding(w.double(), ids), lambda: flce.embedding(w, ids.to(torch.int16)),
                 lambda: flce.embedding(w.t(), ids), lambda: flce.embedding(w, ids.expand(3, 4)[:, ::2]),
                 lambda: flce.embedding(w[0], ids), lambda: flce.embedding(w, ids, out=gy.float()),
                 lambda: flce.embedding(w, ids, out=gy[:3]), lambda: flce.embedding(w, ids, out=w[:4]),
                 lambda: flce.embedding(w, ids, status=ids), lambda: flce.embedding(w, ids.cpu()),
                 lambda: flce.embedding_backward(gy, ids), lambda: flce.embedding_backward(gy, ids[:3], 20),
                 lambda: flce.embedding_backward(gy, ids, 20, accumulate=True),
                 lambda: flce.embedding_backward(gy, ids, 21, grad_weight_out=grad),
                 lambda: flce.embedding_backward(gy, ids, grad_weight_out=grad.bfloat16()),
                 lambda: flce.embedding_backward(gy, ids, grad_weight_out=grad[:, :15]),
                 lambda: flce.embedding_backward(gy, ids, 20, padding_index=20),
                 lambda: flce.embedding_backward(gy, ids, 0), lambda: flce.embedding_backward(gy.double(), ids, 20)):
        with pytest.raises(flce.FlceError):
            call()
