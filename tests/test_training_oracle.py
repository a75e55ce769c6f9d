"""The 64-bit definitions the norm and optimiser tests compare with, checked on
their own: gradients against central differences, closed forms, and the 8-bit
format against its table."""
import numpy as np
import pytest
import torch

from oracle import training_oracle as T


def _rows(n, h, seed):
    rng = np.random.default_rng(seed)
    return rng.normal(size=(n, h)) + 0.3, 1 + 0.2 * rng.normal(size=h), 0.1 * rng.normal(size=h), rng


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("n,h", [(1, 2), (3, 7), (5, 16)])
def test_norm_gradients_are_the_differences(n, h, rms):
    s, w, b, rng = _rows(n, h, 10 * n + h)
    gy, gs = rng.normal(size=(n, h)), rng.normal(size=(n, h))

    def objective(s, w, b):
        return (T.norm_forward(s, w, b, 1e-3, rms)[0] * gy).sum() + (s * gs).sum()

    _, mean, rstd = T.norm_forward(s, w, b, 1e-3, rms)
    grads = T.norm_backward(gy, s, w, mean, rstd, gs, rms)
    step = 1e-5
    for k, (x, got) in enumerate(zip((s, w, b), grads)):
        for i in np.ndindex(x.shape):
            args = [s, w, b]
            args[k] = x.copy()
            args[k][i] += step
            up = objective(*args)
            args[k][i] -= 2 * step
            # central differences: error of the order step^2 plus rounding 1e-16 / step
            assert abs((up - objective(*args)) / (2 * step) - got[i]) < 1e-7 * (1 + abs(got[i]))


def test_norm_closed_forms():
    s, w, b, _ = _rows(4, 33, 1)
    y, mean, rstd = T.norm_forward(s, None, None, 0.0, False)
    assert np.allclose(y.mean(1), 0, atol=1e-14) and np.allclose((y * y).mean(1), 1)
    y2, _, _ = T.norm_forward(3 * s + 5, None, None, 0.0, False)
    assert np.allclose(y, y2)
    y3, m3, r3 = T.norm_forward(s, None, None, 0.0, True)
    assert np.allclose((y3 * y3).mean(1), 1) and (m3 == 0).all()
    # moving along s itself does not change y, so grad_s is at right angles to s (rms) and to 1 (layer)
    g, _, _ = T.norm_backward(w * s, s, w, m3, r3, None, True)
    assert np.allclose((g * s).sum(1), 0, atol=1e-10)
    g, _, _ = T.norm_backward(w * s, s, w, mean, rstd, None, False)
    assert np.allclose(g.sum(1), 0, atol=1e-10)


def test_adamw_matches_torch_in_64_bits():
    rng = np.random.default_rng(3)
    p = torch.tensor(rng.normal(size=17), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(17), np.zeros(17)
    for t in range(1, 6):
        g = rng.normal(size=17)
        p.grad = torch.from_numpy(g)
        opt.step()
        q, m, v = T.adamw(q, g, m, v, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, decay=0.1, step=t)
        assert np.allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_e4m3_table_and_rounding():
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(values, T.e4m3_values().astype(np.float32), equal_nan=True)
    rng = np.random.default_rng(4)
    x = (rng.normal(size=1000) * np.exp(4 * rng.normal(size=1000))).astype(np.float32)
    code, scale = T.encode(x, None, False)
    inverse = np.float32(1) / scale
    y = (x * np.repeat(inverse, 256)[:1000]).astype(np.float32)
    want = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(code, want)


def test_stochastic_rounding_is_unbiased_and_in_between():
    x = np.abs(np.random.default_rng(5).normal(size=256)).astype(np.float32) ** 4
    total = np.zeros(256)
    reps = 2000
    y = None
    for t in range(reps):
        code, scale = T.encode(x, T.rounding_bits(77, t, 0, 256) >> np.uint64(16), False)
        y = (x * (np.float32(1) / scale[0])).astype(np.float64)
        got = T.e4m3_values()[code]
        assert (np.abs(got - y) <= T.e4m3_spacing(y) * (1 + 1e-6)).all()
        total += got
    # the mean of `reps` roundings: a standard error of at most spacing / 2 / sqrt(reps) each; 256 of them within 5
    assert (np.abs(total / reps - y) <= 5 * T.e4m3_spacing(y) / 2 / np.sqrt(reps)).all()


def test_encode_edges():
    x = np.zeros(600, np.float32)
    x[1], x[2], x[3], x[300], x[301] = np.inf, np.nan, 1.0, 1e-3, 1e-12
    code, scale = T.encode(x, None, True)
    assert code[1] == code[2] == 0x7F and code[3] == 0x7E and code[0] == 0
    assert code[301] == 1 and code[300] == 0x7E      # above 0, held as the smallest number
    assert scale[0] == np.float32(1 / 448) and scale[2] == 0
