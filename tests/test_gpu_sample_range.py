"""rfpx_sample at the ends of what its settings and logits may be, with the
expectations and tolerances of test_gpu_sample.py: a weight is off by half of
2^-s and 3e-14 of itself whatever the temperature, since a weight goes by the
difference of two logits (exact in 64 bits) and not by their size."""
import numpy as np
import pytest

from test_gpu_sample import Expected, f32, sample, torch

pytestmark = pytest.mark.gpu

# largest logit over temperature from 10^7 to 10^12: there adjacent fp32 numbers
# are from 1 to 10^5 weights of e apart, and products of them are rounded by bins
COLD = [1e-6, 3e-7, 1e-7, 3e-8, 1e-8, 1e-9, 5e-10, 1e-10, 2e-11]


def below(x, steps):
    """The fp32 number so many steps below."""
    x = np.float32(x)
    for _ in range(steps):
        x = np.nextafter(x, np.float32(-np.inf))
    return x


def cold_rows(n, rows, rng):
    """Rows whose largest logits are neighbours: the largest, the next ones
    below it, some of them twice, and others by far below."""
    x = (rng.normal(size=(rows, n)) - 20).astype(np.float32)
    for i in range(rows):
        top = np.float32(rng.uniform(2, 20) * (1 if i % 2 else -0.5))
        x[i] -= 20
        at = rng.permutation(n)[:8]
        x[i, at] = [below(top, k) for k in (0, 1, 1, 2, 3, 4, 4, 9)]
    return x


@pytest.mark.parametrize("n", [500, 32000, 70000])
@pytest.mark.parametrize("t", COLD)
def test_neighbours_at_low_temperatures(t, n):
    T = torch()
    rng = np.random.default_rng(n + int(-1000 * np.log10(t)))
    rows = 16
    host = cold_rows(n, rows, rng)
    x = T.tensor(host, device="cuda")
    for k, p, m in ((0, 1.0, 0.0), (5, 1.0, 0.0), (400, 1.0, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.35)):
        u = rng.random(rows).astype(np.float32)
        tokens, probs = sample(x, u, [t] * rows, [k] * rows, [f32(p)] * rows, [f32(m)] * rows)
        for i in range(rows):
            e = Expected(host[i].astype(np.float64), f32(t), k, f32(p), f32(m))
            e.check(tokens[i], probs[i], u[i])


@pytest.mark.parametrize("n", [1000, 30000, 131072])
@pytest.mark.parametrize("large", [6.0, -6.0, 2.0 ** 28, -(2.0 ** 27)])
def test_many_neighbours_of_one_logit(large, n):
    """One largest logit and the whole row one step of fp32 below: each of them
    weighs next to nothing, all of them together enough to be drawn."""
    T = torch()
    step = float(np.float32(large)) - float(below(large, 1))
    host = np.full((6, n), below(large, 1), np.float32)
    top = [0, n // 2, n - 1, n // 3, 7, 1]
    host[np.arange(6), top] = np.float32(large)
    u = np.array([0.0, 0.5, 1 - 2.0 ** -20, 0.999, 1 - 2.0 ** -14, 1 - 2.0 ** -24], np.float32)
    x = T.tensor(host, device="cuda")
    for octaves in (3, 12, 18, 22):
        t = f32(step / (octaves * np.log(2)))
        tokens, probs = sample(x, u, [t] * 6)
        for i in range(6):
            e = Expected(host[i].astype(np.float64), t)
            e.check(tokens[i], probs[i], u[i])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [300, 5000, 30000, 70001])
def test_infinite_temperature(n, dtype):
    """All tokens weigh the same and min_p, of 1 and more too, cuts none of them:
    the place drawn is a whole number.  Logits of any size, and tokens at -inf."""
    T = torch()
    rng = np.random.default_rng(n)
    inf = float("inf")
    base = rng.normal(size=n) * 3
    some = np.where(rng.random(n) < 0.3, -inf, base)
    x = T.tensor(np.stack([base, some, base * 1e38 / 12]), device="cuda").to(getattr(T, dtype))
    host = x.double().cpu().numpy()
    u = np.array([0.0, 0.375, 0.9990234375], np.float32)
    for m in (1.0, 3.0, inf, 0.5, 1e-30):
        for k, p in ((0, 1.0), (0, 0.5), (400, 1.0), (100, 1.0), (400, 0.5)):
            tokens, probs = sample(x, u, [inf] * 3, [k] * 3, [p] * 3, [m] * 3)
            for i in range(3):
                order = np.argsort(-host[i], kind="stable")[:int((host[i] > -inf).sum())]
                order = order[:k] if 0 < k < order.size else order
                stays = order.size if p == 1 else -(-order.size // 2)
                assert tokens[i] == order[int(float(u[i]) * stays)], (m, k, p, i)
                assert probs[i] == f32(1 / stays), (m, k, p, i)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [300, 30000, 70001])
def test_min_p_at_temperatures_of_any_size(n, dtype):
    """min_p alone, and with cuts besides, from where the largest logit alone
    weighs anything to where all weigh the same."""
    T = torch()
    rng = np.random.default_rng(n + 1)
    x = T.tensor(rng.normal(size=(4, n)) * 3, device="cuda").to(getattr(T, dtype))
    host = x.double().cpu().numpy()
    u = rng.random(4).astype(np.float32)
    for t in (1e-30, 1e-12, 1e-4, 0.05, 1e4, 1e30, 3e38):
        for m in (1.0, 2.0, 0.30000001):
            for k, p in ((0, 1.0), (400, 1.0), (0, 0.625)):
                tokens, probs = sample(x, u, [t] * 4, [k] * 4, [p] * 4, [m] * 4)
                for i in range(4):
                    Expected(host[i], f32(t), k, f32(p), f32(m)).check(tokens[i], probs[i], u[i])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [600, 40000])
def test_the_lowest_temperatures(n, dtype):
    """Logits as small as a temperature of 2^-100 count as any; below, only the
    largest weighs anything."""
    T = torch()
    rng = np.random.default_rng(n + 2)
    x = T.tensor(-rng.random((4, n)) * 8, device="cuda").to(getattr(T, dtype)) * 2.0 ** -100
    x[:, 5] = 0.0
    x[:2, 9] = 0.0
    host = x.double().cpu().numpy()
    u = np.array([0.3, 0.9, 0.3, 0.9], np.float32)
    for t in (2.0 ** -99, 1.2 * 2.0 ** -100, 2.0 ** -100):
        for k, p in ((0, 1.0), (3, 1.0), (0, 0.6)):
            tokens, probs = sample(x, u, [t] * 4, [k] * 4, [f32(p)] * 4)
            for i in range(4):
                Expected(host[i], f32(t), k, f32(p)).check(tokens[i], probs[i], u[i])
    for t in (f32(0.99 * 2.0 ** -100), 2.0 ** -130, 2.0 ** -149):
        tokens, probs = sample(x, u, [t] * 4)
        assert tokens == [5, 9, 5, 5] and probs == [0.5, 0.5, 1.0, 1.0]
