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
