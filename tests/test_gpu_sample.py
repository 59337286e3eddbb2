"""rfpx_sample (include/rfpx_verify.h) against a plain implementation in 64
bits.

Tolerances.  With n tokens a weight is off by half of 2^-s (s = 50 up to 4096
tokens, one less for each doubling) and by 3e-14 of itself (the series' 7e-15,
the exponent's rounding: |x| <= 64 at 2^-53, and the reference's own); a sum
of up to n of them by e = n 2^-(s+1) + 3e-14 of itself.  The token drawn is
right if u times the whole lies between the sums before and with it, give or
take 2 e (the whole is off by e, the running sum by e); cuts by top_p and min_p
have to be clear of e, which the inputs are, except where weights are equal
whole numbers, where nothing is rounded.  Its probability is off by its own
rounding and the whole's, and by half a step of fp32.
"""
from fractions import Fraction

import numpy as np
import pytest

import block_quantized_expert_amd as bqe

pytestmark = pytest.mark.gpu


def torch():
    import torch as t
    return t


def bits(n):
    return 62 - max(12, (n - 1).bit_length())


class Expected:
    """What a row may give: order, sums and the whole, in 64 bits."""

    def __init__(self, x, t=1.0, k=0, p=1.0, m=0.0):
        x = np.asarray(x, np.float64)
        n = x.size
        real = np.nonzero(x > -np.inf)[0]
        self.empty = real.size == 0
        self.n = n
        if self.empty:
            return
        order = real[np.argsort(-x[real], kind="stable")]
        self.greedy = not t > 0 or k == 1
        if self.greedy:
            order = order[:1]
        top = x[order[0]]
        with np.errstate(invalid="ignore", over="ignore"):
            d = np.where(x[order] == top, 0.0, x[order] - top)
            z = np.where(np.isneginf(d), -np.inf, d / t) if t > 0 else d
        w = np.exp(z)
        if 0 < k < order.size:
            order, w = order[:k], w[:k]
        s = bits(n)
        self.e = lambda whole: n * 2.0 ** -(s + 1) + 3e-14 * whole
        upto = np.cumsum(w)
        if p < 1:
            target = max(p, 0.0) * upto[-1]
            keep = min(int(np.searchsorted(upto, target)) + 1, w.size) if target > 0 else 1
            near = np.abs(upto - target).min()
            self.clear = target == 0 or ((w == 1) | (w == 0)).all() or near > 2 * self.e(upto[-1])
            order, w, upto = order[:keep], w[:keep], upto[:keep]
        else:
            self.clear = True
        if m > 0:
            m = min(m, 1.0)
            self.clear &= bool(((np.abs(w - m) > 2 * self.e(1.0)) | ((w == m) & (w == 1))).all())
            keep = int((w >= m).sum())
            order, w, upto = order[:keep], w[:keep], upto[:keep]
        self.order, self.w, self.upto, self.whole = order, w, upto, upto[-1]
        self.rank = {int(j): i for i, j in enumerate(order)}

    def check(self, token, prob, u):
        if self.empty:
            assert token == -1 and prob == 0
            return
        assert self.clear, "a cut of this input lies within the rounding"
        u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -40)
        assert token in self.rank, f"token {token} is cut"
        i = self.rank[token]
        at, e = u * self.whole, 2 * self.e(self.whole)
        assert self.upto[i] - self.w[i] - e <= at <= self.upto[i] + e, \
            f"u at {at}, token from {self.upto[i] - self.w[i]} to {self.upto[i]}"
        want = self.w[i] / self.whole
        tol = want * (2.0 ** -24 + 6e-14) + (1 + self.n * want) * 2.0 ** -(bits(self.n) + 1) / self.whole + 2.0 ** -149
        assert abs(prob - want) <= tol * (1 + 2.0 ** -20), (prob, want)


def device(v, dtype):
    t = torch()
    return None if v is None else t.tensor(np.asarray(v), device="cuda").to(dtype)


def sample(x, u, t=None, k=None, p=None, m=None, **kw):
    """Tokens and probabilities of logits x (a device tensor)."""
    T = torch()
    rows = x.shape[0]
    probs = T.full((rows,), -7.0, device="cuda")
    tokens = bqe.rfpx_sample(x, device(u, T.float32), device(t, T.float32), device(k, T.int32), device(p, T.float32),
                             device(m, T.float32), probs=probs, **kw)
    return tokens.cpu().tolist(), probs.cpu().tolist()


def f32(v):
    return float(np.float32(v))


def settings(rows, rng):
    """Of every row: a temperature and cuts, none, one or several of them."""
    made = []
    for i in range(rows):
        t = f32(rng.choice([0.3, 0.7, 1.0, 1.0, 1.5, 4.0]))
        k = int(rng.choice([0, 0, -3, 1, 2, 5, 40, 63, 64, 65, 300, 1 << 20]))
        p = f32(rng.choice([1.0, 1.0, 0.99, 0.9, 0.5, 0.1, 0.0, -1.0, 2.0]))
        m = f32(rng.choice([0.0, 0.0, 0.0, 0.01, 0.1, 0.6, 1.0, 3.0, -1.0]))
        if i % 7 == 6:
            t = 0.0
        made.append((t, k, p, m))
    return made


SIZES = [1, 2, 7, 63, 64, 65, 255, 1000, 4097, 32003, 131072, 200001]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", SIZES)
def test_settings(n, dtype):
    T = torch()
    rng = np.random.default_rng(n)
    rows = 21
    x = T.tensor(rng.normal(size=(rows, n)) * rng.choice([0.5, 2.0, 6.0], size=(rows, 1)), device="cuda").to(
        getattr(T, dtype))
    # rows apart, and not on 16 bytes
    wide = T.full((rows, n + 5), 50.0, device="cuda", dtype=x.dtype)
    wide[:, 3:3 + n] = x
    u = rng.random(rows).astype(np.float32)
    s = settings(rows, rng)
    tokens, probs = sample(wide[:, 3:3 + n], u, *zip(*s))
    host = x.double().cpu().numpy()
    for i in range(rows):
        Expected(host[i], *s[i]).check(tokens[i], probs[i], u[i])
    again = sample(x, u, *zip(*s))
    assert again == (tokens, probs)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_no_settings(dtype):
    T = torch()
    rng = np.random.default_rng(3)
    x = T.tensor(rng.normal(size=(9, 5003)) * 2, device="cuda").to(getattr(T, dtype))
    u = rng.random(9).astype(np.float32)
    tokens, probs = sample(x, u)
    for i in range(9):
        Expected(x[i].double().cpu().numpy()).check(tokens[i], probs[i], u[i])
    # one by one, and without probabilities, the same
    alone = [bqe.rfpx_sample(x[i:i + 1], device(u[i:i + 1], T.float32)).item() for i in range(9)]
    assert alone == tokens


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [3, 64, 65, 700, 4096, 4097, 9001, 131072, 1 << 20])
def test_equal_logits(n, dtype):
    """Nothing is rounded here: places are whole numbers.  Rows of many equal
    logits are longer than the list of a row's tokens in question."""
    T = torch()
    x = T.full((10, n), 2.5, device="cuda").to(getattr(T, dtype))
    u = np.array([0, 0.25, 0.5, 0.999, 1 - 2.0 ** -24, 0.3, 0.7, 0.1, 0.6, 1.0], np.float32)
    k = [0, 0, max(2, n // 2), 0, 0, max(2, n // 3), 0, max(2, n - 1), n, 0]
    p = [1, 1, 1, 0.5, 1, 0.75, 0.125, 0.9, 0.25, 0.3]
    tokens, probs = sample(x, u, [1.0] * 10, k, p, [0.5] * 10)
    for i in range(10):
        m = k[i] if 0 < k[i] < n else n
        cut = Fraction(f32(p[i])) * m
        m = max(1, -(-cut.numerator // cut.denominator)) if p[i] < 1 else m
        at = min(Fraction(float(u[i])), Fraction(2 ** 64 - 1, 2 ** 64)) * m
        assert tokens[i] == at.numerator // at.denominator, (i, tokens[i])
        assert probs[i] == f32(1 / m)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [4097, 131072])
def test_two_levels(n, dtype):
    """Half of the row at one logit and half 2^-6 of that weight below, mixed:
    ties by index, many of them, above and below the cut."""
    T = torch()
    rng = np.random.default_rng(n)
    high = rng.random(n) < 0.5
    low = -6 * np.log(2.0)
    x = T.tensor(np.where(high, 0.0, -4.0), device="cuda").to(getattr(T, dtype)).expand(8, n).contiguous()
    t = f32(-4.0 / low)
    u = np.array([0.0, 0.2, 0.9, 0.99, 0.999, 0.5, 0.05, 0.7], np.float32)
    k = [0, 0, 0, 0, 0, int(high.sum()) + 100, 100, int(high.sum())]
    p = [1, 1, 1, 1, 0.995, 1, 1, 1]
    tokens, probs = sample(x, u, [t] * 8, k, p)
    for i in range(8):
        Expected(x[i].double().cpu().numpy(), t, k[i], f32(p[i])).check(tokens[i], probs[i], u[i])


def test_numbers_that_are_no_logits():
    T = torch()
    inf, nan = float("inf"), float("nan")
    n = 300
    base = np.linspace(-3, 3, n)
    rows = {
        "none": np.full(n, -inf), "all nan": np.full(n, nan),
        "one": np.where(np.arange(n) == 17, 1.0, -inf),
        "masked": np.where(np.arange(n) % 3 == 0, base, -inf),
        "nan among": np.where(np.arange(n) % 5 == 0, nan, base),
        "lowest": np.where(np.arange(n) % 2 == 0, -3.3895313892515355e38, base),
        "all lowest": np.full(n, -3.3895313892515355e38),
        "inf": np.where(np.isin(np.arange(n), (5, 250)), inf, base),
        "far apart": np.where(np.arange(n) == 9, 3.3895313892515355e38, -3.3895313892515355e38),
        "zeros": np.where(np.arange(n) % 2 == 0, -0.0, 0.0),
    }
    for dtype in (T.float32, T.bfloat16):
        x = T.tensor(np.stack(list(rows.values())), device="cuda").to(dtype)
        host = x.double().cpu().numpy()
        for t, k, p, m in [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (-1.0, 7, 0.5, 0.0), (1.0, 7, 1.0, 0.0),
                           (1.0, 0, 0.77, 0.0), (1.0, 0, 1.0, 0.123), (1e30, 0, 1.0, 0.0), (2.0 ** -140, 0, 0.9, 0.0)]:
            for u in (0.0, 0.4321, 1 - 2.0 ** -24):
                r = len(rows)
                tokens, probs = sample(x, [u] * r, [t] * r, [k] * r, [f32(p)] * r, [f32(m)] * r)
                for i, name in enumerate(rows):
                    print(name, t, k, p, m, u, tokens[i], probs[i])
                    Expected(host[i], f32(t), k, f32(p), f32(m)).check(tokens[i], probs[i], f32(u))


def test_settings_that_are_no_numbers():
    """NaN: no cut, the first token, u = 0; an infinite temperature: all tokens alike."""
    T = torch()
    nan, inf = float("nan"), float("inf")
    x = T.linspace(3, -3, 500, device="cuda").expand(6, 500).contiguous()
    u = [0.5, nan, -2.0, 7.0, 0.5, 0.25]
    t = [nan, 1.0, 1.0, 1.0, inf, inf]
    k = [0, 0, 0, 3, 0, 100]
    p = [1.0, nan, 1.0, nan, 1.0, 1.0]
    m = [0.0, nan, 0.0, nan, 0.0, 1.0]
    tokens, probs = sample(x, u, t, k, p, m)
    assert tokens == [0, 0, 0, 2, 250, 25]
    assert probs[0] == 1 and probs[4] == f32(1 / 500) and probs[5] == f32(1 / 100)


def test_bins_that_hold_much():
    """All logits within less than one of the row's bins, so that the row itself is
    searched, in both types; and rows where only the far tail is left."""
    T = torch()
    rng = np.random.default_rng(8)
    n = 50000
    for dtype in (T.float32, T.bfloat16):
        x = T.tensor(rng.random((6, n)) * 0.1 + 8, device="cuda").to(dtype)
        u = rng.random(6).astype(np.float32)
        s = [(1.0, 0, 1.0, 0.0), (1.0, 30000, 1.0, 0.0), (1.0, 0, f32(0.3), 0.0), (1.0, 20000, f32(0.9), f32(0.96)),
             (50.0, 70, f32(0.5), 0.0), (1.0, 2, 1.0, 0.0)]
        tokens, probs = sample(x, u, *zip(*s))
        for i in range(6):
            Expected(x[i].double().cpu().numpy(), *s[i]).check(tokens[i], probs[i], u[i])


def bad_rows(n):
    inf, nan = float("inf"), float("nan")
    base = np.linspace(-3, 3, n)
    at = np.arange(n)
    return {
        "none": np.full(n, -inf), "one": np.where(at == n - 2, 1.0, -inf), "last": np.where(at < n - 9000, -inf, base),
        "masked": np.where(at % 3 == 0, base, -inf), "nan among": np.where(at % 5 == 0, nan, base),
        "lowest": np.where(at % 2 == 0, -3.3895313892515355e38, base), "all lowest": np.full(n, -3.3895313892515355e38),
        "inf": np.where(np.isin(at, (5, n - 7)), inf, base),
        "far apart": np.where(at == 9, 3.3895313892515355e38, -3.3895313892515355e38),
        "large": base * 1e30, "large and equal": np.where(at % 4 == 0, 2.0 ** 100, base),
    }


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [40000, 131073])
def test_numbers_that_are_no_logits_in_long_rows(n, dtype):
    """As above, where rows are cut into slices, some of them without tokens."""
    T = torch()
    rows = bad_rows(n)
    x = T.tensor(np.stack(list(rows.values())), device="cuda").to(getattr(T, dtype))
    host = x.double().cpu().numpy()
    r = len(rows)
    for t, k, p, m in [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 7, 1.0, 0.0), (1.0, 0, 0.77, 0.0),
                       (1.0, 0, 1.0, 0.123), (1.0, 300, 0.5, 0.9), (1e30, 0, 1.0, 0.0), (2.0 ** -140, 0, 0.9, 0.0)]:
        u = 0.4321
        tokens, probs = sample(x, [u] * r, [t] * r, [k] * r, [f32(p)] * r, [f32(m)] * r)
        for i, name in enumerate(rows):
            print(name, t, k, p, m, tokens[i], probs[i])
            Expected(host[i], f32(t), k, f32(p), f32(m)).check(tokens[i], probs[i], f32(u))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_slices_that_list_too_much(dtype):
    """Long rows whose first few, or tokens of some weight, are more than a
    slice lists: in every slice, in one, and beside slices without any."""
    T = torch()
    rng = np.random.default_rng(31)
    n = 131072
    flat = np.full(n, 1.5)
    one = rng.normal(size=n)
    one[20000:24000] = 6.0
    rare = np.full(n, -np.inf)
    rare[50000:53000] = 2.0
    rare[90000:90010] = np.linspace(1, 3, 10)
    near = 8 + rng.random(n) * 0.5
    rows = [flat, one, rare, near] * 6
    s = [(1.0, 50, 1.0, 0.0), (1.0, 250, f32(0.5), 0.0), (1.0, 0, 1.0, f32(0.01)), (1.0, 0, f32(0.9), f32(0.3)),
         (0.7, 3000, f32(0.8), f32(0.2)), (2.0, 200, f32(0.99), f32(0.6))]
    s = [x for x in s for _ in range(4)]
    x = T.tensor(np.stack(rows), device="cuda").to(getattr(T, dtype))
    u = rng.random(24).astype(np.float32)
    tokens, probs = sample(x, u, *zip(*s))
    for i in range(24):
        Expected(x[i].double().cpu().numpy(), *s[i]).check(tokens[i], probs[i], u[i])


@pytest.mark.parametrize("dtype,n,rows", [("float32", 33000, 1100), ("bfloat16", 40001, 530), ("float32", 1 << 20, 3),
                                          ("bfloat16", (1 << 20) - 7, 3)])
def test_more_rows_than_are_done_at_once(dtype, n, rows):
    T = torch()
    g = T.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(rows)
    x = (T.randn((rows, n), generator=g, device="cuda") * 2).to(getattr(T, dtype))
    u = rng.random(rows).astype(np.float32)
    s = settings(rows, rng)
    tokens, probs = sample(x, u, *zip(*s))
    for i in [*range(0, rows, 97), rows - 1, *range(min(rows, 511), min(rows, 514))]:
        Expected(x[i].double().cpu().numpy(), *s[i]).check(tokens[i], probs[i], u[i])


def test_many_rows_draw_as_they_weigh():
    """4000 equally spaced numbers draw every token as often as it weighs, within one."""
    T = torch()
    n, rows = 40, 4000
    x = T.linspace(0, 4, n, device="cuda").expand(rows, n).contiguous()
    u = (np.arange(rows) + 0.5) / rows
    tokens, _ = sample(x, u.astype(np.float32))
    w = np.exp(np.linspace(0, 4, n))
    w /= w.sum()
    assert np.abs(np.bincount(tokens, minlength=n) - rows * w).max() <= 2


def test_captured_on_streams_and_two_at_once():
    """A captured call on other logits, settings and numbers, replayed between
    eager work; and calls on two streams with workspaces of their own."""
    T = torch()
    rows, n = 5, 131072
    g = T.Generator(device="cuda").manual_seed(4)
    x = T.zeros((rows, n), device="cuda")
    u, temp, p = T.zeros(rows, device="cuda"), T.ones(rows, device="cuda"), T.ones(rows, device="cuda")
    k = T.zeros(rows, dtype=T.int32, device="cuda")
    tokens, probs = T.zeros(rows, dtype=T.int32, device="cuda"), T.zeros(rows, device="cuda")
    ws = T.empty(bqe.rfpx_sample_workspace_bytes(rows, n, x.dtype), dtype=T.uint8, device="cuda")

    def step():
        bqe.rfpx_sample(x, u, temp, k, p, tokens=tokens, probs=probs, ws=ws)

    side = T.cuda.Stream()
    side.wait_stream(T.cuda.current_stream())
    with T.cuda.stream(side):
        step()
    T.cuda.current_stream().wait_stream(side)
    graph = T.cuda.CUDAGraph()
    with T.cuda.graph(graph):
        step()
    for i in range(6):
        x.copy_(T.randn((rows, n), generator=g, device="cuda") * 3)
        u.copy_(T.rand(rows, generator=g, device="cuda"))
        k.fill_(50 * i)
        p.fill_(1 - 0.1 * i)
        ws.random_(0, 256, generator=g)
        tokens.fill_(-5)
        graph.replay()
        T.cuda.synchronize()
        probs2 = T.zeros_like(probs)
        want = bqe.rfpx_sample(x, u, temp, k, p, probs=probs2)
        assert T.equal(tokens, want) and T.equal(probs, probs2)
        _ = (x @ x.T).sum().item()
    a, b = T.cuda.Stream(), T.cuda.Stream()
    y = x.flip(0).contiguous()
    want_x, want_y = bqe.rfpx_sample(x, u), bqe.rfpx_sample(y, u)
    for s in (a, b):
        s.wait_stream(T.cuda.current_stream())
    for _ in range(5):
        got_x, got_y = bqe.rfpx_sample(x, u, stream=a), bqe.rfpx_sample(y, u, stream=b)
    T.cuda.synchronize()
    assert T.equal(got_x, want_x) and T.equal(got_y, want_y)


def test_wrapper_refusals():
    T = torch()
    x, u = T.zeros((2, 8), device="cuda"), T.zeros(2, device="cuda")
    for bad in (dict(logits=x[0]), dict(logits=x.T), dict(logits=x.half()), dict(logits=x.cpu()), dict(u=u.double()),
                dict(u=u[:1]), dict(top_k=u), dict(temperature=T.zeros(3, device="cuda")), dict(tokens=u),
                dict(probs=u.double())):
        kw = dict(dict(logits=x, u=u), **bad)
        with pytest.raises(ValueError):
            bqe.rfpx_sample(kw.pop("logits"), kw.pop("u"), **kw)
    for bad in (dict(logits=x[:1].expand(2, 8)), dict(ws=T.empty(16, dtype=T.uint8, device="cuda"))):
        kw = dict(dict(logits=x, u=u), **bad)
        with pytest.raises(bqe.RfpxError):
            bqe.rfpx_sample(kw.pop("logits"), kw.pop("u"), **kw)
    assert bqe.rfpx_sample(x[:0], u[:0]).shape == (0,)


@pytest.mark.parametrize("seed", [1, 2])
def test_many_long_rows_again_and_again(seed):
    """As many rows as fill the chip several times over, in one call: every
    row has the token and the probability that it has in a call of its own, run
    after run (sums of many workgroups that share compute units)."""
    T = torch()
    g = T.Generator("cuda").manual_seed(seed)
    rows, n = 512, 65536
    x = T.randn((rows, n), generator=g, device="cuda") * 2.2
    u = T.rand(rows, generator=g, device="cuda")
    p = T.where(T.arange(rows, device="cuda") % 2 == 0, 1.0, 0.9).float()
    one_probs = T.empty(rows, device="cuda")
    one = T.cat([bqe.rfpx_sample(x[r:r + 1], u[r:r + 1], top_p=p[r:r + 1], probs=one_probs[r:r + 1])
                 for r in range(rows)])
    for _ in range(8):
        probs = T.empty(rows, device="cuda")
        tokens = bqe.rfpx_sample(x, u, top_p=p, probs=probs)
        assert T.equal(tokens, one) and T.equal(probs, one_probs)
    for r in range(0, rows, 37):
        e = Expected(x[r].cpu().numpy(), p=float(p[r]))
        assert e.clear
        e.check(int(one[r]), float(one_probs[r]), float(u[r]))
