"""Attention over the FP4 cache (include/rfpx_attn.h) at the edges of what a
caller may hand in, with the rows and tolerances of test_gpu_attn.py.

Where scores are so large that only the best token of a row has any weight,
the row is that token's values: the numerators of the others are 0, its own and
the sum of them are the same number (or, in k_attn_chunk, that number rounded to
bf16 and itself), so that the output is off by at most 2 u(bf16) of the value (4
u32 in fp32), by the offset's removal (256 u32 of 31 units, as everywhere) and
by its own type's rounding.
"""
import numpy as np
import pytest

import block_quantized_expert_amd as bqe
from test_gpu_attn import U32, UBF, Case, attend64, check_lse, check_out, dt, f64, torch, units

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- large scores

@pytest.mark.parametrize("d,scale", [(64, 0.125), (128, 1.0), (128, 128 ** -0.5)])
@pytest.mark.parametrize("low", [2.0 ** 30, 2.0 ** 40, 2.0 ** 90])
def test_many_rows_end_at_any_score(d, scale, low):
    """Scores of 2^30 and more, where the room that k_attn_chunk leaves above a
    row's maximum is lost to rounding: every tile is done with, and the rows of
    ordinary scores in the same waves are right."""
    t = torch()
    # 64 splits with a tile or none in each, and one split of several tiles
    for hk, heads, plan in ((2, 16, 65536), (128, 256, 1024)):
        c = Case([300], [40], hk, d, 64, t.bfloat16, seed=d, capacity=plan)
        g = t.Generator(device="cuda").manual_seed(int(100 * scale))
        q = t.randn((c.rows, heads, d), generator=g, device="cuda") * 1.3
        q[:, 1::2] *= low * (1 + t.rand((c.rows, heads // 2, 1), generator=g, device="cuda"))
        q = q.to(t.bfloat16)
        z = t.zeros((c.rows, heads), device="cuda")
        out = bqe.rfpx_attn_forward(c.cache, c.planned(plan), q, scale, lse=z)
        heads_seen = 16  # of the first kv heads: the plain form takes its time
        (k, v), = c.values()
        c.hk = heads_seen * hk // heads
        c.values = lambda: [(k[:, :c.hk], v[:, :c.hk])]
        ref = attend64(c, q[:, :heads_seen], scale)
        even = {n: x[:, 0:heads_seen:2] for n, x in ref.items() if n not in ("w", "dw")}
        check_out(out[:, 0:heads_seen:2], even, t.bfloat16, slice(0, c.rows))
        check_lse(z[:, 0:heads_seen:2], even, slice(0, c.rows))


def peaked(n, hk, d, page, dtype, cols, capacity, seed):
    """A sequence of n slots whose keys lie along one pattern a head, between
    one and two of it, but for one four times as long and one a quarter: for a
    query along the pattern the long one is best by far, for one against it the
    short one.  Neither stands in the first tiles, so that the running maximum
    moves."""
    t = torch()
    c = Case([n], [cols], hk, d, page, dtype, seed=seed, capacity=capacity)
    g = t.Generator(device="cuda").manual_seed(seed + 1)
    signs = t.randint(0, 2, (1, hk, d), generator=g, device="cuda") * 2.0 - 1
    size = 1 + t.rand((n, hk, 1), generator=g, device="cuda")
    size[n // 2], size[n // 2 + 7] = 8.0, 0.25
    k = (signs * size).to(dtype)
    bqe.rfpx_kv_append(c.cache, c.fill, k, c.v_in)
    return c, signs


def check_peaked(c, signs, heads, dtype, low, high, scale, batch, seed):
    """Rows whose best score is 2^low .. 2^high in size (as powers of two that
    the softmax takes), of either sign."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    rows, group = c.rows, heads // c.hk
    (k, v), = c.values()
    # the best score of a query of ones is 8 d, or 0.25 d against the pattern
    sign = t.randint(0, 2, (rows, heads, 1), generator=g, device="cuda") * 2.0 - 1
    best = c.d * t.where(sign > 0, 8.0, 0.25) * scale * 1.4426950408889634
    want = 2.0 ** (low + (high - low) * t.rand((rows, heads, 1), generator=g, device="cuda", dtype=t.float64))
    spread = 0.9 + 0.2 * t.rand((rows, heads, c.d), generator=g, device="cuda")
    q = (signs.repeat_interleave(group, 1) * sign * spread * (want / best)).to(dtype)
    out, z = t.full_like(q, 7.0), t.full((rows, heads), 7.0, device="cuda")
    bqe.rfpx_attn_forward(c.cache, batch, q, scale, out=out, lse=z)
    o, z, bf = f64(out), f64(z), dtype == t.bfloat16
    kk = t.from_numpy(k).cuda()
    q64 = q.double().view(rows, c.hk, group, c.d)
    s = t.stack([(q64[:, h].reshape(rows * group, c.d) @ kk[:, h].T).view(rows, group, -1) for h in range(c.hk)], 1)
    s = s.reshape(rows, heads, -1) * scale
    seen = len(k) - rows + t.arange(rows, device="cuda").view(-1, 1, 1)
    s = s.masked_fill(t.arange(len(k), device="cuda") > seen, -float("inf"))
    (top, second), (at, _) = (x.unbind(-1) for x in s.topk(2, -1))
    # the best token leads by a tenth of its score, which is beyond any rounding of it
    assert bool((top - second > 0.1 * top.abs()).all()) and bool((top.abs() * 1.44 > 2.0 ** (low - 1)).all())
    top, at = top.cpu().numpy(), at.cpu().numpy()
    head = np.arange(heads)[None] // group
    vv, uu = v[at, head], units(v)[at, head]
    tol = (3 * UBF if bf else 5 * U32) * np.abs(vv) + 256 * U32 * 31 * uu
    err = np.abs(o - vv)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} values off, worst {np.nanmax(err / tol):.3g}"
    # lse is the best score: the products' roundings, and the offset's (beyond
    # fp32 an infinity)
    big = scale * np.abs(f64(q)).sum(-1) * 31 * units(k).max()
    with np.errstate(invalid="ignore"):
        near = np.abs(z - top) <= 256 * U32 * big + 2.0 ** -21 * np.abs(top)
    assert (near | (np.isinf(z) & (np.abs(top) > 2.0 ** 127) & (np.sign(z) == np.sign(top)))).all()


# 16 rows and 32, one workgroup of eight waves, four waves with both joins, heads
# of 256; and the path of many rows in 64 splits and whole
PATHS = [(2, 8, 128, 1, 0), (2, 16, 64, 3, 0), (2, 16, 128, 3, 0), (2, 8, 128, 1, 1500), (2, 8, 64, 5, 4096),
         (2, 8, 256, 2, 700), (2, 16, 64, 10, 65536), (2, 16, 128, 10, 65536), (128, 128, 128, 80, 1024)]


@pytest.mark.parametrize("low,high,scale", [
    (20, 20.6, 0.125), (23.5, 24.5, 1.0), (30, 30.6, 0.125), (30, 30.6, 128 ** -0.5), (33, 33.6, 1.0), (60, 60.6, 0.125),
    (100, 100.6, 1.0), (131, 131.6, 1e29)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,heads,d,cols,plan", PATHS)
def test_scores_of_any_size(hk, heads, d, cols, plan, dtype, low, high, scale):
    c, signs = peaked(700, hk, d, 64, dt(dtype), cols, max(plan, 700), seed=d)
    check_peaked(c, signs, heads, dt(dtype), low, high, scale, c.planned(plan), seed=int(100 * low))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,heads,d,cols,plan", PATHS[1:6] + [(2, 8, 64, 20, 65536), (128, 128, 128, 66, 1024)])
def test_large_values_under_rising_scores(hk, heads, d, cols, plan, dtype):
    """Values of 2^85 while a row's scores rise by 25 powers of two a tile of 64
    tokens: numerators and sums stay in fp32's range, and so does the output."""
    t = torch()
    n = 400
    c = Case([n], [cols], hk, d, 64, dt(dtype), seed=d, capacity=max(plan, n))
    g = t.Generator(device="cuda").manual_seed(3)
    signs = t.randint(0, 2, (1, hk, d), generator=g, device="cuda") * 2.0 - 1
    k = signs * (1 + 6 * t.arange(n, device="cuda").view(n, 1, 1) / n)
    bqe.rfpx_kv_append(c.cache, c.fill, k.to(dt(dtype)), (c.v_in.float() * 2.0 ** 85).to(dt(dtype)))
    # a score of size s is s * 25.6 powers of two: 25.6 * 6 * 64 / 400 a tile
    q = signs.repeat_interleave(heads // hk, 1) * t.ones((c.rows, heads, d), device="cuda") * (25.6 / 1.4427 / d)
    q = q.to(dt(dtype))
    z = t.zeros((c.rows, heads), device="cuda")
    out = bqe.rfpx_attn_forward(c.cache, c.planned(plan), q, 1.0, lse=z)
    (kk, vv), = c.values()
    few = min(hk, 4)  # heads: the plain form takes its time
    h = few * heads // hk
    c.hk, c.values = few, lambda: [(kk[:, :few], vv[:, :few])]
    ref = attend64(c, q[:, :h], 1.0)
    check_out(out[:, :h], ref, dt(dtype), slice(0, c.rows))
    check_lse(z[:, :h], ref, slice(0, c.rows))
    assert bool(t.isfinite(out).all())


# ------------------------------------------------------------------ streams

def test_side_stream_while_the_current_one_is_busy():
    """Calls on a side stream while the current one still has writes queued to
    blocks of memory that have gone back to the allocator: the calls' outputs
    and workspaces are other memory."""
    t = torch()
    c = Case([3000, 700], [3, 2], 2, 128, 64, t.bfloat16)
    q = t.randn((5, 8, 128), device="cuda").to(t.bfloat16)
    pos = t.arange(5, dtype=t.int32, device="cuda")
    rope = bqe.Rope(128)
    x = t.randn((64, 256), device="cuda")
    side = t.cuda.Stream()

    def run(stream=None):
        return (bqe.rfpx_attn_forward(c.cache, c.batch, q, stream=stream),
                *bqe.rfpx_qk_norm_rope(q, q[:, :2], pos, rope=rope, stream=stream),
                *bqe.rfpx_kv_unpack(c.cache, c.batch, 5, stream=stream), bqe.rfpx_pack(4, x, stream=stream))

    want = run()
    ws = bqe.rfpx_attn_workspace_bytes(c.cache, c.batch, 8, 5)
    t.cuda.synchronize()
    shapes = [(y.shape, y.dtype) for y in want] + [((ws,), t.uint8)]
    for _ in range(3):
        t.cuda._sleep(20_000_000)
        for shape, dtype in shapes:
            t.empty(shape, dtype=dtype, device="cuda").fill_(7)  # queued behind the sleep, and given back at once
        got = run(side)
        t.cuda.synchronize()
        for a, b in zip(got, want):
            assert t.equal(a, b)


# ----------------------------------------------------------------- eviction

@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1, None])
@pytest.mark.parametrize("at", [0, 2])
def test_evict_beside_a_sequence_with_pages_outside(at, bad):
    """The page that moves go to, or come from, lies outside the pool in one
    sequence: its weights and positions move alone, no byte of the pool does,
    and the other sequence is cut as ever."""
    t = torch()
    made = []
    for broken in (False, True):
        c = Case([96, 96], [96, 96], 2, 64, 32, t.float32, seed=5)
        acc = t.arange(96, dtype=t.float32, device="cuda").expand(2, 2, 96).contiguous()
        pos = t.arange(96, dtype=t.int32, device="cuda").expand(2, 2, 96).contiguous() + 7
        mine = c.table[0].clone()
        if broken:
            c.table[0, at] = c.cache.n_pages if bad is None else bad
        before = c.cache.pool.view(c.cache.n_pages, -1).clone()
        ao, po, lo = bqe.rfpx_kv_evict(c.cache, c.fill, 32, 0, acc, pos)
        assert lo.tolist() == [32, 32]
        pool = c.cache.pool.view(c.cache.n_pages, -1)
        # slots 64 .. 95 are the best 32, and go to 0 .. 31, in order
        for b in range(2):
            assert t.equal(ao[b, :, :32], t.arange(64.0, 96.0, device="cuda").expand(2, 32))
            assert t.equal(po[b, :, :32], t.arange(71, 103, dtype=t.int32, device="cuda").expand(2, 32))
        if broken:
            assert t.equal(pool[mine.long()], before[mine.long()])
        made.append(pool[c.table[1].long()].clone())
    assert t.equal(*made)


# ------------------------------------------------------- plans and the data

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,heads,d,cols,told,plan", [
    (2, 16, 64, 100, 10, 65536), (2, 16, 128, 70, 9, 65536), (128, 128, 64, 300, 66, 1024), (2, 4, 128, 60, 1, 0),
    (1, 3, 256, 40, 2, 300)])
def test_more_columns_than_planned(hk, heads, d, cols, told, plan, dtype):
    """A workgroup's second turn at row blocks, in both kernels: splits, whole
    sequences, and the fewest row blocks."""
    t = torch()
    c = Case([330, 20], [cols, 3], hk, d, 64, dt(dtype), seed=d, capacity=max(plan, 330))
    g = t.Generator(device="cuda").manual_seed(2)
    q = (t.randn((c.rows, heads, d), generator=g, device="cuda") * 1.3).to(dt(dtype))
    z = t.zeros((c.rows, heads), device="cuda")
    small = bqe.KvBatch(c.table, c.batch.lens, c.batch.starts, told, max(plan, 1))
    out = bqe.rfpx_attn_forward(c.cache, small, q, lse=z)
    few = 1 if hk > 2 else hk  # kv heads: the plain form takes its time
    values, h = [(k[:, :few], v[:, :few]) for k, v in c.values()], few * heads // hk
    c.hk, c.values = few, lambda: values
    ref = attend64(c, q[:, :h], d ** -0.5)
    check_out(out[:, :h], ref, dt(dtype), slice(0, c.rows))
    check_lse(z[:, :h], ref, slice(0, c.rows))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("d,heads,plan", [(64, 4, 0), (64, 20, 0), (256, 4, 0), (128, 20, 1500), (64, 40, 65536), (128, 40, 65536)])
def test_nan_block_in_a_tile_that_all_rows_see(d, heads, plan, dtype):
    """Far before the columns: every row of the head gets the values' NaN in its
    block, and the keys' NaN everywhere."""
    t = torch()
    c = Case([400], [4], 2, d, 64, dt(dtype), seed=d, capacity=max(plan, 400))
    k, v = c.k_in.clone(), c.v_in.clone()
    v[17, 0, 33] = float("nan")
    k[40, 1, d - 1] = float("inf")
    bqe.rfpx_kv_append(c.cache, c.fill, k, v)
    q = t.randn((4, heads, d), device="cuda").to(dt(dtype))
    z = t.zeros((4, heads), device="cuda")
    out = bqe.rfpx_attn_forward(c.cache, c.planned(plan), q, lse=z)
    g = heads // 2
    assert bool(out[:, :g, 32:64].isnan().all()) and bool(out[:, g:].isnan().all())
    keep = [i for i in range(d) if not 32 <= i < 64]
    assert bool(out[:, :g, keep].isfinite().all())
    assert bool(z[:, :g].isfinite().all()) and bool(z[:, g:].isnan().all())


# ------------------------------------------------------------------ weights

def weights_batch(c, kernel, group, max_len=None):
    """The batch as planned for k_attn_weights ("few") or k_attn_weights_chunk
    ("many": 256 rows of a sequence and no more than 16 tokens to each)."""
    cols = -(-256 // group) if kernel == "many" else max(1, min(c.cols))
    return bqe.KvBatch(c.table, c.batch.lens, c.batch.starts, cols, max(c.lens) if max_len is None else max_len)


def check_weights(c, got, start, decay, ref, heads=None):
    """got = decay * start + the weights of ref (its scores' errors three times:
    the score's own, lse's and the product's)."""
    for b, n in enumerate(c.lens):
        for h in range(c.hk) if heads is None else heads:
            want = decay * f64(start)[b, h, :n] + ref["w"][b][h]
            tol = 3 * ref["dw"][b][h] + 2.0 ** -20 * ref["w"][b][h] + 4 * U32 * want + 1e-30
            err = np.abs(f64(got)[b, h, :n] - want)
            assert (err <= tol).all(), (b, h, np.nanmax(err / tol))


KERNELS = [(k, d, n) for k in ("few", "many") for d in (64, 128, 256) for n in ("bfloat16", "float32")]


@pytest.mark.parametrize("kernel,d,dtype", KERNELS)
@pytest.mark.parametrize("told", [None, 1, 64])
def test_weights_rows_outside_strides_and_plans(kernel, d, dtype, told):
    """Queries that are slices of wider rows, rows before the first sequence and
    behind the last, sequences longer than planned."""
    t = torch()
    hk, group = 2, 3
    c = Case([300, 0, 70, 161], [30, 2, 5, 7], hk, d, 32, dt(dtype), seed=d, gap=2)
    g = t.Generator(device="cuda").manual_seed(6)
    rows = c.rows + 3
    wide = (t.randn((rows, 8, d), generator=g, device="cuda") * 1.3).to(dt(dtype))
    q = wide[:, 1:1 + hk * group]
    z = t.full((rows, hk * group), float("nan"), device="cuda")
    wide[:2], wide[c.rows:] = float("nan"), float("nan")  # not read
    bqe.rfpx_attn_forward(c.cache, c.batch, q, lse=z)
    assert bool(z[:2].isnan().all()) and bool(z[c.rows:].isnan().all())
    acc = t.rand((4, hk, c.per * 32), generator=g, device="cuda")
    got = bqe.rfpx_attn_weights(c.cache, weights_batch(c, kernel, group, told), q, z, acc, 0.75,
                                acc_out=t.full_like(acc, -3.0))
    ref = attend64(c, q.nan_to_num(), d ** -0.5)
    check_weights(c, got, acc, 0.75, ref)
    for b, n in enumerate(c.lens):
        assert bool((got[b, :, n:] == -3).all())


@pytest.mark.parametrize("kernel,d,dtype", KERNELS)
def test_weights_over_pages_outside(kernel, d, dtype):
    """Slots without a page receive nothing: their weight only decays."""
    t = torch()
    hk, group = 2, 2
    c = Case([200, 40], [9, 3], hk, d, 32, dt(dtype), seed=d)
    vals = c.values()
    c.table[0, 1], c.table[0, 4], c.table[1, 0] = -1, c.cache.n_pages, 2 ** 31 - 1
    q = t.randn((12, 4, d), device="cuda").to(dt(dtype))
    z = t.zeros((12, 4), device="cuda")
    bqe.rfpx_attn_forward(c.cache, c.batch, q, lse=z)
    acc = t.rand((2, hk, c.per * 32), device="cuda")
    start = acc.clone()
    bqe.rfpx_attn_weights(c.cache, weights_batch(c, kernel, group), q, z, acc, 0.5)
    c.values = lambda: vals
    ref = attend64(c, q, d ** -0.5, seen=lambda b, j: j // 32 not in ((1, 4) if b == 0 else (0,)))
    check_weights(c, acc, start, 0.5, ref)
    assert t.equal(acc[1, :, :32], start[1, :, :32] * 0.5) and t.equal(acc[0, :, 32:64], start[0, :, 32:64] * 0.5)


@pytest.mark.parametrize("kernel,d,dtype", KERNELS)
def test_weights_beside_nan(kernel, d, dtype):
    """A NaN key reaches the head's slots through the rows that see it and no
    others; a row of lse -inf gives nothing; NaN values give nothing either."""
    t = torch()
    hk, group, n = 2, 2, 200
    c = Case([n, 50], [9, 3], hk, d, 64, dt(dtype), seed=d)
    vals = c.values()
    k, v = c.k_in[n - 9:n].clone(), c.v_in[n - 9:n].clone()
    k[8, 1, 5], v[2, 0, 40] = float("nan"), float("inf")  # the last column's key of head 1
    step = c.make([n, 50], [0, 9, 9], 9)
    bqe.rfpx_kv_append(c.cache, step, k, v)
    q = t.randn((12, 4, d), device="cuda").to(dt(dtype))
    z = t.zeros((12, 4), device="cuda")
    bqe.rfpx_attn_forward(c.cache, c.batch, q, lse=z)
    assert bool(z[8, 2:].isnan().all()) and int(z.isnan().sum()) == 2
    acc = t.rand((2, hk, c.per * 64), device="cuda")
    b = weights_batch(c, kernel, group)
    got = bqe.rfpx_attn_weights(c.cache, b, q, z, acc, 1.0, acc_out=t.zeros_like(acc))
    c.values = lambda: vals
    ref = attend64(c, q, d ** -0.5)
    check_weights(c, got, acc, 1.0, ref, heads=[0])
    assert bool(got[0, 1, :n].isnan().all()) and bool(got[1].isfinite().all())
    # without the row that sees it
    z[8, 2:] = -float("inf")
    got = bqe.rfpx_attn_weights(c.cache, b, q, z, acc, 1.0, acc_out=t.zeros_like(acc))
    ref["w"][0][1], ref["dw"][0][1] = 0, 0
    kk = vals[0][0]
    for i in range(8):
        for h in (2, 3):
            m = n - 9 + i + 1
            s = d ** -0.5 * (kk[:m, 1] @ f64(q)[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            ref["w"][0][1, :m] += p
            ref["dw"][0][1, :m] += (2 * ref["ds"][i, h] + 2.0 ** -22) * p
    check_weights(c, got, acc, 1.0, ref)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_captured_weights_of_many_rows(dtype):
    """A captured chunk with k_attn_weights_chunk, replayed with other lengths
    and columns, against the eager calls and, each time, against 64 bits."""
    t = torch()
    hk, group, d, page, rows = 2, 8, 64, 32, 80
    c = Case([300, 200], [40, 40], hk, d, page, dt(dtype), capacity=512)
    batch = c.make(c.lens, c.starts, 40, 320)  # 320 rows a sequence, 320 tokens
    g = t.Generator(device="cuda").manual_seed(9)
    q = t.randn((rows, hk * group, d), generator=g, device="cuda").to(dt(dtype))
    out, lse = t.zeros_like(q), t.zeros((rows, hk * group), device="cuda")
    acc, acc_out = t.rand((2, hk, c.per * page), generator=g, device="cuda"), t.zeros((2, hk, c.per * page), device="cuda")
    ws = t.empty(bqe.rfpx_attn_workspace_bytes(c.cache, batch, hk * group, rows), dtype=t.uint8, device="cuda")

    def step(out, lse, acc_out, ws=None):
        bqe.rfpx_attn_forward(c.cache, batch, q, out=out, lse=lse, ws=ws)
        bqe.rfpx_attn_weights(c.cache, batch, q, lse, acc, 0.5, acc_out=acc_out)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(out, lse, acc_out, ws)
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(out, lse, acc_out, ws)
    values = c.values()
    for lens, starts in (([300, 200], [0, 40, 80]), ([250, 33], [0, 40, 73]), ([64, 80], [0, 3, 80]), ([31, 0], [0, 64, 64]),
                         ([300, 200], [0, 40, 80])):
        batch.lens.copy_(t.tensor(lens, dtype=t.int32))
        batch.starts.copy_(t.tensor(starts, dtype=t.int32))
        for x in (out, lse, acc_out):
            x.fill_(3)
        graph.replay()
        o2, z2, a2 = t.full_like(out, 3), t.full_like(lse, 3), t.full_like(acc_out, 3)
        step(o2, z2, a2)
        t.cuda.synchronize()
        assert t.equal(out, o2) and t.equal(lse, z2) and t.equal(acc_out, a2), lens
        assert bool((out[starts[-1]:] == 3).all())
        c.lens, c.starts, c.cols, c.rows = lens, starts, [b - a for a, b in zip(starts, starts[1:])], starts[-1]
        c.values = lambda: [(k[:n], v[:n]) for (k, v), n in zip(values, lens)]
        ref = attend64(c, q, d ** -0.5)
        check_out(out, ref, dt(dtype), slice(0, c.rows))
        check_lse(lse, ref, slice(0, c.rows))
        check_weights(c, acc_out, acc, 0.5, ref)
        _ = (q.float() @ q.float().transpose(1, 2)).sum().item()  # eager work between


# ------------------------------------------------------------- rows and data

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("plan", [0, 65536])
def test_fewer_rows_than_the_batch_says(plan, dtype):
    """starts tells of 40 + 30 columns, the tensors end after 50 rows: columns
    keep their slots, the rest is neither read nor written."""
    t = torch()
    hk, heads, d = 2, 16, 64
    c = Case([200, 90], [40, 30], hk, d, 32, dt(dtype), seed=1, capacity=max(plan, 200))
    g = t.Generator(device="cuda").manual_seed(8)
    batch = c.planned(plan)
    q = (t.randn((70, heads, d), generator=g, device="cuda") * 1.3).to(dt(dtype))
    whole, zw = t.zeros_like(q), t.zeros((70, heads), device="cuda")
    bqe.rfpx_attn_forward(c.cache, batch, q, out=whole, lse=zw)
    out, z = t.full_like(q, 7.0), t.full((70, heads), 7.0, device="cuda")
    bqe.rfpx_attn_forward(c.cache, batch, q[:50], out=out[:50], lse=z[:50])
    assert t.equal(out[:50], whole[:50]) and t.equal(z[:50], zw[:50])
    assert bool((out[50:] == 7).all()) and bool((z[50:] == 7).all())
    # weights of the rows that are there, by both kernels: the others' lse says that they see nothing
    zw[50:] = -float("inf")
    for kernel in ("few", "many"):
        b = weights_batch(c, kernel, heads // hk)
        acc = t.rand((2, hk, c.per * 32), generator=g, device="cuda")
        a = bqe.rfpx_attn_weights(c.cache, b, q, zw, acc, acc_out=t.zeros_like(acc))
        assert t.equal(bqe.rfpx_attn_weights(c.cache, b, q[:50], z[:50], acc, acc_out=t.zeros_like(acc)), a)
    # append and unpack
    k = t.randn((70, hk, d), generator=g, device="cuda").to(dt(dtype))
    before, _ = bqe.rfpx_kv_unpack(c.cache, c.batch, 70)
    bqe.rfpx_kv_append(c.cache, c.batch, k[:50], k[:50])
    got, _ = bqe.rfpx_kv_unpack(c.cache, c.batch, 70)
    want = bqe.rfpx_unpack(4, bqe.rfpx_pack(4, k[:50].float().reshape(-1, d)), 50 * hk, d).view(50, hk, d)
    assert t.equal(got[:50], want) and t.equal(got[50:], before[50:])
    short = t.full_like(got, 5.0)
    bqe.rfpx_kv_unpack(c.cache, c.batch, 50, short[:50], short[:50].clone())
    assert t.equal(short[:50], got[:50]) and bool((short[50:] == 5).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,heads,d,cols,plan", PATHS)
def test_bad_queries_reach_no_other_row(hk, heads, d, cols, plan, dtype):
    """A query of NaN and one of infinities among ordinary ones: NaN for
    themselves, and the rows beside them within their bounds."""
    t = torch()
    cols = max(cols, 3)
    c = Case([300], [cols], hk, d, 64, dt(dtype), seed=d, capacity=max(plan, 300))
    g = t.Generator(device="cuda").manual_seed(4)
    q = (t.randn((cols, heads, d), generator=g, device="cuda") * 1.3).to(dt(dtype))
    q[0, 0, 5], q[1, 1, :] = float("nan"), float("inf")
    z = t.zeros((cols, heads), device="cuda")
    out = bqe.rfpx_attn_forward(c.cache, c.planned(plan), q, lse=z)
    assert bool(out[0, 0].isnan().all()) and bool(out[1, 1].isnan().all()) and bool(z[0, 0].isnan()) and bool(z[1, 1].isnan())
    few = 2 if hk > 2 else hk  # kv heads: the plain form takes its time
    (k, v), = c.values()
    h = few * heads // hk
    c.hk, c.values = few, lambda: [(k[:, :few], v[:, :few])]
    clean = q[:, :h].clone()
    clean[0, 0], clean[1, 1] = 0, 0
    ref = attend64(c, clean, d ** -0.5)
    out, z = out[:, :h].clone(), z[:, :h].clone()
    for i in (0, 1):
        out[i, i], z[i, i] = t.from_numpy(ref["out"][i, i]).to(out), float(ref["lse"][i, i])
    check_out(out, ref, dt(dtype), slice(0, cols))
    check_lse(z, ref, slice(0, cols))


def test_negative_lengths_are_none():
    t = torch()
    c = Case([40, 33], [2, 2], 2, 64, 32, t.bfloat16)
    b = c.make([-5, -2 ** 31], c.starts, 2, 40)
    q = t.randn((4, 4, 64), device="cuda").to(t.bfloat16)
    z = t.zeros((4, 4), device="cuda")
    before = c.cache.pool.clone()
    bqe.rfpx_kv_append(c.cache, b, q[:, :2], q[:, :2])
    assert t.equal(c.cache.pool, before)
    assert bool((bqe.rfpx_attn_forward(c.cache, b, q, lse=z) == 0).all()) and bool((z == -float("inf")).all())
    acc = t.rand((2, 2, 64), device="cuda")
    start, pos = acc.clone(), t.zeros((2, 2, 64), dtype=t.int32, device="cuda")
    bqe.rfpx_attn_weights(c.cache, b, q, z, acc, 0.5)
    _, _, lens = bqe.rfpx_kv_evict(c.cache, b, 1, 0, acc, pos)
    assert t.equal(acc, start) and lens.tolist() == [0, 0] and t.equal(c.cache.pool, before)
