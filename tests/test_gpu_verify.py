"""Trees of drafted tokens (include/rfpx_verify.h but for rfpx_sample): masks,
attention, acceptance and the cache's commit, against plain implementations,
attention in 64 bits on the values that the cache holds.

Tolerances of attention are those of test_gpu_attn.py, whose kernels these are:
what a row sees changes which terms are summed, not how.  Everything else is
whole numbers and bytes, and equal.
"""
import random

import numpy as np
import pytest

import block_quantized_expert_amd as bqe
from test_gpu_attn import U32, Case, check_lse, check_out, dt, f64, torch, units

pytestmark = pytest.mark.gpu
UNTOUCHED = -12345


def ints(x):
    t = torch()
    return t.tensor(x, dtype=t.int32, device="cuda")


def batch_of(lens, starts, cols=None, max_len=None):
    """A batch for the calls that need no cache."""
    t = torch()
    n = len(lens)
    cols = max([b - a for a, b in zip(starts, starts[1:])] + [1]) if cols is None else cols
    return bqe.KvBatch(t.zeros((n, 1), dtype=t.int32, device="cuda"), ints(lens), ints(starts), cols,
                       max_len or max(list(lens) + [1]))


def tree(n, shape, rng):
    """Parents of n columns."""
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1] + [0] * (n - 1)
    if shape == "forest":
        return [-1 if i == 0 or rng.random() < 0.3 else rng.randrange(i) for i in range(n)]
    if shape == "bad":  # numbers that are no column before this one
        return [rng.choice([-1, -7, i, i + 1, n, 1 << 30, -(1 << 31), rng.randrange(max(1, i))]) for i in range(n)]
    return [-1] + [rng.randrange(max(0, i - 9), i) for i in range(1, n)] if n else []


def line_of(parents, i):
    line = []
    while True:
        line.append(i)
        p = parents[i]
        if not 0 <= p < i:
            return line[::-1]
        i = p


def words_of(columns, words):
    made = [0] * words
    for j in columns:
        if j < 32 * words:
            made[j // 32] |= 1 << (j % 32)
    return [w - (1 << 32) if w >> 31 else w for w in made]


# ----------------------------------------------------------------- masks

@pytest.mark.parametrize("sizes,shape,words", [
    ([1], "chain", 1), ([16], "tree", 1), ([32, 33, 0, 1, 64, 65], "tree", 3), ([1024], "chain", 32),
    ([1024, 1000], "tree", 32), ([257, 3], "star", 9), ([100, 70, 40], "forest", 4), ([100, 70, 40], "bad", 4),
    ([90, 200], "tree", 2), ([5, 6], "tree", 32), ([0, 0], "tree", 1), ([300] * 70, "tree", 10)])
@pytest.mark.parametrize("based", [True, False])
def test_masks(sizes, shape, words, based):
    t = torch()
    rng = random.Random(len(sizes) + words)
    gap = 3
    starts = [gap]
    for n in sizes:
        starts.append(starts[-1] + n)
    rows = starts[-1] + 5
    parents = [rng.randrange(-2, 5) for _ in range(rows)]
    for first, n in zip(starts, sizes):
        parents[first:first + n] = tree(n, shape, rng)
    lens = [n + rng.randrange(0, 1000) for n in sizes]
    base = [rng.randrange(0, 1 << 20) for _ in sizes]
    b = batch_of(lens, starts)
    masks = t.full((rows, words), UNTOUCHED, dtype=t.int32, device="cuda")
    pos = t.full((rows,), UNTOUCHED, dtype=t.int32, device="cuda")
    bqe.rfpx_tree_masks(b, ints(parents), ints(base) if based else None, masks=masks, positions=pos)
    want, wpos = [[UNTOUCHED] * words for _ in range(rows)], [UNTOUCHED] * rows
    for s, (first, n) in enumerate(zip(starts, sizes)):
        for i in range(n):
            line = line_of(parents[first:first + n], i)
            want[first + i] = words_of(line, words)
            wpos[first + i] = (base[s] if based else lens[s] - n) + len(line) - 1
    assert masks.tolist() == want and pos.tolist() == wpos


def test_masks_of_fewer_rows_and_more_columns():
    """Rows past the tensors, and columns past what a tree may have, are left."""
    t = torch()
    parents = ints(tree(1500, "chain", None))
    masks = t.full((1500, 32), UNTOUCHED, dtype=t.int32, device="cuda")
    pos = t.full((1500,), UNTOUCHED, dtype=t.int32, device="cuda")
    bqe.rfpx_tree_masks(batch_of([1500], [0, 1500], cols=1024), parents, masks=masks, positions=pos)
    assert pos.tolist() == list(range(1024)) + [UNTOUCHED] * 476
    assert (masks[1024:] == UNTOUCHED).all() and masks[1023].tolist() == [-1] * 32
    short = t.full((7, 1), UNTOUCHED, dtype=t.int32, device="cuda")
    both = t.full((14, 1), UNTOUCHED, dtype=t.int32, device="cuda")
    b = batch_of([20, 20], [0, 5, 12])
    bqe.rfpx_tree_masks(b, parents[:7].contiguous(), masks=short)
    bqe.rfpx_tree_masks(b, ints([-1, 0, 1, 2, 3, -1, 0, 1, 2, 3, 4, 5, -1, -1]), masks=both)
    assert short[:5].tolist() == both[:5].tolist() and short[5:].tolist() == [[1], [2]]  # (5 is no column before 1)
    assert both[12:].tolist() == [[UNTOUCHED]] * 2
    m, p = bqe.rfpx_tree_masks(b, parents[:0])
    assert m.shape == (0, 1) and p.shape == (0,)


# ------------------------------------------------------------- attention

def attend64(case, q, scale, sees, heads_of=None):
    """out, lse and the bounds of their errors in 64 bits; sees(b, i): the
    slots that column i of sequence b sees."""
    q = f64(q)
    heads = q.shape[1]
    g = heads // case.hk
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    mag, ds_, do = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape)
    for b, (k, v) in enumerate(case.values()):
        for i in range(case.cols[b]):
            at = np.array(sorted(sees(b, i)), np.int64)
            if not at.size:
                continue
            row = case.starts[b] + i
            for h in heads_of or range(heads):
                kk, vv = k[at, h // g], v[at, h // g]
                s = scale * (kk @ q[row, h])
                z = s.max() + np.log(np.exp(s - s.max()).sum())
                p = np.exp(s - z)
                out[row, h], lse[row, h] = p @ vv, z
                mag[row, h] = p @ np.abs(vv)
                big = scale * (31 * units(kk) @ np.abs(q[row, h])).max()
                ds = 256 * U32 * big + 2.0 ** -22 * (1 + np.abs(s).max())
                ds_[row, h] = ds
                do[row, h] = 2 * ds * mag[row, h] + 256 * U32 * 31 * (p @ units(vv))
    return dict(out=out, lse=lse, mag=mag, ds=ds_, do=do)


def seen_by_tree(case, parents):
    """What a column sees: the context and its line."""
    def sees(b, i):
        n = case.cols[b]
        context = case.lens[b] - n
        if context + i < 0:
            return []
        line = line_of(parents[case.starts[b]:case.starts[b] + n], i)
        return [*range(max(0, context)), *[context + j for j in line if context + j >= 0]]
    return sees


def forward(case, heads, dtype, masks, plan=0, gap_rows=0, seed=1, lse=True):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    rows = case.rows + gap_rows
    q = (t.randn((rows, heads, case.d), generator=g, device="cuda") * 1.3).to(dtype)
    out = t.full_like(q, 7.0)
    z = t.full((rows, heads), 7.0, device="cuda")
    scale = case.d ** -0.5
    bqe.rfpx_attn_tree_forward(case.cache, case.planned(plan) if plan else case.batch, q, masks, scale, out=out,
                               lse=z if lse else None)
    return q, out, z, scale


FORMS = [  # lens, cols, kv heads, group, head_dim, page, plan
    ([1], [1], 1, 1, 64, 32, 0),                                # one column over itself
    ([16], [16], 2, 4, 128, 64, 0),                             # a tree and no context
    ([37, 5, 70, 64], [5, 5, 7, 1], 2, 4, 128, 64, 0),          # trees that end inside tiles and pages
    ([333, 12, 95], [33, 0, 40], 1, 3, 64, 32, 0),              # masks of two words, none at one
    ([700], [64], 1, 8, 128, 64, 0), ([1100, 1000], [130, 33], 2, 2, 64, 64, 0),
    ([300], [20], 1, 7, 256, 128, 0), ([90], [9], 8, 2, 256, 32, 0),
    ([2000, 60], [7, 60], 2, 4, 128, 256, 131071),              # many splits, most of them empty
    ([500], [40], 2, 8, 128, 64, 65536),                        # the kernel of many rows
    ([1300, 37, 250], [30, 37, 17], 8, 8, 64, 32, 65536),
    ([300, 37], [16, 9], 2, 4, 128, 64, 65536), ([310, 90], [16, 16], 2, 4, 64, 32, 65536),  # blocks of 32 rows
    ([17 + i % 90 for i in range(70)], [16 - i % 3 for i in range(70)], 2, 4, 64, 32, 1000),  # ... in one launch
    ([17 + i % 90 for i in range(70)], [16 - i % 3 for i in range(70)], 2, 4, 128, 64, 1000),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("lens,cols,hk,group,d,page,plan", FORMS)
def test_attention_of_a_tree(lens, cols, hk, group, d, page, plan, dtype):
    t = torch()
    rng = random.Random(sum(lens))
    c = Case(lens, cols, hk, d, page, dt(dtype), seed=sum(cols), gap=2, capacity=plan or None)
    parents = [-1] * 2 + [p for n in cols for p in tree(n, "tree", rng)] + [-1] * 3
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    q, out, z, scale = forward(c, hk * group, dt(dtype), masks, plan, gap_rows=3)
    ref = attend64(c, q, scale, seen_by_tree(c, parents))
    rows = slice(c.starts[0], c.rows)
    check_out(out, ref, dt(dtype), rows)
    check_lse(z, ref, rows)
    assert (out[c.rows:] == 7).all() and (z[c.rows:] == 7).all() and (out[:2] == 7).all() and (z[:2] == 7).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,group,d,cols,plan", [(2, 4, 128, 33, 0), (1, 2, 256, 40, 0), (2, 8, 64, 70, 65536),
                                                  (2, 8, 128, 45, 65536)])
def test_attention_of_any_bits(hk, group, d, cols, plan, dtype):
    """Bits that are no tree's: columns that see later ones and not themselves,
    nothing but the context, or (without a context) nothing at all; bits of
    columns that there are not, and columns without bits."""
    t = torch()
    rng = random.Random(d + cols)
    words = 2
    lens = [cols, 100 + cols, 20]
    sizes = [cols, cols - 6, 31]  # the last one's first columns have no slots
    c = Case(lens, [cols, cols - 6, 20], hk, d, 64, dt(dtype), seed=cols, capacity=plan or None)
    c.cols, c.starts = sizes, [0, sizes[0], sizes[0] + sizes[1], sum(sizes)]
    c.rows = sum(sizes)
    c.batch = c.make(lens, c.starts, max(sizes))
    named = [[j for j in range(32 * words) if rng.random() < 0.3] for _ in range(c.rows)]
    for r in (0, 5, sizes[0] + 2, sizes[0] + sizes[1] + 15):
        named[r] = []
    masks = ints([words_of(x, words) for x in named])
    q, out, z, scale = forward(c, hk * group, dt(dtype), masks, plan)

    def sees(b, i):
        context = lens[b] - sizes[b]
        if context + i < 0:
            return []
        return [*range(max(0, context)),
                *[context + j for j in named[c.starts[b] + i] if j < sizes[b] and context + j >= 0]]

    ref = attend64(c, q, scale, sees)
    check_out(out, ref, dt(dtype), slice(0, c.rows))
    check_lse(z, ref, slice(0, c.rows))
    for r in (0, 5, sum(sizes[:2]), sum(sizes[:2]) + 10):
        assert (out[r] == 0).all() and (z[r] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("hk,heads,d,plan", [(1, 4, 64, 0), (2, 8, 128, 0), (1, 4, 256, 0), (2, 16, 128, 65536),
                                             (2, 16, 64, 65536)])
def test_attention_beside_nan(hk, heads, d, plan, dtype):
    """Columns whose keys or values are not finite reach those that see them."""
    t = torch()
    n, context = 40, 67
    rng = random.Random(d)
    c = Case([context + n], [n], hk, d, 32, dt(dtype), seed=d, capacity=plan or None)
    parents = tree(n, "tree", rng)
    nan_k, nan_v = 11, 23
    k, v = c.k_in[context:].clone(), c.v_in[context:].clone()
    k[nan_k], v[nan_v, :, 40] = float("nan"), float("inf")
    bqe.rfpx_kv_append(c.cache, c.batch, k, v)
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    q, out, z, scale = forward(c, heads, dt(dtype), masks, plan)
    clean = Case([context + n], [n], hk, d, 32, dt(dtype), seed=d)
    ref = attend64(clean, q, scale, seen_by_tree(c, parents))
    lines = [line_of(parents, i) for i in range(n)]
    fine = [i for i in range(n) if nan_k not in lines[i] and nan_v not in lines[i]]
    assert 0 < len(fine) < n
    check_out(out, ref, dt(dtype), fine)
    check_lse(z, ref, [i for i in range(n) if nan_k not in lines[i]])
    for i in range(n):
        if nan_k in lines[i]:
            assert t.isnan(out[i]).all() and t.isnan(z[i]).all()
        elif nan_v in lines[i]:  # the block of value 40
            assert t.isnan(out[i, :, 32:64]).all() and not t.isnan(out[i, :, :32]).any()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("heads,plan", [(4, 0), (32, 65536)])
def test_attention_over_bad_pages(heads, plan, dtype):
    """Pages outside the pool hold nothing, of the context and of the tree."""
    lens, cols = [150, 40], [40, 10]
    rng = random.Random(2)
    c = Case(lens, cols, 2, 128, 32, dt(dtype), seed=5, capacity=plan or None)
    values = c.values()
    c.values = lambda: values
    c.table[0, 1], c.table[0, 4], c.table[1, 0] = -1, 1 << 30, c.cache.n_pages
    parents = [p for n in cols for p in tree(n, "tree", rng)]
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    q, out, z, scale = forward(c, heads, dt(dtype), masks, plan)
    sees = seen_by_tree(c, parents)
    gone = {0: {1, 4}, 1: {0}}
    ref = attend64(c, q, scale, lambda b, i: [s for s in sees(b, i) if s // 32 not in gone[b]])
    check_out(out, ref, dt(dtype), slice(0, c.rows))
    check_lse(z, ref, slice(0, c.rows))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_chain_is_attention_forward(dtype):
    """A tree that is a chain: the same bits as rfpx_attn_forward gives."""
    t = torch()
    c = Case([700, 33], [8, 5], 2, 128, 64, dt(dtype), seed=3)
    masks, pos = bqe.rfpx_tree_masks(c.batch, ints(tree(8, "chain", None) + tree(5, "chain", None)))
    q, out, z, scale = forward(c, 8, dt(dtype), masks)
    z2 = t.zeros_like(z)
    want = bqe.rfpx_attn_forward(c.cache, c.batch, q, scale, lse=z2)
    assert t.equal(out, want) and t.equal(z, z2)
    assert pos.tolist() == [*range(692, 700), *range(28, 33)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_attention_strides_and_rows(dtype):
    """Queries and outputs as slices of wider rows, more rows than the batch
    has, fewer than it says, and a longer mask than needed."""
    t = torch()
    c = Case([200, 90], [30, 20], 2, 128, 64, dt(dtype), seed=9)
    rng = random.Random(4)
    parents = tree(30, "tree", rng) + tree(20, "tree", rng)
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents), mask_words=5)
    q, out, z, scale = forward(c, 8, dt(dtype), masks)
    wide, wide_out = (t.full((50, 3, 8, 128), 3.0, device="cuda").to(dt(dtype)) for _ in range(2))
    wide[:, 1] = q
    bqe.rfpx_attn_tree_forward(c.cache, c.batch, wide[:, 1], masks, scale, out=wide_out[:, 2])
    assert t.equal(wide_out[:, 2], out) and (wide_out[:, :2] == 3).all()
    few = bqe.rfpx_attn_tree_forward(c.cache, c.batch, q[:37].contiguous(), masks[:37].contiguous(), scale)
    ref = attend64(c, q, scale, seen_by_tree(c, parents))
    check_out(few, ref, dt(dtype), slice(0, 37))
    assert bqe.rfpx_attn_tree_forward(c.cache, c.batch, q[:0], masks[:0], scale).shape == (0, 8, 128)


def test_attention_past_32_bits():
    """A pool of more than 4 GiB, a table of more slots than the sequence has."""
    t = torch()
    page, hk, d = 256, 8, 128
    pages = (5 << 30) // (page * hk * d * 17 // 16)
    cache = bqe.KvCache(hk, d, page, pages)
    cache.pool.fill_(255)
    n, length = 17, 600
    table = ints([[pages - 1, 3, pages - 7, 5]])
    g = t.Generator(device="cuda").manual_seed(1)
    k, v = (t.randn((length, hk, d), generator=g, device="cuda") for _ in range(2))
    fill = bqe.KvBatch(table, ints([length]), ints([0, length]), length, length)
    bqe.rfpx_kv_append(cache, fill, k, v)
    c = Case([length], [n], hk, d, page, t.float32, seed=1)
    c.cache, c.fill, c.batch = cache, fill, bqe.KvBatch(table, ints([length]), ints([0, n]), n, length)
    parents = tree(n, "tree", random.Random(1))
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    q, out, z, scale = forward(c, hk, t.bfloat16, masks)
    ref = attend64(c, q, scale, seen_by_tree(c, parents))
    check_out(out, ref, t.bfloat16, slice(0, n))
    check_lse(z, ref, slice(0, n))
    # ... and a path that moves there
    before = bqe.rfpx_kv_unpack(cache, c.batch, n)
    bqe.rfpx_kv_commit(cache, c.batch, ints([[0, 4, 9, 16]]), ints([4]))
    after = bqe.rfpx_kv_unpack(cache, c.batch, n)
    for x, y in zip(before, after):
        assert t.equal(y[:4], x[[0, 4, 9, 16]]) and t.equal(y[4:], x[4:])


# ------------------------------------------------------------ acceptance

def accept64(parents, tokens, drawn, cols):
    line = [0] if parents else []
    while line and len(line) < cols:
        below = [j for j in range(line[-1] + 1, len(parents))
                 if parents[j] == line[-1] and tokens[j] == drawn[line[-1]] and tokens[j] >= 0]
        if not below:
            break
        line.append(below[0])
    return line


@pytest.mark.parametrize("sizes,shape,vocab", [([1], "chain", 5), ([16], "tree", 3), ([0, 1, 2, 33], "tree", 2),
                                               ([1024], "chain", 1), ([1024, 1024], "tree", 2), ([300], "star", 400),
                                               ([100, 50], "forest", 3), ([100, 50, 20], "bad", 2),
                                               ([64] * 300, "tree", 2)])
@pytest.mark.parametrize("cols", [None, 1, 3, 1024])
def test_accept(sizes, shape, vocab, cols):
    t = torch()
    rng = random.Random(len(sizes) * 7 + vocab)
    starts = [4]
    for n in sizes:
        starts.append(starts[-1] + n)
    rows = starts[-1] + 3
    parents, tokens, drawn = ([rng.randrange(vocab) for _ in range(rows)] for _ in range(3))
    for first, n in zip(starts, sizes):
        parents[first:first + n] = tree(n, shape, rng)
    for i in range(0, rows, 13):
        tokens[i] = drawn[i] = -1  # no tokens: they confirm nothing
    lens = [n + rng.randrange(0, 50) for n in sizes]
    b = batch_of(lens, starts)
    width = cols or max(sizes)
    path = t.full((len(sizes), width), UNTOUCHED, dtype=t.int32, device="cuda")
    got, counts, following, after = bqe.rfpx_tree_accept(b, ints(parents), ints(tokens), ints(drawn), path=path)
    assert got is path
    for s, (first, n) in enumerate(zip(starts, sizes)):
        p = [x if 0 <= x < i else -1 for i, x in enumerate(parents[first:first + n])]
        line = accept64(p, tokens[first:first + n], drawn[first:first + n], width)
        assert path[s].tolist() == line + [-1] * (width - len(line)), s
        assert counts[s].item() == len(line) and after[s].item() == lens[s] - n + len(line)
        assert following[s].item() == (drawn[first + line[-1]] if line else -1)


def test_accept_in_place_and_fewer_rows():
    t = torch()
    b = batch_of([30, 40], [0, 4, 8])
    parents, tokens, drawn = ints([-1, 0, 1, 2] * 2), ints([9, 1, 2, 3] * 2), ints([1, 2, 3, 4] * 2)
    path, counts, following, after = bqe.rfpx_tree_accept(b, parents[:6].contiguous(), tokens[:6].contiguous(),
                                                          drawn[:6].contiguous())
    assert path.tolist() == [[0, 1, 2, 3], [0, 1, -1, -1]] and counts.tolist() == [4, 2]
    assert following.tolist() == [4, 2] and after.tolist() == [30, 38]
    _, _, _, after = bqe.rfpx_tree_accept(b, parents, tokens, drawn, lens_out=b.lens)
    assert after is b.lens and after.tolist() == [30, 40]
    # lengths below the step's columns
    b = batch_of([2], [0, 4])
    assert bqe.rfpx_tree_accept(b, parents[:4], ints([0, 7, 7, 7]), drawn[:4])[3].tolist() == [0]
    empty = bqe.rfpx_tree_accept(batch_of([5], [0, 0]), parents[:0], tokens[:0], drawn[:0])
    assert [x.tolist() for x in empty] == [[[-1]], [0], [-1], [5]]


# ---------------------------------------------------------------- commit

def places(page, d, t):
    """Bytes of page token t within a slab, in the canonical order of its blocks."""
    nb, half = d // 32, page * d // 2
    at = [(t * 4 + o) * 4 * nb + 4 * b + x for b in range(nb) for o in range(4) for x in range(4)]
    at += [half + t * nb + b for b in range(nb)]
    v = half + page * nb
    at += [v + ((t // 4 * 16 + r) * nb * 4 + (t % 4 // 2 * (nb // 2) + b // 2) * 4 + t % 2 * 2 + b % 2)
           for b in range(nb) for r in range(16)]
    return np.array(at + [v + half + t * nb + b for b in range(nb)])


def commit64(c, pool, table, lens, starts, path, counts, extra):
    """The pool and the arrays after a commit, slot by slot."""
    pool, extra = pool.copy(), [x.copy() for x in extra]
    slabs = pool.reshape(c.cache.n_pages, c.hk, -1)
    for b, (first, end) in enumerate(zip(starts, starts[1:])):
        n = end - first
        context = lens[b] - n
        old, olds = slabs.copy() if n else None, [x.copy() for x in extra]
        for i in range(min(counts[b], n, len(path[b]))):
            j = path[b][i]
            if not i < j < n or context + i < 0:
                continue
            src, dst = context + j, context + i
            for x, o in zip(extra, olds):
                x[b, :, dst] = o[b, :, src]
            ps, pd = table[b][src // c.page], table[b][dst // c.page]
            if 0 <= ps < c.cache.n_pages and 0 <= pd < c.cache.n_pages:
                a, z = places(c.page, c.d, src % c.page), places(c.page, c.d, dst % c.page)
                slabs[pd][:, z] = old[ps][:, a]
    return pool, extra


COMMITS = [  # lens, cols, kv heads, head_dim, page, paths
    ([1], [1], 1, 64, 32, [[0]]),
    ([40], [8], 2, 128, 32, [[0, 1, 2, 3, 4, 5, 6, 7]]),           # all stay
    ([40], [8], 2, 128, 32, [[0, 2, 3, 5, 7]]),                    # slots left and entered
    ([70, 33, 20, 10], [30, 33, 0, 1], 3, 64, 32, [[0, 3, 4, 5, 20, 29], [1, 2, 31, 32], [], [0]]),
    ([600], [200], 1, 256, 64, [[i for i in range(200) if i % 3 != 1]]),   # many turns, all overlapping
    ([2000], [1024], 2, 128, 128, [list(range(1, 1024))]),          # the whole step one slot ahead
    ([90, 300], [64, 64], 8, 128, 256, [[0, 63], [0] + list(range(40, 64))]),
    ([9], [12], 1, 128, 32, [[0, 2, 4, 6, 9, 11]]),                # the first columns have no slots
]


@pytest.mark.parametrize("lens,cols,hk,d,page,paths", COMMITS)
@pytest.mark.parametrize("extra", ["none", "acc", "pos", "both"])
def test_commit(lens, cols, hk, d, page, paths, extra):
    t = torch()
    c = Case(lens, [min(n, x) for n, x in zip(lens, cols)], hk, d, page, t.bfloat16, seed=d + hk)
    starts = [0]
    for n in cols:
        starts.append(starts[-1] + n)
    batch = c.make(lens, starts, max(cols))
    width = min(bqe.TREE_COLS_MAX, max(len(p) for p in paths) + 2)
    path = [p + [-1] * (width - len(p)) for p in paths]
    counts = [len(p) for p in paths]
    slots = (len(lens), hk, c.per * page)
    g = t.Generator(device="cuda").manual_seed(1)
    acc = t.rand(slots, generator=g, device="cuda")
    pos = t.randint(0, 1 << 30, slots, generator=g, device="cuda", dtype=t.int32)
    given = dict(acc=acc if extra in ("acc", "both") else None, pos=pos if extra in ("pos", "both") else None)
    want, arrays = commit64(c, c.cache.pool.cpu().numpy(), c.table.tolist(), lens, starts, path, counts,
                            [x.cpu().numpy() for x in given.values() if x is not None])
    bqe.rfpx_kv_commit(c.cache, batch, ints(path), ints(counts), **given)
    assert np.array_equal(c.cache.pool.cpu().numpy(), want)
    for x, y in zip([x for x in given.values() if x is not None], arrays):
        assert np.array_equal(x.cpu().numpy(), y)


def test_commit_passes_over_what_is_no_column():
    """Entries below their index or past the step, counts past the path or the
    step or negative, pages outside the pool."""
    t = torch()
    lens, cols = [100, 60, 64, 50, 70], [20, 10, 40, 20, 8]
    c = Case(lens, cols, 2, 128, 32, t.bfloat16, seed=2)
    c.table[2, 0], c.table[2, 1] = -1, c.cache.n_pages
    path = [[0, 0, 1, 25, -9, 19], [2, 3, 9, 10, 1 << 30, -1], [1, 9, 30, 31, 38, 39], [5, 6, 7, 8, 9, 10],
            [1, 2, 3, 4, 5, 6]]
    counts = [6, 1 << 30, 6, -4, 2]
    slots = (5, 2, c.per * 32)
    acc = t.rand(slots, device="cuda")
    want, (wacc,) = commit64(c, c.cache.pool.cpu().numpy(), c.table.tolist(), lens, c.starts, path,
                             [max(0, n) for n in counts], [acc.cpu().numpy()])
    bqe.rfpx_kv_commit(c.cache, c.batch, ints(path), ints(counts), acc=acc)
    assert np.array_equal(c.cache.pool.cpu().numpy(), want) and np.array_equal(acc.cpu().numpy(), wacc)


# ---------------------------------------------------------- run together

class Model:
    """One attention layer over a vocabulary: embedded tokens become q, k and v,
    its output the logits, all through the library."""

    def __init__(self, lens, page, vocab=64, heads=4, hk=2, d=64, capacity=256, seed=0):
        t = torch()
        g = t.Generator(device="cuda").manual_seed(seed)
        self.heads, self.hk, self.d, self.vocab = heads, hk, d, vocab
        n, per = len(lens), -(-capacity // page)
        self.cache = bqe.KvCache(hk, d, page, n * per + 2)
        self.cache.pool.fill_(255)
        self.table = t.randperm(n * per + 2, generator=t.Generator().manual_seed(seed))[:n * per].reshape(n, per).int().cuda()
        self.embed = t.randn((vocab, (heads + 2 * hk) * d), generator=g, device="cuda")
        self.head = bqe.DenseMatrix(bqe.RFPX_FP4, vocab, heads * d, bqe.rfpx_pack(
            bqe.RFPX_FP4, t.randn((vocab, heads * d), generator=g, device="cuda") * 0.3))
        self.rope = bqe.Rope(d)
        self.slots = (n, hk, per * page)
        self.pos, self.acc = t.zeros(self.slots, dtype=t.int32, device="cuda"), t.zeros(self.slots, device="cuda")

    def batch(self, lens, starts, cols):
        return bqe.KvBatch(self.table, lens, starts, cols, self.slots[2])

    def rows(self, tokens, positions):
        """Queries, keys and values of tokens at positions."""
        h, hk, d = self.heads, self.hk, self.d
        x = self.embed[tokens.long()]
        q, k = bqe.rfpx_qk_norm_rope(x[:, :h * d].view(-1, h, d), x[:, h * d:(h + hk) * d].view(-1, hk, d), positions,
                                     rope=self.rope)
        return q, k, x[:, (h + hk) * d:].reshape(-1, hk, d)

    def logits(self, out):
        t = torch()
        x = out.reshape(out.shape[0], -1)
        return t.cat([bqe.rfpx_dense_forward(self.head, x[i:i + 8].contiguous()) for i in range(0, x.shape[0], 8)])

    def plain(self, tokens, positions, batch):
        """A step of chains."""
        q, k, v = self.rows(tokens, positions)
        bqe.rfpx_kv_append(self.cache, batch, k, v, positions, self.pos, self.acc)
        return self.logits(bqe.rfpx_attn_forward(self.cache, batch, q))

    def verify(self, tokens, parents, batch, u, **settings):
        """A step of trees: path, counts, next tokens, lengths, and the tokens drawn."""
        masks, positions = bqe.rfpx_tree_masks(batch, parents)
        q, k, v = self.rows(tokens, positions)
        bqe.rfpx_kv_append(self.cache, batch, k, v, positions, self.pos, self.acc)
        logits = self.logits(bqe.rfpx_attn_tree_forward(self.cache, batch, q, masks))
        drawn = bqe.rfpx_sample(logits, u, **settings)
        path, counts, following, lens = bqe.rfpx_tree_accept(batch, parents, tokens, drawn)
        bqe.rfpx_kv_commit(self.cache, batch, path, counts, acc=self.acc, pos=self.pos)
        return path, counts, following, lens, drawn


def start(m, prompts):
    """Prompts into the cache; the token that each continues with."""
    t = torch()
    n = [len(p) for p in prompts]
    starts = [sum(n[:i]) for i in range(len(n) + 1)]
    lens = ints(n)
    tokens = ints([x for p in prompts for x in p])
    logits = m.plain(tokens, ints([i for k in n for i in range(k)]), m.batch(lens, ints(starts), max(n)))
    last = logits[[s - 1 for s in starts[1:]]]
    return lens, bqe.rfpx_sample(last, t.zeros(len(n), device="cuda"), temperature=t.zeros(len(n), device="cuda"))


def test_steps_write_what_plain_decoding_writes():
    """Greedy decoding by trees of drafts, right and wrong ones mixed, against
    one token at a time: the same tokens, and in the end the same cache."""
    t = torch()
    prompts = [[1, 2, 3, 4, 5], [7], [11, 13, 17, 19, 23, 29, 31]]
    steps = 30
    a, b = Model([0] * 3, 32), Model([0] * 3, 32)
    lens, token = start(a, prompts)
    alone = ints([0, 1, 2, 3])
    zero = t.zeros(3, device="cuda")
    want = [[int(x)] for x in token]
    for i in range(steps):
        lens = lens + 1
        token = bqe.rfpx_sample(a.plain(token, lens - 1, a.batch(lens, alone, 1)), zero, temperature=zero)
        for s in range(3):
            want[s].append(int(token[s]))
    lens, token = start(b, prompts)
    got = [[int(x)] for x in token]
    rng = random.Random(3)
    while min(len(x) for x in got) < steps:
        parents, tokens, starts = [], [], [0]
        for s in range(3):
            n = rng.randrange(1, 9)
            mine = tree(n, "tree", rng)
            toks = [got[s][-1]]
            for i in range(1, n):
                ahead = len(got[s]) + len(line_of(mine, i)) - 2
                right = ahead < len(want[s]) and rng.random() < 0.7
                toks.append(want[s][ahead] if right else rng.randrange(b.vocab))
            parents += mine
            tokens += toks
            starts.append(starts[-1] + n)
        n = [y - x for x, y in zip(starts, starts[1:])]
        rows = starts[-1]
        batch = b.batch(lens + ints(n), ints(starts), max(n))
        path, counts, following, lens, _ = b.verify(ints(tokens), ints(parents), batch, t.zeros(rows, device="cuda"),
                                                    temperature=t.zeros(rows, device="cuda"))
        for s in range(3):
            took = [tokens[starts[s] + j] for j in path[s].tolist() if j >= 0]
            got[s] += took[1:] + [int(following[s])]
            # settled tokens are all but the one to come
            assert int(lens[s]) == len(prompts[s]) + len(got[s]) - 1
    for s in range(3):
        m = min(len(got[s]), len(want[s]))
        assert got[s][:m] == want[s][:m]
    for s in range(3):
        m = min(int(lens[s]), len(prompts[s]) + steps)
        one = [t.zeros(1, dtype=t.int32, device="cuda") + m, ints([0, m])]
        views = [bqe.KvBatch(x.table[s:s + 1].contiguous(), *one, m, m) for x in (a, b)]
        for x, y in zip(bqe.rfpx_kv_unpack(a.cache, views[0], m), bqe.rfpx_kv_unpack(b.cache, views[1], m)):
            assert t.equal(x, y)
        assert t.equal(a.pos[s, :, :m], b.pos[s, :, :m])


def test_captured_step():
    """One verify step in a graph, replayed on other trees, drafts, numbers and
    lengths, against the same calls made one by one; eager work in between."""
    t = torch()
    made, cols = [], 12
    for _ in range(2):
        m = Model([0, 0], 32, seed=5)
        m.io = dict(tokens=ints([0] * 24), parents=ints([-1] * 24), starts=ints([0, 12, 24]), lens=ints([20, 30]),
                    u=t.zeros(24, device="cuda"))
        m.b = m.batch(m.io["lens"], m.io["starts"], cols)
        made.append(m)
    temp, p = t.full((24,), 0.8, device="cuda"), t.full((24,), 0.9, device="cuda")

    def step(m):
        r = m.verify(m.io["tokens"], m.io["parents"], m.b, m.io["u"], temperature=temp, top_p=p)
        m.io["lens"].copy_(r[3])
        return r

    A, B = made
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(A)
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        ra = step(A)
    for m in made:
        m.cache.pool.fill_(255)
        m.pos.zero_()
        m.acc.zero_()
        m.io["lens"].copy_(ints([0, 0]))
    rng = random.Random(9)
    for i in range(8):
        n = [rng.randrange(1, 13), rng.randrange(0, 13)]
        parents = tree(n[0], "tree", rng) + tree(n[1], "tree", rng)
        tokens = [rng.randrange(6) for _ in parents]
        fill = 24 - len(parents)
        g = t.Generator(device="cuda").manual_seed(i)
        u = t.rand(24, generator=g, device="cuda")
        for m in made:
            m.io["parents"].copy_(ints(parents + [-1] * fill))
            m.io["tokens"].copy_(ints(tokens + [0] * fill))
            m.io["starts"].copy_(ints([0, n[0], n[0] + n[1]]))
            m.io["lens"].add_(ints(n))
            m.io["u"].copy_(u)
        graph.replay()
        rb = step(B)
        t.cuda.synchronize()
        rows = n[0] + n[1]
        for x, y in zip(ra[:4], rb[:4]):
            assert t.equal(x, y)
        assert t.equal(ra[4][:rows], rb[4][:rows])
        for s in range(2):
            m = int(rb[3][s])
            assert t.equal(A.pos[s, :, :m], B.pos[s, :, :m])
        _ = (u.view(4, 6) @ u.view(6, 4)).sum().item()


def test_streams():
    """A step on a side stream while the current one is busy."""
    t = torch()
    m = Model([0], 32, seed=8)
    lens, token = start(m, [[1, 2, 3]])
    batch = m.batch(lens + 6, ints([0, 6]), 6)
    parents, tokens = ints(tree(6, "tree", random.Random(1))), ints([3, 1, 4, 1, 5, 9])
    u = t.full((6,), 0.4, device="cuda")
    pool = m.cache.pool.clone()
    want = m.verify(tokens, parents, batch, u)
    after = m.cache.pool.clone()
    m.cache.pool.copy_(pool)
    side = t.cuda.Stream()
    t.cuda.synchronize()
    busy = t.randn((4096, 4096), device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    with t.cuda.stream(side):
        got = m.verify(tokens, parents, batch, u)
    t.cuda.synchronize()
    for x, y in zip(want, got):
        assert t.equal(x, y)
    assert t.equal(m.cache.pool, after)
    masks, _ = bqe.rfpx_tree_masks(batch, parents, stream=side)
    side.synchronize()
    assert t.equal(masks, bqe.rfpx_tree_masks(batch, parents)[0])


def test_wrapper_refusals():
    t = torch()
    c = Case([20], [4], 2, 64, 32, t.bfloat16)
    parents = ints([-1, 0, 1, 1])
    masks, _ = bqe.rfpx_tree_masks(c.batch, parents)
    q = t.zeros((4, 4, 64), device="cuda", dtype=t.bfloat16)
    path, counts = ints([[0, 1, 2, 3]]), ints([4])
    slots = (1, 2, c.per * 32)
    for call in (lambda: bqe.rfpx_tree_masks(c.batch, parents.long()),
                 lambda: bqe.rfpx_tree_masks(c.batch, parents, base=ints([0, 0])),
                 lambda: bqe.rfpx_tree_masks(c.batch, parents, masks=masks[:2]),
                 lambda: bqe.rfpx_tree_masks(c.batch, parents.cpu()),
                 lambda: bqe.rfpx_attn_tree_forward(c.cache, c.batch, q, masks[:3]),
                 lambda: bqe.rfpx_attn_tree_forward(c.cache, c.batch, q, masks.float()),
                 lambda: bqe.rfpx_attn_tree_forward(c.cache, c.batch, q, masks[:, 0]),
                 lambda: bqe.rfpx_attn_tree_forward(c.cache, c.batch, q[:, :, :32], masks),
                 lambda: bqe.rfpx_attn_tree_forward(c.cache, c.batch, q, masks, out=q.float()),
                 lambda: bqe.rfpx_tree_accept(c.batch, parents, parents, parents[:3]),
                 lambda: bqe.rfpx_tree_accept(c.batch, parents, parents, parents, counts=ints([0, 0])),
                 lambda: bqe.rfpx_kv_commit(c.cache, c.batch, path.long(), counts),
                 lambda: bqe.rfpx_kv_commit(c.cache, c.batch, path, ints([1, 1])),
                 lambda: bqe.rfpx_kv_commit(c.cache, c.batch, path, counts, acc=t.zeros(slots, dtype=t.int32, device="cuda")),
                 lambda: bqe.rfpx_kv_commit(c.cache, c.batch, path, counts, pos=t.zeros((1, 2, 5), dtype=t.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bqe.RfpxError):
        bqe.rfpx_tree_masks(c.batch, parents, mask_words=33)
    with pytest.raises(bqe.RfpxError):
        bqe.rfpx_tree_masks(batch_of([9000], [0, 2000]), parents)


def test_lengths_are_taken_as_they_stand():
    """Masks and acceptance know no cache: lengths past any pages, and below 0."""
    b = batch_of([1 << 30, -5, 3], [0, 2, 4, 8], max_len=64)
    parents = ints([-1, 0, -1, 0, -1, 0, 1, 2])
    _, pos = bqe.rfpx_tree_masks(b, parents)
    assert pos.tolist() == [(1 << 30) - 2, (1 << 30) - 1, -7, -6, -1, 0, 1, 2]
    tokens, drawn = ints([9, 1, 9, 1, 9, 1, 2, 3]), ints([1, 7, 0, 7, 1, 2, 0, 0])
    path, counts, following, after = bqe.rfpx_tree_accept(b, parents, tokens, drawn)
    assert path.tolist() == [[0, 1, -1, -1], [0, -1, -1, -1], [0, 1, 2, -1]] and counts.tolist() == [2, 1, 3]
    assert following.tolist() == [7, 0, 0] and after.tolist() == [1 << 30, 0, 2]
