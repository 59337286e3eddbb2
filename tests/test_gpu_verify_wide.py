"""Attention of trees of hundreds of columns (include/rfpx_verify.h), masks of
up to 32 words: where they lie in LDS behind the decoded tiles, or in place of
the sums.  Values in 64 bits and tolerances as in test_gpu_verify.py."""
import random

import pytest

import block_quantized_expert_amd as bqe
from test_gpu_attn import Case, check_lse, check_out, dt, torch
from test_gpu_verify import attend64, forward, ints, seen_by_tree, tree, words_of

pytestmark = pytest.mark.gpu


def some(case, ref, out, z, dtype, heads, rows):
    """The checks of some heads and rows."""
    ref = {x: ref[x][:, heads] for x in ref}
    check_out(out[:, heads], ref, dt(dtype), rows)
    check_lse(z[:, heads], ref, rows)


WIDE = [  # lens, cols, kv heads, group, head_dim, page, plan
    ([300 + 37], [300], 2, 2, 128, 64, 0),
    ([1024 + 301], [1024], 2, 2, 128, 64, 65536),           # bf16: the kernel of many rows, 32 words
    ([1024 + 45, 333], [1024, 300], 2, 2, 64, 32, 65536),   # ... and fp32: blocks of 32 rows
    ([1000], [1000], 1, 2, 128, 128, 65536),                # no context
    ([1024 + 7], [1024], 1, 1, 64, 64, 0),
    ([300 + 90], [300], 1, 2, 256, 64, 0),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("lens,cols,hk,group,d,page,plan", WIDE)
def test_wide_trees(lens, cols, hk, group, d, page, plan, dtype):
    rng = random.Random(sum(lens) + d)
    c = Case(lens, cols, hk, d, page, dt(dtype), seed=sum(cols), capacity=plan or None)
    parents = [p for n in cols for p in [-1] + [rng.randrange(max(0, i - 60), i) for i in range(1, n)]]
    masks, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    assert masks.shape[1] == -(-max(cols) // 32)
    heads = [hk * group - 1]
    q, out, z, scale = forward(c, hk * group, dt(dtype), masks, plan)
    some(c, attend64(c, q, scale, seen_by_tree(c, parents), heads), out, z, dtype, heads, slice(0, c.rows))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("words,plan", [(32, 65536), (32, 0), (9, 65536), (9, 0)])
def test_more_columns_than_bits(words, plan, dtype):
    """Columns without a bit are not seen, by themselves neither; they see
    what their own bits name."""
    n, context, hk, group, d = 1100, 50, 2, 2, 128
    rng = random.Random(words)
    c = Case([context + n], [n], hk, d, 64, dt(dtype), seed=words, capacity=plan or None)
    named = [sorted(j for j in {rng.randrange(32 * words) for _ in range(rng.randrange(40))}) for _ in range(n)]
    named[0], named[n - 1] = [], [32 * words - 1]
    masks = ints([words_of(x, words) for x in named])
    q, out, z, scale = forward(c, hk * group, dt(dtype), masks, plan)
    heads = [1]
    ref = attend64(c, q, scale, lambda b, i: [*range(context), *[context + j for j in named[i]]], heads)
    some(c, ref, out, z, dtype, heads, slice(0, n))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("plan", [0, 65536])
def test_longer_masks_than_columns(plan, dtype):
    """Words without columns, whatever stands in them: the same bits as masks
    of as many words as there are columns for."""
    t = torch()
    sizes, context, hk = [40, 33], 77, 2
    rng = random.Random(5)
    c = Case([context + n for n in sizes], sizes, hk, 128, 32, dt(dtype), seed=3, capacity=plan or None)
    parents = [p for n in sizes for p in tree(n, "tree", rng)]
    short, _ = bqe.rfpx_tree_masks(c.batch, ints(parents))
    long = t.randint(-(1 << 31), 1 << 31, (sum(sizes), 32), device="cuda",
                     generator=t.Generator("cuda").manual_seed(1)).int()
    long[:, :2] = short
    long[:40, 1] |= -1 << 8  # columns 40 and on of the first tree, 33 and on of the second: there are none
    long[40:, 1] |= -1 << 1
    want = forward(c, 8 * hk, dt(dtype), short, plan)
    got = forward(c, 8 * hk, dt(dtype), long, plan)
    assert t.equal(got[1], want[1]) and t.equal(got[2], want[2])
