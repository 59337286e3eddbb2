"""Attention over the FP4 cache (include/rfpx_attn.h) against plain
implementations in 64 bits, on the values that the cache holds.

Tolerances.  u(t) is half a step of type t relative to a value: 2^-24 fp32,
2^-8 bf16.
 - Norm and rotation: the sum of squares is a chain of 8 and a tree of at most
   5 additions (14 u32 relative), halved by the root, 3 u32 for the mean, eps
   and root, 1 for the division, 2 products, cos and sin within 4 u32 (angle to
   2^-24 and the function's own step), and two products with one sum: below
   24 u32 of |a| + |b|, the pair's magnitudes before the turn; the output's own
   type adds u(t) of the value.
 - Scores: a code enters as 16 + code and the offset comes off by another
   product, so the terms are at most 31 units (2^(e-127)) each; the products
   are exact and at most 3 * 256 + 24 of them are added, in chains of fp32
   roundings no longer than 32 instructions of 8 steps each.  With
   B = scale * sum |q| * 31 unit, |ds| <= 256 u32 B, taken with the exp's own
   steps (2^-22) and the log2 scaling of the exponent (|s| 2^-22).
 - Output: numerators err by 1 + |ds|; in bf16 by u(bf16) besides, of which
   the denominator, their rounded sum, takes a part off: at most 2 (|ds| + u)
   of A = sum p |v|; the offset's removal adds 256 u32 sum p 31 unit; the
   output's own type u(t) of the value.
"""
import numpy as np
import pytest

import block_quantized_expert_amd as bqe
import oracle
import synth

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


def torch():
    import torch as t
    return t


def u_of(dtype):
    return UBF if dtype == torch().bfloat16 else U32


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """A cache filled through rfpx_kv_append, and its values in 64 bits."""

    def __init__(self, lens, cols, hk, d, page, dtype, seed=0, extra_pages=3, gap=0, capacity=None, scale=1.0):
        t = torch()
        g = t.Generator(device="cuda").manual_seed(seed)
        self.lens, self.cols, self.hk, self.d, self.page = list(lens), list(cols), hk, d, page
        n = len(lens)
        per = max(1, -(-max(list(lens) + [1]) // page))
        if capacity:
            per = max(per, -(-capacity // page))
        total = n * per + extra_pages
        perm = t.randperm(total, generator=t.Generator().manual_seed(seed))
        self.table = perm[:n * per].reshape(n, per).int().cuda()
        self.cache = bqe.KvCache(hk, d, page, total)
        # whatever was there before, NaN scales among it, must not show
        self.cache.pool.fill_(255)
        self.per = per
        self.starts = [gap]
        for c in cols:
            self.starts.append(self.starts[-1] + c)
        self.batch = self.make(self.lens, self.starts, max(max(cols), 1))
        # fill: every sequence whole, then the steps' columns are its last slots
        fill = [0]
        for x in lens:
            fill.append(fill[-1] + x)
        self.fill = self.make(self.lens, fill, max(max(lens), 1))
        rows = fill[-1]
        self.k_in = (t.randn((rows, hk, d), generator=g, device="cuda") * scale).to(dtype)
        self.v_in = (t.randn((rows, hk, d), generator=g, device="cuda") * scale).to(dtype)
        bqe.rfpx_kv_append(self.cache, self.fill, self.k_in, self.v_in)
        self.rows, self.fill_starts = self.starts[-1], fill

    def make(self, lens, starts, cols, plan=0):
        """plan: the length that launches are planned for, if larger."""
        t = torch()
        return bqe.KvBatch(self.table, t.tensor(lens, dtype=t.int32, device="cuda"),
                           t.tensor(starts, dtype=t.int32, device="cuda"), cols, max(list(lens) + [1, plan]))

    def planned(self, plan):
        return self.make(self.lens, self.starts, max(self.cols), plan)

    def values(self):
        """Per sequence: k, v [slots][hk][d] and the units of their blocks."""
        k, v = bqe.rfpx_kv_unpack(self.cache, self.fill, self.fill_starts[-1])
        k, v = f64(k), f64(v)
        return [(k[a:b], v[a:b]) for a, b in zip(self.fill_starts, self.fill_starts[1:])]


def units(x):
    """2^(e-127) of every value's block, from the largest value of a block (at
    least half a unit under 7.5 of them, so at most twice the unit is found)."""
    a = np.abs(x.reshape(*x.shape[:-1], -1, 32)).max(-1)
    with np.errstate(divide="ignore"):
        u = 2.0 ** np.ceil(np.log2(np.maximum(a, 1e-300) / 7.5))
    return np.repeat(np.where(a == 0, 0, u), 32, -1)


def attend64(case, q, scale, seen=None):
    """out, lse, weights, and the bounds of their errors, in 64 bits.
    seen(b, slot): False where the cache does not hold the slot."""
    q = f64(q)
    heads = q.shape[1]
    g = heads // case.hk
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    mag, tol_s, tol_o = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape)
    wts = [np.zeros((case.hk, n)) for n in case.lens]
    wtol = [np.zeros((case.hk, n)) for n in case.lens]
    for b, (k, v) in enumerate(case.values()):
        n = case.cols[b]
        held = np.array([seen is None or seen(b, j) for j in range(case.lens[b])], bool)
        for i in range(n):
            m = case.lens[b] - n + i + 1
            if m <= 0:
                continue
            ok = held[:m]
            if not ok.any():
                continue
            row = case.starts[b] + i
            for h in range(heads):
                kk, vv = k[:m, h // g][ok], v[:m, h // g][ok]
                s = scale * (kk @ q[row, h])
                z = s.max() + np.log(np.exp(s - s.max()).sum())
                p = np.exp(s - z)
                out[row, h], lse[row, h] = p @ vv, z
                mag[row, h] = p @ np.abs(vv)
                big = scale * (31 * units(kk) @ np.abs(q[row, h])).max()
                ds = 256 * U32 * big + 2.0 ** -22 * (1 + np.abs(s).max())
                tol_s[row, h] = ds
                tol_o[row, h] = 2 * ds * mag[row, h] + 256 * U32 * 31 * (p @ units(vv))
                idx = np.nonzero(ok)[0]
                wts[b][h // g][idx] += p
                wtol[b][h // g][idx] += 2 * ds * p + 2.0 ** -22 * p
    return dict(out=out, lse=lse, mag=mag, ds=tol_s, do=tol_o, w=wts, dw=wtol)


def check_out(got, ref, dtype, rows):
    o = f64(got)[rows]
    u = u_of(dtype)
    tol = ref["do"][rows] + (2 * UBF * ref["mag"][rows] if dtype == torch().bfloat16 else 0) \
        + u * (1 + 2.0 ** -6) * np.abs(ref["out"][rows]) + 1e-30
    err = np.abs(o - ref["out"][rows])
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the bound"


def check_lse(got, ref, rows):
    z, r = f64(got)[rows], ref["lse"][rows]
    empty = np.isneginf(r)
    assert (np.isneginf(z) == empty).all()
    tol = 2 * ref["ds"][rows] + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, r)))
    d = np.abs(np.where(empty, 0, z) - np.where(empty, 0, r))
    assert (d <= tol).all(), np.max(d / tol)


def attend(case, heads, dtype, seed=1, scale=None, gap_rows=0, batch=None, lse=True):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    rows = case.rows + gap_rows
    q = (t.randn((rows, heads, case.d), generator=g, device="cuda") * 1.3).to(dtype)
    out = t.full_like(q, 7.0)
    z = t.full((rows, heads), 7.0, device="cuda") if lse else None
    scale = case.d ** -0.5 if scale is None else scale
    bqe.rfpx_attn_forward(case.cache, batch or case.batch, q, scale, out=out, lse=z)
    return q, out, z, scale


DTYPES = ["bfloat16", "float32"]


def dt(name):
    return getattr(torch(), name)


# -------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hk,d,page", [(1, 64, 32), (3, 128, 64), (2, 256, 128), (8, 128, 256)])
def test_append_is_rfpx_pack_and_its_layout(hk, d, page, dtype):
    t = torch()
    lens = [1, 37, page, 2 * page + 5]
    c = Case(lens, lens, hk, d, page, dt(dtype), seed=d + hk)
    k, v = bqe.rfpx_kv_unpack(c.cache, c.fill, sum(lens))
    nb = d // 32
    for x, got in ((c.k_in, k), (c.v_in, v)):
        flat = x.float().reshape(-1, d).contiguous()
        blocks = bqe.rfpx_pack(bqe.RFPX_FP4, flat)
        want = bqe.rfpx_unpack(bqe.RFPX_FP4, blocks, flat.shape[0], d).view(x.shape)
        assert t.equal(got, want)
    # the bytes of a few tokens at the places that the layout gives them
    slabs = c.cache.pool.view(-1, hk, page * d * 17 // 16).cpu().numpy()
    half = page * d // 2
    for b, n in enumerate(lens):
        for slot in {0, n // 2, n - 1}:
            for h in range(hk):
                slab = slabs[int(c.table[b, slot // page]), h]
                tok, row = slot % page, c.fill_starts[b] + slot
                for x, first in ((c.k_in, 0), (c.v_in, half + page * nb)):
                    blk = bqe.rfpx_pack(bqe.RFPX_FP4, x[row, h].float().view(1, d)).cpu().numpy().reshape(nb, 17)
                    for i in range(nb):
                        assert slab[first + half + tok * nb + i] == blk[i, 16]
                        for r in range(16):
                            at = tok * d // 2 + (r // 4 * nb + i) * 4 + r % 4 if first == 0 else \
                                first + (tok // 4 * 16 + r) * 4 * nb + (tok % 4 // 2 * (nb // 2) + i // 2) * 4 \
                                + tok % 2 * 2 + i % 2
                            assert slab[at] == blk[i, r]


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_unpack_types_agree(kind):
    t = torch()
    c = Case([50], [50], 2, 128, 32, t.float32)
    k, v = bqe.rfpx_kv_unpack(c.cache, c.fill, 50)
    k2, v2 = (t.empty((50, 2, 128), dtype=dt(kind), device="cuda") for _ in range(2))
    bqe.rfpx_kv_unpack(c.cache, c.fill, 50, k2, v2)
    assert t.equal(k2.float(), k) and t.equal(v2.float(), v)


def test_append_edges():
    t = torch()
    hk, d, page = 2, 64, 32
    c = Case([70, 3], [4, 3], hk, d, page, t.float32, gap=2, capacity=96)
    before = c.cache.pool.clone()
    rows = c.rows + 5
    k = t.randn((rows, hk, d), device="cuda")
    v = t.randn((rows, hk, d), device="cuda")
    k[2, 0, :32] = 0
    k[2, 0, 33] = float("nan")
    v[3, 1, 5] = float("inf")
    v[4, 1, 40:64] = 0
    v[4, 1, 32:40] = 1e-42  # under the smallest normal number
    k[5, 0, 0] = 3.4e38
    # 7.5 and its multiples are where the exponent steps; 0.5 steps are ties
    k[6, 0, :32] = t.arange(32, device="cuda") * 0.25
    k[6, 0, 31] = 7.5
    pos = t.full((2, hk, 96), -5, dtype=t.int32, device="cuda")
    acc = t.full((2, hk, 96), 9.0, device="cuda")
    where = t.arange(100, 100 + rows, dtype=t.int32, device="cuda")
    bqe.rfpx_kv_append(c.cache, c.batch, k, v, where, pos, acc)
    k2, v2 = t.full_like(k, 5.0), t.full_like(v, 5.0)
    bqe.rfpx_kv_unpack(c.cache, c.batch, rows, k2, v2)
    # rows before the first sequence and behind the last
    for r in list(range(2)) + list(range(c.rows, rows)):
        assert bool((k2[r] == 5).all() and (v2[r] == 5).all())
    assert bool(k2[2, 0, 32:].isnan().all()) and bool((k2[2, 0, :32].abs() < 1e-37).all())
    assert bool(v2[3, 1, :32].isnan().all()) and not bool(v2[3, 1, 32:].isnan().any())
    for x, y, r in ((k, k2, 4), (v, v2, 4), (k, k2, 5), (k, k2, 6), (v, v2, 8)):
        want = bqe.rfpx_unpack(4, bqe.rfpx_pack(4, x[r].contiguous()), hk, d)
        assert t.equal(y[r], want), r
    # positions and weights at the new slots only
    for b, (n, ln) in enumerate(((4, 70), (3, 3))):
        new = t.arange(96, device="cuda")
        new = (new >= ln - n) & (new < ln)
        first = c.starts[b]
        for h in range(hk):
            assert pos[b, h][new].tolist() == list(range(100 + first, 100 + first + n))
            assert bool((pos[b, h][~new] == -5).all() and (acc[b, h][new] == 0).all() and (acc[b, h][~new] == 9).all())
    # only the new tokens' bytes changed
    slabs = c.cache.pool.view(-1, hk, page * d * 17 // 16)
    old = before.view_as(slabs)
    used = {int(c.table[0, 2]), int(c.table[1, 0])}
    for p in range(slabs.shape[0]):
        assert t.equal(slabs[p], old[p]) == (p not in used)


def test_append_drops_what_has_no_place():
    """Columns of negative slot, bad pages, lengths past the table's end."""
    t = torch()
    hk, d, page = 2, 128, 32
    c = Case([40, 2], [40, 2], hk, d, page, t.float32)
    c.table[0, 1] = c.cache.n_pages  # behind the pool
    before = c.cache.pool.clone()
    b = c.make([40, 2], [0, 40, 45], 40)  # five columns, two slots
    k, v = t.randn((45, hk, d), device="cuda"), t.randn((45, hk, d), device="cuda")
    bqe.rfpx_kv_append(c.cache, b, k, v)
    k2, v2 = t.full_like(k, 5.0), t.full_like(v, 5.0)
    bqe.rfpx_kv_unpack(c.cache, b, 45, k2, v2)
    assert bool((k2[32:43] == 5).all()) and not bool((k2[:32] == 5).any()) and not bool((k2[43:] == 5).any())
    want = bqe.rfpx_unpack(4, bqe.rfpx_pack(4, k[43:].reshape(-1, d)), 2 * hk, d).view(2, hk, d)
    assert t.equal(k2[43:], want)
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        c.table[0, :] = bad
        c.table[1, :] = bad
        kept = c.cache.pool.clone()
        bqe.rfpx_kv_append(c.cache, b, k, v)
        assert t.equal(c.cache.pool, kept)
    assert before.shape == c.cache.pool.shape
    # lens past the table's end count as its end
    c = Case([64], [64], hk, d, page, t.float32)
    b = c.make([1000], [0, 3], 3)
    bqe.rfpx_kv_append(c.cache, b, k[:3], v[:3])
    k3, _ = bqe.rfpx_kv_unpack(c.cache, c.fill, 64)
    assert t.equal(k3[61:], bqe.rfpx_unpack(4, bqe.rfpx_pack(4, k[:3].reshape(-1, d)), 3 * hk, d).view(3, hk, d))


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 200, 5000])
def test_many_sequences(n):
    """The search of a row's sequence over one, two and three levels, empty
    sequences among them."""
    t = torch()
    r = np.random.default_rng(n)
    cols = r.integers(0, 3, n)
    cols[-1] = 1
    starts = [0] + list(np.cumsum(cols))
    table = t.arange(n, dtype=t.int32, device="cuda").view(n, 1)
    cache = bqe.KvCache(1, 64, 32, n)
    cache.pool.zero_()
    b = bqe.KvBatch(table, t.full((n,), 9, dtype=t.int32, device="cuda"),
                    t.tensor(starts, dtype=t.int32, device="cuda"), 2, 9)
    rows = starts[-1]
    k = t.randn((rows, 1, 64), device="cuda")
    v = t.randn((rows, 1, 64), device="cuda")
    bqe.rfpx_kv_append(cache, b, k, v)
    k2, v2 = bqe.rfpx_kv_unpack(cache, b, rows)
    assert t.equal(k2.view(-1, 64), bqe.rfpx_unpack(4, bqe.rfpx_pack(4, k.view(-1, 64)), rows, 64))
    assert t.equal(v2.view(-1, 64), bqe.rfpx_unpack(4, bqe.rfpx_pack(4, v.view(-1, 64)), rows, 64))


# ------------------------------------------------------------ norm and rope

def norm_rope64(x, w, pos, rope, eps):
    x = f64(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w)
    y, mag = x.copy(), np.abs(x)
    if rope is not None and rope.dim:
        h = rope.dim // 2
        inv = np.array([rope._freq[i] for i in range(h)])
        ang = f64(pos)[:, None, None] * inv
        i = np.arange(h)
        a, b = (i, i + h) if rope.style == 0 else (2 * i, 2 * i + 1)
        y[..., a] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang)
        y[..., b] = x[..., a] * np.sin(ang) + x[..., b] * np.cos(ang)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def check_rows(got, ref, mag, dtype):
    tol = 24 * U32 * mag + u_of(dtype) * (1 + 2.0 ** -6) * np.abs(ref) + 1e-37
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the bound"


@pytest.mark.parametrize("x_dtype,o_dtype", [("float32", "bfloat16"), ("bfloat16", "bfloat16"), ("float32", "float32"),
                                             ("bfloat16", "float32")])
@pytest.mark.parametrize("n,h,hk,d,rot,style", [
    (1, 1, 1, 64, 64, 0), (5, 32, 8, 128, 128, 0), (3, 7, 1, 256, 256, 1), (9, 4, 2, 128, 64, 0),
    (4, 5, 5, 128, 50, 0), (6, 2, 1, 64, 2, 1), (130, 6, 3, 64, 30, 1), (2, 40, 3, 256, 192, 0), (7, 3, 3, 128, 0, 0)])
def test_norm_rope(n, h, hk, d, rot, style, x_dtype, o_dtype):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(n + d)
    # slices of one projection's rows
    qkv = (t.randn((n, (h + 2 * hk) * d + 64), generator=g, device="cuda") * 2).to(dt(x_dtype))
    q, k = qkv[:, :h * d].view(n, h, d), qkv[:, h * d:(h + hk) * d].view(n, hk, d)
    qw, kw = (1 + 0.3 * t.randn(d, generator=g, device="cuda") for _ in range(2))
    pos = t.randint(0, 1 << 20, (n,), generator=g, device="cuda").int()
    pos[0] = 2 ** 31 - 1
    rope = bqe.Rope(rot, theta=10000.0, style=style)
    qo, ko = bqe.rfpx_qk_norm_rope(q, k, pos, qw, kw, 1e-6, rope, out_dtype=dt(o_dtype))
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        ref, mag = norm_rope64(x, w, pos, rope, 1e-6)
        check_rows(got, ref, mag, dt(o_dtype))


def test_norm_rope_forms():
    t = torch()
    n, h, hk, d = 6, 4, 2, 128
    x = t.randn((n, h + hk, d), device="cuda")
    w = t.rand(d, device="cuda") + 0.5
    pos = t.tensor([0, 5, -1, 7, -9, 100000], dtype=t.int32, device="cuda")
    rope = bqe.Rope(d)
    live = np.array([0, 1, 3, 5])
    # in place, padding rows left as they were, no norm for k
    y = x.clone()
    q, k = y[:, :h], y[:, h:]
    a, b = bqe.rfpx_qk_norm_rope(q, k, pos, w, None, 1e-5, rope, q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and b.data_ptr() == k.data_ptr()
    for got, src, wt in ((q, x[:, :h], w), (k, x[:, h:], None)):
        ref, mag = norm_rope64(src, wt, pos, rope, 1e-5)
        check_rows(got[live], ref[live], mag[live], t.float32)
        assert t.equal(got[[2, 4]], src[[2, 4]])
    # one of the two alone; no rope; frequencies of the caller's own
    own = bqe.Rope(8, inv_freq=[0.0, 1.0, -2.5, 1e-9])
    only, none = bqe.rfpx_qk_norm_rope(x, None, pos.abs(), w, None, 0.0, own)
    assert none is None
    ref, mag = norm_rope64(x, w, pos.abs(), own, 0.0)
    check_rows(only, ref, mag, t.float32)
    _, only = bqe.rfpx_qk_norm_rope(None, x, pos.abs(), None, w)
    ref, mag = norm_rope64(x, w, pos.abs(), None, 1e-6)
    check_rows(only, ref, mag, t.float32)
    # nothing to normalize: a head of zeros stays zeros
    z, _ = bqe.rfpx_qk_norm_rope(t.zeros_like(x), None, pos.abs(), w, None, 1e-6, rope)
    assert bool((z == 0).all())
    # no rows at all
    e, _ = bqe.rfpx_qk_norm_rope(x[:0], None, pos[:0], w, None, 1e-6, rope)
    assert e.shape[0] == 0


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,cols,hk,group,d,page", [
    ([1], [1], 1, 1, 64, 32),
    ([2, 31, 32, 33], [1, 1, 1, 1], 2, 4, 128, 32),
    ([1021], [1], 2, 4, 128, 64),
    ([700, 5, 129], [8, 5, 3], 1, 8, 128, 64),
    ([257, 64], [4, 1], 3, 3, 64, 128),
    ([300, 513], [2, 7], 2, 2, 256, 256),
    ([90], [5], 1, 16, 256, 32),
    ([4099], [3], 1, 7, 128, 256),
    ([200, 40], [130, 40], 2, 4, 128, 64),
    ([333], [100], 1, 3, 64, 32),
    ([150], [150], 1, 2, 256, 64),
    ([500, 70, 64], [17, 70, 33], 2, 4, 128, 32),
    ([1500], [66], 1, 5, 64, 256),
    ([40, 1200], [9, 9], 2, 16, 128, 64),
])
def test_attention(lens, cols, hk, group, d, page, dtype):
    t = torch()
    c = Case(lens, cols, hk, d, page, dt(dtype), seed=len(lens) + d)
    q, out, z, scale = attend(c, hk * group, dt(dtype))
    ref = attend64(c, q, scale)
    rows = slice(0, c.rows)
    check_out(out, ref, dt(dtype), rows)
    check_lse(z, ref, rows)
    # the same bits again, and without lse
    q2, out2, _, _ = attend(c, hk * group, dt(dtype), lse=False)
    assert t.equal(q, q2) and t.equal(out, out2)


# rows of a sequence and planned lengths that take the path of many rows, with
# and without splits; most splits of the short sequences have nothing to do
@pytest.mark.parametrize("lens,cols,hk,group,d,page,plan", [
    ([500, 70, 64], [17, 70, 33], 2, 4, 128, 32, 16384),
    ([1500, 3, 0, 700], [66, 5, 9, 14], 2, 5, 64, 256, 16384),
    ([40, 1200], [9, 9], 2, 16, 128, 64, 65536),
    ([100, 64, 1, 65], [35, 20, 1, 35], 32, 2, 128, 64, 1024),
    ([130, 64, 257, 65], [70, 64, 3, 35], 32, 1, 64, 32, 1024),
])
def test_attention_many_rows(lens, cols, hk, group, d, page, plan):
    t = torch()
    c = Case(lens, cols, hk, d, page, t.bfloat16, seed=d, gap=2, capacity=plan)
    q, out, z, scale = attend(c, hk * group, t.bfloat16, batch=c.planned(plan), gap_rows=3)
    ref = attend64(c, q, scale)
    rows = slice(2, c.rows)
    check_out(out, ref, t.bfloat16, rows)
    check_lse(z, ref, rows)
    for part in (slice(0, 2), slice(c.rows, None)):
        assert bool((out[part] == 7).all()) and bool((z[part] == 7).all())
    _, out2, _, _ = attend(c, hk * group, t.bfloat16, batch=c.planned(plan), gap_rows=3, lse=False)
    assert t.equal(out, out2)
    # scores far apart, and a maximum that comes late
    c = Case([300, 90], [40, 40], 2, d, page, t.bfloat16, seed=7, capacity=65536, scale=6.0)
    q, out, z, scale = attend(c, 8, t.bfloat16, batch=c.planned(65536), scale=1.0)
    ref = attend64(c, q, scale)
    check_out(out, ref, t.bfloat16, slice(0, c.rows))
    check_lse(z, ref, slice(0, c.rows))


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_rows_that_see_nothing(dtype):
    """No slots at all, fewer slots than columns, no columns, rows outside."""
    t = torch()
    c = Case([0, 2, 40, 33], [3, 5, 0, 2], 2, 128, 32, dt(dtype), gap=3)
    q, out, z, scale = attend(c, 6, dt(dtype), gap_rows=4)
    ref = attend64(c, q, scale)
    check_out(out, ref, dt(dtype), slice(3, c.rows))
    check_lse(z, ref, slice(3, c.rows))
    assert bool((out[3:6] == 0).all()) and bool((out[6:9] == 0).all())
    assert bool((z[3:9] == -float("inf")).all())
    for part in (slice(0, 3), slice(c.rows, None)):
        assert bool((out[part] == 7).all()) and bool((z[part] == 7).all())


@pytest.mark.parametrize("n,heads,plan", [(60, 4, 0), (1500, 4, 0), (90, 40, 65536), (3000, 40, 65536)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_nan_reaches_those_who_see_it(dtype, n, heads, plan):
    t = torch()
    c = Case([n, 50], [4, 2], 2, 128, 32, dt(dtype), capacity=plan)
    bad_k, bad_v = c.k_in[n - 4:n].clone(), c.v_in[n - 4:n].clone()
    bad_v[2, 0, 40] = float("nan")   # column 2's values of head 0, block 1
    bad_k[3, 1, 7] = float("inf")    # column 3's keys of head 1
    k, v = t.cat([bad_k, c.k_in[-2:]]), t.cat([bad_v, c.v_in[-2:]])
    bqe.rfpx_kv_append(c.cache, c.batch, k, v)
    q, out, z, scale = attend(c, heads, dt(dtype), batch=c.planned(plan))
    g = heads // 2  # query heads of a kv head
    o = out.float().cpu().numpy()
    assert np.isfinite(o[:2]).all() and np.isfinite(o[4:]).all()
    assert np.isnan(o[2:4, :g, 32:64]).all()
    keep = np.ones(128, bool)
    keep[32:64] = False
    assert np.isfinite(o[2:4, :g][..., keep]).all()
    assert np.isfinite(o[2, g:]).all() and np.isnan(o[3, g:]).all()
    zz = z.cpu().numpy()
    assert np.isnan(zz[3, g:]).all() and np.isfinite(zz[:3]).all() and np.isfinite(zz[3, :g]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,plan", [(4, 0), (70, 65536)])
def test_attention_bad_pages_hold_nothing(dtype, heads, plan):
    c = Case([200, 40], [2, 3], 2, 128, 32, dt(dtype), capacity=plan)
    ref_vals = c.values()
    c.table[0, 1], c.table[0, 4] = -1, c.cache.n_pages
    c.table[1, :] = 2 ** 31 - 1
    c.values = lambda: ref_vals
    q, out, z, scale = attend(c, heads, dt(dtype), batch=c.planned(plan))
    ref = attend64(c, q, scale, seen=lambda b, j: b == 0 and j // 32 not in (1, 4))
    check_out(out, ref, dt(dtype), slice(0, c.rows))
    check_lse(z, ref, slice(0, c.rows))
    assert bool((out[2:] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,plan", [(64, 1100), (128, 1500), (128, 2048), (256, 300), (256, 1500)])
def test_attention_splits_without_tokens(d, plan, dtype):
    """9, 12, 16, 3 and 12 splits, of which the short sequence leaves most
    empty, in a workspace of NaN: none of it reaches a row."""
    t = torch()
    c = Case([40, 700, 0], [2, 3, 1], 2, d, 64, dt(dtype), seed=plan, capacity=plan)
    step = c.planned(plan)
    q, out, z, scale = attend(c, 6, dt(dtype), batch=step)
    ref = attend64(c, q, scale)
    check_out(out, ref, dt(dtype), slice(0, c.rows))
    check_lse(z, ref, slice(0, c.rows))
    ws = t.full((bqe.rfpx_attn_workspace_bytes(c.cache, step, 6, c.rows),), 255, dtype=t.uint8, device="cuda")
    assert t.equal(bqe.rfpx_attn_forward(c.cache, step, q, scale, ws=ws), out)


def test_attention_lengths_past_the_plan():
    """max_cols and max_len are for planning alone, and lens past the table's
    end counts as its end."""
    t = torch()
    c = Case([640, 96], [20, 3], 2, 128, 32, t.bfloat16)
    small = bqe.KvBatch(c.table, c.batch.lens, c.batch.starts, 1, 1)
    q, out, z, scale = attend(c, 8, t.bfloat16, batch=small)
    ref = attend64(c, q, scale)
    check_out(out, ref, t.bfloat16, slice(0, c.rows))
    big = c.make([2 ** 31 - 1, 96], c.starts, 20)
    _, out2, _, _ = attend(c, 8, t.bfloat16, batch=big)
    check_out(out2, ref, t.bfloat16, slice(0, c.rows))


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_extreme_scores(dtype):
    """One token far above the rest, and scores in the hundreds."""
    t = torch()
    c = Case([500], [2], 1, 128, 64, dt(dtype), scale=6.0)
    q, out, z, scale = attend(c, 4, dt(dtype), scale=1.0)
    ref = attend64(c, q, scale)
    check_out(out, ref, dt(dtype), slice(0, 2))
    check_lse(z, ref, slice(0, 2))
    # tiny scores: an even mean
    q, out, z, scale = attend(c, 4, dt(dtype), scale=1e-20)
    check_out(out, attend64(c, q, scale), dt(dtype), slice(0, 2))


def test_attention_strided_rows():
    t = torch()
    c = Case([100, 30], [3, 2], 2, 64, 32, t.bfloat16)
    g = t.Generator(device="cuda").manual_seed(5)
    wide = t.randn((5, 8 * 64 + 24), generator=g, device="cuda").to(t.bfloat16)
    q = wide[:, 8:8 + 6 * 64].view(5, 6, 64)
    out = t.zeros((5, 9, 64), dtype=t.bfloat16, device="cuda")
    bqe.rfpx_attn_forward(c.cache, c.batch, q, out=out[:, 2:8])
    plain = bqe.rfpx_attn_forward(c.cache, c.batch, q.contiguous())
    assert t.equal(out[:, 2:8], plain) and bool((out[:, :2] == 0).all() and (out[:, 8:] == 0).all())


def test_cache_past_32_bits():
    """Pages behind 4 GiB of pool."""
    t = torch()
    hk, d, page = 2, 256, 256
    n_pages = (5 << 30) // (hk * page * d * 17 // 16)
    c = Case([300], [2], hk, d, page, t.bfloat16)
    pool = t.empty(bqe.rfpx_kv_pool_bytes(hk, d, page, n_pages), dtype=t.uint8, device="cuda")
    cache = bqe.KvCache(hk, d, page, n_pages, pool=pool)
    table = t.tensor([[n_pages - 1, n_pages - 2]], dtype=t.int32, device="cuda")
    fill = bqe.KvBatch(table, c.fill.lens, c.fill.starts, 300, 300)
    bqe.rfpx_kv_append(cache, fill, c.k_in, c.v_in)
    step = bqe.KvBatch(table, c.batch.lens, c.batch.starts, 2, 300)
    q, out, _, scale = attend(c, 4, t.bfloat16)
    assert t.equal(bqe.rfpx_attn_forward(cache, step, q, scale), out)


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,cols,hk,group,d,page", [
    ([1], [1], 1, 1, 64, 32), ([700, 5, 129], [8, 5, 3], 2, 4, 128, 64), ([90], [5], 1, 16, 256, 32),
    ([200, 40], [130, 40], 2, 3, 128, 128), ([0, 3, 64], [2, 5, 1], 2, 2, 64, 32),
    ([500, 70, 0, 65], [17, 70, 9, 33], 2, 4, 128, 32), ([330], [66], 1, 5, 64, 256), ([150], [150], 1, 2, 256, 64),
    # rows enough for the path of many
    ([500, 70, 0, 65, 33], [130, 70, 9, 33, 3], 2, 4, 128, 32), ([97], [90], 1, 6, 64, 64), ([140], [140], 1, 4, 256, 128)])
def test_weights(lens, cols, hk, group, d, page, dtype):
    t = torch()
    c = Case(lens, cols, hk, d, page, dt(dtype), seed=3)
    q, out, z, scale = attend(c, hk * group, dt(dtype))
    cap = c.per * page
    acc = t.rand((len(lens), hk, cap), device="cuda")
    kept = acc.clone()
    got = bqe.rfpx_attn_weights(c.cache, c.batch, q, z, acc, 0.75, scale, acc_out=t.full_like(acc, -3.0))
    ref = attend64(c, q, scale)
    assert t.equal(acc, kept)
    # lse's own error reaches every weight of its row
    for b, n in enumerate(lens):
        want = 0.75 * f64(kept)[b, :, :n] + ref["w"][b]
        tol = 3 * ref["dw"][b] + 2.0 ** -20 * ref["w"][b] + 4 * U32 * want + 1e-30
        err = np.abs(f64(got)[b, :, :n] - want)
        assert (err <= tol).all(), np.max(err / tol)
        assert bool((got[b, :, n:] == -3).all())
    # in place
    again = bqe.rfpx_attn_weights(c.cache, c.batch, q, z, acc, 0.75, scale)
    assert again.data_ptr() == acc.data_ptr()
    for b, n in enumerate(lens):
        assert t.equal(acc[b, :, :n], got[b, :, :n]) and t.equal(acc[b, :, n:], kept[b, :, n:])


# ----------------------------------------------------------------- eviction

def evict_plain(lens, keep, recent, acc, pos, tokens):
    """tokens: what every slot holds, [seqs][hk][slots] of anything."""
    acc2, pos2, tok2, lens2 = acc.copy(), pos.copy(), tokens.copy(), []
    for b, n in enumerate(lens):
        lens2.append(min(n, keep))
        for h in range(acc.shape[1]):
            if n <= keep:
                continue
            w, p = acc[b, h, :n], pos[b, h, :n].astype(np.int64)
            edge = p.max() - recent

            def rank(j):
                a = w[j]
                return (0, 0.0, j) if p[j] > edge else (1, -a, j) if a == a else (2, 0.0, j)
            best = sorted(range(n), key=rank)[:keep]
            kept = set(best)
            holes = [j for j in range(keep) if j not in kept]
            for dst, src in zip(holes, sorted(j for j in best if j >= keep)):
                acc2[b, h, dst], pos2[b, h, dst], tok2[b, h, dst] = w[src], pos[b, h, src], tokens[b, h, src]
    return acc2, pos2, tok2, lens2


@pytest.mark.parametrize("lens,keep,recent,hk,d,page,kind", [
    ([100, 64, 65, 3], 64, 16, 2, 128, 32, "spread"), ([1000], 1, 0, 3, 64, 64, "spread"),
    ([700, 10], 333, 400, 1, 256, 128, "spread"), ([513, 400], 200, 50, 2, 128, 256, "ties"),
    ([300], 299, 0, 2, 64, 32, "nan"), ([5000, 4000], 1500, 100, 2, 64, 64, "ties"),
    ([129], 40, 129, 1, 64, 32, "spread"), ([40, 0], 100, 5, 2, 64, 32, "spread"), ([64], 20, 3, 2, 64, 32, "negative"),
    ([33000, 9000], 20000, 700, 1, 64, 256, "ties"), ([9000], 8500, 10, 2, 128, 128, "spread")])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(lens, keep, recent, hk, d, page, kind, in_place):
    t = torch()
    c = Case(lens, lens, hk, d, page, t.float32, seed=keep)
    cap = c.per * page
    r = np.random.default_rng(keep)
    acc = np.exp(3 * r.standard_normal((len(lens), hk, cap))).astype(np.float32)
    if kind == "ties":
        acc = np.round(np.minimum(acc, 3)).astype(np.float32)
        acc[..., ::7] = -0.0
    if kind == "nan":
        acc[..., ::3] = np.nan
        acc[..., 1::9] = np.inf
        acc[..., 2::11] = -np.inf
    if kind == "negative":
        acc = -acc
    pos = r.permuted(np.broadcast_to(np.arange(cap, dtype=np.int32) * 2 - 50, acc.shape), axis=-1)
    before = c.cache.pool.clone()
    # what every slot of every head holds: its token's first key value
    vals = c.values()
    tokens = np.zeros((len(lens), hk, cap, 2 * d))
    for b, (k, v) in enumerate(vals):
        if lens[b]:
            tokens[b, :, :lens[b]] = np.concatenate([k, v], -1).transpose(1, 0, 2)
    a, p = t.from_numpy(acc).cuda(), t.from_numpy(np.ascontiguousarray(pos)).cuda()
    if in_place:
        ao, po, lo = bqe.rfpx_kv_evict(c.cache, c.fill, keep, recent, a, p)
        assert lo.data_ptr() == c.fill.lens.data_ptr()
    else:
        ao, po, lo = t.full_like(a, -7), t.full_like(p, -7), t.full_like(c.fill.lens, -7)
        bqe.rfpx_kv_evict(c.cache, c.fill, keep, recent, a, p, ao, po, lo)
        assert c.fill.lens.tolist() == lens
    acc2, pos2, tok2, lens2 = evict_plain(lens, keep, recent, acc, pos, tokens)
    assert lo.tolist() == lens2
    left = c.make(lens2, [0] + list(np.cumsum(lens2)), max(lens2))
    k, v = (f64(x) for x in bqe.rfpx_kv_unpack(c.cache, left, sum(lens2)))
    at = 0
    for b, n in enumerate(lens2):
        assert np.array_equal(ao[b, :, :n].cpu().numpy(), acc2[b, :, :n], equal_nan=True)
        assert np.array_equal(po[b, :, :n].cpu().numpy(), pos2[b, :, :n])
        got = np.concatenate([k[at:at + n], v[at:at + n]], -1).transpose(1, 0, 2)
        assert np.array_equal(got, tok2[b, :, :n])
        at += n
        rest = (slice(None), slice(n, None))
        if in_place:
            assert np.array_equal(ao[b][rest].cpu().numpy(), acc[b][rest], equal_nan=True)
        else:
            assert bool((ao[b][rest] == -7).all() and (po[b][rest] == -7).all())
    if all(n <= keep for n in lens):
        assert t.equal(before, c.cache.pool)


def test_evict_bad_pages_move_nothing():
    t = torch()
    c = Case([96], [96], 1, 64, 32, t.float32)
    acc = t.arange(96, dtype=t.float32, device="cuda").view(1, 1, 96).contiguous()
    pos = t.arange(96, dtype=t.int32, device="cuda").view(1, 1, 96).contiguous()
    c.table[0, 2] = -3
    before = c.cache.pool.clone()
    ao, po, lo = bqe.rfpx_kv_evict(c.cache, c.fill, 32, 0, acc, pos)
    assert t.equal(before, c.cache.pool) and lo.tolist() == [32]
    assert ao[0, 0, :32].tolist() == [float(x) for x in range(64, 96)]


# ---------------------------------------------------------------- together

def layer_step(P, x, rows):
    """One decode step as a user writes it: projection, norm and rotation,
    append, attention with its weights, projection, experts."""
    t = torch()
    qkv = bqe.rfpx_dense_forward(P["wqkv"], x)
    h, hk, d = P["h"], P["cache"].n_kv_heads, P["cache"].head_dim
    q, k, v = (qkv[:, a * d:b * d].view(rows, b - a, d) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    q, k = bqe.rfpx_qk_norm_rope(q, k, P["positions"], P["qw"], P["kw"], 1e-6, P["rope"])
    bqe.rfpx_kv_append(P["cache"], P["batch"], k, v, P["positions"], P["pos"], P["acc"])
    o = bqe.rfpx_attn_forward(P["cache"], P["batch"], q, lse=P["lse"])
    bqe.rfpx_attn_weights(P["cache"], P["batch"], q, P["lse"], P["acc"])
    y = bqe.rfpx_dense_forward(P["wo"], o.view(rows, h * d))
    return q, k, v, o, bqe.moe_layer_forward(P["moe"], y)


def layer_setup(rows, seqs=2, cap=128):
    t = torch()
    lay = synth.gen_layer(synth.WORKLOADS[synth.TINY], 0, threads=4)
    width, h, hk, d = lay.d, 4, 2, 64
    g = t.Generator(device="cuda").manual_seed(11)

    def dense(r, c):
        w = t.randn((r, c), generator=g, device="cuda") * c ** -0.5
        return bqe.DenseMatrix(bqe.RFPX_FP4, r, c, bqe.rfpx_pack(bqe.RFPX_FP4, w))
    per = cap // 32
    table = t.randperm(seqs * per, generator=t.Generator().manual_seed(2)).view(seqs, per).int().cuda()
    shape = (seqs, hk, cap)
    return dict(h=h, wqkv=dense((h + 2 * hk) * d, width), wo=dense(width, h * d), moe=bqe.upload_layer(lay),
                qw=t.rand(d, generator=g, device="cuda") + 0.5, kw=t.rand(d, generator=g, device="cuda") + 0.5,
                rope=bqe.Rope(d), cache=bqe.KvCache(hk, d, 32, seqs * per), table=table, width=width,
                pos=t.zeros(shape, dtype=t.int32, device="cuda"), acc=t.zeros(shape, device="cuda"),
                lse=t.zeros((rows, h), device="cuda"), positions=t.zeros(rows, dtype=t.int32, device="cuda"),
                batch=bqe.KvBatch(table, t.zeros(seqs, dtype=t.int32, device="cuda"),
                                  t.tensor([0, rows // 2, rows], dtype=t.int32, device="cuda"), rows // 2, cap))


def test_run_together():
    """Steps of two sequences through projection, rotation, cache, attention
    and experts, with an eviction between, against 64 bits on the values that
    the cache holds."""
    t = torch()
    rows, keep, recent = 4, 20, 6
    P = layer_setup(rows)
    P["cache"].pool.fill_(255)
    g = t.Generator(device="cuda").manual_seed(4)
    lens, total = 0, 0
    for step in range(14):
        lens, total = lens + 2, total + 2
        P["batch"].lens.fill_(lens)
        P["positions"].copy_(t.tensor([total - 2, total - 1] * 2, dtype=t.int32))
        x = t.randn((rows, P["width"]), generator=g, device="cuda")
        before = P["acc"].clone()
        q, k, v, o, y = layer_step(P, x, rows)
        c = Case.__new__(Case)
        c.lens, c.cols, c.hk, c.d, c.page = [lens, lens], [2, 2], 2, 64, 32
        c.cache, c.table, c.starts, c.rows = P["cache"], P["table"], [0, 2, 4], 4
        c.fill_starts = [0, lens, 2 * lens]
        c.fill = c.make(c.lens, c.fill_starts, lens)
        ref = attend64(c, q, 64 ** -0.5)
        check_out(o, ref, t.float32, slice(0, rows))
        # the new slots hold what rfpx_pack makes of k and v
        kk, vv = bqe.rfpx_kv_unpack(P["cache"], P["batch"], rows)
        assert t.equal(kk.view(-1, 64), bqe.rfpx_unpack(4, bqe.rfpx_pack(4, k.reshape(-1, 64)), 8, 64))
        assert t.equal(vv.view(-1, 64), bqe.rfpx_unpack(4, bqe.rfpx_pack(4, v.reshape(-1, 64)), 8, 64))
        before[:, :, lens - 2:lens] = 0
        for b in range(2):
            want = f64(before)[b, :, :lens] + ref["w"][b]
            assert (np.abs(f64(P["acc"])[b, :, :lens] - want) <= 3 * ref["dw"][b] + 2.0 ** -20 * want).all()
        assert bool(t.isfinite(y).all())
        if lens > keep:
            bqe.rfpx_kv_evict(P["cache"], P["batch"], keep, recent, P["acc"], P["pos"])
            assert P["batch"].lens.tolist() == [keep, keep]
            kept = P["pos"][:, :, :keep].cpu().numpy()
            for row in kept.reshape(-1, keep):
                assert len(set(row)) == keep and set(range(total - recent, total)) <= set(row)
            lens = keep
    assert lens == keep and total == 28


def test_captured_steps_follow_device_lengths():
    """One captured step (rotation, append, attention, weights, eviction)
    replayed as the sequences grow, against the eager calls; eager work and
    synchronizations between the replays."""
    t = torch()
    rows, keep = 4, 24
    made = []
    for _ in range(2):
        P = layer_setup(rows)
        P["cache"].pool.fill_(255)
        P["q"] = t.zeros((rows, P["h"], 64), device="cuda", dtype=t.bfloat16)
        P["k"], P["v"] = (t.zeros((rows, 2, 64), device="cuda", dtype=t.bfloat16) for _ in range(2))
        P["ws"] = t.empty(bqe.rfpx_attn_workspace_bytes(P["cache"], P["batch"], P["h"], rows), dtype=t.uint8,
                          device="cuda")
        P["ews"] = t.empty(bqe.rfpx_kv_evict_workspace_bytes(P["cache"], P["batch"], keep), dtype=t.uint8,
                           device="cuda")
        P["out"], P["qo"], P["ko"] = t.zeros_like(P["q"]), t.zeros_like(P["q"]), t.zeros_like(P["k"])
        made.append(P)

    def step(P):
        bqe.rfpx_qk_norm_rope(P["q"], P["k"], P["positions"], P["qw"], P["kw"], 1e-6, P["rope"], P["qo"], P["ko"])
        bqe.rfpx_kv_append(P["cache"], P["batch"], P["ko"], P["v"], P["positions"], P["pos"], P["acc"])
        bqe.rfpx_attn_forward(P["cache"], P["batch"], P["qo"], out=P["out"], lse=P["lse"], ws=P["ws"])
        bqe.rfpx_attn_weights(P["cache"], P["batch"], P["qo"], P["lse"], P["acc"])
        bqe.rfpx_kv_evict(P["cache"], P["batch"], keep, 4, P["acc"], P["pos"], ws=P["ews"])

    A, B = made
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(A)  # before the capture, on the capture's stream
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(A)
    for P in made:
        P["acc"].zero_()
        P["pos"].zero_()
        P["batch"].lens.zero_()
        P["cache"].pool.fill_(255)
    for i in range(20):
        g = t.Generator(device="cuda").manual_seed(i)
        q, k, v = (t.randn(A[n].shape, generator=g, device="cuda").to(t.bfloat16) for n in ("q", "k", "v"))
        for P in made:
            P["q"].copy_(q)
            P["k"].copy_(k)
            P["v"].copy_(v)
            P["batch"].lens.add_(2)
            P["positions"].copy_(t.tensor([2 * i, 2 * i + 1] * 2, dtype=t.int32))
        graph.replay()
        step(B)
        t.cuda.synchronize()
        n = int(B["batch"].lens[0])
        assert A["batch"].lens.tolist() == B["batch"].lens.tolist() == [min(2 * i + 2, keep)] * 2
        for name in ("out", "lse"):
            assert t.equal(A[name], B[name]), (i, name)
        assert t.equal(A["acc"][:, :, :n], B["acc"][:, :, :n]) and t.equal(A["pos"][:, :, :n], B["pos"][:, :, :n])
        _ = (q.float() @ q.float().transpose(1, 2)).sum().item()  # eager work between


def test_captured_chunk_follows_device_lengths():
    """A captured chunk (append, attention of many rows, its weights) replayed
    with other lengths and fewer columns than it was captured with."""
    t = torch()
    hk, g, d, page, cap, rows = 2, 8, 128, 64, 65536, 80
    c = Case([900, 700], [40, 40], hk, d, page, t.bfloat16, capacity=cap)
    batch = c.planned(cap)
    gen = t.Generator(device="cuda").manual_seed(9)
    q = t.randn((rows, hk * g, d), generator=gen, device="cuda").to(t.bfloat16)
    k, v = (t.randn((rows, hk, d), generator=gen, device="cuda").to(t.bfloat16) for _ in range(2))
    out, lse = t.zeros_like(q), t.zeros((rows, hk * g), device="cuda")
    acc, acc_out = t.zeros((2, hk, c.per * page), device="cuda"), t.zeros((2, hk, c.per * page), device="cuda")
    ws = t.empty(bqe.rfpx_attn_workspace_bytes(c.cache, batch, hk * g, rows), dtype=t.uint8, device="cuda")

    def step(out, lse, acc_out, ws=None):
        bqe.rfpx_kv_append(c.cache, batch, k, v)
        bqe.rfpx_attn_forward(c.cache, batch, q, out=out, lse=lse, ws=ws)
        bqe.rfpx_attn_weights(c.cache, batch, q, lse, acc, 1.0, acc_out=acc_out)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(out, lse, acc_out, ws)
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(out, lse, acc_out, ws)
    for lens, starts in (([900, 700], [0, 40, 80]), ([950, 33], [0, 40, 73]), ([400, 80], [0, 3, 80]),
                         ([64, 0], [0, 64, 64]), ([900, 700], [0, 40, 80])):
        batch.lens.copy_(t.tensor(lens, dtype=t.int32))
        batch.starts.copy_(t.tensor(starts, dtype=t.int32))
        for x in (out, lse, acc_out):
            x.fill_(3)
        graph.replay()
        o2, z2, a2 = t.full_like(out, 3), t.full_like(lse, 3), t.full_like(acc_out, 3)
        step(o2, z2, a2)
        t.cuda.synchronize()
        # (950 slots reach tokens that were never appended, which read as NaN)
        for x, y in ((out, o2), (lse, z2), (acc_out, a2)):
            assert t.allclose(x, y, rtol=0.0, atol=0.0, equal_nan=True), lens
        assert bool((out[starts[-1]:] == 3).all())
        _ = (q.float() @ q.float().transpose(1, 2)).sum().item()  # eager work between


def test_other_stream_and_two_at_once():
    t = torch()
    c = Case([900, 300], [3, 2], 2, 128, 64, t.bfloat16)
    q, out, z, scale = attend(c, 8, t.bfloat16)
    t.cuda.synchronize()
    s1, s2 = t.cuda.Stream(), t.cuda.Stream()
    a = [bqe.rfpx_attn_forward(c.cache, c.batch, q, scale, stream=s) for s in (s1, s2, s1, s2)]
    s1.synchronize()
    s2.synchronize()
    for x in a:
        assert t.equal(x, out)


def test_wrapper_refusals():
    t = torch()
    c = Case([40], [2], 2, 128, 32, t.bfloat16)
    q = t.zeros((2, 4, 128), dtype=t.bfloat16, device="cuda")
    lse = t.zeros((2, 4), device="cuda")
    acc = t.zeros((1, 2, 64), device="cuda")
    for bad in (q.half(), q.transpose(0, 1), q[..., :64], q.cpu(), q[0]):
        with pytest.raises(ValueError):
            bqe.rfpx_attn_forward(c.cache, c.batch, bad)
    with pytest.raises(ValueError):
        bqe.rfpx_attn_forward(c.cache, c.batch, q, lse=lse[:1])
    with pytest.raises(ValueError):
        bqe.rfpx_attn_forward(c.cache, c.batch, q, out=q.float())
    with pytest.raises(ValueError):
        bqe.rfpx_attn_weights(c.cache, c.batch, q, lse, acc[..., :60])
    with pytest.raises(ValueError):
        bqe.rfpx_kv_append(c.cache, c.batch, q, q)
    with pytest.raises(ValueError):
        bqe.rfpx_kv_evict(c.cache, c.batch, 8, 2, acc, acc)
    with pytest.raises(bqe.RfpxError):
        bqe.rfpx_attn_forward(c.cache, c.batch, t.zeros((2, 5, 128), dtype=t.bfloat16, device="cuda"))
    with pytest.raises(bqe.RfpxError):
        bqe.rfpx_kv_evict(c.cache, c.batch, 0, 2, acc, acc.int())
    with pytest.raises(bqe.RfpxError):
        bqe.KvCache(2, 100, 32, 1)
    with pytest.raises(ValueError):
        bqe.KvBatch(c.table.long(), c.batch.lens, c.batch.starts, 1, 1)


def test_no_rows():
    """A step without columns: nothing is written, and weights only decay."""
    t = torch()
    c = Case([40], [0], 2, 128, 32, t.bfloat16)
    none = t.empty((0, 4, 128), dtype=t.bfloat16, device="cuda")
    before = c.cache.pool.clone()
    bqe.rfpx_kv_append(c.cache, c.batch, none[:, :2], none[:, :2])
    assert t.equal(before, c.cache.pool)
    assert bqe.rfpx_attn_forward(c.cache, c.batch, none).shape == (0, 4, 128)
    acc = t.rand((1, 2, 64), device="cuda")
    want = acc.clone()
    want[..., :40] *= 0.5
    bqe.rfpx_attn_weights(c.cache, c.batch, none, t.empty((0, 4), device="cuda"), acc, 0.5)
    assert t.equal(acc, want)
