"""What is measured of the attention operators over a 4-bit key/value cache:
cases, inputs, their plain forms in elementary torch operations, and their
values in 64 bits.

The cache is a pool of pages.  A page holds, for every kv head, a slab of
page tokens: codes of the keys, their scales, codes of the values, their
scales.  A head's D values of a token are D/32 blocks of 32 codes
(value (c - 7.5) * 2^(e-127), two codes to a byte, the even one in the low
half), laid out as

  keys    [token][octet of a block: 4][block: D/32][4 bytes]
  values  [token / 4][byte of a block: 16][pair: 2][block / 2][token & 1][block & 1]
  scales  [token][block] (one byte e each)

so that a matrix instruction's operands are read as they stand.
"""
import math
import random

import torch

own = False

STYLE_HALF, STYLE_PAIRS = 0, 1


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the q=5 verify step's query and key rows, slices of one fp32 projection
        dict(name="norm rope verify q5", kind="norm_rope", dtype="float32", out="bfloat16", rows=5, heads=32,
             kv_heads=8, dim=128, rot=128, style=STYLE_HALF),
        # a 2048-token prefill chunk, half of each head rotated in neighbouring pairs
        dict(name="norm rope chunk 2048", kind="norm_rope", dtype="bfloat16", out="bfloat16", rows=2048, heads=32,
             kv_heads=8, dim=128, rot=64, style=STYLE_PAIRS),
        # 16 sequences in decode, up to 4 verify columns each
        dict(name="append verify 16 seqs", kind="append", dtype="bfloat16", seqs=16, cols=4, length=2000, ragged=True,
             kv_heads=8, dim=128, page=64),
        # a 2048-token chunk behind a prompt's first part, in fp32 as a projection leaves it
        dict(name="append chunk 2048", kind="append", dtype="float32", seqs=1, cols=2048, length=5000, ragged=False,
             kv_heads=8, dim=128, page=64),
        # one column of one short conversation: latency
        dict(name="attend 1 column, 1021", kind="attend", dtype="bfloat16", seqs=1, cols=1, length=1021, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64),
        # a batch in decode, every sequence at its own length, fp32 as a projection leaves it
        dict(name="attend 16 seqs to 8192", kind="attend", dtype="float32", seqs=16, cols=1, length=8192, ragged=True,
             heads=32, kv_heads=8, dim=64, page=32),
        # q=5 verify columns against one long context
        dict(name="attend q5, 131071", kind="attend", dtype="bfloat16", seqs=1, cols=5, length=131071, ragged=False,
             heads=32, kv_heads=8, dim=128, page=256),
        # a 2048-token prefill chunk at the end of an 8192-token context
        dict(name="attend chunk 2048 of 8192", kind="attend", dtype="bfloat16", seqs=1, cols=2048, length=8192,
             ragged=False, heads=32, kv_heads=8, dim=128, page=64),
        # q=4 verify columns of four sequences, with the weight that each cached token receives
        dict(name="weights 4 seqs q4, 16384", kind="weights", dtype="bfloat16", seqs=4, cols=4, length=16384,
             ragged=True, heads=32, kv_heads=8, dim=128, page=128),
        # a first 2048-token chunk with its weights
        dict(name="weights chunk 2048", kind="weights", dtype="bfloat16", seqs=1, cols=2048, length=2048, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64),
        # 8 sequences that have grown 128 tokens past their budget
        dict(name="evict 8 seqs 4224 to 4096", kind="evict", seqs=8, length=4224, keep=4096, recent=256, kv_heads=8,
             dim=128, page=64),
        # a long prompt cut to its budget once
        dict(name="evict 32768 to 8192", kind="evict", seqs=1, length=32768, keep=8192, recent=1024, kv_heads=8,
             dim=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["norm_rope", "append", "attend", "attend", "weights", "evict"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if kind == "norm_rope":
        rot = rng.choice([dim, dim // 2, dim - 2 * rng.randrange(1, dim // 4)])
        rows = _log_int(rng, 1, 2048 * 40 * 128 // ((heads + kv_heads) * dim))
        return dict(kind=kind, dtype=dtype, out=rng.choice([dtype, "bfloat16"]), rows=min(rows, 8192), heads=heads,
                    kv_heads=kv_heads, dim=dim, rot=rot, style=rng.choice([STYLE_HALF, STYLE_PAIRS]))
    seqs = _log_int(rng, 1, 16)
    if kind == "append":
        cols = rng.choice([_log_int(rng, 1, 8), _log_int(rng, 9, max(9, 2048 // seqs))])
        return dict(kind=kind, dtype=dtype, seqs=seqs, cols=cols, length=cols + _log_int(rng, 1, 6000),
                    ragged=rng.random() < 0.5, kv_heads=kv_heads, dim=dim, page=page)
    if kind == "evict":
        length = _log_int(rng, 64, max(64, 8 * 4224 * 8 // (seqs * kv_heads)))
        length = min(length, 32768)
        keep = rng.randrange(1, length + length // 8)
        return dict(kind=kind, seqs=seqs, length=length, keep=keep, recent=rng.randrange(0, keep + 1) // 2,
                    kv_heads=kv_heads, dim=dim, page=page)
    if rng.random() < 0.75:
        cols = rng.randrange(1, 9)
    else:
        cols, seqs = _log_int(rng, 9, 2048), min(seqs, 2)
    # tokens of the cache at most those of the longest listed one, products at most those of the listed chunk
    most = min(131071 * 8 * 128 // (seqs * kv_heads * dim), 2048 * 8192 * 32 * 128 // (seqs * cols * heads * dim))
    length = max(cols, _log_int(rng, 1, max(1, min(most, 131071))))
    return dict(kind=kind, dtype=dtype, seqs=seqs, cols=cols, length=length, ragged=rng.random() < 0.5, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page)


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def _quantize(x):
    """FP4 blocks of x [.., D]: codes uint8 [.., D], scales uint8 [.., D/32]."""
    w = x.double().unflatten(-1, (-1, 32))
    a = w.abs().amax(-1)
    mant, power = torch.frexp(a / 7.5)
    up = power.double() - (mant == 0.5).double()  # ceil(log2(a / 7.5))
    e = (127 + up).clamp(1, 254)
    c = torch.round(w * torch.exp2(127 - e).unsqueeze(-1) + 7.5).clamp(0, 15)
    zero = a == 0
    e = torch.where(zero, torch.zeros_like(e), e)
    c = torch.where(zero.unsqueeze(-1), torch.zeros_like(c), c)
    return c.to(torch.uint8).flatten(-2), e.to(torch.uint8)


def _values(codes, scales):
    """fp32 values of codes [.., D] and scales [.., D/32]."""
    c = codes.float().unflatten(-1, (-1, 32)) - 7.5
    return (c * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _slab_parts(page, dim):
    half = page * dim // 2
    s = page * dim // 32
    return [half, s, half, s]


def _pages(k, v):
    """Slabs [pages][heads][bytes] of k, v [pages][page tokens][heads][D]."""
    (kc, ks), (vc, vs) = _quantize(k), _quantize(v)
    n, page, heads, dim = k.shape
    nb = dim // 32

    def rows(c):  # the canonical bytes, [pages][heads][token][block][16]
        return (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(1, 2).unflatten(-1, (nb, 16))

    kb = rows(kc).unflatten(-1, (4, 4)).transpose(3, 4).reshape(n, heads, -1)
    vb = rows(vc).reshape(n, heads, page // 4, 2, 2, nb // 2, 2, 16).permute(0, 1, 2, 7, 3, 5, 4, 6)
    return torch.cat([kb, ks.transpose(1, 2).reshape(n, heads, -1), vb.reshape(n, heads, -1),
                      vs.transpose(1, 2).reshape(n, heads, -1)], -1)


def _cached(pool, table, page, heads, dim):
    """fp32 keys and values [seqs][heads][tokens][D] of the pages in table [seqs][n]."""
    nb, (b, n) = dim // 32, table.shape
    got = pool.view(-1, heads, sum(_slab_parts(page, dim)))[table.long()].transpose(1, 2)
    kb, ks, vb, vs = got.split(_slab_parts(page, dim), -1)
    kb = kb.reshape(b, heads, n * page, 4, nb, 4).transpose(3, 4).reshape(b, heads, n * page, -1)
    vb = vb.reshape(b, heads, n * page // 4, 16, 2, nb // 2, 2, 2).permute(0, 1, 2, 4, 6, 5, 7, 3)
    vb = vb.reshape(b, heads, n * page, -1)

    def codes(x):
        return torch.stack([x & 15, x >> 4], -1).flatten(-2)

    return (_values(codes(kb), ks.reshape(b, heads, n * page, nb)),
            _values(codes(vb), vs.reshape(b, heads, n * page, nb)))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _sizes(case):
    """Length and columns of every sequence: the case's own, or spread below
    them (the first sequence has them in full)."""
    b, length, cols = case["seqs"], case["length"], case.get("cols", 0)
    if not case.get("ragged"):
        return [length] * b, [cols] * b
    r = random.Random(b * 1000003 + length * 17 + cols)
    n = [cols] + [r.randint(1 if cols <= 8 else cols // 2, cols) for _ in range(b - 1)]
    lens = [length] + [max(n[i], r.randint(max(1, length // 4), length)) for i in range(1, b)]
    return lens, n


def _batch(case, seed):
    """Sequence lengths, column starts and a shuffled page table."""
    g = torch.Generator().manual_seed(seed + 1000)
    lens, n = _sizes(case)
    starts = [sum(n[:i]) for i in range(len(n) + 1)]
    b, per = len(n), -(-case["length"] // case["page"])
    total = b * per + 3
    table = torch.randperm(total, generator=g)[:b * per].reshape(b, per)
    return dict(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), table=table.int().cuda(), total=total,
                rows=starts[-1], max_cols=max(n), max_len=case["length"])


def _pool(case, total, g):
    shape = (min(total, max(1, (1 << 27) // (case["page"] * case["kv_heads"] * case["dim"]))), case["page"],
             case["kv_heads"], case["dim"])
    made, at = [], 0
    while at < total:  # a part at a time: the generator's values take 32 times the pool's bytes
        n = min(shape[0], total - at)
        k = torch.randn((n,) + shape[1:], generator=g, device="cuda")
        v = torch.randn((n,) + shape[1:], generator=g, device="cuda")
        made.append(_pages(k, v))
        at += n
    return torch.cat(made).reshape(-1)


def prepare(case, seed):
    g, kind = _gen(seed), case["kind"]
    s = dict(case)
    if kind == "norm_rope":
        n, d, hq, hk = case["rows"], case["dim"], case["heads"], case["kv_heads"]
        # a projection's rows: queries, keys and values side by side
        qkv = torch.randn(n, (hq + 2 * hk) * d, generator=g, device="cuda") * 3
        s["qkv"] = qkv.to(_dtype(case["dtype"]))
        s["positions"] = (torch.randint(0, 1 << 20, (1,), generator=g, device="cuda")
                          + torch.arange(n, device="cuda")).int()
        s["q_weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        s["eps"] = 1e-6
        if own:
            import block_quantized_expert_amd as bqe
            s["rope"] = bqe.Rope(case["rot"], theta=10000.0, style=case["style"])
        return s
    b = _batch(case, seed)
    s.update(b)
    s["pool"] = _pool(case, b["total"], g)
    shape = (case["seqs"], case["kv_heads"], b["table"].shape[1] * case["page"])
    if kind == "append":
        shape = (b["rows"], case["kv_heads"], case["dim"])
        s["k"] = torch.randn(shape, generator=g, device="cuda").to(_dtype(case["dtype"]))
        s["v"] = torch.randn(shape, generator=g, device="cuda").to(_dtype(case["dtype"]))
    elif kind == "evict":
        slots = torch.arange(shape[2], device="cuda").expand(shape)
        # the weight that a token has gathered: a few large, many next to nothing, some none
        acc = torch.exp(2.5 * torch.randn(shape, generator=g, device="cuda"))
        s["acc"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.05, torch.zeros_like(acc), acc)
        # earlier evictions have mixed the order of all but the newest tokens
        mixed = torch.rand(shape, generator=g, device="cuda").masked_fill_(
            slots >= case["length"] * 3 // 4, 2.0).sort(dim=-1, stable=True).indices
        s["pos"] = (mixed * 3 + 7).int()
        s["acc_out"], s["pos_out"] = torch.zeros_like(s["acc"]), torch.zeros_like(s["pos"])
        s["lens_out"] = torch.zeros_like(b["lens"])
    else:
        q = torch.randn((b["rows"], case["heads"], case["dim"]), generator=g, device="cuda") * 1.5
        s["q"] = q.to(_dtype(case["dtype"]))
        s["scale"] = case["dim"] ** -0.5
        if kind == "weights":
            s["acc"] = torch.rand(shape, generator=g, device="cuda")
            s["acc_out"] = torch.zeros_like(s["acc"])
            s["decay"] = 0.9375
    if own:
        import block_quantized_expert_amd as bqe
        s["cache"] = bqe.KvCache(case["kv_heads"], case["dim"], case["page"], s["total"], pool=s["pool"])
        s["batch"] = bqe.KvBatch(s["table"], s["lens"], s["starts"], max_cols=b["max_cols"], max_len=b["max_len"])
    return s


# ------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rot, style):
    part, rest = x[..., :rot], x[..., rot:]
    if style == STYLE_HALF:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([part, rest], -1)


def _plain_norm_rope(s):
    n, d, hq, hk = s["rows"], s["dim"], s["heads"], s["kv_heads"]
    angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(x, cos, sin, s["rot"], s["style"]).to(_dtype(s["out"]))

    return {"q": one(s["qkv"][:, :hq * d].view(n, hq, d), s["q_weight"]),
            "k": one(s["qkv"][:, hq * d:(hq + hk) * d].view(n, hk, d), s["k_weight"])}


def _rows_of(s):
    """Sequence, column and slot of every row."""
    row = torch.arange(s["rows"], device="cuda")
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, row, right=True) - 1
    n = starts[1:] - starts[:-1]
    col = row - starts[seq]
    return seq, col, s["lens"].long()[seq] - n[seq] + col


def _plain_append(s):
    # the cache's bytes at the rows' slots change, and what they hold comes back
    heads, dim, page = s["kv_heads"], s["dim"], s["page"]
    seq, _, slot = _rows_of(s)
    at = s["table"].long()[seq, slot // page]
    pool = s["pool"].view(-1, heads, sum(_slab_parts(page, dim)))
    nb, t = dim // 32, slot % page
    back = []
    for x, key in ((s["k"], True), (s["v"], False)):
        c, e = _quantize(x)
        first = 0 if key else page * (dim // 2 + nb)
        by = (c[..., 0::2] | (c[..., 1::2] << 4)).unflatten(-1, (nb, 16))
        if key:
            by, off = by.unflatten(-1, (4, 4)).transpose(2, 3).flatten(2), torch.arange(dim // 2, device="cuda")
            off = first + t.unsqueeze(-1) * (dim // 2) + off
        else:
            by = by.unflatten(2, (nb // 2, 2)).permute(0, 1, 4, 2, 3).flatten(2)  # [rows][heads][byte][block]
            r = torch.arange(16, device="cuda").view(1, 16, 1, 1)
            bp = torch.arange(nb // 2, device="cuda").view(1, 1, -1, 1)
            z, u = torch.arange(2, device="cuda"), t.view(-1, 1, 1, 1)
            off = ((u // 4 * 16 + r) * 2 + u % 4 // 2) * (nb // 2) * 4 + bp * 4 + u % 2 * 2 + z
            off = first + off.flatten(1)
        h = torch.arange(heads, device="cuda").view(1, -1, 1)
        pool[at.view(-1, 1, 1), h, off.unsqueeze(1)] = by
        off = first + page * dim // 2 + t.unsqueeze(-1) * nb + torch.arange(nb, device="cuda")
        pool[at.view(-1, 1, 1), h, off.unsqueeze(1)] = e
        back.append(_values(c, e))
    return {"k": back[0], "v": back[1]}


def _plain_attend(s, weights):
    b, hk, g, d, cols = s["seqs"], s["kv_heads"], s["heads"] // s["kv_heads"], s["dim"], s["max_cols"]
    k, v = _cached(s["pool"], s["table"], s["page"], hk, d)
    length = k.shape[2]
    seq, col, slot = _rows_of(s)
    q = torch.zeros((b, cols, hk * g, d), device="cuda")
    q[seq, col] = s["q"].float()
    last = torch.full((b, cols), -1, device="cuda")
    last[seq, col] = slot
    q = q.view(b, cols, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, cols * g, d)
    last = last.view(b, 1, cols, 1).expand(b, 1, cols, g).reshape(b, 1, cols * g, 1)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_(torch.arange(length, device="cuda") > last, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    out = torch.matmul(p, v).view(b, hk, cols, g, d).permute(0, 2, 1, 3, 4).reshape(b, cols, hk * g, d)
    lse = (top + total.log()).view(b, hk, cols, g).permute(0, 2, 1, 3).reshape(b, cols, hk * g)
    r = {"out": out[seq, col].to(_dtype(s["dtype"])), "lse": lse[seq, col]}
    if weights:
        held = torch.arange(length, device="cuda") < s["lens"].view(-1, 1, 1)
        r["acc"] = torch.where(held, s["acc"] * s["decay"] + p.sum(2), s["acc_out"])
    return r


def _plain_evict(s):
    keep, page, dim, heads = s["keep"], s["page"], s["dim"], s["kv_heads"]
    acc, pos, nb = s["acc"], s["pos"], s["dim"] // 32
    b, _, cap = acc.shape
    slot = torch.arange(cap, device="cuda").expand(acc.shape)
    held = slot < s["lens"].view(-1, 1, 1)
    newest = torch.where(held, pos, torch.full_like(pos, -1)).amax(-1, keepdim=True).long()
    safe = held & (pos.long() > newest - s["recent"])
    worth = torch.where(safe, torch.full_like(acc, math.inf), acc)
    worth = torch.where(held, worth, torch.full_like(acc, -math.inf))
    order = worth.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(held).scatter_(-1, order[..., :keep], True) & held
    hole = ~kept & held & (slot < keep)
    late = kept & (slot >= keep)
    # the n-th late slot goes into the n-th hole
    to = torch.where(hole, slot, torch.full_like(slot, cap)).sort(-1).values
    nth = (late.long().cumsum(-1) - 1).clamp(min=0)
    to = torch.gather(to, -1, nth)
    q, h, src = late.nonzero(as_tuple=True)
    dst = to[q, h, src]
    stays = held & (slot < keep)
    acc2, pos2 = torch.where(stays, acc, s["acc_out"]), torch.where(stays, pos, s["pos_out"])
    acc2[q, h, dst], pos2[q, h, dst] = acc[q, h, src], pos[q, h, src]
    pool = s["pool"].view(-1, heads, sum(_slab_parts(page, dim)))

    def place(j):
        t = (j % page).unsqueeze(-1)
        half = page * dim // 2
        k = t * (dim // 2) + torch.arange(dim // 2, device="cuda")
        ks = half + t * nb + torch.arange(nb, device="cuda")
        r = torch.arange(16, device="cuda").view(1, 16, 1, 1)
        bp = torch.arange(nb // 2, device="cuda").view(1, 1, -1, 1)
        z, u = torch.arange(2, device="cuda"), t.view(-1, 1, 1, 1)
        v = ((u // 4 * 16 + r) * 2 + u % 4 // 2) * (nb // 2) * 4 + bp * 4 + u % 2 * 2 + z
        v = half + page * nb + v.flatten(1)
        vs = 2 * half + page * nb + t * nb + torch.arange(nb, device="cuda")
        return s["table"].long()[q, j // page].unsqueeze(-1), h.unsqueeze(-1), torch.cat([k, ks, v, vs], -1)

    pool[place(dst)] = pool[place(src)]
    return {"acc": acc2, "pos": pos2, "lens": s["lens"].clamp(max=keep), "pool": s["pool"]}


def run(s):
    kind = s["kind"]
    if not own:
        if kind == "norm_rope":
            return _plain_norm_rope(s)
        if kind == "append":
            return _plain_append(s)
        if kind == "evict":
            return _plain_evict(s)
        return _plain_attend(s, kind == "weights")
    import block_quantized_expert_amd as bqe
    if kind == "norm_rope":
        n, d, hq, hk = s["rows"], s["dim"], s["heads"], s["kv_heads"]
        q, k = bqe.rfpx_qk_norm_rope(s["qkv"][:, :hq * d].view(n, hq, d), s["qkv"][:, hq * d:(hq + hk) * d].view(n, hk, d),
                                     s["positions"], s["q_weight"], s["k_weight"], s["eps"], s["rope"],
                                     out_dtype=_dtype(s["out"]))
        return {"q": q, "k": k}
    cache, batch = s["cache"], s["batch"]
    if kind == "append":
        bqe.rfpx_kv_append(cache, batch, s["k"], s["v"])
        k, v = bqe.rfpx_kv_unpack(cache, batch, s["rows"])
        return {"k": k, "v": v}
    if kind == "evict":
        acc, pos, lens = bqe.rfpx_kv_evict(cache, batch, s["keep"], s["recent"], s["acc"], s["pos"],
                                           acc_out=s["acc_out"], pos_out=s["pos_out"],
                                           lens_out=s["lens_out"])
        return {"acc": acc, "pos": pos, "lens": lens, "pool": s["pool"]}
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    r = {"out": bqe.rfpx_attn_forward(cache, batch, s["q"], s["scale"], lse=lse), "lse": lse}
    if kind == "weights":
        r["acc"] = bqe.rfpx_attn_weights(cache, batch, s["q"], lse, s["acc"], s["decay"], s["scale"],
                                         acc_out=s["acc_out"])
    return r


# -------------------------------------------------------------------- work

def work(case):
    kind, d = case["kind"], case["dim"]
    size = 4 if case.get("dtype") == "float32" else 2
    if kind == "norm_rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": n * (size + (4 if case["out"] == "float32" else 2)) + 8 * d + 4 * case["rows"], "flops": 8 * n}
    token = case["kv_heads"] * d * 17 / 16  # bytes of a token's keys and values
    lens, cols = _sizes(case)
    if kind == "append":  # the rows, their blocks in the cache, and the values read back
        n = sum(cols) * case["kv_heads"] * d
        return {"bytes": n * 2 * (size + 4) + sum(cols) * token * 2, "flops": 10 * n}
    if kind == "evict":  # weights and positions of all, those of the kept ones, and the blocks that move
        gone = max(0, case["length"] - case["keep"])
        moved = gone * case["keep"] / max(1, case["length"])
        n = case["seqs"] * case["kv_heads"]
        return {"bytes": n * 8 * (case["length"] + min(case["keep"], case["length"])) + case["seqs"] * moved * token * 2,
                "flops": n * case["length"]}
    pairs = case["heads"] * sum(n * (length - (n - 1) / 2) for length, n in zip(lens, cols))
    r = {"bytes": sum(lens) * token + sum(cols) * case["heads"] * (d * size * 2 + 4), "flops": 4 * pairs * d}
    if kind == "weights":
        r["bytes"] += sum(lens) * case["kv_heads"] * 8
    return r


# ------------------------------------------------- the definition, 64 bits

def _slab_values(slab, tokens, page, dim, key):
    """Values [tokens][D] of one sequence and head in 64 bits, each code read
    at the place that the layout gives it.  slab: uint8 [pages][bytes]."""
    nb = dim // 32
    j = torch.arange(tokens, device="cuda").view(-1, 1)
    d = torch.arange(dim, device="cuda").view(1, -1)
    t, block, i = j % page, d // 32, d % 32
    if key:
        at = t * (dim // 2) + (i // 8 * nb + block) * 4 + i % 8 // 2
    else:
        at = page * (dim // 2 + nb) + ((t // 4 * 16 + i // 2) * nb * 4 + (t % 4 // 2 * (nb // 2) + block // 2) * 4
                                       + t % 2 * 2 + block % 2)
    code = (slab[j // page, at] >> (4 * (i % 2)).to(torch.uint8)) & 15
    first = page * dim // 2 + (0 if key else page * (dim // 2 + nb))
    e = slab[j // page, first + t * nb + block]
    return (code.double() - 7.5) * torch.exp2(e.double() - 127)


def _exact_attend(case, s):
    hk, g, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    pool = s["pool"].view(s["total"], hk, -1)
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.zeros((s["rows"], hk * g, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["rows"], hk * g), dtype=torch.float64, device="cuda")
    acc = s["acc_out"].double() if case["kind"] == "weights" else None
    for b in range(case["seqs"]):
        n, first = starts[b + 1] - starts[b], starts[b]
        pages = s["table"][b].long()
        seen = lens[b] - n + torch.arange(n, device="cuda").repeat_interleave(g).view(-1, 1)
        for h in range(hk):
            slab = pool[pages, h]
            k = _slab_values(slab, lens[b], case["page"], d, True)
            v = _slab_values(slab, lens[b], case["page"], d, False)
            mine = slice(h * g, (h + 1) * g)
            q = s["q"][first:first + n, mine].double().reshape(n * g, d)
            x = (q @ k.T) * s["scale"]
            x[torch.arange(lens[b], device="cuda") > seen] = -math.inf
            z = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - z)
            out[first:first + n, mine] = (p @ v).view(n, g, d)
            lse[first:first + n, mine] = z.view(n, g)
            if acc is not None:
                acc[b, h, :lens[b]] = s["acc"][b, h, :lens[b]].double() * s["decay"] + p.sum(0)
    r = {"out": out, "lse": lse}
    if acc is not None:
        r["acc"] = acc
    return r


def _exact_norm_rope(case, s):
    n, d, rot = case["rows"], case["dim"], case["rot"]
    inv = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    turn = torch.polar(torch.ones((n, 1, rot // 2), dtype=torch.float64, device="cuda"),
                       s["positions"].double().view(n, 1, 1) * inv)
    r, at = {}, 0
    for name, heads in (("q", case["heads"]), ("k", case["kv_heads"])):
        x = s["qkv"][:, at:at + heads * d].double().view(n, heads, d)
        at += heads * d
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + s["eps"]) * s[name + "_weight"].double()
        i = torch.arange(rot // 2, device="cuda")
        a, b = (i, i + rot // 2) if case["style"] == STYLE_HALF else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., a], x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
        r[name] = x
    return r


def _exact_append(case, s):
    r = {}
    for name in ("k", "v"):
        x = s[name].double().cpu().reshape(-1, 32)
        a = x.abs().amax(-1)
        e = torch.ceil(torch.log2(a / 7.5))
        e = torch.where(torch.exp2(e - 1) >= a / 7.5, e - 1, torch.where(torch.exp2(e) < a / 7.5, e + 1, e))
        unit = torch.exp2(e.clamp(-126, 127)).unsqueeze(-1)
        half = (torch.round(x / unit + 7.5).clamp(0, 15) - 7.5) * unit
        half[a == 0] = -7.5 * 2.0 ** -127
        r[name] = half.reshape(s[name].shape)
    return r


def _exact_evict(case, s):
    acc, pos = s["acc"].cpu(), s["pos"].cpu()
    lens, keep = s["lens"].tolist(), case["keep"]
    acc2, pos2 = torch.zeros(acc.shape, dtype=torch.float64), torch.zeros_like(pos)
    for b in range(case["seqs"]):
        n = lens[b]
        for h in range(case["kv_heads"]):
            w, p = acc[b, h, :n].tolist(), pos[b, h, :n].tolist()
            edge = max(p) - case["recent"]
            best = sorted(range(n), key=lambda j: (p[j] <= edge, -w[j] if p[j] <= edge else 0.0, j))[:keep]
            kept = set(best)
            m = min(n, keep)
            acc2[b, h, :m], pos2[b, h, :m] = acc[b, h, :m].double(), pos[b, h, :m]
            holes = [j for j in range(m) if j not in kept]
            for dst, src in zip(holes, sorted(j for j in best if j >= keep)):
                acc2[b, h, dst], pos2[b, h, dst] = w[src], p[src]
    return {"acc": acc2, "pos": pos2, "lens": s["lens"].clamp(max=keep), "pool": None}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm_rope":
        return _exact_norm_rope(case, s)
    if kind == "append":
        return _exact_append(case, s)
    if kind == "evict":
        return _exact_evict(case, s)
    return _exact_attend(case, s)
