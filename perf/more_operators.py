"""What is measured of the operators that verify a tree of drafted tokens:
cases, inputs, their plain forms in elementary torch operations, and their
values in 64 bits.

A step brings every sequence a tree of columns.  Column 0 is the token that
was settled last, the others are drafts; parents[j] < j is the column that
column j follows (-1: none).  In order, a step
  masks   turns parents into ancestor bits and positions,
  attend  lets every column see the context and its own ancestors,
  sample  draws a token from every column's logits,
  accept  follows the drafts that the drawn tokens confirm,
  commit  moves their keys and values together in the cache.

The cache is a pool of pages of 4-bit blocks.  A page holds, for every kv
head, a slab of page tokens; a head's D values of a token are D/32 blocks of
32 codes (value (c - 7.5) * 2^(e-127), two codes to a byte, the even one in
the low half), laid out as

  keys    [token][octet of a block: 4][block: D/32][4 bytes]
  scales  [token][block] (one byte e each)
  values  [token / 4][byte of a block: 16][pair: 2][block / 2][token & 1][block & 1]
  scales  [token][block]
"""
import math
import random

import torch

own = False

VOCAB = 32000  # of drafted and drawn tokens where no logits say it


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a step of one conversation, a small tree: latency
        dict(name="masks 1 tree of 16", kind="masks", seqs=1, cols=16, ragged=False),
        # a large batch, each sequence with a tree of its own size
        dict(name="masks 64 trees to 256", kind="masks", seqs=64, cols=256, ragged=True),
        # one short conversation with 16 drafts: latency
        dict(name="attend tree 16, 1021", kind="attend", dtype="bfloat16", seqs=1, cols=16, length=1021, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64),
        # a batch of small trees, every sequence at its own length, fp32 as a projection leaves it
        dict(name="attend 8 trees, to 8192", kind="attend", dtype="float32", seqs=8, cols=12, length=8192, ragged=True,
             heads=32, kv_heads=8, dim=64, page=32),
        # a wide tree at the end of one long context
        dict(name="attend tree 64, 131071", kind="attend", dtype="bfloat16", seqs=1, cols=64, length=131071,
             ragged=False, heads=32, kv_heads=8, dim=128, page=256),
        # one column, nucleus sampling, fp32 logits as a projection leaves them: latency
        dict(name="sample 1 row 32000", kind="sample", dtype="float32", rows=1, vocab=32000, filters="top_p"),
        # the columns of one wide tree, or of a batch; each request with settings of its own
        dict(name="sample 64 rows 131072", kind="sample", dtype="bfloat16", rows=64, vocab=131072, filters="mixed"),
        # a large batch of trees
        dict(name="sample 512 rows 131072", kind="sample", dtype="float32", rows=512, vocab=131072, filters="mixed"),
        # a step of one conversation: latency
        dict(name="accept 1 tree of 16", kind="accept", seqs=1, cols=16, ragged=False),
        dict(name="accept 64 trees to 256", kind="accept", seqs=64, cols=256, ragged=True),
        # one layer's cache after a step of one conversation
        dict(name="commit 1 tree of 16", kind="commit", seqs=1, cols=16, depth=5, length=1021, ragged=False,
             kv_heads=8, dim=128, page=64),
        # ... and of a batch, long drafts
        dict(name="commit 64 trees of 64", kind="commit", seqs=64, cols=64, depth=12, length=600, ragged=True,
             kv_heads=8, dim=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["masks", "attend", "attend", "attend", "sample", "sample", "sample", "accept", "commit"])
    ragged = rng.random() < 0.5
    if kind in ("masks", "accept"):
        return dict(kind=kind, seqs=_log_int(rng, 1, 64), cols=_log_int(rng, 2, 256), ragged=ragged)
    if kind == "sample":
        vocab = _log_int(rng, 1000, 200000)
        return dict(kind=kind, dtype=rng.choice(["bfloat16", "float32"]),
                    rows=_log_int(rng, 1, min(512, 512 * 131072 // vocab)), vocab=vocab,
                    filters=rng.choice(["mixed", "mixed", "none", "top_k", "top_p", "min_p"]))
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    if kind == "commit":
        cols = _log_int(rng, 2, 256)
        return dict(kind=kind, seqs=_log_int(rng, 1, 64), cols=cols, depth=rng.randrange(1, min(cols, 16) + 1),
                    length=cols + _log_int(rng, 1, 500), ragged=ragged, kv_heads=kv_heads, dim=dim, page=page)
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    seqs, cols = _log_int(rng, 1, 16), _log_int(rng, 2, 128)
    # tokens of the cache and products at most those of the longest listed one
    most = min(131071 * 8 * 128 // (seqs * kv_heads * dim), 131071 * 64 * 32 * 128 // (seqs * cols * heads * dim))
    length = max(cols, _log_int(rng, 1, max(1, min(most, 131071))))
    return dict(kind=kind, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]), seqs=seqs, cols=cols, length=length,
                ragged=ragged, heads=heads, kv_heads=kv_heads, dim=dim, page=page)


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _sizes(case):
    """Length and columns of every sequence: the case's own, or spread below
    them (the first sequence has them in full)."""
    b, length, cols = case["seqs"], case.get("length", 2000), case["cols"]
    if not case["ragged"]:
        return [length] * b, [cols] * b
    r = random.Random(b * 1000003 + length * 17 + cols)
    n = [cols] + [r.randint(1, cols) for _ in range(b - 1)]
    return [length] + [max(n[i], r.randint(max(1, length // 4), length)) for i in range(1, b)], n


def _trees(n, rng):
    """Parents of all columns: level by level, every column below one of the
    level before, as a draft model lays them out."""
    parents = []
    for size in n:
        level, at = [0], 1
        mine = [-1]
        while at < size:
            width = min(size - at, rng.randint(1, 2 + size // 6))
            mine += sorted(rng.choice(level) for _ in range(width))
            level = list(range(at, at + width))
            at += width
        parents += mine
    return parents


def _drawn(parents, starts, rng):
    """Drafted tokens, and the tokens drawn at every column: a walk from the
    root, each step of which is confirmed four times in five."""
    tokens = [rng.randrange(VOCAB) for _ in parents]
    drawn = [rng.randrange(VOCAB) for _ in parents]
    for first, end in zip(starts, starts[1:]):
        at = 0
        while True:
            below = [j for j in range(at + 1, end - first) if parents[first + j] == at]
            if not below or rng.random() > 0.8:
                break
            child = rng.choice(below)
            drawn[first + at] = tokens[first + child]
            at = child
    return tokens, drawn


def _paths(n, depth, width, rng):
    """Columns that stay, up to `depth` of each tree.  None of them lies in a
    place that another one moves to, so that every pass moves the same."""
    path, counts = [], []
    for size in n:
        count = rng.randint(min(2, size, depth), min(size, depth))
        moved = min(count - 1, size - count)
        mine = list(range(count - moved)) + sorted(rng.sample(range(count, size), moved))
        counts.append(count)
        path.append(mine + [-1] * (width - count))
    return path, counts


def _slab_parts(page, dim):
    half, s = page * dim // 2, page * dim // 32
    return [half, s, half, s]


def _pool(case, total, g):
    """A pool of random codes, scales of values of about 1."""
    page, dim = case["page"], case["dim"]
    n, half, s = total * case["kv_heads"], *_slab_parts(page, dim)[:2]
    made = []
    for k in range(4):
        lo, hi, size = ((0, 256, half), (124, 126, s))[k % 2]
        made.append(torch.randint(lo, hi, (n, size), generator=g, device="cuda", dtype=torch.uint8))
    return torch.cat(made, -1).reshape(-1)


def _settings(case, rng):
    """Temperature, top_k, top_p and min_p of every row."""
    rows, f = case["rows"], case["filters"]
    t = [rng.choice([0.6, 0.8, 1.0, 1.0, 1.3]) for _ in range(rows)]
    k, p, m = [0] * rows, [1.0] * rows, [0.0] * rows
    for i in range(rows):
        pick = rng.choice(["top_k", "top_p", "both", "min_p", "none", "greedy"]) if f == "mixed" else f
        if pick in ("top_k", "both"):
            k[i] = rng.choice([8, 20, 50, 64, 200])
        if pick in ("top_p", "both"):
            p[i] = rng.choice([0.8, 0.9, 0.95, 0.99])
        if pick == "min_p":
            m[i] = rng.choice([0.02, 0.05, 0.1])
        if pick == "greedy":
            t[i] = 0.0
    return t, k, p, m


def prepare(case, seed):
    g, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)
    kind, s = case["kind"], dict(case)
    if kind == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a language model's logits: most tokens far below a few, padding and forbidden tokens at -inf
        x = 2.2 * torch.randn((rows, vocab), generator=g, device="cuda")
        few = torch.randint(0, vocab, (rows, 24), generator=g, device="cuda")
        x.scatter_add_(1, few, 4 + 8 * torch.rand((rows, 24), generator=g, device="cuda"))
        x[:, vocab - vocab // 100:] = -math.inf
        s["logits"] = x.to(_dtype(case["dtype"]))
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        t, k, p, m = _settings(case, rng)
        s["temperature"], s["top_p"], s["min_p"] = (torch.tensor(v, device="cuda") for v in (t, p, m))
        s["top_k"] = _ints(k)
        return s
    lens, n = _sizes(case)
    starts = [sum(n[:i]) for i in range(len(n) + 1)]
    page = case.get("page", 64)
    b, per = len(n), -(-case.get("length", 2000) // page)
    total = b * per + 3
    table = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 1000))[:b * per].reshape(b, per)
    s.update(lens=_ints(lens), starts=_ints(starts), table=table.int().cuda(), rows=starts[-1], max_cols=max(n),
             max_len=max(lens), per=per)
    if kind in ("masks", "attend", "accept"):
        parents = _trees(n, rng)
        s["parents"] = _ints(parents)
        s["words"] = -(-max(n) // 32)
    if kind == "masks":
        # positions go on where the context's end, whatever an eviction has cut from the cache
        s["base"] = s["lens"] + torch.randint(0, 1 << 18, (b,), generator=g, device="cuda", dtype=torch.int32)
    elif kind == "accept":
        tokens, drawn = _drawn(parents, starts, rng)
        s["tokens"], s["drawn"] = _ints(tokens), _ints(drawn)
    else:
        s["pool"] = _pool(case, total, g)
    if kind == "commit":
        path, counts = _paths(n, case["depth"], max(n), rng)
        s["path"], s["counts"] = _ints(path), _ints(counts)
        shape = (b, case["kv_heads"], per * page)
        s["acc"] = torch.rand(shape, generator=g, device="cuda")
        s["pos"] = torch.randint(0, 1 << 20, shape, generator=g, device="cuda", dtype=torch.int32)
    if kind == "attend":
        q = torch.randn((s["rows"], case["heads"], case["dim"]), generator=g, device="cuda") * 0.7
        s["q"] = q.to(_dtype(case["dtype"]))
        s["scale"] = case["dim"] ** -0.5
        s["masks"] = _words(_seen(s), s["words"])[_rows_of(s)[:2]]
    if own:
        import block_quantized_expert_amd as bqe
        if "pool" in s:
            s["cache"] = bqe.KvCache(case["kv_heads"], case["dim"], page, total, pool=s["pool"])
        s["batch"] = bqe.KvBatch(s["table"], s["lens"], s["starts"], max_cols=s["max_cols"], max_len=s["max_len"])
    return s


# ------------------------------------------------------------- plain forms

def _rows_of(s):
    """Sequence, column and slot of every row."""
    row = torch.arange(s["rows"], device="cuda")
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, row, right=True) - 1
    n = starts[1:] - starts[:-1]
    col = row - starts[seq]
    return seq, col, s["lens"].long()[seq] - n[seq] + col


def _padded(s, x, fill):
    seq, col, _ = _rows_of(s)
    out = torch.full((s["seqs"], s["max_cols"]), fill, dtype=x.dtype, device="cuda")
    out[seq, col] = x
    return out


def _seen(s):
    """[sequence][column][column]: 1 where the second is the first or an
    ancestor of it: the sum of all powers of the parent matrix, by squaring."""
    parents = _padded(s, s["parents"], -1)
    cols = s["max_cols"]
    up = (parents.unsqueeze(-1) == torch.arange(cols, device="cuda")).float()
    seen = torch.eye(cols, device="cuda") + up
    for _ in range(max(1, cols - 1).bit_length()):
        up = up @ up
        seen = seen + seen @ up
    return seen > 0


def _words(bits, words):
    """int32 words of truth values [..][n], bit j % 32 of word j / 32."""
    bits = torch.nn.functional.pad(bits, (0, 32 * words - bits.shape[-1])).unflatten(-1, (words, 32))
    return (bits.long() << torch.arange(32, device="cuda")).sum(-1).int()


def _plain_masks(s):
    seq, col, _ = _rows_of(s)
    seen = _seen(s)[seq, col]
    return {"masks": _words(seen, s["words"]), "positions": s["base"][seq] + seen.sum(-1, dtype=torch.int32) - 1}


def _values(codes, scales):
    """fp32 values of codes [.., D] and scales [.., D/32]."""
    c = codes.float().unflatten(-1, (-1, 32)) - 7.5
    return (c * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


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


def _plain_attend(s):
    b, hk, g, d, cols = s["seqs"], s["kv_heads"], s["heads"] // s["kv_heads"], s["dim"], s["max_cols"]
    k, v = _cached(s["pool"], s["table"], s["page"], hk, d)
    length = k.shape[2]
    seq, col, slot = _rows_of(s)
    q = torch.zeros((b, cols, hk * g, d), device="cuda")
    q[seq, col] = s["q"].float()
    q = q.view(b, cols, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, cols * g, d)
    # what every column sees: the context, and the columns that its bits name
    bits = ((s["masks"].unsqueeze(-1) >> torch.arange(32, device="cuda")) & 1).bool().flatten(1)
    context = slot - col
    sees = torch.zeros((b, cols, length), dtype=torch.bool, device="cuda")
    at = torch.arange(length, device="cuda") - context.unsqueeze(-1)
    named = torch.gather(bits, 1, at.clamp(0, bits.shape[1] - 1)) & (at < bits.shape[1])
    sees[seq, col] = (at < 0) | (named & (at + context.unsqueeze(-1) < s["lens"].long()[seq].unsqueeze(-1)))
    sees = sees.view(b, 1, cols, 1, length).expand(b, 1, cols, g, length).reshape(b, 1, cols * g, length)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~sees, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    out = torch.matmul(p, v).view(b, hk, cols, g, d).permute(0, 2, 1, 3, 4).reshape(b, cols, hk * g, d)
    lse = (top + total.log()).view(b, hk, cols, g).permute(0, 2, 1, 3).reshape(b, cols, hk * g)
    return {"out": out[seq, col].to(_dtype(s["dtype"])), "lse": lse[seq, col]}


def _plain_sample(s):
    # whether a token is the one that u falls on is a matter of the last bits: 64 of them
    x, index = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    t = s["temperature"].double().unsqueeze(-1)
    rank = torch.arange(x.shape[1], device="cuda")
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(t > 0, t, torch.ones_like(t)))
    w = torch.where(t > 0, w, (rank == 0).double())
    k = s["top_k"].unsqueeze(-1)
    w = torch.where((k <= 0) | (rank < k), w, torch.zeros_like(w))
    upto = w.cumsum(-1)
    # the shortest beginning that reaches top_p of it all, and of that what min_p leaves
    p = s["top_p"].double().unsqueeze(-1)
    w = torch.where((p >= 1) | (upto - w < p * upto[:, -1:]) | (rank == 0), w, torch.zeros_like(w))
    w = torch.where(w < s["min_p"].double().unsqueeze(-1), torch.zeros_like(w), w)
    upto = w.cumsum(-1)
    total = upto[:, -1:]
    at = (upto <= s["u"].double().unsqueeze(-1) * total).sum(-1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(-1, keepdim=True) - 1)
    return {"tokens": torch.gather(index, 1, at)[:, 0].int(), "probs": (torch.gather(w, 1, at) / total)[:, 0].float()}


def _plain_accept(s):
    seq, col, _ = _rows_of(s)
    b, cols = s["seqs"], s["max_cols"]
    parents, tokens, drawn = (_padded(s, s[x], -1) for x in ("parents", "tokens", "drawn"))
    column = torch.arange(cols, device="cuda").expand(b, cols)
    above = parents.clamp(min=0).long()
    fits = (parents >= 0) & (tokens == torch.gather(drawn, 1, above))
    # of a column's children that fit the first one alone
    first = torch.full((b, cols), cols, device="cuda").scatter_reduce(
        1, above, torch.where(fits, column, torch.full_like(column, cols)), "amin")
    fits &= torch.gather(first, 1, above) == column
    fits[:, 0] = True
    real = torch.zeros((b, cols), dtype=torch.bool, device="cuda")
    real[seq, col] = True
    stays = real & ~(_seen(s) & ~fits.unsqueeze(1)).any(-1)
    counts = stays.sum(-1)
    path = torch.where(stays, column, torch.full_like(column, cols)).sort(-1).values
    last = torch.gather(path, 1, (counts - 1).unsqueeze(-1))
    path = torch.where(path == cols, torch.full_like(path, -1), path)
    n = s["starts"][1:] - s["starts"][:-1]
    return {"path": path.int(), "counts": counts.int(), "next": torch.gather(drawn, 1, last)[:, 0],
            "lens": s["lens"] - n + counts.int()}


def _plain_commit(s):
    page, dim, heads, nb = s["page"], s["dim"], s["kv_heads"], s["dim"] // 32
    column = torch.arange(s["max_cols"], device="cuda")
    q, i = (column < s["counts"].unsqueeze(-1)).nonzero(as_tuple=True)
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    dst, src = first[q] + i, first[q] + s["path"].long()[q, i]
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
        h = torch.arange(heads, device="cuda").view(1, -1, 1)
        at = s["table"].long()[q, j // page].view(-1, 1, 1)
        return at, h, torch.cat([k, ks, v, vs], -1).unsqueeze(1)

    pool[place(dst)] = pool[place(src)]
    for x in (s["acc"], s["pos"]):
        x[q, :, dst] = x[q, :, src]
    return {"pool": s["pool"], "acc": s["acc"], "pos": s["pos"]}


def run(s):
    kind = s["kind"]
    if not own:
        return {"masks": _plain_masks, "attend": _plain_attend, "sample": _plain_sample, "accept": _plain_accept,
                "commit": _plain_commit}[kind](s)
    import block_quantized_expert_amd as bqe
    if kind == "masks":
        masks, positions = bqe.rfpx_tree_masks(s["batch"], s["parents"], base=s["base"])
        return {"masks": masks, "positions": positions}
    if kind == "attend":
        lse = torch.empty(s["q"].shape[:2], device="cuda")
        return {"out": bqe.rfpx_attn_tree_forward(s["cache"], s["batch"], s["q"], s["masks"], s["scale"], lse=lse),
                "lse": lse}
    if kind == "sample":
        probs = torch.empty(s["rows"], device="cuda")
        tokens = bqe.rfpx_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                                 probs=probs)
        return {"tokens": tokens, "probs": probs}
    if kind == "accept":
        path, counts, following, lens = bqe.rfpx_tree_accept(s["batch"], s["parents"], s["tokens"], s["drawn"])
        return {"path": path, "counts": counts, "next": following, "lens": lens}
    bqe.rfpx_kv_commit(s["cache"], s["batch"], s["path"], s["counts"], acc=s["acc"], pos=s["pos"])
    return {"pool": s["pool"], "acc": s["acc"], "pos": s["pos"]}


# -------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    size = 4 if case.get("dtype") == "float32" else 2
    if kind == "sample":  # every logit; its difference from the largest, scaling, exponential and sum
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * 28, "flops": 4 * n}
    lens, n = _sizes(case)
    rows = sum(n)
    if kind == "masks":
        return {"bytes": rows * (4 + 4 * -(-max(n) // 32) + 4) + case["seqs"] * 12, "flops": rows}
    if kind == "accept":
        return {"bytes": rows * 12 + case["seqs"] * (max(n) + 6) * 4, "flops": rows}
    d = case["dim"]
    token = case["kv_heads"] * d * 17 / 16  # bytes of a token's keys and values
    if kind == "commit":  # of every moved token its blocks, weights and positions, read and written
        moved = sum(min(size, case["depth"]) // 2 for size in n)
        return {"bytes": 2 * moved * (token + case["kv_heads"] * 8) + case["seqs"] * (case["depth"] + 4) * 4, "flops": 0}
    # every column sees the context and, of the tree, some of its columns
    pairs = case["heads"] * sum(c * (length - c + math.log2(c) + 1) for length, c in zip(lens, n))
    return {"bytes": sum(lens) * token + rows * (case["heads"] * (d * size * 2 + 4) + 4 * -(-max(n) // 32)),
            "flops": 4 * pairs * d}


# ------------------------------------------------- the definition, 64 bits

def _ancestors(parents):
    """The columns from the root to each column of one tree."""
    lines = []
    for j, p in enumerate(parents):
        lines.append((lines[p] if p >= 0 else []) + [j])
    return lines


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
    pool = s["pool"].view(-1, hk, sum(_slab_parts(case["page"], d)))
    lens, starts, parents = s["lens"].tolist(), s["starts"].tolist(), s["parents"].tolist()
    out = torch.zeros((s["rows"], hk * g, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["rows"], hk * g), dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        first, n = starts[b], starts[b + 1] - starts[b]
        context = lens[b] - n
        hidden = torch.ones((n, lens[b]), dtype=torch.bool)
        hidden[:, :context] = False
        for i, line in enumerate(_ancestors(parents[first:first + n])):
            for j in line:
                hidden[i, context + j] = False
        hidden = hidden.cuda().repeat_interleave(g, 0)
        for h in range(hk):
            slab = pool[s["table"][b].long(), h]
            k = _slab_values(slab, lens[b], case["page"], d, True)
            v = _slab_values(slab, lens[b], case["page"], d, False)
            mine = slice(h * g, (h + 1) * g)
            x = (s["q"][first:first + n, mine].double().reshape(n * g, d) @ k.T) * s["scale"]
            x[hidden] = -math.inf
            z = torch.logsumexp(x, -1, keepdim=True)
            out[first:first + n, mine] = (torch.exp(x - z) @ v).view(n, g, d)
            lse[first:first + n, mine] = z.view(n, g)
    return {"out": out, "lse": lse}


def _exact_sample(case, s):
    tokens, probs = [], []
    for i in range(case["rows"]):
        x = s["logits"][i].double()
        t, u, k = s["temperature"][i].item(), s["u"][i].item(), s["top_k"][i].item()
        p, m = s["top_p"][i].item(), s["min_p"][i].item()
        order = torch.argsort(-x, stable=True)
        order = order[:1] if t == 0 else order[:k] if k > 0 else order
        share = torch.exp((x[order] - x[order[0]]) / t) if t else torch.ones_like(x[:1])
        if p < 1:
            before = torch.cumsum(share, 0) / share.sum()
            order = order[:int((before < p).sum()) + 1]
            share = share[:order.numel()]
        keep = int((share >= m).sum())
        upto = torch.cumsum(share[:keep], 0)
        at = min(int(torch.searchsorted(upto, u * upto[-1], right=True)), keep - 1)
        tokens.append(int(order[at]))
        probs.append((share[at] / upto[-1]).item())
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "probs": torch.tensor(probs, dtype=torch.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "attend":
        return _exact_attend(case, s)
    if kind == "sample":
        return _exact_sample(case, s)
    starts = s["starts"].tolist()
    if kind == "commit":
        acc, pos = s["acc"].double().cpu(), s["pos"].cpu()
        for b, n in enumerate(s["counts"].tolist()):
            context = s["lens"][b].item() - (starts[b + 1] - starts[b])
            for i, j in enumerate(s["path"][b].tolist()[:n]):
                acc[b, :, context + i], pos[b, :, context + i] = acc[b, :, context + j], pos[b, :, context + j]
        return {"pool": None, "acc": acc, "pos": pos}
    r = {"masks": [], "positions": [], "path": [], "counts": [], "next": [], "lens": []}
    for b, (first, end) in enumerate(zip(starts, starts[1:])):
        parents = s["parents"][first:end].tolist()
        if kind == "masks":
            for line in _ancestors(parents):
                word = [sum(1 << (j % 32) for j in line if j // 32 == w) for w in range(s["words"])]
                r["masks"].append([w - (1 << 32) if w >> 31 else w for w in word])
                r["positions"].append(s["base"][b].item() + len(line) - 1)
            continue
        tokens, drawn, line = s["tokens"][first:end].tolist(), s["drawn"][first:end].tolist(), [0]
        while True:
            below = [j for j, p in enumerate(parents) if p == line[-1] and tokens[j] == drawn[line[-1]]]
            if not below:
                break
            line.append(below[0])
        r["path"].append(line + [-1] * (s["max_cols"] - len(line)))
        r["counts"].append(len(line))
        r["next"].append(drawn[line[-1]])
        r["lens"].append(s["lens"][b].item() - (end - first) + len(line))
    names = ("masks", "positions") if kind == "masks" else ("path", "counts", "next", "lens")
    return {x: torch.tensor(r[x], dtype=torch.int32) for x in names}
