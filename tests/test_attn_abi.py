"""include/rfpx_attn.h on the host: exports, sizes and every refusal.  These
calls never reach the GPU."""
import ctypes as C
import os
import re

import pytest

import block_quantized_expert_amd as bqe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, SHAPE, ALIGN, WS = -1, -2, -3, -5
P = 0x10000  # stands for a device pointer that no refused call reads


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bqe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return bqe.lib()


def test_exports_every_declared_function(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rfpx_attn.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(rfpx_\w+)\s*\(", src))
    assert declared == set(bqe.ATTN_SYMBOLS)
    for name in declared:
        assert hasattr(lib, name), name


def test_pool_bytes(lib):
    # 17/16 bytes a value pair: 64 tokens x 8 heads x 128 values, keys and values
    assert lib.rfpx_kv_pool_bytes(8, 128, 64, 10) == 10 * 8 * 64 * 136
    assert lib.rfpx_kv_pool_bytes(1, 64, 32, 1) == 32 * 68
    assert lib.rfpx_kv_pool_bytes(1024, 256, 256, 100000) == 100000 * 1024 * 256 * 272
    for bad in ((0, 128, 64, 1), (1025, 128, 64, 1), (8, 96, 64, 1), (8, 128, 48, 1), (8, 128, 64, 0),
                (8, 128, 16, 1), (-1, 128, 64, 1)):
        assert lib.rfpx_kv_pool_bytes(*bad) == 0


def cache(**kw):
    d = dict(n_kv_heads=8, head_dim=128, page_tokens=64, n_pages=10, pool=P, pool_bytes=10 * 8 * 64 * 136)
    d.update(kw)
    return bqe.KvCacheC(*[d[k] for k in ("n_kv_heads", "head_dim", "page_tokens", "n_pages", "pool", "pool_bytes")])


def batch(**kw):
    d = dict(n_seqs=2, pages_per_seq=4, max_cols=4, max_len=200, page_table=P, lens=P, starts=P)
    d.update(kw)
    return bqe.KvBatchC(*[d[k] for k in ("n_seqs", "pages_per_seq", "max_cols", "max_len", "page_table", "lens",
                                        "starts")])


BAD_CACHE = [(dict(pool=None), ARG), (dict(pool=P + 128), ALIGN), (dict(pool_bytes=10 * 8 * 64 * 136 - 1), WS),
             (dict(head_dim=80), SHAPE), (dict(page_tokens=512), SHAPE), (dict(n_pages=0), SHAPE)]
BAD_BATCH = [(dict(n_seqs=0), SHAPE), (dict(n_seqs=65536), SHAPE), (dict(pages_per_seq=0), SHAPE),
             (dict(pages_per_seq=(1 << 24) + 1), SHAPE), (dict(max_cols=-1), SHAPE), (dict(max_len=-1), SHAPE),
             (dict(page_table=None), ARG), (dict(lens=None), ARG), (dict(starts=None), ARG),
             (dict(lens=P + 2), ALIGN)]


def refused(lib, fn, st, *args):
    assert getattr(lib, fn)(*args) == st, (fn, lib.rfpx_last_error())
    assert fn.encode() in lib.rfpx_last_error()


def append(lib, c=None, b=None, **kw):
    d = dict(k=P, ks=1024, v=P, vs=1024, xt=1, n=5, positions=None, pos=None, acc=None)
    d.update(kw)
    return (C.byref(c or cache()), C.byref(b or batch()), *[d[k] for k in ("k", "ks", "v", "vs", "xt", "n",
                                                                          "positions", "pos", "acc")], None)


def unpack(lib, c=None, b=None, **kw):
    d = dict(n=5, k=P, v=P, ot=0)
    d.update(kw)
    return (C.byref(c or cache()), C.byref(b or batch()), *[d[k] for k in ("n", "k", "v", "ot")], None)


def forward(lib, c=None, b=None, **kw):
    d = dict(q=P, qs=4096, xt=1, h=32, n=5, scale=0.1, out=2 * P, os=4096, lse=None, ws=P, wsb=1 << 40)
    d.update(kw)
    return (C.byref(c or cache()), C.byref(b or batch()),
            *[d[k] for k in ("q", "qs", "xt", "h", "n", "scale", "out", "os", "lse", "ws", "wsb")], None)


def weights(lib, c=None, b=None, **kw):
    d = dict(q=P, qs=4096, xt=1, h=32, n=5, scale=0.1, lse=P, decay=1.0, acc=P, acc_out=P)
    d.update(kw)
    return (C.byref(c or cache()), C.byref(b or batch()),
            *[d[k] for k in ("q", "qs", "xt", "h", "n", "scale", "lse", "decay", "acc", "acc_out")], None)


def evict(lib, c=None, b=None, **kw):
    d = dict(keep=100, recent=10, acc=P, pos=P, acc_out=P, pos_out=P, lens_out=P, ws=P, wsb=1 << 40)
    d.update(kw)
    return (C.byref(c or cache()), C.byref(b or batch()),
            *[d[k] for k in ("keep", "recent", "acc", "pos", "acc_out", "pos_out", "lens_out", "ws", "wsb")], None)


@pytest.mark.parametrize("fn,make", [("rfpx_kv_append", append), ("rfpx_kv_unpack", unpack),
                                     ("rfpx_attn_forward", forward), ("rfpx_attn_weights", weights),
                                     ("rfpx_kv_evict", evict)])
def test_cache_and_batch_refusals(lib, fn, make):
    for kw, st in BAD_CACHE:
        refused(lib, fn, st, *make(lib, c=cache(**kw)))
    for kw, st in BAD_BATCH:
        refused(lib, fn, st, *make(lib, b=batch(**kw)))
    args = list(make(lib))
    args[0] = None
    refused(lib, fn, ARG, *args)


def test_append_and_unpack_refusals(lib):
    for kw, st in [(dict(k=None), ARG), (dict(v=None), ARG), (dict(xt=2), ARG), (dict(n=-1), SHAPE),
                   (dict(n=(1 << 20) + 1), SHAPE), (dict(k=P + 8), ALIGN), (dict(ks=1028), ALIGN),
                   (dict(ks=1016), SHAPE), (dict(vs=0), SHAPE), (dict(pos=P), ARG),
                   (dict(pos=P + 2, positions=P), ALIGN), (dict(acc=P + 1), ALIGN)]:
        refused(lib, "rfpx_kv_append", st, *append(lib, **kw))
    for kw, st in [(dict(k=None), ARG), (dict(ot=3), ARG), (dict(n=-1), SHAPE), (dict(v=P + 4), ALIGN)]:
        refused(lib, "rfpx_kv_unpack", st, *unpack(lib, **kw))
    # nothing to do is no error, and nothing is launched
    assert lib.rfpx_kv_append(*append(lib, n=0)) == 0
    assert lib.rfpx_kv_unpack(*unpack(lib, n=0)) == 0
    assert lib.rfpx_attn_forward(*forward(lib, n=0)) == 0


def test_attention_refusals(lib):
    shared = [(dict(q=None), ARG), (dict(xt=-1), ARG), (dict(h=0), SHAPE), (dict(h=33), SHAPE),
              (dict(h=1032), SHAPE), (dict(n=-1), SHAPE), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
              (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(q=P + 2), ALIGN),
              (dict(qs=4095), ALIGN), (dict(qs=2048), SHAPE)]
    for kw, st in shared + [(dict(out=None), ARG), (dict(out=P), ARG), (dict(os=8), SHAPE), (dict(ws=None), ARG),
                            (dict(ws=P + 16), ALIGN), (dict(wsb=0), WS), (dict(lse=P + 2), ALIGN)]:
        refused(lib, "rfpx_attn_forward", st, *forward(lib, **kw))
    for kw, st in shared + [(dict(lse=None), ARG), (dict(acc=None), ARG), (dict(acc_out=None), ARG),
                            (dict(decay=float("nan")), ARG), (dict(acc=P + 2), ALIGN)]:
        refused(lib, "rfpx_attn_weights", st, *weights(lib, **kw))


def test_evict_refusals(lib):
    for kw, st in [(dict(keep=0), SHAPE), (dict(recent=-1), SHAPE), (dict(acc=None), ARG), (dict(pos=None), ARG),
                   (dict(acc_out=None), ARG), (dict(lens_out=None), ARG), (dict(ws=None), ARG), (dict(ws=P + 4), ALIGN),
                   (dict(wsb=100), WS), (dict(pos_out=P + 1), ALIGN)]:
        refused(lib, "rfpx_kv_evict", st, *evict(lib, **kw))
    assert lib.rfpx_kv_evict_workspace_bytes(C.byref(cache()), C.byref(batch()), 0) == 0
    n = lib.rfpx_kv_evict_workspace_bytes(C.byref(cache()), C.byref(batch(page_table=None)), 100)
    assert n >= 2 * 8 * 4 * 64 * 4


def test_attention_workspace_depends_on_sizes_alone(lib):
    one = lib.rfpx_attn_workspace_bytes(C.byref(cache()), C.byref(batch()), 32, 5)
    bare = lib.rfpx_attn_workspace_bytes(C.byref(cache(pool=None)), C.byref(batch(lens=None, starts=None)), 32, 5)
    assert one == bare >= 256
    assert lib.rfpx_attn_workspace_bytes(C.byref(cache()), C.byref(batch()), 12, 5) == 0


def test_norm_rope_refusals(lib):
    freq = (C.c_double * 64)(*[0.5] * 64)

    def call(**kw):
        d = dict(q=P, qs=4096, h=32, k=P, ks=1024, hk=8, d=128, xt=1, n=5, positions=P, qw=P, kw=P, eps=1e-6,
                 rope=bqe.RopeC(128, 0, C.cast(freq, C.c_void_p)), qo=P, qos=4096, ko=P, kos=1024, ot=1)
        d.update(kw)
        r = d["rope"]
        return (*[d[k] for k in ("q", "qs", "h", "k", "ks", "hk", "d", "xt", "n", "positions", "qw", "kw", "eps")],
                C.byref(r) if r is not None else None, *[d[k] for k in ("qo", "qos", "ko", "kos", "ot")], None)

    f = C.cast(freq, C.c_void_p)
    nan = (C.c_double * 64)(*[float("nan")] * 64)
    for kw, st in [(dict(q=None), ARG), (dict(ko=None), ARG), (dict(xt=5), ARG), (dict(ot=-1), ARG),
                   (dict(d=96), SHAPE), (dict(h=0, hk=0), SHAPE), (dict(h=1025), SHAPE), (dict(n=-1), SHAPE),
                   (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(positions=None), ARG),
                   (dict(positions=P + 2), ALIGN), (dict(qw=P + 4), ALIGN), (dict(qs=4100), ALIGN),
                   (dict(qs=4088), SHAPE), (dict(kos=8), SHAPE), (dict(ot=0), ARG),
                   (dict(qos=8192), ARG),
                   (dict(rope=bqe.RopeC(63, 0, f)), SHAPE), (dict(rope=bqe.RopeC(130, 0, f)), SHAPE),
                   (dict(rope=bqe.RopeC(-2, 0, f)), SHAPE), (dict(rope=bqe.RopeC(64, 2, f)), ARG),
                   (dict(rope=bqe.RopeC(64, 0, None)), ARG),
                   (dict(rope=bqe.RopeC(64, 0, C.cast(nan, C.c_void_p))), ARG)]:
        refused(lib, "rfpx_qk_norm_rope", st, *call(**kw))
    assert lib.rfpx_qk_norm_rope(*call(n=0)) == 0


def test_rope_frequencies():
    r = bqe.Rope(64, theta=500.0)
    assert r._freq[0] == 1.0 and abs(r._freq[31] - 500.0 ** (-62 / 64)) < 1e-15
    with pytest.raises(ValueError):
        bqe.Rope(64, inv_freq=[1.0])
    assert bqe.Rope(0).c.dim == 0
