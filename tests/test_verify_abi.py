"""include/rfpx_verify.h on the host: exports, sizes and every refusal.  These
calls never reach the GPU."""
import ctypes as C
import os
import re

import pytest

import block_quantized_expert_amd as bqe
from test_attn_abi import ALIGN, ARG, BAD_BATCH, BAD_CACHE, P, SHAPE, WS, batch, cache, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bqe.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return bqe.lib()


def test_exports_every_declared_function(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rfpx_verify.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(rfpx_\w+)\s*\(", src))
    assert declared == set(bqe.VERIFY_SYMBOLS)
    for name in declared:
        assert hasattr(lib, name), name
    assert f"RFPX_TREE_COLS_MAX {bqe.TREE_COLS_MAX}\n" in src


def args(names, defaults, kw, c=None, b=None, cached=False):
    d = dict(defaults)
    d.update(kw)
    head = (C.byref(c or cache()),) if cached else ()
    return (*head, C.byref(b or batch()), *[d[k] for k in names.split()], None)


def masks(c=None, b=None, **kw):
    return args("n parents base words masks positions", dict(n=5, parents=P, base=None, words=1, masks=P, positions=P),
                kw, b=b)


def accept(c=None, b=None, **kw):
    return args("n parents tokens drawn cols path counts next lens_out",
                dict(n=5, parents=P, tokens=P, drawn=P, cols=4, path=P, counts=P, next=P, lens_out=P), kw, b=b)


def commit(c=None, b=None, **kw):
    return args("cols path counts acc pos", dict(cols=4, path=P, counts=P, acc=P, pos=P), kw, c, b, cached=True)


def forward(c=None, b=None, **kw):
    return args("q qs xt h n scale masks words out os lse ws wsb",
                dict(q=P, qs=4096, xt=1, h=32, n=5, scale=0.1, masks=P, words=1, out=2 * P, os=4096, lse=None, ws=P,
                     wsb=1 << 40), kw, c, b, cached=True)


@pytest.mark.parametrize("fn,make", [("rfpx_attn_tree_forward", forward), ("rfpx_kv_commit", commit)])
def test_cache_and_batch_refusals(lib, fn, make):
    for kw, st in BAD_CACHE:
        refused(lib, fn, st, *make(c=cache(**kw)))
    for kw, st in BAD_BATCH:
        refused(lib, fn, st, *make(b=batch(**kw)))
    for at in (0, 1):
        a = list(make())
        a[at] = None
        refused(lib, fn, ARG, *a)


@pytest.mark.parametrize("fn,make", [("rfpx_tree_masks", masks), ("rfpx_tree_accept", accept)])
def test_batch_refusals(lib, fn, make):
    for kw, st in [(dict(n_seqs=0), SHAPE), (dict(n_seqs=65536), SHAPE), (dict(max_cols=-1), SHAPE),
                   (dict(max_cols=1025), SHAPE), (dict(lens=None), ARG), (dict(starts=None), ARG),
                   (dict(lens=P + 2), ALIGN), (dict(starts=P + 1), ALIGN)]:
        refused(lib, fn, st, *make(b=batch(**kw)))
    a = list(make())
    a[0] = None
    refused(lib, fn, ARG, *a)


def test_tree_refusals(lib):
    for kw, st in [(dict(n=-1), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(words=0), SHAPE), (dict(words=33), SHAPE),
                   (dict(parents=None), ARG), (dict(masks=None), ARG), (dict(parents=P + 2), ALIGN),
                   (dict(base=P + 2), ALIGN), (dict(masks=P + 1), ALIGN), (dict(positions=P + 2), ALIGN)]:
        refused(lib, "rfpx_tree_masks", st, *masks(**kw))
    assert lib.rfpx_tree_masks(*masks(n=0, parents=None, masks=None)) == 0
    for kw, st in [(dict(n=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=1025), SHAPE), (dict(parents=None), ARG),
                   (dict(tokens=None), ARG), (dict(drawn=None), ARG), (dict(path=None), ARG), (dict(counts=None), ARG),
                   (dict(next=None), ARG), (dict(path=P + 2), ALIGN), (dict(lens_out=P + 1), ALIGN),
                   (dict(tokens=P + 3), ALIGN)]:
        refused(lib, "rfpx_tree_accept", st, *accept(**kw))
    for kw, st in [(dict(cols=0), SHAPE), (dict(cols=1025), SHAPE), (dict(path=None), ARG), (dict(counts=None), ARG),
                   (dict(acc=P + 2), ALIGN), (dict(pos=P + 2), ALIGN), (dict(path=P + 1), ALIGN)]:
        refused(lib, "rfpx_kv_commit", st, *commit(**kw))


def test_tree_attention_refusals(lib):
    for kw, st in [(dict(q=None), ARG), (dict(xt=2), ARG), (dict(h=33), SHAPE), (dict(n=-1), SHAPE),
                   (dict(scale=0.0), ARG), (dict(q=P + 2), ALIGN), (dict(qs=2048), SHAPE), (dict(out=P), ARG),
                   (dict(ws=None), ARG), (dict(ws=P + 16), ALIGN), (dict(wsb=0), WS), (dict(lse=P + 2), ALIGN),
                   (dict(masks=None), ARG), (dict(masks=P + 2), ALIGN), (dict(words=0), SHAPE), (dict(words=33), SHAPE)]:
        refused(lib, "rfpx_attn_tree_forward", st, *forward(**kw))
    assert lib.rfpx_attn_tree_forward(*forward(n=0, masks=None)) == 0


def test_sample_refusals(lib):
    names = "logits stride xt n vocab u t k p m tokens probs ws wsb".split()
    d = dict(logits=P, stride=1000, xt=0, n=3, vocab=1000, u=P, t=P, k=P, p=P, m=P, tokens=P, probs=P, ws=P, wsb=1 << 40)

    def call(**kw):
        return (*[{**d, **kw}[x] for x in names], None)

    for kw, st in [(dict(logits=None), ARG), (dict(u=None), ARG), (dict(tokens=None), ARG), (dict(xt=2), ARG),
                   (dict(xt=-1), ARG), (dict(n=-1), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(vocab=0), SHAPE),
                   (dict(vocab=(1 << 20) + 1), SHAPE), (dict(stride=999), SHAPE), (dict(stride=-1000), SHAPE),
                   (dict(stride=1 << 41), SHAPE),
                   (dict(logits=P + 2), ALIGN), (dict(logits=P + 1, xt=1), ALIGN), (dict(u=P + 2), ALIGN),
                   (dict(t=P + 1), ALIGN), (dict(k=P + 2), ALIGN), (dict(p=P + 2), ALIGN), (dict(m=P + 2), ALIGN),
                   (dict(tokens=P + 2), ALIGN), (dict(probs=P + 2), ALIGN), (dict(ws=None), ARG),
                   (dict(ws=P + 64), ALIGN), (dict(wsb=0), WS)]:
        refused(lib, "rfpx_sample", st, *call(**kw))
    assert lib.rfpx_sample(*call(n=0, logits=None)) == 0
    for bad in ((-1, 1000, 0), (3, 0, 0), (3, (1 << 20) + 1, 1), (3, 1000, 7)):
        assert lib.rfpx_sample_workspace_bytes(*bad) == 0
    for xt in (0, 1):
        assert lib.rfpx_sample_workspace_bytes(0, 1, xt) >= 256
        assert lib.rfpx_sample_workspace_bytes(1, 1 << 20, xt) >= 256


def test_tree_workspace_depends_on_sizes_alone(lib):
    one = lib.rfpx_attn_tree_workspace_bytes(C.byref(cache()), C.byref(batch()), 32, 5)
    bare = lib.rfpx_attn_tree_workspace_bytes(C.byref(cache(pool=None)), C.byref(batch(lens=None, starts=None)), 32, 5)
    assert one == bare >= 256
    assert lib.rfpx_attn_tree_workspace_bytes(C.byref(cache()), C.byref(batch()), 12, 5) == 0
    assert b"rfpx_attn_tree_workspace_bytes" in lib.rfpx_last_error()
