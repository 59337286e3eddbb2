"""Which stream's memory the binding takes for a call on a stream (CPU: the
library and torch's streams are stood in for).  The allocator orders the uses of
a block along the stream that it was taken on, so that every tensor made inside
a call must be taken on the stream that the call runs on."""
import contextlib

import pytest
import torch

import block_quantized_expert_amd as bqe


class Stream:
    cuda_stream = 1
    device_index = -1  # where CPU tensors say they are


class Lib:
    """Answers every size with 256 and every call with success."""

    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith(("_bytes", "_words")) else b"" if name == "rfpx_last_error" else 0


@pytest.fixture
def world(monkeypatch):
    here, made, noted = Stream(), [], []
    now = [here]

    @contextlib.contextmanager
    def on(stream):
        if stream is None:
            yield
            return
        now.append(stream)
        yield
        now.pop()

    def recorded(make):
        def f(*a, **kw):
            kw.pop("device", None)
            t = make(*a, **kw)
            made.append((t, now[-1]))
            return t
        return f

    monkeypatch.setattr(bqe, "_lib", Lib())
    monkeypatch.setattr(bqe, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded(torch.Tensor.new_empty), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: noted.append((t.data_ptr(), s)), raising=False)
    return here, made, noted


def tensor(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype)


def layer():
    return bqe.MoeLayer(32, 32, 4, 2, tensor(4, 32), tensor(256, dtype=torch.uint8), [[4, 4, 4]] * 5)


def dense():
    return bqe.DenseMatrix(4, 32, 32, tensor(256, dtype=torch.uint8))


def cache():
    return bqe.KvCache(2, 64, 32, 4, pool=tensor(256, dtype=torch.uint8))


def batch():
    i = torch.int32
    return bqe.KvBatch(tensor(1, 2, dtype=i), tensor(1, dtype=i), tensor(2, dtype=i), 1, 32)


CALLS = {
    "rfpx_pack": lambda s: bqe.rfpx_pack(4, tensor(2, 32), stream=s),
    "rfpx_pack_weighted": lambda s: bqe.rfpx_pack_weighted(4, tensor(2, 32), tensor(32), stream=s),
    "rfpx_pack_codes": lambda s: bqe.rfpx_pack_codes(4, tensor(2, 32, dtype=torch.uint8),
                                                     tensor(2, 1, dtype=torch.int16), stream=s),
    "rfpx_unpack": lambda s: bqe.rfpx_unpack(4, tensor(34, dtype=torch.uint8), 2, 32, stream=s),
    "moe_image_build": lambda s: bqe.moe_image_build(32, 32, 1, [[4, 4, 4]], [tensor(17, dtype=torch.uint8)] * 3, stream=s),
    "moe_image_validate": lambda s: bqe.moe_image_validate(layer(), stream=s),
    "moe_image_unpack": lambda s: bqe.moe_image_unpack(layer(), 0, 0, stream=s),
    "moe_route_topk": lambda s: bqe.moe_route_topk(layer(), tensor(3, 32), stream=s),
    "moe_layer_forward": lambda s: bqe.moe_layer_forward(layer(), tensor(3, 32), stream=s),
    "moe_prefill_forward": lambda s: bqe.moe_prefill_forward(layer(), tensor(3, 32), stream=s),
    "DenseMatrix": lambda s: bqe.DenseMatrix(4, 32, 32, tensor(256, dtype=torch.uint8), stream=s).image,
    "DenseMatrix.unpack": lambda s: dense().unpack(stream=s),
    "rfpx_dense_forward": lambda s: bqe.rfpx_dense_forward(dense(), tensor(3, 32), stream=s),
    "rfpx_qk_norm_rope": lambda s: bqe.rfpx_qk_norm_rope(tensor(1, 4, 64), tensor(1, 2, 64), tensor(1, dtype=torch.int32),
                                                         stream=s),
    "rfpx_kv_unpack": lambda s: bqe.rfpx_kv_unpack(cache(), batch(), 1, stream=s),
    "rfpx_attn_forward": lambda s: bqe.rfpx_attn_forward(cache(), batch(), tensor(1, 4, 64), stream=s),
    "rfpx_kv_evict": lambda s: bqe.rfpx_kv_evict(cache(), batch(), 1, 0, tensor(1, 2, 64),
                                                 tensor(1, 2, 64, dtype=torch.int32), stream=s),
    "rfpx_stream_read": lambda s: bqe.rfpx_stream_read(tensor(64), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_taken_on_the_calls_stream(world, name):
    here, made, noted = world
    if name in ("DenseMatrix.unpack", "rfpx_dense_forward"):  # the matrix is made on the current stream
        CALLS["DenseMatrix"](None)
        skip = len(made)
        made.clear()
    else:
        skip = 0
    side = Stream()
    result = CALLS[name](side)
    taken = [(t, s) for t, s in made[skip:]]
    assert taken, "the call takes no memory of its own"
    assert all(s is side for _, s in taken), [s is here for _, s in taken]
    # what comes back may be used on the stream that the caller is on
    mine = {t.data_ptr() for t, _ in taken}
    for t in result if isinstance(result, tuple) else (result,):
        if t.data_ptr() in mine:
            assert (t.data_ptr(), here) in noted


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(world, name):
    here, made, noted = world
    CALLS[name](None)
    assert made and all(s is here for _, s in made) and not noted


@pytest.mark.parametrize("validate", [True, False])
def test_upload_waits_for_its_stream(world, monkeypatch, validate):
    """The image is checked on the stream that builds it, and that stream is
    waited for before the canonical bytes go."""
    here, made, _ = world
    waited, checked = [], []
    side = Stream()
    monkeypatch.setattr(Stream, "synchronize", lambda self: waited.append(self), raising=False)

    def validate_on(l, report=None, stream=None):
        checked.append(stream)
        return torch.zeros(4, dtype=torch.int32)
    monkeypatch.setattr(bqe, "moe_image_validate", validate_on)

    class Synthetic:
        import numpy as np
        d = f = 32
        E, k = 1, 1
        fmts = [[4, 4, 4]] * 2
        blob = np.zeros(6 * 544, np.uint8)
        offsets = np.arange(6) * 544
        wr = np.zeros((1, 32), np.float32)

        def mat(self, e, m):
            return self.blob[:544]
    bqe.upload_layer(Synthetic(), device="cpu", stream=side, validate=validate)
    assert waited == [side] and checked == ([side] if validate else [])


@pytest.mark.parametrize("at", [0, 1, 2])
def test_a_batch_lies_on_one_device(world, at):
    i = torch.int32
    t = [tensor(1, 2, dtype=i), tensor(1, dtype=i), tensor(2, dtype=i)]
    bqe.KvBatch(*t, 1, 32)
    t[at] = t[at].to("meta")
    with pytest.raises(ValueError, match="one device"):
        bqe.KvBatch(*t, 1, 32)


@pytest.mark.parametrize("name", ["rfpx_qk_norm_rope", "rfpx_kv_unpack", "rfpx_attn_forward", "rfpx_kv_evict"])
def test_a_stream_of_another_device_is_refused(world, name):
    other = Stream()
    other.device_index = 1
    with pytest.raises(ValueError, match="current device"):
        CALLS[name](other)
