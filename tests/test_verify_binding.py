"""The binding of the verification calls (CPU: the library and torch's streams
are stood in for): whose memory a call takes, streams of other devices, shapes."""
import pytest
import torch

import block_quantized_expert_amd as bqe
from test_binding_streams import Stream, batch, cache, tensor, world  # noqa: F401  (world: a fixture)

I32 = torch.int32

CALLS = {
    "rfpx_tree_masks": lambda s: bqe.rfpx_tree_masks(batch(), tensor(1, dtype=I32), stream=s),
    "rfpx_attn_tree_forward": lambda s: bqe.rfpx_attn_tree_forward(cache(), batch(), tensor(1, 4, 64),
                                                                   tensor(1, 1, dtype=I32), stream=s),
    "rfpx_sample": lambda s: bqe.rfpx_sample(tensor(3, 32), tensor(3), stream=s),
    "rfpx_tree_accept": lambda s: bqe.rfpx_tree_accept(batch(), *(tensor(1, dtype=I32),) * 3, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_taken_on_the_calls_stream(world, name):  # noqa: F811
    here, made, noted = world
    side = Stream()
    result = CALLS[name](side)
    assert made and all(s is side for _, s in made)
    mine = {t.data_ptr() for t, _ in made}
    for t in result if isinstance(result, tuple) else (result,):
        assert t.data_ptr() in mine and (t.data_ptr(), here) in noted


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(world, name):  # noqa: F811
    here, made, noted = world
    CALLS[name](None)
    assert made and all(s is here for _, s in made) and not noted


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(world, name):  # noqa: F811
    other = Stream()
    other.device_index = 1
    with pytest.raises(ValueError, match="current device"):
        CALLS[name](other)


def test_a_commit_on_another_devices_stream_is_refused(world):  # noqa: F811
    other = Stream()
    other.device_index = 1
    with pytest.raises(ValueError, match="current device"):
        bqe.rfpx_kv_commit(cache(), batch(), tensor(1, 1, dtype=I32), tensor(1, dtype=I32), stream=other)


@pytest.mark.parametrize("call", [
    lambda: bqe.rfpx_tree_masks(batch(), tensor(1, dtype=I32), masks=tensor(1, dtype=I32)),
    lambda: bqe.rfpx_tree_accept(batch(), *(tensor(1, dtype=I32),) * 3, path=tensor(1, dtype=I32)),
    lambda: bqe.rfpx_kv_commit(cache(), batch(), tensor(1, dtype=I32), tensor(1, dtype=I32)),
    lambda: bqe.rfpx_attn_tree_forward(cache(), batch(), tensor(1, 4, 64), tensor(1, dtype=I32)),
    lambda: bqe.rfpx_sample(tensor(32), tensor(1)),
    lambda: bqe.rfpx_sample(tensor(2, 32), tensor(1)),
    lambda: bqe.rfpx_sample(tensor(32, 2).T, tensor(2)),
    lambda: bqe.rfpx_tree_accept(batch(), tensor(1), *(tensor(1, dtype=I32),) * 2),
], ids=["masks", "path", "commit path", "attention masks", "one row", "few u", "strides", "parents of floats"])
def test_shapes_and_types_are_refused(world, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()
