"""Where the paged cache's operators take memory from for work on a caller's
stream, as tests/test_stream_memory.py asks of the others."""
import pytest
import torch

import reduction_codec_amd as rca
from tests.test_stream_memory import Stream, streams, zeros  # noqa: F401 (a fixture)

TOKENS, HEADS, KV, D = 2, 4, 2, 128


def place():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return (*rca.mxfp4_cache_new(1, KV, 16, D, "cpu"), i32([[0]]), i32([2]), i32([0, 2]))


CALLS = {
    "mxfp4_cache_append": lambda s: rca.mxfp4_cache_append(zeros(TOKENS, KV, D), zeros(TOKENS, KV, D), *place(),
                                                           q=zeros(TOKENS, HEADS, D), stream=s),
    "mxfp4_cache_read": lambda s: rca.mxfp4_cache_read(*place(), TOKENS, D, stream=s),
    "mxfp4_cache_attention": lambda s: rca.mxfp4_cache_attention(zeros(TOKENS, HEADS, D), *place(), lse=True, stream=s),
}


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(rca, "_head_rows", lambda t, name, index: (*t.shape, t.shape[1] * t.shape[2]))


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(name, streams):  # noqa: F811
    current, side, made = streams
    CALLS[name](side)
    assert made() and all(pool is side and told == [current] for pool, told in made()), made()


@pytest.mark.parametrize("name", CALLS)
def test_without_another_stream_nothing_is_told(name, streams):  # noqa: F811
    current, side, made = streams
    CALLS[name](None)
    first = len(made())
    CALLS[name](current)
    assert len(made()) == 2 * first > 0 and all(pool is current and not told for pool, told in made())


@pytest.mark.parametrize("name", CALLS)
def test_another_devices_stream_is_refused_before_anything_is_allocated(name, streams):  # noqa: F811
    _, _, made = streams
    with pytest.raises(ValueError, match="stream is on"):
        CALLS[name](Stream(torch.device("meta")))
    assert not made()
