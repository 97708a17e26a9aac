"""A cache's bytes tell page * d alone: rows of another width are refused where the caller names the page."""
import pytest
import torch

import reduction_codec_amd as rca

PAGE, KV, D = 32, 2, 128


def calls(dev, d, page):
    """The three calls with rows of width d on a cache of pages of 32 tokens of 128 values, with the page named or not."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    place = (*rca.mxfp4_cache_new(3, KV, PAGE, D, dev), i32([[1, 2]]), i32([40]), i32([0, 2]))
    rows = torch.ones(2, KV, d, device=dev)
    more = {} if page is None else {"page": page}
    return [lambda: rca.mxfp4_cache_append(rows, rows, *place, q=rows, **more),
            lambda: rca.mxfp4_cache_read(*place, 2, d, **more),
            lambda: rca.mxfp4_cache_attention(rows, *place, **more)]


@pytest.fixture
def on_the_cpu(monkeypatch):
    """The binding's checks without a GPU: calls end before the library is asked."""
    monkeypatch.setattr(rca, "_head_rows", lambda t, name, index: (*t.shape, t.shape[1] * t.shape[2]))
    monkeypatch.setattr(rca, "_check_dev", lambda *a: None)
    monkeypatch.setattr(rca, "_check_on", lambda *a: None)
    monkeypatch.setattr(rca, "_launch", lambda *a: None)


@pytest.mark.parametrize("d,page,fits", [(D, PAGE, True), (D, None, True), (D, 64, False), (D, 0, False), (64, PAGE, False),
                                         (256, PAGE, False), (64, 64, True), (64, None, True)])
def test_rows_of_another_width(on_the_cpu, d, page, fits):
    for call in calls("cpu", d, page):
        if fits:
            call()
        else:
            with pytest.raises(ValueError, match="a page of the cache holds"):
                call()


@pytest.mark.gpu
def test_on_the_gpu():
    dev = torch.device("cuda:0")
    for call in calls(dev, D, PAGE):
        call()
    for call in calls(dev, 64, PAGE) + calls(dev, D, 16):
        with pytest.raises(ValueError, match="a page of the cache holds"):
            call()


@pytest.mark.parametrize("pages,kv,page,d", [(4, 2, 8, 256), (4, 2, 48, 128), (4, 2, 1, 2048), (4, 2, 131072, 64), (4, 2, 0, 64),
                                             (4, 2, 64, 32), (4, 2, 256, 80), (4, 2, 32, 0), (4, 2, 16, 64), (4, 0, 32, 64),
                                             (-1, 2, 32, 64)])
def test_no_cache_that_the_calls_would_refuse_is_made(pages, kv, page, d):
    with pytest.raises(ValueError):
        rca.mxfp4_cache_new(pages, kv, page, d, "cpu")


@pytest.mark.parametrize("d,least", [(64, 32), (96, 64), (128, 16), (192, 32), (256, 16)])
def test_caches_of_every_width(d, least):
    for page in (least, 2 * least, 4096):
        k, v = rca.mxfp4_cache_new(2, 3, page, d, "cpu")
        assert k.shape == v.shape == (2, 3, page * d // 2048 * 1088) and not k.any()
    assert rca.mxfp4_cache_new(0, 3, least, d, "cpu")[0].shape[0] == 0


def test_a_window_past_64_bits_is_no_window(on_the_cpu, monkeypatch):
    """Positions end at 2^30: the library is handed no more than it can hold."""
    seen = []
    monkeypatch.setattr(rca, "_launch", lambda what, dev, stream, *args: seen.append(args[8]))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    place = (*rca.mxfp4_cache_new(3, KV, PAGE, D, "cpu"), i32([[1, 2]]), i32([40]), i32([0, 2]))
    for window in (0, 5, 1 << 31, (1 << 64) + 5):
        rca.mxfp4_cache_attention(torch.ones(2, KV, D), *place, window=window)
    assert seen[:2] == [0, 5] and all((1 << 30) < w < (1 << 64) for w in seen[2:])
