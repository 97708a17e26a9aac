"""The workspace of attention over the cache: 0 for heads and widths that the call refuses, whatever they are, without a GPU."""
import pytest

import reduction_codec_amd as rca


def size(tokens=10, heads=8, kv=2, d=128):
    return rca.lib().rc_mxfp4_cache_attention_workspace(tokens, heads, kv, d)


@pytest.mark.parametrize("bad", [{"heads": 0}, {"heads": 0, "kv": 1 << 32}, {"heads": 0, "kv": 3 << 32}, {"heads": 0, "kv": 1 << 40},
                                 {"heads": 0, "kv": 70000}, {"kv": 0}, {"kv": 1 << 32}, {"heads": 65536}, {"heads": 7},
                                 {"d": 0}, {"d": 80}, {"d": 512}, {"d": (1 << 32) + 128}], ids=str)
def test_refused_sizes_take_none(bad):
    assert size(**bad) == 0


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_more_rows_and_heads_take_no_less(d):
    for kv, group in ((1, 1), (2, 4), (8, 4), (1100, 1), (65535, 1)):
        sizes = [size(n, kv * group, kv, d) for n in (0, 1, 16, 17, 128, 129, 5000, (1 << 31) - 1, 1 << 40)]
        assert sizes == sorted(sizes) and sizes[0] > 0
