"""A rotation has a row for every position that a kernel may read: the table's, and the first one for tokens before it,
even if the table has no columns. (A misaligned k stands for what would be accepted: nothing is launched.)"""
import pytest

import reduction_codec_amd as rca
from tests.test_cache_refusals import M, append


@pytest.mark.parametrize("columns,positions,status", [(0, 0, rca.ERR_RANGE), (0, 1, rca.ERR_ALIGN), (1, 15, rca.ERR_RANGE),
                                                      (1, 16, rca.ERR_ALIGN), (4, 0, rca.ERR_RANGE), (4, 64, rca.ERR_ALIGN)])
def test_rows(columns, positions, status):
    assert append(k=M, c_max_pages=columns, positions=positions) == status
    assert append(k=M, c_max_pages=columns, positions=positions, rotation=None) == rca.ERR_ALIGN
    assert append(k=M, c_max_pages=columns, positions=positions, rot=0) == rca.ERR_ALIGN
