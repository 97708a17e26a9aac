"""Offsets that do not ascend within the rows there are: attention does nothing, rather than what sequences that overlap
would add up to; in order but out of range, they are clamped."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def place(offsets, tokens, seed=1):
    seqs, page, columns = len(offsets) - 1, 16, 20
    g = torch.Generator().manual_seed(seed)
    plan = ref.Plan([(0, columns * page)] * min(seqs, 8), page, wider=0)
    cache = [c.to(DEV) for c in ref.random_cache(plan, 2, 128, 3, poison=False)[:2]]
    table = torch.randint(0, plan.pages, (seqs, columns), generator=g, dtype=torch.int32).to(DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return (*cache, table, i32([columns * page] * seqs), i32(offsets)), torch.randn(tokens, 8, 128, generator=g).to(torch.bfloat16).to(DEV)


BAD = {"few": ([0, 40, 10, 60], 60), "rows": ([0, 400, 100, 600], 600), "last": ([0, 5, 9, 3], 60), "negative": ([0, -5, 20], 20),
       "past the first 128": (list(range(300)) + [250, 310], 320), "all": ([0, 300] * 200, 300),
       "both ways": ([300, 0, 300, 0, 1], 300)}


@pytest.mark.parametrize("case", BAD)
@pytest.mark.parametrize("most", [None, 1, 300])
def test_nothing_is_written(case, most):
    offsets, tokens = BAD[case]
    if case == "negative":
        offsets = [3, -5, 20]
    state, q = place(offsets, tokens)
    out = torch.full_like(q, 7.0)
    rca.mxfp4_cache_attention(q, *state, max_query=most, out=out)
    assert (out == 7.0).all()
    state[-1].copy_(state[-1].sort().values)                 # in order, it is answered
    rca.mxfp4_cache_attention(q, *state, max_query=most, out=out)
    first, last = max(0, state[-1][0].item()), min(tokens, state[-1][-1].item())
    assert (out[first:last] != 7.0).any(2).all() and (out[:first] == 7.0).all() and (out[last:] == 7.0).all()


def test_bounds_that_are_out_of_range_but_in_order_are_clamped():
    state, q = place([-7, -3, 5, 5, 1 << 30, (1 << 31) - 1], 40)
    want, _ = place([0, 0, 5, 5, 40, 40], 40)
    assert torch.equal(rca.mxfp4_cache_attention(q, *state), rca.mxfp4_cache_attention(q, *want))
