"""Attention whose values take the place of dense queries: the same bits as beside them."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref
from tests.test_cache_refusals import A, attend
from tests.test_gpu_cache_attention import DECODE, FEW, PROMPTS

MIXED = [(1, 300), (140, 170), (0, 9), (300, 300), (1, 1), (129, 700)]
LONG = [(1, 30000)]
CHUNK = [(200, 9000)]


@pytest.mark.parametrize("tokens,stride,status", [(3, 512, rca.ERR_ALIGN), (3, 520, rca.ERR_UNSUPPORTED),
                                                  (3, 1024, rca.ERR_UNSUPPORTED), (1, 520, rca.ERR_ALIGN)])
def test_queries_that_lie_apart_are_refused(tokens, stride, status):
    """(A misaligned workspace stands for what would be accepted.)"""
    assert attend(tokens=tokens, out=A, q=A, qs=stride, ws=A + 4) == status
    assert attend(tokens=tokens, out=2 * A, q=A, qs=stride, ws=A + 4) == rca.ERR_ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS, MIXED, LONG, CHUNK],
                         ids=["one", "few", "prompts", "mixed", "long", "chunk"])
def test_in_place(spec, dtype):
    dev = torch.device("cuda:0")
    plan = ref.Plan(spec, 16, before=2, behind=3)
    cache = [c.to(dev) for c in ref.random_cache(plan, 2, 128, 5)[:2]]
    g = torch.Generator().manual_seed(1)
    q = torch.randn(plan.tokens, 8, 128, generator=g).to(dtype).to(dev)
    for most in (None, 1, 300):
        want = q.clone()
        _, lse = rca.mxfp4_cache_attention(q, *cache, *plan.tensors(dev), out=want, max_query=most, lse=True)
        got = q.clone()
        out, ls = rca.mxfp4_cache_attention(got, *cache, *plan.tensors(dev), out=got, max_query=most, lse=True)
        assert out is got and torch.equal(got, want)         # rows of no sequence too
        mine = torch.tensor([at is not None for at in plan.rows()], device=dev)
        assert torch.equal(ls[mine], lse[mine])
