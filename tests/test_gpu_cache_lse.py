"""The log-sum-exp of attention over the cache is FP32's own, whatever type the queries have: its bound is that of
tests/cache_reference.py without what the weights are rounded by before they are multiplied."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref
from tests.test_gpu_cache_attention import DECODE, FEW, LEAST, PROMPTS

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MIXED = [(1, 300), (140, 170), (0, 9), (170, 170), (1, 1)]
LONG = [(1, 9000), (1, 3), (1, 20000)]
CHUNK = [(200, 3000)]


def check(plan, heads, kv, d, dtype, causal=True, window=0, scale=None, most=None):
    """Weights sum to one, so that what rounding them adds to the bound of the logarithm is that rounding itself."""
    kc, vc, kvals, vvals = ref.random_cache(plan, kv, d, 1)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(plan.tokens, heads, d, generator=g).to(dtype)
    _, lse = rca.mxfp4_cache_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), *plan.tensors(DEV), scale=scale, causal=causal,
                                       window=window, max_query=most, lse=True)
    _, want, _, tol = ref.attention(plan, q, kvals, vvals, d ** -0.5 if scale is None else scale, causal, window)
    mine = torch.tensor([at is not None for at in plan.rows()], dtype=torch.bool)
    seen = mine[:, None] & torch.isfinite(want)
    off = (lse.cpu().double() - want).abs()[seen] / (tol - ref.WEIGHT[dtype])[seen]
    assert seen.any() and off.max() <= 1, off.max().item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS, MIXED, LONG, CHUNK], ids=["one", "few", "prompts", "mixed", "long", "chunk"])
def test_lse_is_fp32s_own(dtype, spec):
    check(ref.Plan(spec, 16), 4, 2, 128, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", sorted(LEAST))
def test_every_width(dtype, d):
    for spec in (DECODE, MIXED):
        check(ref.Plan(spec, LEAST[d]), 4, 2, d, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_scores_of_any_size(dtype, scale):
    """The maximum moves late and early, and the sum that the logarithm is formed of with it."""
    for spec in (DECODE, FEW, MIXED):
        check(ref.Plan(spec, 16), 4, 2, 128, dtype, scale=scale)


def test_windows_and_every_row_seeing_all():
    for spec, most in ((DECODE, 1), (MIXED, None), (MIXED, 170)):
        check(ref.Plan(spec, 16), 4, 2, 128, torch.bfloat16, window=37, most=most)
        check(ref.Plan(spec, 16), 4, 2, 128, torch.bfloat16, causal=False, most=most)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("spec", [DECODE, MIXED, LONG], ids=["one", "mixed", "long"])
def test_values_are_the_same_without_it(dtype, spec):
    plan = ref.Plan(spec, 16)
    cache = [c.to(DEV) for c in ref.random_cache(plan, 2, 128, 1)[:2]]
    q = torch.randn(plan.tokens, 4, 128, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    out, _ = rca.mxfp4_cache_attention(q, *cache, *plan.tensors(DEV), lse=True)
    assert torch.equal(out, rca.mxfp4_cache_attention(q, *cache, *plan.tensors(DEV)))
