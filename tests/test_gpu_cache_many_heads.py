"""More heads in the cache than workgroups that the card holds at once."""
import pytest
import torch

from tests import cache_reference as ref
from tests import test_gpu_cache_append as append
from tests import test_gpu_cache_attention as attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spec", [[(1, 40), (1, 3)], [(1, 40), (40, 70)]], ids=["one", "mixed"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention(dtype, spec):
    attention.run(ref.Plan(spec, 32), 1100, 1100, 64, dtype)


@pytest.mark.parametrize("d", [64, 96])
def test_append_and_read(d):
    append.check(ref.Plan([(1, 40), (2, 5)], 64), 1100, 1100, d, torch.bfloat16, 64, False)
