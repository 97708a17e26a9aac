"""Attention by both ways to share a tile, and by both at once, over every state that a sequence can be in; the plans
are those of tests/cache_forms.py, which a CPU test asks the library's rules about."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_forms as forms
from tests import cache_reference as ref
from tests.test_gpu_cache_attention import LEAST, TYPES, compare, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", sorted(LEAST))
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 7), (True, 150), (False, 0)])
def test_every_state(d, dtype, causal, window):
    run(forms.awkward(LEAST[d]), 2, 1, d, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [1, 10, 300])
def test_every_state_whatever_the_hint(dtype, most):
    run(forms.awkward(), 2, 2, 128, dtype, max_query=most)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spec", forms.ALONE)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 33), (False, 0)])
def test_a_sequence_by_itself(spec, dtype, causal, window):
    for d in (64, 128, 256):
        run(forms.alone(forms.ALONE[spec], LEAST[d], before=2, behind=1), 2, 2, d, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_heads_than_workgroups_fit_and_both_kernels(dtype):
    """Heads all over the range against the plain statement, which all of them would take minutes of."""
    kv, d = 1100, 64
    some = sorted({*range(0, kv, 37), 511, 512, 767, 768, 1023, 1024, kv - 1})
    plan = ref.Plan(forms.MANY_HEADS, 32, seed=2)
    kc, vc, kvals, vvals = ref.random_cache(plan, kv, d, 3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(plan.tokens, kv, d, generator=g).to(dtype)
    out, lse = rca.mxfp4_cache_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), *plan.tensors(DEV), lse=True)
    out, lse = out.cpu(), lse.cpu()
    want = ref.attention(plan, q[:, some], kvals[:, some], vvals[:, some], d ** -0.5)
    compare(plan, out[:, some].contiguous(), lse[:, some].contiguous(), want, dtype)
