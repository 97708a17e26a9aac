"""From 1024 tokens on a workgroup takes several turns over a token's heads: what is appended, turned and read is bit
for bit what calls of fewer tokens, whose heads stand side by side, append, turn and read."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_forms as forms
from tests import cache_reference as ref
from tests.test_gpu_cache_append import LEAST, rotation, rows

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def in_parts(plan, most):
    """[(rows, sequence, length after them)] of calls of one sequence's next tokens each."""
    out = []
    for s, (new, length) in enumerate(zip(plan.new, plan.lengths)):
        for a in range(0, new, most):
            b = min(new, a + most)
            out.append((slice(plan.offsets[s] + a, plan.offsets[s] + b), s, length - new + b))
    return out


def check(spec, heads, kv, d, dtype, rot, interleaved):
    plan = ref.Plan(spec, LEAST[d], seed=d, before=2, behind=3)
    q, k, v = rows(plan, heads, kv, d, dtype, 5)
    turn = rotation(plan, rot, 7).to(DEV) if rot else None
    cache = [c.to(DEV) for c in ref.random_cache(plan, kv, d, 11, poison=False)[:2]]
    table, lengths, offsets = plan.tensors(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    whole, parts = [c.clone() for c in cache], [c.clone() for c in cache]
    new = lambda n: torch.full((plan.tokens, n, d), 7.0, dtype=dtype, device=DEV)  # noqa: E731
    one, two = [new(heads), new(kv), new(kv)], [new(heads), new(kv), new(kv)]
    rca.mxfp4_cache_append(k, v, *whole, table, lengths, offsets, q=q, rotation=turn, interleaved=interleaved, q_out=one[0])
    rca.mxfp4_cache_read(*whole, table, lengths, offsets, plan.tokens, d, dtype, k=one[1], v=one[2])
    for at, s, length in in_parts(plan, 300):
        place = *parts, table[s:s + 1], i32(length), i32(0, at.stop - at.start)
        rca.mxfp4_cache_append(k[at], v[at], *place, q=q[at], rotation=turn, interleaved=interleaved, q_out=two[0][at])
    for at, s, length in in_parts(plan, 300):
        place = *parts, table[s:s + 1], i32(length), i32(0, at.stop - at.start)
        rca.mxfp4_cache_read(*place, at.stop - at.start, d, dtype, k=two[1][at], v=two[2][at])
    assert all(torch.equal(a, b) for a, b in zip(whole + one, parts + two))
    assert not torch.equal(whole[0], cache[0]) and (one[0][:2] == 7.0).all() and (one[0][-3:] == 7.0).all()


@pytest.mark.parametrize("d", sorted(LEAST))
@pytest.mark.parametrize("heads,kv", forms.HEADS)
@pytest.mark.parametrize("rot", ["none", "half", "all"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_width_and_rotation(d, heads, kv, rot, interleaved):
    check(forms.TOKENS[2], heads, kv, d, torch.bfloat16, {"none": 0, "half": d // 32 * 16, "all": d}[rot], interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("spec", forms.TOKENS, ids=[str(sum(n for n, _ in s)) for s in forms.TOKENS])
def test_either_side_of_the_border(spec, dtype):
    for d in (64, 96, 128, 256):
        check(spec, *forms.HEADS[1], d, dtype, 64, False)
