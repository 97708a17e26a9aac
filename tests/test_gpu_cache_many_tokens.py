"""More tokens in a call than a grid's first dimension takes: the last ones are
appended, read and answered as they are alone, and what belongs to no sequence
stays as it was."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref
from tests.test_gpu_cache_attention import compare

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, PAGE, FRONT = 64, 32, (1 << 22) - 8


@pytest.fixture(scope="module")
def both():
    plan = ref.Plan([(8, 50), (35, 35)], PAGE, seed=1, before=5)
    kc, vc, kv, vv = ref.random_cache(plan, 1, D, 2, poison=False)
    table, lengths, offsets = plan.tensors(DEV)
    return plan, (kc, vc), (kv, vv), (table, lengths), offsets


@pytest.mark.parametrize("rot", [0, 64, 32])
def test_append(both, rot):
    plan, cache, _, state, offsets = both
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(plan.tokens, 3, D, generator=g).to(torch.bfloat16).to(DEV)
    turn = torch.randn(plan.max_pages * PAGE, rot, generator=g).to(DEV) if rot else None
    many = torch.zeros(FRONT + plan.tokens, 3, D, dtype=torch.bfloat16, device=DEV)
    many[FRONT:] = rows
    got = []
    for x, off in ((rows, offsets), (many, offsets + FRONT)):
        c = [t.to(DEV) for t in cache]
        q_out = torch.full((x.shape[0], 1, D), 7.0, dtype=torch.bfloat16, device=DEV)
        q, k, v = x.split(1, 1)
        rca.mxfp4_cache_append(k, v, *c, *state, off, q=q, rotation=turn, q_out=q_out)
        got.append(c + [q_out[-plan.tokens:]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (q_out[:FRONT + 5] == 7.0).all()


def test_read(both):
    plan, cache, values, state, offsets = both
    c = [t.to(DEV) for t in cache]
    k, v = (torch.full((FRONT + plan.tokens, 1, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rca.mxfp4_cache_read(*c, *state, offsets + FRONT, FRONT + plan.tokens, D, k=k, v=v)
    for got, vals in zip((k, v), values):
        assert (got[:FRONT + 5] == 7.0).all()
        for i, at in enumerate(plan.rows()):
            if at is not None:
                assert torch.equal(got[FRONT + i, 0].cpu().double(), vals[plan.page_at(*at), 0, at[1] % PAGE])


def test_attention(both):
    plan, cache, values, state, offsets = both
    c = [t.to(DEV) for t in cache]
    g = torch.Generator().manual_seed(4)
    q = torch.randn(plan.tokens, 1, D, generator=g).to(torch.bfloat16)
    many = torch.zeros(FRONT + plan.tokens, 1, D, dtype=torch.bfloat16, device=DEV)
    many[FRONT:] = q.to(DEV)
    out = torch.full_like(many, 7.0)
    _, lse = rca.mxfp4_cache_attention(many, *c, *state, offsets + FRONT, lse=True, out=out)
    compare(plan, out[FRONT:].cpu(), lse[FRONT:].cpu(), ref.attention(plan, q, *values, D ** -0.5), torch.bfloat16)
    assert (out[:FRONT] == 7.0).all()
