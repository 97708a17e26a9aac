"""The plain statements that the cache's tests go by agree with the oracle and with torch."""
import numpy as np
import pytest
import torch

import oracle
from tests import cache_reference as ref


def test_pack_is_the_oracles():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4 * 2048, generator=g) * torch.exp2(torch.randint(-140, 120, (4 * 2048,), generator=g).float())
    x[:64] = 0
    x[64:128:2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25] * 4)[:32]
    x[65:128:2] = 4.0
    want = oracle.quantize_pack(oracle.MXFP4, x.numpy())
    assert np.array_equal(ref.pack(x.numpy()).numpy(), want)


def test_narrow_rounds_once():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(1 << 16, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-30, 10, (1 << 16,), generator=g).double())
    x[:1000] = (1 + 2.0 ** -11) * (1 + 2.0 ** -30)               # just above the middle of two fp16 values
    assert np.array_equal(ref.narrow(x, torch.float16).numpy(), x.numpy().astype(np.float16))
    y = ref.narrow(x, torch.bfloat16).double()
    for step in (-1, 1):
        z = (y.to(torch.bfloat16).view(torch.int16) + step).view(torch.bfloat16).double()
        assert ((y - x).abs() <= (z - x).abs()).all()


def test_turning_keeps_lengths_and_both_orders_agree():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 64, generator=g).double()
    a = torch.rand(5, 16, generator=g) * 6
    rot = torch.cat([a.cos(), a.sin()], 1)
    y = ref.turn(x, rot, 2, False)
    assert torch.allclose(y[:, :32].norm(dim=1), x[:, :32].norm(dim=1)) and torch.equal(y[:, 32:], x[:, 32:])
    mixed = torch.arange(32).view(2, 16).t().reshape(-1)
    z = ref.turn(x[:, torch.cat([mixed, torch.arange(32, 64)])], rot, 2, True)
    assert torch.equal(z[:, torch.argsort(mixed)], y[:, :32])


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attention_is_torchs(causal, window):
    plan = ref.Plan([(3, 20), (2, 7)], 64)
    _, _, k, v = ref.random_cache(plan, 2, 64, 1)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(5, 4, 64, generator=g)
    out, lse, tol, _ = ref.attention(plan, q, k, v, 0.125, causal, window)
    for s, (m, n, a) in enumerate([(3, 20, 0), (2, 7, 3)]):
        kk, vv = (x[plan.table[s][0]][:, :n].repeat_interleave(2, 0) for x in (k, v))
        at = torch.arange(n - m, n)[:, None] - torch.arange(n)
        seen = (at >= 0) if causal else torch.ones_like(at, dtype=torch.bool)
        if window:
            seen &= at < window
        want = torch.nn.functional.scaled_dot_product_attention(q[a:a + m].double().transpose(0, 1), kk, vv,
                                                                attn_mask=seen, scale=0.125)
        assert torch.allclose(out[a:a + m], want.transpose(0, 1), rtol=1e-12, atol=1e-12)
    assert (tol[:5] > 0).all() and torch.isfinite(lse).all()
