"""Positions up to 2^30, the most that a table has: a token's place and what it sees there."""
import math

import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, PAGE, PAGES = 64, 65536, 16384


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_last_token_of_the_longest_sequence(dtype, window):
    """Keys of zero: every weight is 1 and out is the mean of the values that are there, the last page's. A sum of n
    terms is off by (n + 8) 2^-23 of their magnitudes, out once more by half a step of its type."""
    g = torch.Generator().manual_seed(1)
    kc, vc = rca.mxfp4_cache_new(2, 1, PAGE, D, DEV)
    v_host = torch.randint(0, 256, (vc.shape[-1] // 1088, 1088), generator=g, dtype=torch.uint8)
    v_host[:, 1024:] = v_host[:, 1024:] % 3 + 126
    vc[1, 0] = v_host.view(-1).to(DEV)
    table = torch.full((1, PAGES), -1, dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    place = kc, vc, table, i32([1 << 30]), i32([0, 1])
    x = torch.randn(1, 3, D, generator=g).to(dtype)
    q, k, v = x.to(DEV).split([1, 1, 1], 1)
    rca.mxfp4_cache_append(torch.zeros_like(k), v, *place)
    got_k, got_v = rca.mxfp4_cache_read(*place, 1, D, dtype=torch.float32)
    vals = ref.values(vc[1, 0]).view(PAGE, D)
    last = ref.values(ref.pack(torch.cat([x[0, 2].double(), torch.zeros(2048 - D).double()]).numpy()))[:D]
    assert (got_k == 0).all() and torch.equal(got_v[0, 0].cpu().double(), last) and torch.equal(vals[-1], last)
    assert torch.equal(vc[1, 0, :-1088].cpu(), v_host.view(-1)[:-1088]) and (vc[0] == 0).all()
    out, lse = rca.mxfp4_cache_attention(q, *place, window=window, lse=True)
    seen = vals[-window:] if window else vals
    n, want = seen.shape[0], seen.mean(0)
    bound = 2 * (n + 8) * 2.0 ** -23 * seen.abs().mean(0)
    bound = bound + (want.abs() + bound) * torch.finfo(dtype).eps / 2
    assert ((out[0, 0].cpu().double() - want).abs() <= bound).all()
    assert abs(lse.item() - math.log(n)) <= (n + 8) * 2.0 ** -23 + 2.0 ** -22 * (math.log(n) + 1)
