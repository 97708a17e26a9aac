"""Keys and values that are not finite, in blocks of any codes and scales, under both ways to share a tile: what
reaches the rows that see them, and that nothing reaches the others; and the smallest scale, 2^-127."""
import functools
import math

import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref
from tests import test_gpu_cache_attention as attention
from tests.test_gpu_cache_attention import HALF, TYPES

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
KV, D, BLOCK = 2, 128, 1
SPEC = [(140, 170), (1, 40), (150, 150)]                     # 140 and 150 rows a head of the cache or more, and one
HIDDEN = [0, 5, 63, 100, 165]                                # positions of the first sequence, its first and last steps' among them


@functools.lru_cache(None)
def setting(dtype, sign="any"):
    plan = ref.Plan(SPEC, 16)
    q = torch.randn(plan.tokens, 4, D, generator=torch.Generator().manual_seed(9)).to(dtype)
    q = {"any": q, "positive": q.abs(), "negative": -q.abs(), "-1": -torch.ones_like(q)}[sign]
    return plan, ref.random_cache(plan, KV, D, 5), q


@functools.lru_cache(None)
def clean(dtype, sign="any", window=0, hidden=None):
    """The plain statement of the cache as it was, and without the first sequence's token `hidden`."""
    plan, cache, q = setting(dtype, sign)
    return ref.attention(plan if hidden is None else _Hidden(plan, hidden), q, *cache[2:], D ** -0.5, True, window)


def place(c, plan, seq, pos):
    """Block BLOCK of a token: its tile, and its number in it."""
    b = pos % plan.page * (D // 32) + BLOCK
    return c.view(plan.pages, KV, -1, ref.TILE_BYTES)[plan.page_at(seq, pos), :, b // 64], b % 64


def with_block(cache, plan, which, pos, codes, byte):
    """The cache with a block of the first sequence's token given these codes and this scale."""
    c = cache[which].clone()
    t, b = place(c, plan, 0, pos)
    t[:, b * 16:b * 16 + 16] = codes
    t[:, 1024 + b] = byte
    vals = [cache[2], cache[3]]
    vals[which] = ref.values(c).view(vals[which].shape)
    both = [cache[0], cache[1]]
    both[which] = c
    return both, vals


def sees(plan, pos, window):
    return torch.tensor([s == 0 and p >= pos and (window == 0 or p < pos + window) for s, p in plan.rows()])


def answer(plan, q, both, most, window):
    got, lse = rca.mxfp4_cache_attention(q.to(DEV), *(c.to(DEV) for c in both), *plan.tensors(DEV), window=window,
                                         max_query=most, lse=True)
    return got.cpu().double(), lse.cpu().double()


def near(got, out, tol, dtype):
    half, least = HALF[dtype]
    return (got - out).abs() <= tol + (out.abs() + tol) * half + least


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [None, 1, 150])
@pytest.mark.parametrize("byte,first", [(253, 4), (254, 2), (255, 0)])
def test_a_value_reaches_its_place_in_the_rows_that_see_it_and_its_block_at_most(dtype, most, byte, first):
    """Codes of all magnitudes side by side: under 2^126 those from 4 on are infinite, under 2^127 from 2 on."""
    plan, cache, q = setting(dtype)
    codes = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2, dtype=torch.uint8)
    for pos, window in [(p, 0) for p in HIDDEN] + [(63, 20)]:
        both, vals = with_block(cache, plan, 1, pos, codes, byte)
        bad = ~torch.isfinite(vals[1][plan.page_at(0, pos), 0, pos % 16])
        magnitudes = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6] * 4)
        assert torch.equal(bad[32:64], (magnitudes >= first) | (byte == 255)) and bad.sum() == bad[32:64].sum()
        got, lse = answer(plan, q, both, most, window)
        out, ls, tol, lse_tol = clean(dtype, window=window)
        row = sees(plan, pos, window)
        assert row.any() and not torch.isfinite(got[row][:, :, bad]).any()
        fine = torch.ones_like(got, dtype=torch.bool)
        fine[row, :, 32:64] = False
        assert near(got, out, tol, dtype)[fine].all()
        assert ((lse - ls).abs() <= lse_tol).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [None, 1, 150])
@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("sign", ["any", "positive", "negative", "-1"])
def test_a_key_spoils_the_rows_that_see_it_or_counts_for_nothing(dtype, most, byte, sign):
    """An infinite key gives scores of either infinity, or NaN: the row's values and lse are not finite, or they are
    those without the key."""
    plan, cache, q = setting(dtype, sign)
    for pos, window in ((5, 0), (100, 0), (63, 20)):
        both, _ = with_block(cache, plan, 0, pos, torch.full((16,), 0x77, dtype=torch.uint8), byte)
        got, lse = answer(plan, q, both, most, window)
        out, ls, tol, lse_tol = clean(dtype, sign, window)
        row = sees(plan, pos, window)
        assert near(got, out, tol, dtype)[~row].all() and ((lse - ls).abs() <= lse_tol)[~row].all()
        spoilt = ~torch.isfinite(got)
        if sign == "positive" or byte == 255:
            assert spoilt[row].all() and not torch.isfinite(lse[row]).any()
            continue
        assert (spoilt.all(2) == spoilt.any(2)).all() and (spoilt.any(2) == ~torch.isfinite(lse)).all()
        without = clean(dtype, sign, window, pos)
        left = row[:, None] & ~spoilt.any(2)
        assert near(got, without[0], without[2], dtype)[left].all()
        assert ((lse - without[1]).abs() <= without[3])[left].all()


class _Hidden:
    """A plan of which a token of the first sequence is not there."""

    def __init__(self, plan, pos):
        self.plan, self.pos = plan, pos

    def __getattr__(self, name):
        return getattr(self.plan, name)

    def page_at(self, s, pos):
        return -1 if (s, pos) == (0, self.pos) else self.plan.page_at(s, pos)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [None, 1, 150])
def test_a_query_that_is_not_finite_stays_in_its_row(dtype, most):
    """The other rows are held to their bound and not to their bits: the 32 rows of a wave move their maxima together,
    and this row's score, which no maximum is large enough for, moves theirs at every step. A weight is then formed
    under another maximum m': e^(s - m') rounded, for e^(s - m) rounded and multiplied by e^(m - m') rounded. Both are
    within the roundings that the bound counts for each weight and sum, and need not be the same."""
    plan, both, q = setting(dtype)
    cache, q = [c.to(DEV) for c in both[:2]], q.to(DEV)
    out, ls, tol, lse_tol = clean(dtype)
    for row in (7, 130, 140, 200):
        for bad in (math.nan, math.inf, -math.inf):
            p = q.clone()
            p[row, 1, 3] = bad
            got, lse = (t.cpu().double() for t in rca.mxfp4_cache_attention(p, *cache, *plan.tensors(DEV), max_query=most,
                                                                            lse=True))
            assert not torch.isfinite(got[row, 1]).any() and not torch.isfinite(lse[row, 1])
            others = torch.ones_like(lse, dtype=torch.bool)
            others[row, 1] = False
            assert near(got, out, tol, dtype)[others].all() and ((lse - ls).abs() <= lse_tol)[others].all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", [0, 1], ids=["keys", "values"])
def test_the_smallest_scale(dtype, which):
    """Scale bytes of 0 under codes that are not zero: 2^-127."""
    plan = ref.Plan(SPEC, 16)
    cache = list(ref.random_cache(plan, KV, D, 3))
    least = ref.random_cache(plan, KV, D, 4, exponents=(-127, -127))
    assert (least[which].view(plan.pages, KV, -1, ref.TILE_BYTES)[..., 1024:] != 1).all() and (least[2 + which] != 0).any()
    cache[which], cache[2 + which] = least[which], least[2 + which]
    attention.run(plan, 4, KV, D, dtype, cache=cache)
