"""Attention over a paged cache held in MXFP4 against the plain statement in binary64,
within the rounding that its arithmetic allows. What no row sees has NaN scales."""
import math

import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
LEAST = {64: 32, 96: 64, 128: 16, 192: 32, 256: 16}
# half an ulp of a value and of the smallest subnormal
HALF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
        torch.float32: (2.0 ** -24, 2.0 ** -150)}
DECODE = [(1, 1), (1, 2), (1, 17), (1, 31), (1, 32), (1, 33), (1, 300), (0, 50), (1, 129), (0, 0), (1, 1000)]
FEW = [(3, 3), (2, 40), (5, 129), (0, 9), (7, 200), (4, 513), (1, 64)]
PROMPTS = [(150, 150), (1, 90), (33, 300), (0, 10), (130, 391), (17, 17)]


def run(plan, heads, kv, d, dtype, seed=1, causal=True, window=0, scale=None, max_query=None, poison=True,
        exponents=(-3, 1), qstd=1.0, cache=None):
    kc, vc, kv_, vv = cache or ref.random_cache(plan, kv, d, seed, poison=poison, exponents=exponents)
    g = torch.Generator().manual_seed(seed + 100)
    q = (torch.randn(plan.tokens, heads, d, generator=g) * qstd).to(dtype)
    out = torch.full((plan.tokens, heads, d), 7.0, dtype=dtype, device=DEV)
    got, lse = rca.mxfp4_cache_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), *plan.tensors(DEV), scale=scale, causal=causal,
                                         window=window, max_query=max_query, lse=True, out=out)
    assert got is out
    sc = d ** -0.5 if scale is None else scale
    want = ref.attention(plan, q, kv_, vv, sc, causal, window)
    compare(plan, got.cpu(), lse.cpu(), want, dtype)
    return got, lse


def compare(plan, got, lse, want, dtype):
    out, ls, tol, lse_tol = want
    half, least = HALF[dtype]
    mine = torch.tensor([at is not None for at in plan.rows()], dtype=torch.bool)
    assert (got[~mine] == 7.0).all()                         # rows of no sequence stay as they were
    off = (got.double() - out).abs()[mine]
    bound = (tol + (out.abs() + tol) * half + least)[mine]
    worst = (off / bound.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1, worst
    empty = torch.isinf(ls) & mine[:, None]
    assert torch.equal(torch.isneginf(lse) & mine[:, None], empty) and (got[empty] == 0).all()
    seen = mine[:, None] & ~empty
    assert ((lse.double() - ls).abs()[seen] <= lse_tol[seen]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", sorted(LEAST))
@pytest.mark.parametrize("spec", [DECODE, FEW], ids=["one", "few"])
def test_few_rows(d, dtype, spec):
    run(ref.Plan(spec, LEAST[d], seed=d), 8, 2, d, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", sorted(LEAST))
@pytest.mark.parametrize("window", [0, 37])
def test_prompts(d, dtype, window):
    run(ref.Plan(PROMPTS, LEAST[d], seed=d), 4, 2, d, dtype, window=window)


@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS], ids=["one", "few", "prompts"])
@pytest.mark.parametrize("dtype", TYPES)
def test_every_row_sees_all(dtype, spec):
    run(ref.Plan(spec, 16), 6, 3, 128, dtype, causal=False)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 17, 40])
@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS[:3]], ids=["one", "few", "prompts"])
def test_heads_of_a_group(group, spec):
    run(ref.Plan(spec, 16), 2 * group, 2, 128, torch.bfloat16)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 1000, 1 << 40])
@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS], ids=["one", "few", "prompts"])
def test_windows(window, spec):
    run(ref.Plan(spec, 32), 8, 2, 64, torch.bfloat16, window=window)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("spec", [DECODE, PROMPTS], ids=["one", "prompts"])
def test_pages(page, spec):
    run(ref.Plan(spec, page, seed=page), 8, 1, 128, torch.bfloat16)


@pytest.mark.parametrize("hint", [None, 1, 5, 150, 100000])
def test_the_hint_changes_nothing_but_speed(hint):
    run(ref.Plan(PROMPTS, 16), 8, 2, 128, torch.bfloat16, max_query=hint)
    run(ref.Plan(DECODE, 16), 8, 2, 128, torch.bfloat16, max_query=hint)


@pytest.mark.parametrize("dtype", TYPES)
def test_padding_more_rows_than_tokens_and_missing_pages(dtype):
    plan = ref.Plan([(4, 40), (6, 2), (3, -5), (5, 50), (40, 60)], 16, before=3, behind=9)
    plan.table[0][1] = plan.pages                            # sixteen tokens are not there
    plan.table[3] = [-1] * plan.max_pages                    # none is
    plan.lengths[4] = 5000                                   # counts as the table's
    for causal, window in ((True, 0), (True, 7), (False, 0)):
        run(plan, 4, 2, 128, dtype, causal=causal, window=window)


def test_one_token_split_over_the_card():
    for n in (4000, 20001, 70000):
        run(ref.Plan([(1, n)], 64, seed=n), 8, 2, 64, torch.bfloat16)
    run(ref.Plan([(1, 9000), (1, 3), (1, 20000), (1, 1)], 16), 4, 1, 128, torch.float32)


def test_a_chunk_split_over_the_card():
    run(ref.Plan([(65, 3000)], 16), 2, 1, 128, torch.bfloat16)
    run(ref.Plan([(65, 3000), (200, 200)], 64), 4, 2, 96, torch.float16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spec", [DECODE, PROMPTS], ids=["one", "prompts"])
def test_peaked_scores(dtype, spec):
    """Scores up to some hundreds: all but one weight vanish, the maximum moves late and early."""
    run(ref.Plan(spec, 16), 4, 2, 128, dtype, qstd=12.0)
    run(ref.Plan(spec, 16), 4, 2, 128, dtype, scale=-0.5)
    run(ref.Plan(spec, 16), 4, 2, 128, dtype, scale=0.0)


@pytest.mark.parametrize("exponents", [(-126, -120), (-60, -40), (40, 60), (-30, 30)])
@pytest.mark.parametrize("spec", [DECODE, FEW, PROMPTS], ids=["one", "few", "prompts"])
def test_scales_of_any_size(exponents, spec):
    """Values' scales at both ends of the range; keys' of ordinary size."""
    for dtype in TYPES:
        plan = ref.Plan(spec, 16)
        kc, _, kv_, _ = ref.random_cache(plan, 2, 128, 3)
        _, vc, _, vv = ref.random_cache(plan, 2, 128, 4, exponents=exponents)
        if dtype == torch.float16 and exponents[1] > 13:
            continue                                         # results that fp16 does not hold
        run(plan, 4, 2, 128, dtype, cache=(kc, vc, kv_, vv))
    plan = ref.Plan(spec, 16)
    kc, _, kv_, _ = ref.random_cache(plan, 2, 128, 3, exponents=exponents)
    _, vc, _, vv = ref.random_cache(plan, 2, 128, 4)
    run(plan, 4, 2, 128, torch.float32, cache=(kc, vc, kv_, vv), scale=2.0 ** -max(0, exponents[1]) / 12)


def _without(cache, plan, kv, d, seq, pos, which, byte, block=1):
    """The cache with one token's block given the scale `byte`."""
    c = cache[which].clone().view(plan.pages, kv, -1, ref.TILE_BYTES)
    b = pos % plan.page * (d // 32) + block
    c[plan.page_at(seq, pos), :, b // 64, 1024 + b % 64] = byte
    c[plan.page_at(seq, pos), :, b // 64, b % 64 * 16:b % 64 * 16 + 16] = 0x77       # largest values
    return c.view(cache[which].shape)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
@pytest.mark.parametrize("byte", [255, 254], ids=["nan", "inf"])
@pytest.mark.parametrize("heads", [2, 8])
def test_what_is_not_finite_reaches_the_rows_that_see_it_alone(dtype, which, byte, heads):
    """A key or value of a token in the midst of a prompt: what the plain statement, which takes for a row what it
    sees alone, gives as finite is finite and within the rounding, and what it does not is not."""
    plan, kv, d = ref.Plan([(60, 75), (40, 40)], 16), 2, 128
    cache = ref.random_cache(plan, kv, d, 5)
    pos = 41
    bad = _without(cache, plan, kv, d, 0, pos, which, byte)
    vals = [cache[2], cache[3]]
    vals[which] = ref.values(bad).view(vals[which].shape)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(plan.tokens, heads, d, generator=g).abs().to(dtype)
    caches = [cache[0].to(DEV), cache[1].to(DEV)]
    caches[which] = bad.to(DEV)
    for window in (0, 9):
        got, lse = rca.mxfp4_cache_attention(q.to(DEV), *caches, *plan.tensors(DEV), window=window, lse=True)
        out, ls, tol, lse_tol = ref.attention(plan, q, *vals, d ** -0.5, True, window)
        fine = torch.isfinite(out)
        sees = torch.tensor([not s and p >= pos and (window == 0 or p < pos + window) for s, p in plan.rows()])
        assert fine[~sees].all() and not fine[sees].all()    # of the statement itself
        got, lse = got.cpu().double(), lse.cpu().double()
        assert not torch.isfinite(got[~fine]).any()
        half, least = HALF[dtype]
        bound = tol + (out.abs() + tol) * half + least
        assert ((got - out).abs()[fine] <= bound[fine]).all()
        fine = torch.isfinite(ls)
        assert ((lse - ls).abs()[fine] <= lse_tol[fine]).all() and not torch.isfinite(lse[~fine]).any()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_query_that_is_not_finite_stays_in_its_row(dtype):
    plan = ref.Plan([(20, 50), (1, 40)], 16)
    cache = [c.to(DEV) for c in ref.random_cache(plan, 2, 128, 5)[:2]]
    g = torch.Generator().manual_seed(9)
    q = torch.randn(plan.tokens, 4, 128, generator=g).to(dtype).to(DEV)
    clean = rca.mxfp4_cache_attention(q, *cache, *plan.tensors(DEV))
    for bad in (math.nan, math.inf, -math.inf):
        p = q.clone()
        p[7, 1, 3] = bad
        got = rca.mxfp4_cache_attention(p, *cache, *plan.tensors(DEV))
        assert not torch.isfinite(got[7, 1]).any()
        got[7, 1] = clean[7, 1]
        assert torch.equal(got, clean)


def test_results_repeat_bit_for_bit():
    plan = ref.Plan([(1, 5000), (40, 700), (1, 3), (9, 90)], 16)
    cache = [c.to(DEV) for c in ref.random_cache(plan, 2, 128, 5)[:2]]
    q = torch.randn(plan.tokens, 8, 128, device=DEV).to(torch.bfloat16)
    first = rca.mxfp4_cache_attention(q, *cache, *plan.tensors(DEV), lse=True)
    for _ in range(5):
        again = rca.mxfp4_cache_attention(q, *cache, *plan.tensors(DEV), lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_queries_that_are_part_of_a_wider_tensor():
    plan = ref.Plan(FEW, 16)
    cache = [c.to(DEV) for c in ref.random_cache(plan, 2, 128, 5)[:2]]
    qkv = torch.randn(plan.tokens, 12, 128, device=DEV).to(torch.bfloat16)
    got = rca.mxfp4_cache_attention(qkv[:, :8], *cache, *plan.tensors(DEV))
    assert torch.equal(got, rca.mxfp4_cache_attention(qkv[:, :8].contiguous(), *cache, *plan.tensors(DEV)))


def test_many_sequences():
    run(ref.Plan([(i % 3, 5 + i % 37 + i % 3) for i in range(300)], 16, seed=3), 2, 1, 128, torch.bfloat16)
    run(ref.Plan([(1 if i % 41 == 0 else 0, i % 50 + 1) for i in range(5000)], 16, wider=0), 2, 1, 128, torch.bfloat16)


def test_no_tokens_and_no_sequences():
    kc, vc = rca.mxfp4_cache_new(1, 2, 16, 128, DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.zeros(0, 4, 128, device=DEV)
    assert rca.mxfp4_cache_attention(q, kc, vc, i32(0)[None], i32(5), i32(0, 0)).shape == (0, 4, 128)
    q = torch.full((3, 4, 128), 2.0, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    rca.mxfp4_cache_attention(q, kc, vc, none.view(0, 1), none, i32(0), out=out)
    assert (out == 7.0).all()
    empty = torch.zeros(2, 0, dtype=torch.int32, device=DEV)                         # a table without columns
    out = rca.mxfp4_cache_attention(q, kc, vc, empty, i32(5, 5), i32(0, 1, 3))
    assert (out == 0).all()
    kc, vc = rca.mxfp4_cache_new(0, 2, 16, 128, DEV)                                 # and a cache without pages
    out, lse = rca.mxfp4_cache_attention(q, kc, vc, i32(0, 0)[:, None], i32(5, 5), i32(0, 1, 3), lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
