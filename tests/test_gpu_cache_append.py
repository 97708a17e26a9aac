"""Appending to a cache held in MXFP4 writes the bytes of the plain statement, turns
queries to their correctly rounded values, and leaves everything else as it was;
the rows read back are the cache's."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
LEAST = {64: 32, 96: 64, 128: 16, 192: 32, 256: 16}
# (new, length): one token at the start, behind a page's end, sequences without new tokens, whole prompts, a page filled
SPEC = [(1, 1), (1, 130), (0, 40), (70, 70), (16, 128), (3, 67), (0, 0), (5, 64), (2, 65)]


def rotation(plan, r, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(plan.max_pages * plan.page, r // 2, generator=g, dtype=torch.float64) * 6.3
    return torch.cat([a.cos(), a.sin()], 1).float()


def rows(plan, heads, kv, d, dtype, seed, scale=1.0):
    """q, k and v as parts of one fused projection's output."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(plan.tokens, heads + 2 * kv, d, generator=g) * scale
    x[:, -1, :32] = 0                                        # a block of zeros
    x[::2, heads, :] *= 64
    return x.to(dtype).to(DEV).split([heads, kv, kv], 1)


def check(plan, heads, kv, d, dtype, rot, interleaved, seed=5, scale=1.0):
    q, k, v = rows(plan, heads, kv, d, dtype, seed, scale)
    r = rotation(plan, rot, 7) if rot else None
    kc, vc, _, _ = ref.random_cache(plan, kv, d, 11, poison=False)
    gk, gv = kc.to(DEV), vc.to(DEV)
    kept = torch.full((plan.tokens, heads, d), 7.0, dtype=dtype, device=DEV)
    got = rca.mxfp4_cache_append(k, v, gk, gv, *plan.tensors(DEV), q=q, rotation=None if r is None else r.to(DEV),
                                 interleaved=interleaved, q_out=kept)
    assert got is kept
    want_k = ref.appended(plan, kc, k.cpu(), d, r, interleaved)
    want_v = ref.appended(plan, vc, v.cpu(), d)
    assert torch.equal(gk.cpu(), want_k) and torch.equal(gv.cpu(), want_v)
    for i, at in enumerate(plan.rows()):
        want = torch.full((heads, d), 7.0, dtype=dtype) if at is None else \
            ref.narrow(ref.turn(q[i].cpu().double(), r, max(at[1], 0), interleaved), dtype)
        assert bool((got[i].cpu() == want).all()), (i, at)
    rk, rv = (torch.full((plan.tokens, kv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    rca.mxfp4_cache_read(gk, gv, *plan.tensors(DEV), plan.tokens, d, dtype, k=rk, v=rv)
    for c, got in ((want_k, rk), (want_v, rv)):
        vals = ref.values(c).view(plan.pages, kv, plan.page, d)
        for i, at in enumerate(plan.rows()):
            page = -1 if at is None else plan.page_at(*at)
            want = torch.full((kv, d), 7.0, dtype=dtype) if at is None else torch.zeros(kv, d, dtype=dtype) \
                if page < 0 else vals[page, :, at[1] % plan.page].to(dtype)
            assert bool((got[i].cpu() == want).all()), (i, at)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", sorted(LEAST))
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_width_and_type(d, dtype, interleaved):
    check(ref.Plan(SPEC, LEAST[d], seed=d), 6, 3, d, dtype, d, interleaved)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 96])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_a_head_is_turned(rot, interleaved):
    check(ref.Plan(SPEC, 64, seed=rot), 2, 1, 96, torch.bfloat16, rot, interleaved)


@pytest.mark.parametrize("page", [16, 32, 128])
def test_pages(page):
    check(ref.Plan(SPEC, page, seed=page), 8, 1, 128, torch.float16, 64, False)


def test_rows_of_no_sequence_and_more_tokens_than_length():
    """Padding before and behind; a sequence with more rows than its length (positions below zero)."""
    plan = ref.Plan([(4, 20), (6, 2), (3, -5)], 16, before=3, behind=5)
    check(plan, 4, 2, 128, torch.bfloat16, 128, False)


def test_lengths_beyond_the_table_and_pages_that_are_not_there():
    plan = ref.Plan([(4, 40), (5, 33), (6, 20)], 16, wider=0)
    plan.lengths[0] = 1000                                   # counts as the table's 48
    plan.table[1][2] = plan.pages                            # a page past the last
    plan.table[2][0] = -3
    check(plan, 4, 2, 128, torch.bfloat16, 128, False)


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e30])
def test_extreme_values(scale):
    check(ref.Plan(SPEC, 16), 2, 2, 128, torch.float32, 128, False, scale=scale)


def test_many_sequences():
    check(ref.Plan([(i % 3, 5 + i % 37 + i % 3) for i in range(300)], 16, seed=3), 2, 1, 128, torch.bfloat16, 64, True)


def test_more_than_4096_sequences():
    """The bounds are searched in three rounds of 64."""
    plan = ref.Plan([(1 if i % 41 == 0 else 0, 1) for i in range(5000)], 16, wider=0)
    check(plan, 1, 1, 128, torch.bfloat16, 0, False)


def test_what_is_not_turned_is_quantize_packs():
    """A page filled in order is the stream that quantize_pack writes."""
    plan = ref.Plan([(32, 32)], 32, spare=0, wider=0)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(32, 2, 64, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    kc, vc = rca.mxfp4_cache_new(1, 2, 32, 64, DEV)
    assert rca.mxfp4_cache_append(k, v, kc, vc, *plan.tensors(DEV)) is None
    for x, c in ((k, kc), (v, vc)):
        assert torch.equal(rca.quantize_pack(x.transpose(0, 1).contiguous(), rca.MXFP4), c.view(-1))


def test_a_cache_of_more_than_4_gib():
    """Pages whose bytes lie past 2^32."""
    page, d, kv = 64, 128, 8
    pages = (1 << 32) // (kv * ref.stream_bytes(page, d)) + 3
    kc = torch.zeros(pages, kv, ref.stream_bytes(page, d), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 64, 128], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(128, kv, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    rca.mxfp4_cache_append(k, v, kc, vc, table, lengths, offsets)
    for c, x in ((kc, k), (vc, v)):
        for p, s in ((pages - 1, 0), (0, 64)):
            want = rca.quantize_pack(x[s:s + 64].transpose(0, 1).contiguous(), rca.MXFP4)
            assert torch.equal(c[p].reshape(-1), want)
        assert not c[1:-1].any()
    q = torch.randn(128, kv, d, generator=g).to(torch.bfloat16).to(DEV)
    got = rca.mxfp4_cache_attention(q, kc, vc, table, lengths, offsets)
    small = [c[[pages - 1, 0]].contiguous() for c in (kc, vc)]
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    assert torch.equal(got, rca.mxfp4_cache_attention(q, *small, table, lengths, offsets))
