"""fp16 rows on weights as the packer writes them: blocks of zeros have the
scale 2^-127, and so has the padding after the last weight.  fp16 holds them
like the rest, so rows are multiplied as they are and an infinity in a row
comes out as one wherever its weight is not zero."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_forms
from tests.test_gpu_grouped_forms import held, offsets, on_gpu, product, whole

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
# sizes of more than 16 rows a workgroup: with fewer, rows are cut into two terms always
SHAPES = pytest.mark.parametrize("shape", [s for s in op_forms.SHAPES if not op_forms.forms(
    "fp16", op_forms.rows_of(s[0]), len(s[0]), s[1], s[2])["forward"][0].startswith("16x")], ids=op_forms.label)


def packed_weights(experts, n, k, seed, zeros=0.0):
    """Whole numbers (the largest of each block 6, so all are exact), a share of their blocks zero; packed, and the values."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.tensor([0.0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device=DEV)[
        torch.randint(0, 11, (experts, n, k // 32, 32), generator=g, device=DEV)]
    w[..., 0] = 6.0
    w[torch.rand(experts, n, k // 32, generator=g, device=DEV) < zeros] = 0.0
    w = w.view(experts, n, k)
    packed = rca.quantize_pack(w, rca.MXFP4)
    assert torch.equal(rca.unpack_dequant(packed, rca.MXFP4, w.numel()).view_as(w), w)
    return packed, w


def check(shape, packed, w, seed):
    """Whole numbers exactly, and infinities in some rows as the definition gives them."""
    counts, n, k = shape
    rows, off = op_forms.rows_of(counts), offsets(counts)
    x = whole(rows, k, torch.float16, seed)
    bad = torch.arange(off[0] + 2, off[-1], 61, device=DEV)
    at = bad * 7 % k
    x[bad, at] = torch.where(bad % 2 == 0, float("inf"), float("-inf")).to(torch.float16)
    y = rca.mxfp4_grouped_matmul(x, packed, on_gpu(off), n, out_dtype=torch.float32)
    clean = torch.ones(rows, dtype=torch.bool, device=DEV)
    clean[bad] = False
    finite = x.clone()
    finite[bad, at] = 0
    assert torch.equal(y[clean].double(), product(finite, w, off)[0][clean])
    expert = torch.searchsorted(on_gpu(off)[1:], bad, right=True)
    want = x[bad, at, None].float() * w[expert, :, at]                 # infinite, or NaN where the weight is zero
    assert torch.equal(y[bad].nan_to_num(nan=0.5), want.nan_to_num(nan=0.5))


@pytest.mark.parametrize("zeros", [0.0, 0.02, 1.0])
@SHAPES
def test_packed_weights_with_blocks_of_zeros(shape, zeros):
    counts, n, k = shape
    print(f"case zeros {op_forms.label(shape)} {zeros}", flush=True)
    check(shape, *packed_weights(len(counts), n, k, 1, zeros), 2)


@SHAPES
def test_one_expert_beyond_fp16_leaves_the_others_alone(shape):
    """The second expert's weights need another exponent range; its neighbours in the stream share tiles with it."""
    counts, n, k = shape
    print(f"case neighbours {op_forms.label(shape)}", flush=True)
    _, w = packed_weights(len(counts), n, k, 3)
    w[1] *= 2.0 ** -60                                                 # an empty group: no row uses these weights
    check(shape, rca.quantize_pack(w, rca.MXFP4), w, 4)


@pytest.mark.parametrize("byte", [0, 60, 254, 255])
@SHAPES
def test_scales_beyond_fp16_in_single_blocks(shape, byte):
    """Single blocks with a scale out of fp16's range, with codes and without: the first and the last of an expert, one
    in the middle of its 41st row, the last of its 130th.  Rows of whole numbers are held to the stated bound (their
    sums with such weights are no binary32 numbers); rows of one value each, in the columns of these blocks, are exact
    (where a weight overflows, any value that is not finite)."""
    counts, n, k = shape
    print(f"case scale {byte} {op_forms.label(shape)}", flush=True)
    packed, w = packed_weights(len(counts), n, k, 5)
    rows, off, each = op_forms.rows_of(counts), offsets(counts), k // 32
    x = whole(rows, k, torch.float16, 6)
    one = torch.zeros(rows, k, dtype=torch.float16, device=DEV)
    r = torch.arange(rows, device=DEV)
    at = torch.tensor([0, k - 1, each // 2 * 32 + 5, k - 7], device=DEV)[r % 4]
    one[r, at] = (r % 6 + 1).to(torch.float16)
    expert = torch.searchsorted(on_gpu(off)[1:], r, right=True).clamp(max=len(counts) - 1)
    inside = (r >= off[0]) & (r < off[-1])
    for codes in (True, False):
        p = packed.clone()
        tiles = p.view(-1, 1088)
        for b in (0, n * each - 1, 40 * each + each // 2, 130 * each - 1):
            for e in range(len(counts)):
                block = e * n * each + b
                tiles[block // 64, 1024 + block % 64] = byte
                if not codes:
                    tiles[block // 64, block % 64 * 16:block % 64 * 16 + 16] = 0x80       # zeros of both signs
        v = rca.unpack_dequant(p, rca.MXFP4, w.numel()).view_as(w)
        y = rca.mxfp4_grouped_matmul(x, p, on_gpu(off), n, out_dtype=torch.float32)
        want, mag = product(x, v, off)
        fine = mag < 2.0 ** 100                                        # the others' weights overflow, or are NaN
        held(y[fine], want[fine], mag[fine], k, torch.float32, "whole numbers")
        y = rca.mxfp4_grouped_matmul(one, p, on_gpu(off), n, out_dtype=torch.float32)
        if byte == 255:                                                # NaN, whatever the codes are
            hit = v[expert].isnan().any(2) & inside[:, None]
            assert hit.any() and y[hit].isnan().all()
            y[hit] = 0
            v = v.nan_to_num(nan=0.0)
        else:
            hit = torch.zeros_like(y, dtype=torch.bool)
        weight = v[expert, :, at].double()
        want = torch.where(inside[:, None] & ~hit, one[r, at, None].double() * weight, 0.0)
        over = v[expert].isinf().any(2) & inside[:, None]
        assert torch.equal(y[~over].double(), want.float().double()[~over])
        assert not y[over & weight.isinf()].isfinite().any()
