"""Infinities and NaN in the rows, in every form of every type: what is not
finite stays in its row (its group's rows and columns of the weight gradient),
and everything there that the definition makes infinite or NaN is not finite.
bf16 rows, and fp16 rows in the weight gradient, come out as the definition
has them; where fp16 or fp32 rows are cut into terms an infinity may be NaN."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_forms
from tests.test_gpu_grouped_forms import DTYPES, SHAPES, TYPES, offsets, on_gpu, outer, product, setup, weights, whole

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BAD = [float("inf"), float("-inf"), float("nan")]


def spoil(x, off, step, seed):
    """Every `step`-th row of the groups gets one infinity or NaN; (rows, columns)."""
    r = torch.arange(off[0] + seed, off[-1], step, device=DEV)
    c = r * 11 % x.shape[1]
    x[r, c] = torch.tensor(BAD, device=DEV)[torch.arange(r.numel(), device=DEV) % 3].to(x.dtype)
    return r, c


def same(a, b):
    return torch.equal(a.nan_to_num(nan=0.25), b.nan_to_num(nan=0.25))


@DTYPES
@SHAPES
def test_rows_that_are_not_finite(shape, dtype):
    counts, n, k, rows, off = setup(shape, dtype, "not finite")
    packed, w = weights(len(counts), n, k, 1)
    od = on_gpu(off)
    expert = torch.searchsorted(od[1:], torch.arange(rows, device=DEV), right=True)
    for transpose, width in ((False, k), (True, n)):
        x = whole(rows, width, TYPES[dtype], 2)
        r, c = spoil(x, off, 7, 1)
        if transpose:
            got = rca.mxfp4_grouped_matmul_dx(x, packed, od, k, out_dtype=torch.float32)
            weight = w[expert[r], c]
        else:
            got = rca.mxfp4_grouped_matmul(x, packed, od, n, out_dtype=torch.float32)
            weight = w[expert[r], :, c]
        want = x[r, c, None].float() * weight              # nothing else in the row changes it
        clean = torch.ones(rows, dtype=torch.bool, device=DEV)
        clean[r] = False
        x[r, c] = 0
        assert torch.equal(got[clean].double(), product(x, w, off, transpose)[0][clean])
        if dtype == "bf16":
            assert same(got[r], want)
        assert not got[r].isfinite().any() and got[r][want.isnan()].isnan().all()


@DTYPES
@SHAPES
def test_weight_gradient_of_rows_that_are_not_finite(shape, dtype):
    counts, n, k, rows, off = setup(shape, dtype, "not finite dw")
    t = TYPES[dtype]
    dy, x = whole(rows, n, t, 3), whole(rows, k, t, 4)
    spoil(dy, off, 41, 2)
    spoil(x, off, 53, 5)
    dw = rca.grouped_matmul_dw(dy, x, on_gpu(off))
    for e in range(len(counts)):
        want = outer(dy, x, off, e)[0].float()
        # inf and -inf, or 0 times inf, meet in one sum: NaN there, as in any order of additions
        fine = want.isfinite()
        assert torch.equal(dw[e][fine], want[fine]) and not dw[e][~fine].isfinite().any()
        if dtype != "fp32":
            assert same(dw[e], want)
