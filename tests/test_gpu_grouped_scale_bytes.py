"""The smallest scale, the largest one (weights that overflow to an infinity)
and the NaN scale among ordinary blocks, in every form of every type, forward
and to the rows.  bf16 rows give what the definition gives; rows cut into terms
may give NaN for an infinity."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_forms
from tests.test_gpu_grouped_forms import DTYPES, SHAPES, TYPES, offsets, on_gpu, held, product, setup, weights, whole

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@DTYPES
@SHAPES
def test_scale_bytes(shape, dtype):
    counts, n, k, rows, off = setup(shape, dtype, "scale bytes")
    packed = weights(len(counts), n, k, 1)[0].clone()
    tiles, each = packed.view(-1, 1088), k // 32
    for e in range(len(counts)):                           # in rows 1, 3, 5 and 7 of every expert
        for row, block, byte in ((1, 0, 0), (3, each - 1, 254), (5, each // 2, 255), (7, 0, 252)):
            at = (e * n + row) * each + block
            tiles[at // 64, 1024 + at % 64] = byte
    w = rca.unpack_dequant(packed, rca.MXFP4, len(counts) * n * k).view(len(counts), n, k)
    assert w.isinf().any() and w.isnan().any()
    for transpose, width in ((False, k), (True, n)):
        x = whole(rows, width, TYPES[dtype], 2).abs() + 1  # no zero meets an infinity
        if transpose:
            got = rca.mxfp4_grouped_matmul_dx(x, packed, on_gpu(off), k, out_dtype=torch.float32)
        else:
            got = rca.mxfp4_grouped_matmul(x, packed, on_gpu(off), n, out_dtype=torch.float32)
        large = torch.where(w.isinf() | w.isnan(), torch.zeros_like(w), w).abs() >= 2.0 ** 100
        want, mag = product(x, w, off, transpose)
        # sums of products near binary32's end may overflow in one order and not in another
        near = product(x, large.float(), off, transpose)[0] > 0
        fine = want.isfinite() & ~near
        held(got[fine], want[fine], mag[fine], width, torch.float32, transpose)
        over = ~want.isfinite() & ~near
        assert over.any() and not got[over].isfinite().any() and got[want.isnan()].isnan().all()
        if dtype == "bf16":
            assert torch.equal(got[over].nan_to_num(nan=0.25), want[over].float().nan_to_num(nan=0.25))
