"""fp32 rows whose last bits lie below bfloat16's smallest number, 2^-133, in
every form: values count as its nearest multiple, so one product p = x w is off
by at most 2^-134 |w|, plus the stated bound and one rounding."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_forms
from tests.test_gpu_grouped_forms import SHAPES, offsets, on_gpu, setup, weights

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def tiny(rows, seed):
    """fp32 values of all magnitudes below 2^-100, subnormals among them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    bits = torch.randint(0, 28 << 23, (rows,), generator=g, device=DEV, dtype=torch.int32)
    return (bits | (torch.randint(0, 2, (rows,), generator=g, device=DEV, dtype=torch.int32) << 31)).view(torch.float32)


def within(got, want, other, what):
    tol = other * 2.0 ** -134 + 4 * 2.0 ** -23 * want.abs() + 2.0 ** -149
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (what, float((off / tol).max()))


@SHAPES
def test_rows(shape):
    counts, n, k, rows, off = setup(shape, "fp32", "small")
    packed, w = weights(len(counts), n, k, 1, exponents=(40, 46))
    for transpose, width in ((False, k), (True, n)):
        x = torch.zeros(rows, width, device=DEV)
        r = torch.arange(rows, device=DEV)
        at, v = r * 13 % width, tiny(rows, 2)
        x[r, at] = v
        if transpose:
            got = rca.mxfp4_grouped_matmul_dx(x, packed, on_gpu(off), k)
        else:
            got = rca.mxfp4_grouped_matmul(x, packed, on_gpu(off), n)
        for e in range(len(counts)):
            a, b = off[e], off[e + 1]
            m = (w[e] if transpose else w[e].T)[at[a:b]].double()
            within(got[a:b], v[a:b, None].double() * m, m.abs(), (transpose, e))


@SHAPES
def test_weight_gradient(shape):
    counts, n, k, rows, off = setup(shape, "fp32", "small dw")
    r = torch.arange(rows, device=DEV)
    v = tiny(rows, 3)
    u = torch.randn(rows, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) * 2.0 ** 60
    dy, x = torch.zeros(rows, n, device=DEV), torch.zeros(rows, k, device=DEV)
    dy[r, r % n], x[r, r * 5 % k] = v, u
    dw = rca.grouped_matmul_dw(dy, x, on_gpu(off))
    for e in range(len(counts)):
        a, b = off[e], off[e + 1]
        want, other = (torch.zeros(n, k, dtype=torch.float64, device=DEV) for _ in range(2))
        want[(r % n)[a:b], (r * 5 % k)[a:b]] = v[a:b].double() * u[a:b].double()
        other[(r % n)[a:b], (r * 5 % k)[a:b]] = u[a:b].abs().double()
        within(dw[e], want, other, e)
