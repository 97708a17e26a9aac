"""Every form of the products grouped by expert, at sizes that the launch rules
send to it: ragged groups (empty, of one row, around tile edges), rows of no
expert, several spans and column tiles, partial last ones.

Where results are compared for equality, every partial sum is a binary32
number, so they are the same in any order: small whole numbers, or rows of one
value each, whose bits then all have to arrive.  Random values are held to the
stated bound (N + 3) 2^-23 sum |p| plus one rounding.  References are formed in
binary64 on the GPU."""
import functools
import itertools

import numpy as np
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_forms
from tests import op_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SHAPES = pytest.mark.parametrize("shape", op_forms.SHAPES, ids=op_forms.label)
DTYPES = pytest.mark.parametrize("dtype", TYPES)


@functools.lru_cache(2)
def weights(experts, n, k, seed, exponents=(-2, 2), powers=False):
    """(packed, values as fp32) on the GPU; `powers`: codes of plus and minus 0.5, 1, 2 and 4 only."""
    count = experts * n * k
    tiles = -(-count // 2048)
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 16, (tiles, 2048), generator=g, dtype=torch.uint8, device=DEV)
    if powers:
        codes = torch.tensor([1, 2, 4, 6, 9, 10, 12, 14], dtype=torch.uint8, device=DEV)[(codes & 7).long()]
    scales = torch.randint(127 + exponents[0], 128 + exponents[1], (tiles, 64), generator=g, dtype=torch.uint8, device=DEV)
    packed = torch.cat([codes[:, 0::2] | (codes[:, 1::2] << 4), scales], 1).reshape(-1).contiguous()
    return packed, rca.unpack_dequant(packed, rca.MXFP4, count).view(experts, n, k)


def offsets(counts):
    return [op_forms.BEFORE] + [op_forms.BEFORE + int(v) for v in np.cumsum(counts)]


def on_gpu(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def whole(rows, width, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-6, 7, (rows, width), generator=g, device=DEV).to(dtype)


def product(x, w, off, transpose=False):
    """y (or dx) and the sums of the products' magnitudes, in binary64; rows of no expert 0."""
    y = torch.zeros(x.shape[0], w.shape[2 if transpose else 1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    for e, (a, b) in enumerate(itertools.pairwise(off) if hasattr(itertools, "pairwise") else zip(off, off[1:])):
        if b > a:
            m = w[e].double() if transpose else w[e].double().T.contiguous()
            y[a:b] = x[a:b].double() @ m
            mag[a:b] = x[a:b].double().abs() @ m.abs()
    return y, mag


def outer(dy, x, off, e):
    a, b = off[e], off[e + 1]
    p, q = dy[a:b].double().T.contiguous(), x[a:b].double()
    return p @ q, p.abs() @ q.abs()


def held(got, want, mag, terms, dtype, what):
    tol = (terms + 3) * 2.0 ** -23 * mag + ref.rounding(want, dtype)
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).max()))


def setup(shape, dtype, what):
    counts, n, k = shape
    rows = op_forms.rows_of(counts)
    print(f"case {what} {op_forms.label(shape)} {dtype} {op_forms.forms(dtype, rows, len(counts), n, k)}", flush=True)
    return counts, n, k, rows, offsets(counts)


@DTYPES
@SHAPES
def test_whole_numbers_are_exact(shape, dtype):
    counts, n, k, rows, off = setup(shape, dtype, "whole")
    t, od = TYPES[dtype], on_gpu(off)
    packed, w = weights(len(counts), n, k, 1)
    x, dy = whole(rows, k, t, 2), whole(rows, n, t, 3)
    y = torch.full((rows, n), 7.0, device=DEV)
    dx = torch.full((rows, k), 7.0, device=DEV)
    rca.mxfp4_grouped_matmul(x, packed, od, n, out_dtype=torch.float32, out=y)
    rca.mxfp4_grouped_matmul_dx(dy, packed, od, k, out_dtype=torch.float32, out=dx)
    dw = rca.grouped_matmul_dw(dy, x, od)
    assert torch.equal(y.double(), product(x, w, off)[0])
    assert torch.equal(dx.double(), product(dy, w, off, True)[0])
    for e in range(len(counts)):
        assert torch.equal(dw[e].double(), outer(dy, x, off, e)[0]), e


def one_each(rows, width, dtype, seed):
    """Rows of one value each, with all the bits of its type: fp16 subnormals too, fp32 from 2^-108 on (whose last bit
    is a bfloat16 subnormal)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if dtype == torch.float32:
        bits = torch.randint(0, 1 << 23, (rows,), generator=g, device=DEV, dtype=torch.int32) | 1
        exponent = torch.randint(127 - 108, 127 + 80, (rows,), generator=g, device=DEV, dtype=torch.int32)
        sign = torch.randint(0, 2, (rows,), generator=g, device=DEV, dtype=torch.int32)
        v = (bits | (exponent << 23) | (sign << 31)).view(torch.float32)
    else:
        bits = torch.randint(-1 << 15, 1 << 15, (rows,), generator=g, device=DEV, dtype=torch.int32).to(torch.int16)
        bits[::3] &= -31745 if dtype == torch.float16 else -1          # a third of the fp16 values subnormal
        v = bits.view(dtype)
        if dtype == torch.bfloat16:                                    # products with weights stay normal binary32 numbers
            v = torch.where((v.float().abs() < 2.0 ** -100) | (v.float().abs() > 2.0 ** 100), torch.ones_like(v), v)
        v = torch.where(v.isfinite(), v, torch.ones_like(v))
    x = torch.zeros(rows, width, dtype=dtype, device=DEV)
    at = torch.randint(0, width, (rows,), generator=g, device=DEV)
    x[torch.arange(rows, device=DEV), at] = v
    return x, v, at


@DTYPES
@SHAPES
def test_all_bits_of_the_rows_arrive(shape, dtype):
    """One value a row and weights that are powers of two: every output is one product, exact in binary32."""
    counts, n, k, rows, off = setup(shape, dtype, "bits")
    t, od = TYPES[dtype], on_gpu(off)
    packed, w = weights(len(counts), n, k, 4, exponents=(-3, 3), powers=True)
    for what, width in (("y", k), ("dx", n)):
        x, v, at = one_each(rows, width, t, 5)
        if what == "y":
            got = rca.mxfp4_grouped_matmul(x, packed, od, n, out_dtype=torch.float32)
        else:
            got = rca.mxfp4_grouped_matmul_dx(x, packed, od, k, out_dtype=torch.float32)
        for e in range(len(counts)):
            a, b = off[e], off[e + 1]
            m = (w[e].T if what == "y" else w[e])[at[a:b]].double()
            assert torch.equal(got[a:b].double(), v[a:b, None].double() * m), (what, e)
        assert not got[:off[0]].any() and not got[off[-1]:].any()


@DTYPES
@SHAPES
def test_all_bits_arrive_in_the_weight_gradient(shape, dtype):
    """One value in each row of dy and of x, no two rows of a group at one place: exact for 16-bit types (22 bits at
    most), within the bound of one product for fp32."""
    counts, n, k, rows, off = setup(shape, dtype, "bits of dw")
    t, od = TYPES[dtype], on_gpu(off)
    _, v, _ = one_each(rows, 8, t, 6)
    _, u, _ = one_each(rows, 8, t, 7)
    if dtype == "fp32":                                                # the products stay normal
        u, v = torch.where(u.abs() < 1, 1 / u, u).clamp(-1e30, 1e30), v.clamp(-1.0, 1.0)
        u = torch.where(u.abs() * v.abs() < 2.0 ** -100, torch.ones_like(u), u)
    if dtype == "bf16":
        u = torch.where((u.abs().float() * v.abs().float() < 2.0 ** -100) | (u.abs().float() * v.abs().float() > 2.0 ** 100),
                        torch.ones_like(u), u)
    at_y, at_x = torch.arange(rows, device=DEV) % n, torch.arange(rows, device=DEV) * 5 % k
    dy, x = torch.zeros(rows, n, dtype=t, device=DEV), torch.zeros(rows, k, dtype=t, device=DEV)
    dy[torch.arange(rows, device=DEV), at_y], x[torch.arange(rows, device=DEV), at_x] = v, u
    dw = rca.grouped_matmul_dw(dy, x, od)
    for e in range(len(counts)):
        want = torch.zeros(n, k, dtype=torch.float64, device=DEV)
        a, b = off[e], off[e + 1]
        want[at_y[a:b], at_x[a:b]] = v[a:b].double() * u[a:b].double()
        if dtype == "fp32":
            held(dw[e], want, want.abs(), 1, torch.float32, e)
        else:
            assert torch.equal(dw[e].double(), want), e


@pytest.mark.parametrize("exponents", [(-30, -27), (-16, -12), (12, 16)])
@SHAPES
def test_fp16_rows_on_weights_beyond_fp16(shape, exponents):
    """Weights that fp16 cannot hold, or only as subnormals."""
    counts, n, k, rows, off = setup(shape, "fp16", f"beyond fp16 {exponents}")
    packed, w = weights(len(counts), n, k, 8, exponents=exponents)
    x = whole(rows, k, torch.float16, 9)
    y = rca.mxfp4_grouped_matmul(x, packed, on_gpu(off), n, out_dtype=torch.float32)
    assert torch.equal(y.double(), product(x, w, off)[0])


@DTYPES
@SHAPES
def test_random_values_within_the_bound_and_the_same_again(shape, dtype):
    counts, n, k, rows, off = setup(shape, dtype, "random")
    t, od = TYPES[dtype], on_gpu(off)
    out = list(TYPES.values())[(n // 8 + k // 32) % 3]
    packed, w = weights(len(counts), n, k, 10)
    g = torch.Generator(device=DEV).manual_seed(11)
    rn = lambda width, std: (torch.randn(rows, width, generator=g, device=DEV) * std * torch.exp(  # noqa: E731
        torch.rand(rows, width, generator=g, device=DEV) * 4 - 2)).to(t)
    x, dy = rn(k, 1.0), rn(n, 0.01)
    first = None
    for _ in range(2):
        got = (rca.mxfp4_grouped_matmul(x, packed, od, n, out_dtype=out), rca.mxfp4_grouped_matmul_dx(dy, packed, od, k, out_dtype=out),
               rca.grouped_matmul_dw(dy, x, od, out_dtype=out))
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    held(got[0], *product(x, w, off), k, out, "y")
    held(got[1], *product(dy, w, off, True), n, out, "dx")
    for e in range(len(counts)):
        held(got[2][e], *outer(dy, x, off, e), max(1, counts[e]), out, f"dw {e}")
