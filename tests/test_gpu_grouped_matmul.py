"""Products grouped by expert on MXFP4 weights, against binary64.

Two kinds of inputs: small whole numbers with power-of-two scales, whose sums
are exact in binary32 in any order, so the results must be equal; and random
values, held to the stated bound (N + 3) 2^-23 sum |p| plus one rounding."""
import numpy as np
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = [torch.bfloat16, torch.float16, torch.float32]

# experts' row counts, n, k: single rows, empty experts, groups around tile edges, odd widths
SHAPES = [
    ([1], 8, 32),
    ([0, 1, 0], 64, 64),
    ([1, 1], 4096, 4096),
    ([3, 0, 7, 1], 200, 96),
    ([16, 17, 15, 1], 72, 160),
    ([31, 32, 33], 128, 2048),
    ([63, 64, 65, 0, 129], 136, 224),
    ([255, 257, 0, 1], 264, 288),
    ([700], 1000, 2080),
    ([0, 0, 530, 0], 520, 512),
    ([5] * 70, 24, 64),
]


def offsets_of(counts, first=0):
    return [first] + [first + int(v) for v in np.cumsum(counts)]


def on_gpu(t):
    return t.to(DEV)


def exact_inputs(rows, width, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-6, 7, (rows, width), generator=g).to(dtype)


def random_inputs(rows, width, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g)
    return (x * torch.exp(torch.rand(rows, width, generator=g) * 4 - 2)).to(dtype)


def held(got, want, mag, terms, dtype, what):
    got = got.cpu().double()
    assert got.shape == want.shape, what
    tol = (terms + 3) * 2.0 ** -23 * mag + ref.rounding(want, dtype)
    off = (got - want).abs()
    bad = (off > tol) | got.isnan()
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_whole_numbers_are_exact_in_every_direction(case, dtype):
    counts, n, k = SHAPES[case]
    print(f"case exact {counts[:6]} n={n} k={k} {dtype}", flush=True)
    off = offsets_of(counts)
    rows, experts = off[-1], len(counts)
    packed, w = ref.random_packed(experts, n, k, case, exponents=(-2, 2))
    x, dy = exact_inputs(rows, k, dtype, 100 + case), exact_inputs(rows, n, dtype, 200 + case)
    pd, od, xd, dyd = on_gpu(packed), on_gpu(torch.tensor(off, dtype=torch.int32)), on_gpu(x), on_gpu(dy)
    y = rca.mxfp4_grouped_matmul(xd, pd, od, n, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), ref.grouped(x, w, off)[0])
    dx = rca.mxfp4_grouped_matmul_dx(dyd, pd, od, k, out_dtype=torch.float32)
    assert torch.equal(dx.cpu().double(), ref.grouped_dx(dy, w, off)[0])
    dw = rca.grouped_matmul_dw(dyd, xd, od)
    assert torch.equal(dw.cpu().double(), ref.grouped_dw(dy, x, off)[0])


@pytest.mark.parametrize("exponents", [(-30, -27), (-16, -12), (12, 16)])
@pytest.mark.parametrize("case", [2, 3, 4, 6, 7, 8])
def test_fp16_rows_on_weights_beyond_fp16(case, exponents):
    """Weights that fp16 cannot hold, or only as subnormals: the products are
    formed in another way, exact all the same."""
    counts, n, k = SHAPES[case]
    print(f"case beyond fp16 {counts[:6]} n={n} k={k} {exponents}", flush=True)
    off = offsets_of(counts)
    packed, w = ref.random_packed(len(counts), n, k, case, exponents=exponents)
    x = exact_inputs(off[-1], k, torch.float16, 100 + case)
    y = rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), on_gpu(torch.tensor(off, dtype=torch.int32)), n,
                                 out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), ref.grouped(x, w, off)[0])


@pytest.mark.parametrize("out", DTYPES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("case", [3, 4, 7, 8])
def test_random_values_within_the_bound(case, dtype, out):
    counts, n, k = SHAPES[case]
    print(f"case random {counts[:6]} n={n} k={k} {dtype} -> {out}", flush=True)
    off = offsets_of(counts)
    rows, experts = off[-1], len(counts)
    packed, w = ref.random_packed(experts, n, k, 40 + case)
    x, dy = random_inputs(rows, k, dtype, case), random_inputs(rows, n, dtype, 7 + case) * 0.01
    pd, od, xd, dyd = on_gpu(packed), on_gpu(torch.tensor(off, dtype=torch.int32)), on_gpu(x), on_gpu(dy)
    held(rca.mxfp4_grouped_matmul(xd, pd, od, n, out_dtype=out), *ref.grouped(x, w, off), k, out, "y")
    held(rca.mxfp4_grouped_matmul_dx(dyd, pd, od, k, out_dtype=out), *ref.grouped_dx(dy, w, off), n, out, "dx")
    held(rca.grouped_matmul_dw(dyd, xd, od, out_dtype=out), *ref.grouped_dw(dy, x, off), max(counts), out, "dw")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("first,counts,after", [(3, [2, 0, 5], 4), (70, [1, 130], 65), (0, [0, 0], 9), (5, [0], 0)])
def test_rows_of_no_expert_get_zeros(first, counts, after, dtype):
    print(f"case outside {first} {counts} {after} {dtype}", flush=True)
    n, k = 40, 96
    off = offsets_of(counts, first)
    rows = off[-1] + after
    packed, w = ref.random_packed(len(counts), n, k, 5, exponents=(-2, 2))
    x, dy = exact_inputs(rows, k, dtype, 1), exact_inputs(rows, n, dtype, 2)
    pd, od = on_gpu(packed), on_gpu(torch.tensor(off, dtype=torch.int32))
    y = torch.full((rows, n), 7.0, dtype=torch.float32, device=DEV)
    dx = torch.full((rows, k), 7.0, dtype=torch.float32, device=DEV)
    rca.mxfp4_grouped_matmul(on_gpu(x), pd, od, n, out_dtype=torch.float32, out=y)
    rca.mxfp4_grouped_matmul_dx(on_gpu(dy), pd, od, k, out_dtype=torch.float32, out=dx)
    assert torch.equal(y.cpu().double(), ref.grouped(x, w, off)[0])
    assert torch.equal(dx.cpu().double(), ref.grouped_dx(dy, w, off)[0])
    dw = rca.grouped_matmul_dw(on_gpu(dy), on_gpu(x), od)
    assert torch.equal(dw.cpu().double(), ref.grouped_dw(dy, x, off)[0])


def test_no_rows_and_one_matrix():
    packed, w = ref.random_packed(2, 16, 64, 1)
    od = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    dy = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    assert rca.mxfp4_grouped_matmul(x, on_gpu(packed), od, 16).shape == (0, 16)
    assert rca.mxfp4_grouped_matmul_dx(dy, on_gpu(packed), od, 64).shape == (0, 64)
    assert not rca.grouped_matmul_dw(dy, x, od).any()


def test_a_single_vector_is_the_gemv():
    rows, cols = 96, 2048
    packed, w = ref.random_packed(1, rows, cols, 9, exponents=(-2, 2))
    x = exact_inputs(1, cols, torch.bfloat16, 3)
    od = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    y = rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), od, rows, out_dtype=torch.float32)
    assert torch.equal(y[0], rca.mxfp4_gemv(on_gpu(packed), rows, cols, on_gpu(x[0])))


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_scale_extremes(dtype, rows):
    """Blocks with the smallest scale, the largest ones (weights that overflow to
    infinity) and the NaN scale: rows in fp16 / fp32 see an infinite weight as an
    infinity or a NaN, everything else as IEEE arithmetic gives it."""
    n, k = 64, 128
    special = [(0, 0), (5, 1), (9, 255), (14, 254)]
    packed, w = ref.random_packed(1, n, k, 2, exponents=(-2, 2), special=special)
    w32 = w.to(torch.float32)
    x = exact_inputs(rows, k, dtype, 4).abs() + 1
    od = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), od, n, out_dtype=torch.float32).cpu()
    fine = w32[0].isfinite().all(1) & (w32[0].abs() < 2.0 ** 100).all(1)
    assert fine.sum() >= n - 2
    want, mag = ref.grouped(x, w, [0, rows])
    assert ((y.double() - want).abs()[:, fine] <= ((k + 3) * 2.0 ** -23 * mag + ref.rounding(want, torch.float32))[:, fine]).all()
    assert y[:, 2].isnan().all()                       # block 9: row 2
    if dtype == torch.bfloat16:                        # block 14: row 3, weights up to 6 * 2^127
        assert not y[:, 3].isfinite().any() or not w32[0, 3].isinf().any()


def test_non_finite_rows_stay_in_their_rows():
    n, k, rows = 48, 96, 130
    packed, w = ref.random_packed(1, n, k, 3, exponents=(-2, 2))
    x = exact_inputs(rows, k, torch.bfloat16, 4)
    x[7, 3], x[65, 95], x[129, 0] = float("inf"), float("nan"), float("-inf")
    od = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), od, n, out_dtype=torch.float32).cpu()
    want = torch.full((rows, n), 0.0, dtype=torch.float64)
    for i in range(rows):
        want[i] = (x[i].double()[None] * w[0]).sum(1)
    clean = torch.ones(rows, dtype=torch.bool)
    clean[[7, 65, 129]] = False
    assert torch.equal(y[clean].double(), want[clean])
    assert y[65].isnan().all()
    assert torch.equal(y[7].isnan(), want[7].isnan()) and torch.equal(y[129].isnan(), want[129].isnan())


def test_offsets_that_do_not_ascend_stay_in_bounds():
    """Unspecified values, but nothing outside the buffers: the kernels clamp
    every bound to the rows there are."""
    n, k, rows = 64, 64, 50
    packed, _ = ref.random_packed(3, n, k, 3)
    x = exact_inputs(rows, k, torch.bfloat16, 4)
    for off in ([0, 40, 10, 50], [-5, 20, 2 ** 31 - 1, 3], [60, 70, 80, 90], [0, -2 ** 31, 50, 2]):
        print(f"case offsets {off}", flush=True)
        od = torch.tensor(off, dtype=torch.int32, device=DEV)
        guard = torch.full((rows + 64, n), 3.0, dtype=torch.float32, device=DEV)
        rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), od, n, out_dtype=torch.float32, out=guard[:rows])
        assert (guard[rows:] == 3.0).all()
        dw = rca.grouped_matmul_dw(on_gpu(x), on_gpu(x), od)
        assert dw.shape == (3, n, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_repeats_bit_for_bit(dtype):
    counts, n, k = [120, 3, 400], 512, 1024
    off = offsets_of(counts)
    packed, _ = ref.random_packed(3, n, k, 8)
    x, dy = on_gpu(random_inputs(off[-1], k, dtype, 1)), on_gpu(random_inputs(off[-1], n, dtype, 2))
    pd, od = on_gpu(packed), on_gpu(torch.tensor(off, dtype=torch.int32))
    run = lambda: (rca.mxfp4_grouped_matmul(x, pd, od, n), rca.mxfp4_grouped_matmul_dx(dy, pd, od, k),  # noqa: E731
                   rca.grouped_matmul_dw(dy, x, od))
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """dx and dW against central differences of the forward pass, which is
    linear in x and in W: with whole numbers both are exact."""
    counts, n, k = [5, 0, 9], 16, 64
    off = offsets_of(counts)
    packed, w = ref.random_packed(3, n, k, 12, exponents=(-1, 1))
    od = on_gpu(torch.tensor(off, dtype=torch.int32))
    x, dy = exact_inputs(off[-1], k, torch.float32, 5), exact_inputs(off[-1], n, torch.float32, 6)
    loss = lambda xs: (rca.mxfp4_grouped_matmul(on_gpu(xs), on_gpu(packed), od, n).double().cpu() * dy.double()).sum()  # noqa: E731
    dx = rca.mxfp4_grouped_matmul_dx(on_gpu(dy), on_gpu(packed), od, k).cpu().double()
    dw = rca.grouped_matmul_dw(on_gpu(dy), on_gpu(x), od).cpu().double()
    for seed in range(4):
        step = exact_inputs(off[-1], k, torch.float32, 50 + seed)
        assert float(loss(x + step) - loss(x - step)) / 2 == float((dx * step.double()).sum())
        dstep = torch.randint(-2, 3, w.shape, generator=torch.Generator().manual_seed(seed)).double()
        change = ref.grouped(x, w + dstep, off)[0] - ref.grouped(x, w - dstep, off)[0]
        assert float((change * dy.double()).sum()) / 2 == float((dw * dstep).sum())


def test_more_than_2_to_32_weights():
    """The last expert of a stream of 4.6e9 weights (its code bytes start past
    2^31 and its elements past 2^32)."""
    experts, n, k = 1100, 2048, 2048
    tiles = n * k // 2048
    one, w = ref.random_packed(1, n, k, 6, exponents=(-2, 2))
    packed = torch.zeros(experts * tiles * 1088, dtype=torch.uint8, device=DEV)
    packed[-tiles * 1088:] = on_gpu(one)
    for counts in ([0] * (experts - 1) + [3], [0] * (experts - 1) + [200]):
        off = offsets_of(counts)
        x, dy = exact_inputs(off[-1], k, torch.bfloat16, 1), exact_inputs(off[-1], n, torch.bfloat16, 2)
        od = on_gpu(torch.tensor(off, dtype=torch.int32))
        print(f"case large weights rows={off[-1]}", flush=True)
        y = rca.mxfp4_grouped_matmul(on_gpu(x), packed, od, n, out_dtype=torch.float32)
        assert torch.equal(y.cpu().double(), x.double() @ w[0].T)
        dx = rca.mxfp4_grouped_matmul_dx(on_gpu(dy), packed, od, k, out_dtype=torch.float32)
        assert torch.equal(dx.cpu().double(), dy.double() @ w[0])


def test_more_than_2_to_32_outputs():
    """Rows whose outputs lie past 2^32 elements."""
    n, k, rows = 65536, 32, 70000
    packed, w = ref.random_packed(1, n, k, 6, exponents=(-1, 1))
    x = exact_inputs(rows, k, torch.bfloat16, 1)
    od = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    print("case large outputs", flush=True)
    y = rca.mxfp4_grouped_matmul(on_gpu(x), on_gpu(packed), od, n)
    want = (x[-300:].double() @ w[0].T).to(torch.bfloat16)
    assert torch.equal(y[-300:].cpu(), want)
    dx = rca.mxfp4_grouped_matmul_dx(y, on_gpu(packed), od, k, out_dtype=torch.float32)
    full = want[-8:].double() @ w[0]
    mag = want[-8:].double().abs() @ w[0].abs()
    held(dx[-8:], full, mag, n, torch.float32, "dx")
