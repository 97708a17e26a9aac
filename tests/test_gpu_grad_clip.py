"""Global norm of many tensors and clipping by it, against binary64.

The squares are added in binary64, so the norm is the exact one rounded to
binary32 (2^-23 covers the root and the scale); the factor goes through four
more roundings of binary32 and every value through one product and one
rounding to its type."""
import math

import pytest
import torch

import reduction_codec_amd as rca
from tests import op_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [[1], [0, 1, 0], [7, 4096, 3], [8192, 8193, 8191], [100000], [1] * 300, list(range(1, 220)),
         [4095 * 3, 0, 65536, 17] * 60]


def tensors(sizes, dtypes, seed=0, std=0.01):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.empty(s, device=DEV).normal_(0, std, generator=g).to(dtypes[i % len(dtypes)]) for i, s in enumerate(sizes)]


def check(grads, outs, norm, before, scale, max_norm, eps=1e-6):
    want, factor = ref.clip(before, scale, max_norm, eps)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    for b, o in zip(before, outs):
        w = b.double() * factor
        tol = w.abs() * 10 * ref.U32 + ref.rounding(w, o.dtype)
        assert ((o.double() - w).abs() <= tol).all()


@pytest.mark.parametrize("dtypes", [[d] for d in DTYPES] + [DTYPES], ids=["bf16", "fp16", "fp32", "mixed"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_in_place_and_into_others(case, dtypes):
    print(f"case clip {case} {dtypes}", flush=True)
    for scale, max_norm in ((1.0, 0.05), (0.125, 1e9), (-2.0, 0.5), (1.0, float("inf")), (1.0, 0.0)):
        grads = tensors(SIZES[case], dtypes, seed=case)
        before = [t.clone() for t in grads]
        outs = [torch.full_like(t, 9.0, dtype=DTYPES[(i + case) % 3]) for i, t in enumerate(grads)]
        norm = rca.grad_norm_clip(grads, max_norm, scale=scale, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        check(grads, outs, norm, before, scale, max_norm)
        norm2 = rca.grad_norm_clip(grads, max_norm, scale=scale)
        assert torch.equal(norm, norm2)
        check(grads, grads, norm2, before, scale, max_norm)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_parts_of_one_buffer_at_any_alignment(dtype):
    sizes = [3, 8191, 1, 20001, 5, 8192, 16385, 77]
    flat, other = torch.randn(sum(sizes) + 9, device=DEV).to(dtype), torch.full((sum(sizes) + 9,), 4.0, device=DEV, dtype=dtype)
    for shift_in, shift_out in ((0, 0), (1, 1), (1, 3), (7, 2)):
        at, grads, outs = 0, [], []
        for s in sizes:
            grads.append(flat[shift_in + at:shift_in + at + s])
            outs.append(other[shift_out + at:shift_out + at + s])
            at += s
        other.fill_(4.0)
        norm = rca.grad_norm_clip(grads, 1.0, out=outs)
        check(grads, outs, norm, grads, 1.0, 1.0)
        assert (other[:shift_out] == 4.0).all() and (other[shift_out + at:] == 4.0).all()


def test_under_the_limit_nothing_changes():
    grads = tensors([1000, 37], [torch.bfloat16])
    before = [t.clone() for t in grads]
    norm = rca.grad_norm_clip(grads, 100.0)
    assert float(norm) < 100 and all(torch.equal(a, b) for a, b in zip(grads, before))


def test_values_whose_squares_leave_binary32():
    big = [torch.full((1000,), 1e30, device=DEV), torch.full((10,), 1e-30, device=DEV)]
    norm = rca.grad_norm_clip(big, 1.0)
    assert abs(float(norm) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    assert torch.allclose(big[0], torch.full_like(big[0], 1000 ** -0.5), rtol=1e-6)
    small = [torch.full((1000,), 1e-30, device=DEV)]
    norm = rca.grad_norm_clip(small, 1.0)
    assert abs(float(norm) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6


def test_non_finite_gradients_show():
    for bad in (float("inf"), float("nan")):
        grads = [torch.ones(100, device=DEV), torch.ones(9000, device=DEV, dtype=torch.bfloat16)]
        grads[1][8999] = bad
        norm = rca.grad_norm_clip(grads, 1.0)
        assert (math.isinf if bad == float("inf") else math.isnan)(float(norm))
        assert grads[1][8999].isnan()
        assert (grads[0] == 0).all() if bad == float("inf") else grads[0].isnan().all()


def test_all_empty():
    norm = rca.grad_norm_clip([torch.empty(0, device=DEV), torch.empty(0, 3, device=DEV)], 1.0)
    assert float(norm) == 0.0


def test_order_does_not_show():
    grads = tensors([5000, 300001, 17] * 50, DTYPES, seed=4)
    first = [torch.empty_like(t) for t in grads]
    n1 = rca.grad_norm_clip(grads, 0.1, out=first)
    for _ in range(3):
        again = [torch.empty_like(t) for t in grads]
        assert torch.equal(n1, rca.grad_norm_clip(grads, 0.1, out=again))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_more_than_2_to_32_elements():
    n = (1 << 32) + 12345
    print("case large", flush=True)
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[-1], t[-20000] = 3.0, 4.0
    norm = rca.grad_norm_clip([t], 1.0)
    assert abs(float(norm) - 5.0) < 1e-6
    assert abs(float(t[-1]) - 0.6) < 0.002 and abs(float(t[-20000]) - 0.8) < 0.002
