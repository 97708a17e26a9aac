"""The operators around the codec refuse what they cannot do, with the
documented status and before any HIP call (no GPU is needed), and the binding
with a ValueError."""
import ctypes

import pytest
import torch

import reduction_codec_amd as rca

A, M = 0x10000, 0x10008                     # aligned, misaligned: never dereferenced
BIG = (1 << 40) + 1


def grouped(which, w=A, experts=4, n=64, k=64, off=A, t=3, x=A, rows=8, out_t=3, out=A):
    return getattr(rca.lib(), which)(w, experts, n, k, off, t, x, rows, out_t, out, None)


@pytest.mark.parametrize("which", ["rc_mxfp4_grouped_matmul", "rc_mxfp4_grouped_matmul_dx"])
def test_grouped_matmul(which):
    g = lambda **a: grouped(which, **a)  # noqa: E731
    assert g(t=0) == rca.ERR_UNSUPPORTED and g(out_t=4) == rca.ERR_UNSUPPORTED
    for bad in ({"experts": 0}, {"experts": 65536}, {"n": 0}, {"n": 12}, {"n": (1 << 20) + 8}, {"k": 0}, {"k": 48},
                {"k": (1 << 20) + 32}, {"rows": 1 << 31}, {"experts": 65535, "n": 1 << 20, "k": 1 << 20}):
        assert g(**bad) == rca.ERR_RANGE, bad
    for bad in ("w", "off", "x", "out"):
        assert g(**{bad: None}) == rca.ERR_NULL, bad
        assert g(**{bad: M}) == rca.ERR_ALIGN, bad
    assert g(rows=0, w=None, off=None, x=None, out=None) == rca.OK


def test_grouped_matmul_dw():
    def g(experts=4, n=64, k=64, off=A, t=3, dy=A, x=A, rows=8, dw_t=1, dw=A):
        return rca.lib().rc_grouped_matmul_dw(experts, n, k, off, t, dy, x, rows, dw_t, dw, None)
    assert g(t=9) == rca.ERR_UNSUPPORTED and g(dw_t=0) == rca.ERR_UNSUPPORTED
    assert g(n=4) == rca.ERR_RANGE and g(k=33) == rca.ERR_RANGE and g(experts=0) == rca.ERR_RANGE
    for bad in ("off", "dy", "x", "dw"):
        assert g(**{bad: None}) == rca.ERR_NULL, bad
        assert g(**{bad: M}) == rca.ERR_ALIGN, bad


def test_block_norm():
    def f(t=3, rows=4, d=64, y=A, r=A, w_t=3, post=A, mode=1, gate=A, pre=A, h=A, z=A, stats=A):
        return rca.lib().rc_block_norm(t, rows, d, y, r, w_t, post, mode, gate, pre, 1.0, 1e-6, h, z, stats, None)
    assert f(t=0) == rca.ERR_UNSUPPORTED and f(w_t=7) == rca.ERR_UNSUPPORTED and f(mode=3) == rca.ERR_UNSUPPORTED
    assert f(d=0) == rca.ERR_RANGE and f(d=32769) == rca.ERR_RANGE and f(rows=BIG) == rca.ERR_RANGE
    assert f(rows=0, y=None) == rca.OK
    for bad in ("y", "r", "pre", "h", "z", "gate"):
        assert f(**{bad: None}) == rca.ERR_NULL, bad
    for bad in ("y", "r", "pre", "h", "z", "gate", "post", "stats"):
        assert f(**{bad: M}) == rca.ERR_ALIGN, bad


def test_block_norm_backward():
    def f(t=3, rows=4, d=64, dz=A, dh=A, h=A, stats=A, y=A, w_t=3, post=A, mode=2, gate=A, pre=A, dy=A, dr=A, dpre=A,
          dpost=A, dgate=A, ws=A):
        return rca.lib().rc_block_norm_backward(t, rows, d, dz, dh, h, stats, y, w_t, post, mode, gate, pre, 1.0, dy,
                                                dr, dpre, dpost, dgate, ws, None)
    assert f(t=0) == rca.ERR_UNSUPPORTED and f(w_t=7) == rca.ERR_UNSUPPORTED and f(mode=-1) == rca.ERR_UNSUPPORTED
    assert f(d=0) == rca.ERR_RANGE and f(d=32769) == rca.ERR_RANGE and f(rows=BIG) == rca.ERR_RANGE
    for bad in ("dz", "h", "stats", "y", "gate", "pre", "dy", "dr", "dpre", "dpost", "dgate", "ws"):
        assert f(**{bad: None}) == rca.ERR_NULL, bad
    for bad in ("dz", "dh", "h", "stats", "y", "post", "gate", "pre", "dy", "dr", "dpre", "dpost", "dgate", "ws"):
        assert f(**{bad: M}) == rca.ERR_ALIGN, bad
    assert rca.lib().rc_block_norm_backward_workspace(10, 0) == 0
    assert rca.lib().rc_block_norm_backward_workspace(10, 32769) == 0
    assert rca.lib().rc_block_norm_backward_workspace(10, 100) % 8 == 0


class Grad(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("o", ctypes.c_void_p), ("n", ctypes.c_uint64), ("it", ctypes.c_int32),
                ("ot", ctypes.c_int32)]


def test_grad_norm_clip():
    def f(rows=((A, A, 10, 3, 3),), scale=1.0, max_norm=1.0, eps=1e-6, ws=A, norm=A, null=False):
        arr = (Grad * max(1, len(rows)))(*[Grad(*r) for r in rows])
        return rca.lib().rc_grad_norm_clip(None if null else ctypes.addressof(arr), len(rows), scale, max_norm, eps,
                                           ws, norm, None)
    assert f(max_norm=-1.0) == rca.ERR_RANGE and f(max_norm=float("nan")) == rca.ERR_RANGE
    assert f(eps=-1e-6) == rca.ERR_RANGE and f(rows=((A, A, BIG, 3, 3),)) == rca.ERR_RANGE
    assert f(ws=None) == rca.ERR_NULL and f(norm=None) == rca.ERR_NULL and f(null=True) == rca.ERR_NULL
    assert f(ws=M) == rca.ERR_ALIGN and f(norm=A + 2) == rca.ERR_ALIGN
    assert f(rows=((None, A, 10, 3, 3),)) == rca.ERR_NULL and f(rows=((A, None, 10, 3, 3),)) == rca.ERR_NULL
    assert f(rows=((A, A, 10, 0, 3),)) == rca.ERR_UNSUPPORTED and f(rows=((A, A, 10, 3, 1),)) == rca.ERR_UNSUPPORTED
    assert f(rows=((A + 2, M, 10, 1, 1),)) == rca.ERR_ALIGN and f(rows=((A + 1, M, 10, 3, 3),)) == rca.ERR_ALIGN


def test_binding_refuses():
    cpu = torch.zeros(4, 64)
    off = torch.zeros(3, dtype=torch.int32)
    packed = torch.zeros(1088 * 8, dtype=torch.uint8)
    for call in (lambda: rca.mxfp4_grouped_matmul(cpu, packed, off, 64),
                 lambda: rca.mxfp4_grouped_matmul_dx(cpu, packed, off, 64),
                 lambda: rca.grouped_matmul_dw(cpu, cpu, off),
                 lambda: rca.block_norm(cpu, cpu, cpu[0]),
                 lambda: rca.block_norm_backward(cpu, None, cpu, cpu, cpu, cpu[0]),
                 lambda: rca.grad_norm_clip([cpu], 1.0),
                 lambda: rca.grad_norm_clip([], 1.0)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    dev = torch.device("cuda:0")
    x = torch.zeros(4, 64, device=dev, dtype=torch.bfloat16)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    packed = torch.zeros(1088 * 4, dtype=torch.uint8, device=dev)          # 2 x 64 x 64
    w = torch.ones(64, device=dev)
    bad = [
        lambda: rca.mxfp4_grouped_matmul(x[0], packed, off, 64),             # one dimension
        lambda: rca.mxfp4_grouped_matmul(x, packed, off.long(), 64),
        lambda: rca.mxfp4_grouped_matmul(x, packed, off[:1], 64),
        lambda: rca.mxfp4_grouped_matmul(x, packed[:-1], off, 64),
        lambda: rca.mxfp4_grouped_matmul(x, packed, off, 128),               # packed too short
        lambda: rca.mxfp4_grouped_matmul(x.int(), packed, off, 64),
        lambda: rca.mxfp4_grouped_matmul(x, packed, off, 64, out_dtype=torch.int8),
        lambda: rca.mxfp4_grouped_matmul(x, packed, off, 64, out=torch.empty(4, 65, device=dev)),
        lambda: rca.mxfp4_grouped_matmul(x.t(), packed, off, 64),            # not contiguous
        lambda: rca.grouped_matmul_dw(x, x.float(), off),
        lambda: rca.grouped_matmul_dw(x, x[:3], off),
        lambda: rca.block_norm(x, x[:3], w),
        lambda: rca.block_norm(x, x, w[:63]),
        lambda: rca.block_norm(x, x, w, post_weight=w.bfloat16()),
        lambda: rca.block_norm(x, x, w, gate=w.bfloat16()),
        lambda: rca.block_norm(x, x, w, gate=x.float()),
        lambda: rca.block_norm_backward(x, x, x, torch.zeros(7, device=dev), x, w),
        lambda: rca.grad_norm_clip([x, w], 1.0, out=[x]),
        lambda: rca.grad_norm_clip([x], 1.0, out=[w]),
        lambda: rca.grad_norm_clip([x.t()], 1.0),
        lambda: rca.grad_norm_clip([x.int()], 1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    for call in (lambda: rca.mxfp4_grouped_matmul(x, packed, off, 60),
                 lambda: rca.mxfp4_grouped_matmul(x[:, :40].contiguous(), packed, off, 64)):
        with pytest.raises(rca.CodecError) as e:
            call()
        assert e.value.status == rca.ERR_RANGE
