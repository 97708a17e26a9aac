"""Python binding of the MI355X codec library ``librcodec.so``.

Argument marshalling only: every step of the codec runs in the HIP kernels
behind the C ABI declared in ``include/rcodec.h``.  PyTorch provides device
memory and the current stream; nothing here computes on the CPU, and there is
no fallback: if the library is not built, every call raises.

Entry points (same names as the C ABI, minus the ``rc_`` prefix):

* ``quantize_pack(x, codec)``             -> packed uint8 tensor
* ``unpack_dequant(packed, codec, n, dtype)`` -> tensor of n values
* ``dequant_reduce_requant(streams, codec, n, sum_out=False)``
                                           -> (packed, fp32 sums or None)
* ``tile_bytes(codec)``, ``packed_bytes(codec, n)``, ``copy(dst, src)``

and the operators around a quantized all-reduce:

* ``mxfp4_grouped_matmul(x, w_packed, offsets, n)``, ``mxfp4_grouped_matmul_dx``,
  ``grouped_matmul_dw``               -> products grouped by expert
* ``block_norm(y, residual, pre_weight, ...)``, ``block_norm_backward``
                                           -> norms around a block, gate, residual
* ``grad_norm_clip(grads, max_norm)``  -> global norm of many tensors, clipping

and a paged cache of keys and values held in MXFP4:

* ``mxfp4_cache_new(pages, kv_heads, page, d, device)`` -> (k_cache, v_cache)
* ``mxfp4_cache_append(k, v, k_cache, v_cache, table, lengths, offsets, q=...)``
                                           -> q turned by its positions, or None
* ``mxfp4_cache_attention(q, k_cache, v_cache, table, lengths, offsets)``
                                           -> out, or (out, log-sum-exp)
* ``mxfp4_cache_read(k_cache, v_cache, table, lengths, offsets, tokens, d)``
                                           -> (k, v) as the cache holds them
"""
from __future__ import annotations

import array
import ctypes
import operator
import os

import torch  # must load before librcodec.so: both share torch's HIP runtime

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librcodec.so")

TILE = 2048
BLOCK = 32
MAX_STREAMS = 16
MXFP4_TILE_BYTES = 1088

FMT_INT4, FMT_INT3, FMT_FP8_E4M3, FMT_MXFP4, FMT_FP8_E5M2 = 1, 2, 3, 4, 5
SCALE_FP16, SCALE_FP32, SCALE_E8M0 = 1, 2, 3
DT_FP32, DT_FP16, DT_BF16 = 1, 2, 3
GATE_NONE, GATE_CHANNEL, GATE_FULL = 0, 1, 2
OK, ERR_NULL, ERR_UNSUPPORTED, ERR_ALIGN, ERR_RANGE, ERR_HIP = 0, 1, 2, 3, 4, 5


class Codec(ctypes.Structure):
    """rc_codec: element format, scale type, block size (passed by value)."""
    _fields_ = [("format", ctypes.c_int32), ("scale", ctypes.c_int32), ("block", ctypes.c_int32)]

    def __repr__(self):
        return f"Codec({self.format}, {self.scale}, {self.block})"


INT4 = Codec(FMT_INT4, SCALE_FP16, BLOCK)
INT3 = Codec(FMT_INT3, SCALE_FP16, BLOCK)
FP8 = Codec(FMT_FP8_E4M3, SCALE_FP32, BLOCK)
MXFP4 = Codec(FMT_MXFP4, SCALE_E8M0, BLOCK)
CODECS = {"int4": INT4, "int3": INT3, "fp8": FP8, "mxfp4": MXFP4}


def _all_codecs():
    """Every codec the library supports, by name "<element>_<scale>_b<block>"
    (also accepted wherever a codec is expected)."""
    elems = {"int4": FMT_INT4, "int3": FMT_INT3, "e4m3": FMT_FP8_E4M3, "e5m2": FMT_FP8_E5M2, "e2m1": FMT_MXFP4}
    scales = {"f16": SCALE_FP16, "f32": SCALE_FP32, "e8m0": SCALE_E8M0}
    allowed = {"int4": ("f16", "e8m0"), "int3": ("f16", "e8m0"), "e4m3": ("f32", "f16", "e8m0"),
               "e5m2": ("f32", "f16", "e8m0"), "e2m1": ("e8m0",)}
    return {f"{e}_{sc}_b{b}": Codec(elems[e], scales[sc], b)
            for e, scs in allowed.items() for sc in scs for b in (16, 32, 64)}


ALL_CODECS = _all_codecs()

ABI_VERSION = 3                       # RC_ABI_VERSION of include/rcodec.h
_DTYPES = {torch.float32: DT_FP32, torch.float16: DT_FP16, torch.bfloat16: DT_BF16}
_lib = None


class CodecError(RuntimeError):
    """A non-zero rc_status from the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().rc_status_str(status).decode()} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded librcodec.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                           "(the codec has no CPU fallback)")
    l = ctypes.CDLL(LIB_PATH)
    try:
        l.rc_abi_version.restype, l.rc_abi_version.argtypes = ctypes.c_int, []
        if l.rc_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI version {l.rc_abi_version()}, this binding expects "
                               f"{ABI_VERSION}; rebuild the library")
        _declare(l)
    except AttributeError as e:                          # functions are added without a new version
        raise RuntimeError(f"{LIB_PATH} is older than this binding ({e}); rebuild the library") from None
    _lib = l
    return l


def _declare(l: ctypes.CDLL):
    """The types of the library's functions."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    l.rc_tile_bytes.restype, l.rc_tile_bytes.argtypes = sz, [Codec]
    l.rc_packed_bytes.restype, l.rc_packed_bytes.argtypes = sz, [Codec, sz]
    l.rc_quantize_pack.restype, l.rc_quantize_pack.argtypes = i32, [Codec, i32, vp, sz, vp, vp]
    l.rc_unpack_dequant.restype, l.rc_unpack_dequant.argtypes = i32, [Codec, vp, sz, i32, vp, vp]
    l.rc_dequant_reduce_requant.restype = i32
    l.rc_dequant_reduce_requant.argtypes = [Codec, ctypes.POINTER(vp), i32, sz, vp, vp, vp]
    l.rc_copy.restype, l.rc_copy.argtypes = i32, [vp, vp, sz, vp]
    l.rc_mxfp4_gemv.restype = i32
    l.rc_mxfp4_gemv.argtypes = [vp, sz, sz, i32, vp, i32, vp, vp]
    l.rc_allreduce_emulate.restype = i32
    l.rc_allreduce_emulate.argtypes = [Codec, i32, ctypes.POINTER(vp), i32, sz, i32, vp, vp, vp]
    l.rc_mxfp4_grouped_matmul.restype = i32
    l.rc_mxfp4_grouped_matmul.argtypes = [vp, sz, sz, sz, vp, i32, vp, sz, i32, vp, vp]
    l.rc_mxfp4_grouped_matmul_dx.restype = i32
    l.rc_mxfp4_grouped_matmul_dx.argtypes = [vp, sz, sz, sz, vp, i32, vp, sz, i32, vp, vp]
    l.rc_grouped_matmul_dw.restype = i32
    l.rc_grouped_matmul_dw.argtypes = [sz, sz, sz, vp, i32, vp, vp, sz, i32, vp, vp]
    f32 = ctypes.c_float
    l.rc_block_norm.restype = i32
    l.rc_block_norm.argtypes = [i32, sz, sz, vp, vp, i32, vp, i32, vp, vp, f32, f32, vp, vp, vp, vp]
    l.rc_block_norm_backward_workspace.restype, l.rc_block_norm_backward_workspace.argtypes = sz, [sz, sz]
    l.rc_block_norm_backward.restype = i32
    l.rc_block_norm_backward.argtypes = [i32, sz, sz, vp, vp, vp, vp, vp, i32, vp, i32, vp, vp, f32,
                                         vp, vp, vp, vp, vp, vp, vp]
    l.rc_grad_norm_clip_workspace.restype, l.rc_grad_norm_clip_workspace.argtypes = sz, []
    l.rc_grad_norm_clip.restype, l.rc_grad_norm_clip.argtypes = i32, [vp, sz, f32, f32, f32, vp, vp, vp]
    l.rc_mxfp4_cache_append.restype = i32
    l.rc_mxfp4_cache_append.argtypes = [vp, i32, sz, vp, sz, vp, sz, sz, vp, sz, vp, vp, sz, sz, i32, vp]
    l.rc_mxfp4_cache_read.restype, l.rc_mxfp4_cache_read.argtypes = i32, [vp, sz, i32, vp, vp, vp]
    l.rc_mxfp4_cache_attention_workspace.restype = sz
    l.rc_mxfp4_cache_attention_workspace.argtypes = [sz, sz, sz, sz]
    l.rc_mxfp4_cache_attention.restype = i32
    l.rc_mxfp4_cache_attention.argtypes = [vp, i32, sz, sz, vp, sz, f32, i32, sz, sz, vp, vp, vp, vp]
    l.rc_status_str.restype, l.rc_status_str.argtypes = ctypes.c_char_p, [i32]


def _codec(c) -> Codec:
    if isinstance(c, Codec):
        return c
    if isinstance(c, str):
        return CODECS[c] if c in CODECS else ALL_CODECS[c]
    return Codec(*c)


def _stream(stream, dev: torch.device) -> ctypes.c_void_p:
    """The HIP stream to launch on: the given one (which must belong to the
    tensors' device) or that device's current stream."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return ctypes.c_void_p(stream.cuda_stream)


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _same_device(dev: torch.device, *named):
    for name, t in named:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _new(shape, dtype: torch.dtype, dev: torch.device, stream) -> torch.Tensor:
    """A tensor for work enqueued on `stream` (None: the current one), from
    that stream's memory: a block that the current stream has freed may still
    be read or written by work queued there, which `stream` does not wait for.
    The caller goes on with the tensor on the current stream, so torch's
    allocator is told not to hand it out again before that has finished too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _stream(stream, dev)
    current = torch.cuda.current_stream(dev)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(current)
    return t


def _check_dev(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ok(status: int, what: str):
    if status != OK:
        raise CodecError(status, what)


def tile_bytes(codec) -> int:
    return lib().rc_tile_bytes(_codec(codec))


def packed_bytes(codec, n: int) -> int:
    return lib().rc_packed_bytes(_codec(codec), n)


def quantize_pack(x: torch.Tensor, codec, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Block-quantize the elements of x (bf16 / fp16 / fp32, any shape, taken
    flat) into ``packed_bytes(codec, x.numel())`` bytes."""
    c = _codec(codec)
    _check_dev(x, "x")
    hs = _stream(stream, x.device)
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    n = x.numel()
    if out is None:
        out = _new(packed_bytes(c, n), torch.uint8, x.device, stream)
    _check_dev(out, "out")
    _same_device(x.device, ("out", out))
    if out.numel() < packed_bytes(c, n) or out.dtype != torch.uint8:
        raise ValueError("out must be a uint8 tensor of packed_bytes(codec, n) bytes")
    with torch.cuda.device(x.device):
        _ok(lib().rc_quantize_pack(c, _DTYPES[x.dtype], x.data_ptr(), n, out.data_ptr(), hs),
            "rc_quantize_pack")
    return out


def unpack_dequant(packed: torch.Tensor, codec, n: int, dtype: torch.dtype = torch.float32,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode the first n elements of a packed stream to dtype."""
    c = _codec(codec)
    _check_dev(packed, "packed")
    hs = _stream(stream, packed.device)
    if _nbytes(packed) < packed_bytes(c, n):
        raise ValueError("packed is shorter than packed_bytes(codec, n)")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {dtype}")
    if out is None:
        out = _new(n, dtype, packed.device, stream)
    _check_dev(out, "out")
    _same_device(packed.device, ("out", out))
    if out.numel() < n or out.dtype != dtype:
        raise ValueError("out must hold n elements of dtype")
    with torch.cuda.device(packed.device):
        _ok(lib().rc_unpack_dequant(c, packed.data_ptr(), n, _DTYPES[dtype], out.data_ptr(), hs),
            "rc_unpack_dequant")
    return out


def dequant_reduce_requant(streams, codec, n: int, out: torch.Tensor | None = None,
                           sum_out: bool | torch.Tensor = False, stream=None):
    """Dequantize K packed streams, add them in FP32 in stream order and
    requantize.  Returns (packed, sums) with sums None unless requested."""
    c = _codec(codec)
    streams = list(streams)
    k = len(streams)
    if not 1 <= k <= MAX_STREAMS:
        raise ValueError(f"need 1..{MAX_STREAMS} streams, got {k}")
    need = packed_bytes(c, n)
    dev = streams[0].device if streams and isinstance(streams[0], torch.Tensor) else None
    for j, s in enumerate(streams):
        _check_dev(s, f"streams[{j}]")
        _same_device(dev, (f"streams[{j}]", s))
        if _nbytes(s) < need:
            raise ValueError(f"streams[{j}] is shorter than packed_bytes(codec, n)")
    hs = _stream(stream, dev)
    if out is None:
        out = _new(need, torch.uint8, dev, stream)
    _check_dev(out, "out")
    _same_device(dev, ("out", out))
    if _nbytes(out) < need:
        raise ValueError("out is shorter than packed_bytes(codec, n)")
    sums = None
    if isinstance(sum_out, torch.Tensor):
        sums = sum_out
        _check_dev(sums, "sum_out")
        _same_device(dev, ("sum_out", sums))
        if sums.dtype != torch.float32 or sums.numel() < n:
            raise ValueError("sum_out must hold n float32 values")
    elif sum_out:
        sums = _new(n, torch.float32, dev, stream)
    ptrs = (ctypes.c_void_p * k)(*[s.data_ptr() for s in streams])
    with torch.cuda.device(dev):
        _ok(lib().rc_dequant_reduce_requant(c, ptrs, k, n, out.data_ptr(),
                                            sums.data_ptr() if sums is not None else None, hs),
            "rc_dequant_reduce_requant")
    return out, sums


def allreduce_emulate(msgs, codec, two_shot: bool = True, out: torch.Tensor | None = None,
                      packed_out: bool | torch.Tensor = False, stream=None):
    """Fused one-GPU emulation of a quantized all-reduce of the messages (one
    per emulated rank, same dtype and length).  Returns (out, packed or
    None); see rc_allreduce_emulate in include/rcodec.h."""
    c = _codec(codec)
    msgs = list(msgs)
    k = len(msgs)
    if not 1 <= k <= MAX_STREAMS:
        raise ValueError(f"need 1..{MAX_STREAMS} messages, got {k}")
    dt = msgs[0].dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    n = msgs[0].numel()
    dev = msgs[0].device
    for j, m in enumerate(msgs):
        _check_dev(m, f"msgs[{j}]")
        _same_device(dev, (f"msgs[{j}]", m))
        if m.dtype != dt or m.numel() != n:
            raise ValueError("all messages need the same dtype and length")
    hs = _stream(stream, dev)
    if out is None:
        out = _new(n, dt, dev, stream)
    _check_dev(out, "out")
    _same_device(dev, ("out", out))
    if out.dtype != dt or out.numel() < n:
        raise ValueError("out must hold n elements of the messages' dtype")
    packed = None
    if isinstance(packed_out, torch.Tensor):
        packed = packed_out
        _check_dev(packed, "packed_out")
        _same_device(dev, ("packed_out", packed))
        if packed.numel() < packed_bytes(c, n) or packed.dtype != torch.uint8:
            raise ValueError("packed_out must be a uint8 tensor of packed_bytes(codec, n) bytes")
    elif packed_out:
        packed = _new(packed_bytes(c, n), torch.uint8, dev, stream)
    ptrs = (ctypes.c_void_p * k)(*[m.data_ptr() for m in msgs])
    with torch.cuda.device(dev):
        _ok(lib().rc_allreduce_emulate(c, _DTYPES[dt], ptrs, k, n, 1 if two_shot else 0, out.data_ptr(),
                                       packed.data_ptr() if packed is not None else None, hs),
            "rc_allreduce_emulate")
    return out, packed


def mxfp4_gemv(w_packed: torch.Tensor, rows: int, cols: int, x: torch.Tensor, out_dtype=torch.float32,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = W x with W (rows x cols, row-major) packed by quantize_pack with the
    MXFP4 codec; cols a multiple of 2048.  See rc_mxfp4_gemv."""
    _check_dev(w_packed, "w_packed")
    _check_dev(x, "x")
    _same_device(w_packed.device, ("x", x))
    hs = _stream(stream, w_packed.device)
    if w_packed.dtype != torch.uint8 or w_packed.numel() < packed_bytes(MXFP4, rows * cols):
        raise ValueError("w_packed must hold packed_bytes(MXFP4, rows * cols) bytes")
    if x.dtype not in _DTYPES or x.numel() < cols:
        raise ValueError("x must hold cols fp32 / fp16 / bf16 values")
    if out_dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {out_dtype}")
    if out is None:
        out = _new(rows, out_dtype, x.device, stream)
    _check_dev(out, "out")
    _same_device(w_packed.device, ("out", out))
    if out.dtype != out_dtype or out.numel() < rows:
        raise ValueError("out must hold rows values of out_dtype")
    with torch.cuda.device(w_packed.device):
        _ok(lib().rc_mxfp4_gemv(w_packed.data_ptr(), rows, cols, _DTYPES[x.dtype], x.data_ptr(), _DTYPES[out_dtype],
                                out.data_ptr(), hs), "rc_mxfp4_gemv")
    return out


def copy(dst: torch.Tensor, src: torch.Tensor, stream=None) -> torch.Tensor:
    """Byte copy through the library's 16-byte vector copy kernel."""
    _check_dev(dst, "dst")
    _check_dev(src, "src")
    _same_device(src.device, ("dst", dst))
    hs = _stream(stream, src.device)
    nbytes = _nbytes(src)
    if _nbytes(dst) < nbytes:
        raise ValueError("dst too small")
    with torch.cuda.device(src.device):
        _ok(lib().rc_copy(src.data_ptr(), dst.data_ptr(), nbytes, hs), "rc_copy")
    return dst


# ------------------------------------------- operators around the codec ----

def _dtype(dt: torch.dtype, name: str) -> int:
    if dt not in _DTYPES:
        raise ValueError(f"unsupported {name} dtype {dt}")
    return _DTYPES[dt]


def _check_on(t: torch.Tensor, name: str, index: int):
    """A contiguous tensor on GPU `index`."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous():
        _check_dev(t, name)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _result(out, shape, dtype, dev: torch.device, stream, name: str) -> torch.Tensor:
    """The caller's output, checked, or a new one for work on `stream`."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev) if stream is None else _new(shape, dtype, dev, stream)
    _check_on(out, name, dev.index)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    return out


def _launch(what: str, dev: torch.device, stream, *args):
    """The library's function on the device and stream; its status checked."""
    hs = torch.cuda.current_stream(dev.index).cuda_stream if stream is None else _stream(stream, dev)
    if dev.index == torch.cuda.current_device():
        status = getattr(_lib or lib(), what)(*args, hs)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib or lib(), what)(*args, hs)
    if status != OK:
        raise CodecError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows_of(t: torch.Tensor, name: str, offsets: torch.Tensor):
    _check_dev(t, name)
    _check_on(offsets, "offsets", t.get_device())
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, rows and width")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must hold experts + 1 int32 values")
    return t.shape[0], t.shape[1], offsets.numel() - 1


def _weights(w_packed: torch.Tensor, experts: int, n: int, k: int, dev):
    _check_on(w_packed, "w_packed", dev.index)
    tiles = -(-experts * n * k // TILE)
    if n < 0 or k < 0 or w_packed.dtype != torch.uint8 or w_packed.numel() < tiles * MXFP4_TILE_BYTES:
        raise ValueError("w_packed must hold packed_bytes(MXFP4, experts * n * k) bytes")


def mxfp4_grouped_matmul(x: torch.Tensor, w_packed: torch.Tensor, offsets: torch.Tensor, n: int,
                         out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """y[i] = W_e x[i] for the rows offsets[e] <= i < offsets[e + 1] of x
    (rows x k, sorted by expert): W_e is n x k, all experts one after another
    in one MXFP4 packed stream; offsets int32 on the GPU, experts + 1 values.
    Returns rows x n of out_dtype (x's by default).  See
    rc_mxfp4_grouped_matmul."""
    rows, k, experts = _rows_of(x, "x", offsets)
    dev = x.device
    _weights(w_packed, experts, n, k, dev)
    y_t = x.dtype if out_dtype is None else out_dtype
    xt, yt = _dtype(x.dtype, "x"), _dtype(y_t, "output")
    out = _result(out, (rows, n), y_t, dev, stream, "out")
    _launch("rc_mxfp4_grouped_matmul", dev, stream, w_packed.data_ptr(), experts, n, k, offsets.data_ptr(), xt,
            x.data_ptr(), rows, yt, out.data_ptr())
    return out


def mxfp4_grouped_matmul_dx(dy: torch.Tensor, w_packed: torch.Tensor, offsets: torch.Tensor, k: int,
                            out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """dx[i] = W_e^T dy[i]: the gradient of mxfp4_grouped_matmul's rows, from
    dy (rows x n); rows x k of out_dtype (dy's by default)."""
    rows, n, experts = _rows_of(dy, "dy", offsets)
    dev = dy.device
    _weights(w_packed, experts, n, k, dev)
    dx_t = dy.dtype if out_dtype is None else out_dtype
    yt, xt = _dtype(dy.dtype, "dy"), _dtype(dx_t, "output")
    out = _result(out, (rows, k), dx_t, dev, stream, "out")
    _launch("rc_mxfp4_grouped_matmul_dx", dev, stream, w_packed.data_ptr(), experts, n, k, offsets.data_ptr(),
            yt, dy.data_ptr(), rows, xt, out.data_ptr())
    return out


def grouped_matmul_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                      out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """dW[e] = sum over expert e's rows of dy[i] x[i]^T (experts x n x k): the
    dense gradient of the weights before their cast to MXFP4."""
    rows, n, experts = _rows_of(dy, "dy", offsets)
    dev = dy.device
    _check_on(x, "x", dev.index)
    if x.dim() != 2 or x.shape[0] != rows or x.dtype != dy.dtype:
        raise ValueError("x must have dy's rows and dtype")
    k = x.shape[1]
    t, wt = _dtype(dy.dtype, "dy"), _dtype(out_dtype, "output")
    out = _result(out, (experts, n, k), out_dtype, dev, stream, "out")
    _launch("rc_grouped_matmul_dw", dev, stream, experts, n, k, offsets.data_ptr(), t, dy.data_ptr(),
            x.data_ptr(), rows, wt, out.data_ptr())
    return out


def _norm_weights(like: torch.Tensor, d: int, pre_weight, post_weight, gate):
    """(weight type, gate mode) of a block norm; the gate is None, d values of
    the weights' type, or one per element of `like`, of its type."""
    index = like.get_device()
    _check_on(pre_weight, "pre_weight", index)
    if post_weight is not None:
        _check_on(post_weight, "post_weight", index)
    if gate is not None:
        _check_on(gate, "gate", index)
    wt = _dtype(pre_weight.dtype, "weight")
    if pre_weight.numel() != d or (post_weight is not None and
                                   (post_weight.numel() != d or post_weight.dtype != pre_weight.dtype)):
        raise ValueError("pre_weight and post_weight must hold one value per column, of one dtype")
    if gate is None:
        return wt, GATE_NONE
    if gate.dim() == 1 and gate.numel() == d and gate.dtype == pre_weight.dtype:
        return wt, GATE_CHANNEL
    if gate.shape == like.shape and gate.dtype == like.dtype:
        return wt, GATE_FULL
    raise ValueError("gate must be one value per column of the weights' dtype, or y's shape and dtype")


def _like(t: torch.Tensor, like: torch.Tensor, name: str):
    _check_on(t, name, like.get_device())
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must have y's shape and dtype")


def block_norm(y: torch.Tensor, residual: torch.Tensor, pre_weight: torch.Tensor,
               post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               residual_scale: float = 1.0, eps: float = 1e-6, stats: bool = False,
               h: torch.Tensor | None = None, z: torch.Tensor | None = None, stream=None):
    """Norm of a block's output y, its gate, the scaled residual and the norm
    before the next block, over the last dimension:

        u = post_weight * y / rms(y)  (u = y without post_weight)
        h = residual_scale * residual + gate * u
        z = pre_weight * h / rms(h)

    Returns (h, z, stats): stats is None, or the 2 x rows fp32 values that
    block_norm_backward reads.  h may be the residual and z may be y.  See
    rc_block_norm."""
    _check_dev(y, "y")
    if y.dim() < 1 or y.shape[-1] == 0:
        raise ValueError("y must have a last dimension of at least one value")
    d = y.shape[-1]
    rows = y.numel() // d
    _like(residual, y, "residual")
    wt, mode = _norm_weights(y, d, pre_weight, post_weight, gate)
    t = _dtype(y.dtype, "y")
    dev, shape, dtype = y.device, y.shape, y.dtype
    h = _result(h, shape, dtype, dev, stream, "h")
    z = _result(z, shape, dtype, dev, stream, "z")
    st = _result(None, (2, rows), torch.float32, dev, stream, "stats") if stats else None
    _launch("rc_block_norm", dev, stream, t, rows, d, y.data_ptr(), residual.data_ptr(), wt, _ptr(post_weight),
            mode, _ptr(gate), pre_weight.data_ptr(), residual_scale, eps, h.data_ptr(), z.data_ptr(), _ptr(st))
    return h, z, st


def block_norm_backward(dz: torch.Tensor, dh: torch.Tensor | None, h: torch.Tensor, stats: torch.Tensor,
                        y: torch.Tensor, pre_weight: torch.Tensor, post_weight: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                        dy: torch.Tensor | None = None, dresidual: torch.Tensor | None = None, stream=None):
    """Gradients of block_norm from dz and dh (what reaches h beside z, or
    None), with the forward pass's y, h and stats.  Returns (dy, dresidual,
    dpre, dpost, dgate); dpre, dpost and a channel gate's gradient are fp32, a
    full gate's has y's dtype; dpost and dgate are None where there is no such
    input.  dy may be dz and dresidual may be dh.  See rc_block_norm_backward."""
    _check_dev(y, "y")
    if y.dim() < 1 or y.shape[-1] == 0:
        raise ValueError("y must have a last dimension of at least one value")
    d = y.shape[-1]
    rows = y.numel() // d
    for name, g in (("dz", dz), ("h", h)) + ((("dh", dh),) if dh is not None else ()):
        _like(g, y, name)
    dev = y.device
    _check_on(stats, "stats", dev.index)
    if stats.dtype != torch.float32 or stats.numel() != 2 * rows:
        raise ValueError("stats must hold 2 x rows float32 values")
    wt, mode = _norm_weights(y, d, pre_weight, post_weight, gate)
    t = _dtype(y.dtype, "y")
    dy = _result(dy, y.shape, y.dtype, dev, stream, "dy")
    dr = _result(dresidual, y.shape, y.dtype, dev, stream, "dresidual")
    new = lambda shape, dt: _result(None, shape, dt, dev, stream, "")  # noqa: E731
    dpre = new((d,), torch.float32)
    dpost = new((d,), torch.float32) if post_weight is not None else None
    dgate = None if gate is None else new((d,), torch.float32) if mode == GATE_CHANNEL else new(y.shape, y.dtype)
    ws = new((lib().rc_block_norm_backward_workspace(rows, d),), torch.uint8)
    _launch("rc_block_norm_backward", dev, stream, t, rows, d, dz.data_ptr(), _ptr(dh), h.data_ptr(),
            stats.data_ptr(), y.data_ptr(), wt, _ptr(post_weight), mode, _ptr(gate), pre_weight.data_ptr(),
            residual_scale, dy.data_ptr(), dr.data_ptr(), dpre.data_ptr(), _ptr(dpost), _ptr(dgate), ws.data_ptr())
    return dy, dr, dpre, dpost, dgate


_dtype_of = operator.attrgetter("dtype")


def _tensors(tensors, dev: torch.device, name: str):
    """(addresses, sizes, type codes) of contiguous tensors on `dev`; a few
    hundred of them are looked at per call, hence the maps over C methods."""
    T = torch.Tensor
    try:
        if set(map(T.get_device, tensors)) == {dev.index} and all(map(T.is_contiguous, tensors)):
            return (array.array("Q", map(T.data_ptr, tensors)), array.array("Q", map(T.numel, tensors)),
                    memoryview(array.array("I", map(_DTYPES.__getitem__, map(_dtype_of, tensors)))))
    except (TypeError, KeyError):
        pass
    for j, t in enumerate(tensors):                          # something is refused: say which
        _check_dev(t, f"{name}[{j}]")
        _same_device(dev, (f"{name}[{j}]", t))
        _dtype(t.dtype, f"{name}[{j}]")
    raise ValueError(f"{name} must hold GPU tensors")


def grad_norm_clip(grads, max_norm: float, scale: float = 1.0, eps: float = 1e-6, out=None,
                   norm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Global norm N = |scale| * sqrt(sum of squares) of all the tensors
    (bf16 / fp16 / fp32, mixed, any shapes and alignments), and every tensor
    times scale * min(1, max_norm / (N + eps)): in place, or into the tensors
    of `out` (same sizes, any of the types).  Returns N, one fp32 value on the
    GPU; nothing waits for it.  See rc_grad_norm_clip."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if not grads:
        raise ValueError("need at least one tensor")
    if len(outs) != len(grads):
        raise ValueError("out must hold one tensor for each of grads")
    _check_dev(grads[0], "grads[0]")
    dev = grads[0].device
    desc = array.array("Q", bytes(32 * len(grads)))          # rc_grad: in, out, n, and in_t, out_t as halves
    ptrs, numels, types = _tensors(grads, dev, "grads")
    desc[0::4], desc[2::4] = ptrs, numels
    if outs is grads:
        desc[1::4], out_types = ptrs, types
    else:
        desc[1::4], out_numels, out_types = _tensors(outs, dev, "out")
        if out_numels != numels:
            raise ValueError("each tensor of out must hold as many values as its gradient")
    halves = memoryview(desc).cast("B").cast("I")
    halves[6::8], halves[7::8] = types, out_types
    norm = _result(norm, (1,), torch.float32, dev, stream, "norm")
    ws = _result(None, ((_lib or lib()).rc_grad_norm_clip_workspace(),), torch.uint8, dev, stream, "")
    _launch("rc_grad_norm_clip", dev, stream, desc.buffer_info()[0], len(grads), scale, max_norm, eps, ws.data_ptr(),
            norm.data_ptr())
    return norm


# ------------------------------------------------- a paged cache in MXFP4 ----

def mxfp4_cache_new(pages: int, kv_heads: int, page: int, d: int, device):
    """(k_cache, v_cache) with room for `pages` pages of `page` tokens, all
    zeros: uint8 tensors pages x kv_heads x bytes, where the last dimension is
    the packed stream {MXFP4, E8M0, 32} of one head's page * d values."""
    if d not in (64, 96, 128, 192, 256) or not 16 <= page <= 65536 or page & (page - 1):
        raise ValueError("d must be 64, 96, 128, 192 or 256, and page a power of two from 16 to 65536")
    if page * d % TILE != 0:
        raise ValueError("page * d must be a multiple of 2048")
    if pages < 0 or kv_heads < 1:
        raise ValueError("pages must not be negative, and kv_heads at least 1")
    shape = (pages, kv_heads, page * d // TILE * MXFP4_TILE_BYTES)
    return torch.zeros(shape, dtype=torch.uint8, device=device), torch.zeros(shape, dtype=torch.uint8, device=device)


def _cache(k_cache, v_cache, table, lengths, offsets, d: int, page: int | None) -> array.array:
    """rc_cache of checked tensors, as its eleven 64-bit words.  The bytes of a
    page tell page * d alone, so a d that is not the cache's is seen only
    beside the page that the caller names."""
    _check_dev(k_cache, "k_cache")
    index = k_cache.get_device()
    for name, t in (("v_cache", v_cache), ("table", table), ("lengths", lengths), ("offsets", offsets)):
        _check_on(t, name, index)
    shape = k_cache.shape
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or len(shape) != 3 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be uint8 tensors of one shape, pages x kv_heads x bytes")
    if d <= 0 or shape[2] % MXFP4_TILE_BYTES or shape[2] // MXFP4_TILE_BYTES * TILE % d:
        raise ValueError("a page of one head must be whole MXFP4 tiles of whole rows of d values")
    if table.dtype != torch.int32 or lengths.dtype != torch.int32 or offsets.dtype != torch.int32:
        raise ValueError("table, lengths and offsets must be int32 tensors")
    seqs = lengths.numel()
    if lengths.dim() != 1 or offsets.dim() != 1 or offsets.numel() != seqs + 1 or table.dim() != 2 or \
            table.shape[0] != seqs:
        raise ValueError("need table (sequences x pages), lengths (sequences) and offsets (sequences + 1)")
    tokens = shape[2] // MXFP4_TILE_BYTES * TILE // d
    if page is not None and page != tokens:
        raise ValueError(f"a page of the cache holds {tokens} tokens of {d} values, not {page}")
    return array.array("Q", (k_cache.data_ptr(), v_cache.data_ptr(), shape[0], tokens, shape[1], d,
                             table.data_ptr(), seqs, table.shape[1], lengths.data_ptr(), offsets.data_ptr()))


def _head_rows(t: torch.Tensor, name: str, index: int):
    """(tokens, heads, d, elements from a token to the next) of a tensor whose
    tokens' rows are dense; tokens may lie apart, as parts of a wider tensor do."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions, tokens, heads and values")
    tokens, heads, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and heads > 1):
        raise ValueError(f"the heads of a token of {name} must lie one after another")
    return tokens, heads, d, s0 if tokens > 1 else heads * d


def mxfp4_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       table: torch.Tensor, lengths: torch.Tensor, offsets: torch.Tensor,
                       q: torch.Tensor | None = None, rotation: torch.Tensor | None = None,
                       interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None, page: int | None = None):
    """Write new tokens' keys and values (tokens x kv_heads x d) to the cache,
    keys turned by their positions, and return the queries (tokens x heads x d)
    turned alike, or None without q.  Rows offsets[s] to offsets[s + 1] are the
    last tokens of sequence s, which has lengths[s] with them; token j of it is
    in page table[s, j // page].  rotation: fp32, at least table.shape[1] * page
    rows of the cosines, then the sines of a position's angles:

        angle = position[:, None] * base ** (-torch.arange(r // 2) / (r // 2))  # in float64
        rotation = torch.cat([angle.cos(), angle.sin()], 1).float()             # positions x r

    turning pairs (i, i + r/2) of the first r values of a head, or (2i, 2i + 1)
    if `interleaved`.  k, v and q may be parts of one wider tensor.  page: the
    tokens of a page, if given checked against the cache and k's width (another
    width would otherwise be taken for other pages).  See rc_mxfp4_cache_append."""
    _check_dev(k_cache, "k_cache")
    dev, index = k_cache.device, k_cache.get_device()
    tokens, kv_heads, d, k_stride = _head_rows(k, "k", index)
    vt, vh, vd, v_stride = _head_rows(v, "v", index)
    cache = _cache(k_cache, v_cache, table, lengths, offsets, d, page)
    if (vt, vh, vd) != (tokens, kv_heads, d) or v.dtype != k.dtype or kv_heads != k_cache.shape[1]:
        raise ValueError("k and v must have one shape and dtype, and the cache's heads")
    t, heads, q_stride, positions, rot = _dtype(k.dtype, "k"), 0, 0, 0, 0
    if rotation is not None:
        _check_on(rotation, "rotation", index)
        if rotation.dtype != torch.float32 or rotation.dim() != 2:
            raise ValueError("rotation must be a float32 tensor, positions x values")
        positions, rot = rotation.shape
    if q is not None:
        qt, heads, qd, q_stride = _head_rows(q, "q", index)
        if (qt, qd) != (tokens, d) or q.dtype != k.dtype:
            raise ValueError("q must have k's tokens, width and dtype")
        q_out = _result(q_out, (tokens, heads, d), q.dtype, dev, stream, "q_out")
    _launch("rc_mxfp4_cache_append", dev, stream, cache.buffer_info()[0], t, tokens, k.data_ptr(), k_stride,
            v.data_ptr(), v_stride, heads, _ptr(q), q_stride, None if q is None else q_out.data_ptr(),
            _ptr(rotation), positions, rot, int(interleaved))
    return None if q is None else q_out


def mxfp4_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                     offsets: torch.Tensor, tokens: int, d: int, dtype: torch.dtype = torch.bfloat16,
                     k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None, page: int | None = None):
    """(k, v), tokens x kv_heads x d each: the rows' keys and values as the
    cache holds them, decoded; rows offsets[s] to offsets[s + 1] are the last
    tokens of sequence s (all of them if offsets are the lengths' sums).  page:
    as above.  See rc_mxfp4_cache_read."""
    cache = _cache(k_cache, v_cache, table, lengths, offsets, d, page)
    dev = k_cache.device
    t, shape = _dtype(dtype, "output"), (tokens, k_cache.shape[1], d)
    k, v = _result(k, shape, dtype, dev, stream, "k"), _result(v, shape, dtype, dev, stream, "v")
    _launch("rc_mxfp4_cache_read", dev, stream, cache.buffer_info()[0], tokens, t, k.data_ptr(), v.data_ptr())
    return k, v


def mxfp4_cache_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                          lengths: torch.Tensor, offsets: torch.Tensor, scale: float | None = None,
                          causal: bool = True, window: int = 0, max_query: int | None = None, lse: bool = False,
                          out: torch.Tensor | None = None, stream=None, page: int | None = None):
    """Attention of the queries (tokens x heads x d, heads a multiple of the
    cache's) over their sequences' tokens in the cache, the new ones included:
    rows offsets[s] to offsets[s + 1] stand at the last positions of sequence
    s, and see what is at or before them (`causal`), the last `window` of that
    if window > 0.  scale: 1 / sqrt(d) by default.  max_query: the most rows a
    sequence has, if known (it only helps to choose the kernel).  page: as above.  Returns out
    (like q, dense; out=q if q is), or (out, the fp32 log-sum-exp of tokens x heads).  See
    rc_mxfp4_cache_attention."""
    _check_dev(k_cache, "k_cache")
    dev = k_cache.device
    tokens, heads, d, q_stride = _head_rows(q, "q", k_cache.get_device())
    cache = _cache(k_cache, v_cache, table, lengths, offsets, d, page)
    if window < 0 or (max_query is not None and max_query < 0):
        raise ValueError("window and max_query must not be negative")
    t = _dtype(q.dtype, "q")
    out = _result(out, (tokens, heads, d), q.dtype, dev, stream, "out")
    sums = _result(None, (tokens, heads), torch.float32, dev, stream, "") if lse else None
    ws = _result(None, ((_lib or lib()).rc_mxfp4_cache_attention_workspace(tokens, heads, k_cache.shape[1], d),),
                 torch.uint8, dev, stream, "")
    _launch("rc_mxfp4_cache_attention", dev, stream, cache.buffer_info()[0], t, tokens, heads, q.data_ptr(), q_stride,
            d ** -0.5 if scale is None else scale, int(causal), min(window, 1 << 32), max_query or 0, out.data_ptr(), _ptr(sums),
            ws.data_ptr())
    return (out, sums) if lse else out
