"""Where the binding takes memory from for work on a caller's stream: from that
stream's pool (a block that the current stream freed may still be in use by
work queued there), told to the current stream, which goes on with it.  On the
CPU torch's stream calls and the library are replaced by recorders."""
import array
import contextlib

import pytest
import torch

import reduction_codec_amd as rca

CPU = torch.device("cpu")


class Stream:
    def __init__(self, device=CPU):
        self.device, self.cuda_stream = device, 0


class Library:
    """Every entry point succeeds; sizes come from the library itself."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        real = getattr(self.real, name)
        return real if name.endswith(("bytes", "workspace")) else lambda *args: rca.OK


@pytest.fixture
def streams(monkeypatch):
    """(the current stream, another one, allocations: each (pool, streams told))."""
    current, side = Stream(), Stream()
    inside, made, told = [current], [], {}
    real_empty, library = torch.empty, Library(rca.lib())

    @contextlib.contextmanager
    def use(stream):
        inside.append(stream)
        yield
        inside.pop()

    def empty(*args, **kw):
        t = real_empty(*args, **kw)
        made.append((t, inside[-1]))
        return t

    for target, name, value in (
            (torch.cuda, "current_stream", lambda device=None: inside[-1]), (torch.cuda, "stream", use),
            (torch.cuda, "device", lambda device: contextlib.nullcontext()), (torch.cuda, "current_device", lambda: None),
            (torch, "empty", empty), (rca, "lib", lambda: library), (rca, "_lib", library),
            (rca, "_check_dev", lambda *a: None), (rca, "_check_on", lambda *a: None),
            (rca, "_tensors", lambda ts, dev, name: (array.array("Q", [0] * len(ts)), array.array("Q", [t.numel() for t in ts]),
                                                     memoryview(array.array("I", [1] * len(ts)))))):
        monkeypatch.setattr(target, name, value)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.setdefault(id(t), []).append(s), raising=False)
    return current, side, lambda: [(pool, told.get(id(t), [])) for t, pool in made]


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


ROWS, N, K = 4, 64, 64
OFF = torch.tensor([0, 2, 4], dtype=torch.int32)
CALLS = {
    "quantize_pack": lambda s: rca.quantize_pack(zeros(2048), rca.INT3, stream=s),
    "unpack_dequant": lambda s: rca.unpack_dequant(zeros(896, dtype=torch.uint8), rca.INT3, 2048, stream=s),
    "dequant_reduce_requant": lambda s: rca.dequant_reduce_requant([zeros(896, dtype=torch.uint8)], rca.INT3, 2048,
                                                                   sum_out=True, stream=s),
    "allreduce_emulate": lambda s: rca.allreduce_emulate([zeros(2048)], rca.INT3, packed_out=True, stream=s),
    "mxfp4_gemv": lambda s: rca.mxfp4_gemv(zeros(1088, dtype=torch.uint8), 1, 2048, zeros(2048), stream=s),
    "mxfp4_grouped_matmul": lambda s: rca.mxfp4_grouped_matmul(zeros(ROWS, K), zeros(4 * 1088, dtype=torch.uint8), OFF, N,
                                                               stream=s),
    "mxfp4_grouped_matmul_dx": lambda s: rca.mxfp4_grouped_matmul_dx(zeros(ROWS, N), zeros(4 * 1088, dtype=torch.uint8), OFF,
                                                                     K, stream=s),
    "grouped_matmul_dw": lambda s: rca.grouped_matmul_dw(zeros(ROWS, N), zeros(ROWS, K), OFF, stream=s),
    "block_norm": lambda s: rca.block_norm(zeros(ROWS, N), zeros(ROWS, N), zeros(N), stats=True, stream=s),
    "block_norm_backward": lambda s: rca.block_norm_backward(
        zeros(ROWS, N), None, zeros(ROWS, N), zeros(2, ROWS, dtype=torch.float32), zeros(ROWS, N), zeros(N),
        post_weight=zeros(N), gate=zeros(N), stream=s),
    "grad_norm_clip": lambda s: rca.grad_norm_clip([zeros(8)], 1.0, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(name, streams):
    current, side, made = streams
    CALLS[name](side)
    assert made() and all(pool is side and told == [current] for pool, told in made()), made()


@pytest.mark.parametrize("name", CALLS)
def test_without_another_stream_nothing_is_told(name, streams):
    current, side, made = streams
    CALLS[name](None)
    first = len(made())
    CALLS[name](current)
    assert len(made()) == 2 * first > 0 and all(pool is current and not told for pool, told in made())


@pytest.mark.parametrize("name", CALLS)
def test_another_devices_stream_is_refused_before_anything_is_allocated(name, streams):
    _, _, made = streams
    with pytest.raises(ValueError, match="stream is on"):
        CALLS[name](Stream(torch.device("meta")))
    assert not made()


@pytest.mark.gpu
def test_blocks_freed_by_queued_work_are_left_alone():
    """While the current stream still has work queued on blocks that it freed, an operator on another stream takes none
    of them."""
    dev = torch.device("cuda:0")
    rows, d = 4096, 1024
    y, r = (torch.randn(rows, d, device=dev).to(torch.bfloat16) for _ in range(2))
    pre = torch.ones(d, device=dev, dtype=torch.bfloat16)
    want = [t.clone() for t in rca.block_norm(y, r, pre, stats=True)]
    side = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device=dev)
    sink = torch.zeros(rows, d, dtype=torch.bfloat16, device=dev)
    used = set()
    for _ in range(20):                                    # a queue of products, then writes to blocks of the outputs' size
        a = a @ a * 1e-3
    for _ in range(4):
        blocks = [torch.empty(rows, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        for b in blocks:
            b.fill_(3.0)
            sink += b
            used.add(b.data_ptr())
        del b, blocks
    got = rca.block_norm(y, r, pre, stats=True, stream=side)
    assert not used & {t.data_ptr() for t in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    assert (sink == 24.0).all()


@pytest.mark.gpu
def test_another_stream_inside_a_captured_graph():
    """A graph that forks to a second stream, whose outputs come from that stream's memory: replays with new inputs, with
    eager work on freed blocks in between, equal the eager results."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    y, r, pre = rn(300, 520), rn(300, 520), rn(520)

    def run(stream):
        h, z, st = rca.block_norm(y, r, pre, post_weight=pre, stats=True, stream=stream)
        return [h, z, *rca.block_norm_backward(z, h, h, st, y, pre, post_weight=pre, stream=stream)[:4]]

    main, side = torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev)
    run(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        first = run(side)
        second = run(None)                                 # on the capturing stream, beside the other
        main.wait_stream(side)
    for _ in range(4):
        y.copy_(rn(300, 520))
        r.copy_(rn(300, 520))
        graph.replay()
        torch.cuda.synchronize()
        want = run(None)
        for got in (first, second):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
