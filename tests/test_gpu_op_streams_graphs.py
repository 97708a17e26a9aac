"""The operators around the codec on a caller's stream, under HIP graph capture
(replayed with new inputs, against the eager results), from several host
threads, and together in the example."""
import threading

import pytest
import torch

import reduction_codec_amd as rca
from examples import expert_block
from tests import op_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E, N, K, ROWS = 3, 136, 160, 150


def state(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    packed, _ = ref.random_packed(E, N, K, seed)
    return {"x": rn(ROWS, K), "dy": rn(ROWS, N), "r": rn(ROWS, N), "w": packed.to(DEV), "pre": rn(N), "post": rn(N),
            "gate": rn(N), "off": torch.tensor([0, 40, 40 + 10 * seed, ROWS], dtype=torch.int32, device=DEV)}


def everything(s, stream=None):
    y = rca.mxfp4_grouped_matmul(s["x"], s["w"], s["off"], N, stream=stream)
    h, z, st = rca.block_norm(y, s["r"], s["pre"], post_weight=s["post"], gate=s["gate"], stats=True, stream=stream)
    dy, dr, dpre, dpost, dgate = rca.block_norm_backward(s["dy"], z, h, st, y, s["pre"], post_weight=s["post"],
                                                         gate=s["gate"], stream=stream)
    dx = rca.mxfp4_grouped_matmul_dx(dy, s["w"], s["off"], K, stream=stream)
    dw = rca.grouped_matmul_dw(dy, s["x"], s["off"], stream=stream)
    clipped = [torch.empty_like(t) for t in (dw, dpre, dpost, dgate)]
    norm = rca.grad_norm_clip([dw, dpre, dpost, dgate], 0.5, out=clipped, stream=stream)
    return [y, h, z, st, dy, dr, dx, dw, norm] + clipped


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_side_stream():
    s = state(1)
    want = everything(s)
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = everything(s, stream=side)                       # on `side`, while the current stream is another
    side.synchronize()
    assert same(got, want)
    with torch.cuda.stream(side):
        got = everything(s)
    side.synchronize()
    assert same(got, want)


def test_captured_and_replayed_with_new_inputs():
    s = state(1)
    everything(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(s)
    for seed in (2, 3, 1, 4, 2):
        new = state(seed)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, everything(new)), seed
        torch.cuda.synchronize()


def test_host_threads_on_their_own_streams():
    states = [state(i + 1) for i in range(4)]
    want = [everything(s) for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream(device=DEV)
        for _ in range(5):
            with torch.cuda.stream(stream):
                got = everything(states[i])
            stream.synchronize()
            if not same(got, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_expert_block_example_learns():
    losses = expert_block.train(steps=12, rows=200, ranks=2, experts=4, width=256, hidden=256, log=lambda s: None)
    assert all(x == x for x in losses) and losses[-1] < 0.8 * losses[0], losses
