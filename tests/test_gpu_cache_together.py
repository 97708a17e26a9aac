"""The paged MXFP4 cache as it is used: written and read in turn, captured into
graphs that are replayed with new inputs and lengths, on side streams, from
several host threads, and in a serving step beside the codec's operators."""
import threading

import pytest
import torch

import reduction_codec_amd as rca
from examples import serving_block
from tests import cache_reference as ref
from tests.test_gpu_cache_attention import compare

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HEADS, KV, D, PAGE = 8, 2, 128, 16


def rotation(positions):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2).double() / (D // 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def state(spec, seed, max_pages=80):
    """What a step of sequences (new, length) reads and writes: places are the same whatever the seed."""
    plan = ref.Plan(spec, PAGE, seed=seed)
    plan.table = [r + [-1] * (max_pages - len(r)) for r in plan.table]
    plan.max_pages = max_pages
    g = torch.Generator().manual_seed(seed)
    pages = 200
    cache = [torch.randint(0, 256, (pages, KV, PAGE * D // 2048, 1088), generator=g, dtype=torch.uint8) for _ in range(2)]
    for c in cache:
        c[..., 1024:] = c[..., 1024:] % 3 + 125
    rows = torch.randn(plan.tokens, HEADS + 2 * KV, D, generator=g).to(torch.bfloat16)
    table, lengths, offsets = plan.tensors(DEV)
    return {"k_cache": cache[0].view(pages, KV, -1).to(DEV), "v_cache": cache[1].view(pages, KV, -1).to(DEV),
            "table": table, "lengths": lengths, "offsets": offsets, "rows": rows.to(DEV),
            "rotation": rotation(max_pages * PAGE).to(DEV)}


def everything(s, most=None, stream=None):
    q, k, v = s["rows"].split([HEADS, KV, KV], 1)
    place = s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"]
    q = rca.mxfp4_cache_append(k, v, *place, q=q, rotation=s["rotation"], stream=stream)
    out, lse = rca.mxfp4_cache_attention(q, *place, max_query=most, lse=True, stream=stream)
    k, v = rca.mxfp4_cache_read(*place, s["rows"].shape[0], D, stream=stream)
    return [q, out, lse, k, v]


def results(s, **kw):
    return everything(s, **kw) + [s["k_cache"], s["v_cache"]]


def copy(s):
    return {k: v.clone() for k, v in s.items()}


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


ONE = [(1, 300), (1, 17), (1, 1), (1, 999), (1, 64)]
MIXED = [(1, 300), (40, 40), (3, 500), (0, 9), (129, 700), (1, 1)]
SPECS = {"one": (ONE, 1), "mixed": (MIXED, None), "chunk": ([(257, 900)], 257)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_prompt_in_chunks_and_then_token_by_token(dtype):
    """The cache is the same byte by byte however its tokens come, and so is what each row sees of it."""
    total, cuts = 150, [0, 70, 71, 120, 147, 148, 149, 150]
    plan = ref.Plan([(total, total), (total, total)], PAGE, seed=3)
    table, _, _ = plan.tensors(DEV)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2, total, HEADS + 2 * KV, D, generator=g).to(dtype).to(DEV)
    turn = rotation(plan.max_pages * PAGE).to(DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    outs = []
    for steps in ([0, total], cuts):
        kc, vc = rca.mxfp4_cache_new(plan.pages, KV, PAGE, D, DEV)
        out, sums, turned = [], [], []
        for a, b in zip(steps, steps[1:]):
            n = b - a
            place = kc, vc, table, i32([b, b]), i32([0, n, 2 * n])
            q, k, v = x[:, a:b].reshape(2 * n, -1, D).split([HEADS, KV, KV], 1)
            q = rca.mxfp4_cache_append(k, v, *place, q=q, rotation=turn)
            o, lse = rca.mxfp4_cache_attention(q, *place, lse=True)
            for all_, part in ((out, o), (sums, lse), (turned, q)):
                all_.append(part.view(2, n, HEADS, -1))
        outs.append([kc, vc] + [torch.cat(p, 1).reshape(2 * total, HEADS, -1) for p in (turned, out, sums)])
    whole, parts = outs
    assert torch.equal(whole[0], parts[0]) and torch.equal(whole[1], parts[1]) and torch.equal(whole[2], parts[2])
    kv, vv = (ref.values(c).view(plan.pages, KV, PAGE, D) for c in whole[:2])
    want = ref.attention(plan, whole[2].cpu(), kv, vv, D ** -0.5)
    for o in outs:
        compare(plan, o[3].cpu(), o[4].squeeze(-1).cpu(), want, dtype)


@pytest.mark.parametrize("spec", SPECS)
def test_side_stream(spec):
    spec, most = SPECS[spec]
    s = state(spec, 1)
    want = results(copy(s), most=most)
    mine, other = copy(s), copy(s)
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = results(mine, most=most, stream=side)
    side.synchronize()
    assert same(got, want)
    with torch.cuda.stream(side):
        got = results(other, most=most)
    side.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("spec", SPECS)
def test_captured_and_replayed_with_new_inputs_and_lengths(spec):
    spec, most = SPECS[spec]
    s = state(spec, 1)
    everything(copy(s), most=most)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = results(s, most=most)
    for seed in (2, 3, 1, 4, 2):
        new = state([(a, n + 31 * seed if n > 1 else n) for a, n in spec], seed)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, results(new, most=most)), seed
        torch.cuda.synchronize()


def test_two_graphs_of_one_pool_in_turn():
    """Their workspaces may be the same memory: they run one after another on one stream."""
    a, b = state(ONE, 1), state(MIXED, 2)
    everything(copy(a)), everything(copy(b))
    torch.cuda.synchronize()
    graphs, got, pool = [], [], None
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            got.append([t.clone() for t in results(s)])
        pool = graph.pool()
        graphs.append(graph)
    want = [results(copy(s)) for s in (a, b)]
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same(got[i], want[i]), i


def test_host_threads_on_their_own_streams():
    states = [state(s, i + 1) for i, s in enumerate((ONE, MIXED, SPECS["chunk"][0], MIXED))]
    want = [[t.clone() for t in results(s)] for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream(device=DEV)
        for _ in range(5):
            with torch.cuda.stream(stream):
                got = results(states[i])
            stream.synchronize()
            if not same(got, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_serving_block_example_runs():
    steps, prompts = 3, (70, 1, 33, 130)
    out = serving_block.serve(steps=steps, prompts=prompts, ranks=2, width=256, heads=4, kv_heads=2, d=64, page=32,
                              log=lambda s: None)
    assert [h.shape[0] for h, _ in out] == [sum(prompts)] + [len(prompts)] * steps
    assert all(torch.isfinite(t.float()).all() for pair in out for t in pair)
