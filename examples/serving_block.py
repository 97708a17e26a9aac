"""An attention block of a tensor-parallel model that answers with its keys and
values held in MXFP4.

K emulated ranks share one GPU.  Each holds a slice of the heads, its weights in
MXFP4 and a paged cache of its heads' keys and values; a step runs

    queries, keys and values          mxfp4_grouped_matmul     (each rank)
    keys and values to the cache      mxfp4_cache_append       (each rank)
    attention over the cache          mxfp4_cache_attention    (each rank)
    partial sums of the output        mxfp4_grouped_matmul     (each rank)
    all-reduce of the partial sums    allreduce_emulate        (INT4 payload)
    residual, norm                    block_norm

A batch's prompts go through it first, all rows at once; then it is captured
into a graph whose replays take one row of every sequence.

    python examples/serving_block.py [--steps 32] [--prompts 700 64 1500 200] [--ranks 2]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduction_codec_amd as rca  # noqa: E402


class Rank:
    """heads and kv_heads of width d, weights and cache of one rank."""

    def __init__(self, width, heads, kv_heads, d, pages, page, device, generator):
        self.heads, self.kv_heads, self.d, self.page = heads, kv_heads, d, page
        self.all = heads + 2 * kv_heads
        weights = lambda n, k: rca.quantize_pack(  # noqa: E731
            (torch.randn(n, k, device=device, generator=generator) * k ** -0.5).to(torch.bfloat16), rca.MXFP4)
        self.qkv, self.out = weights(self.all * d, width), weights(width, heads * d)
        self.k_cache, self.v_cache = rca.mxfp4_cache_new(pages, kv_heads, page, d, device)

    def forward(self, x, rotation, state, rows, most):
        qkv = rca.mxfp4_grouped_matmul(x, self.qkv, rows, self.all * self.d).view(-1, self.all, self.d)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        place = self.k_cache, self.v_cache, *state
        q = rca.mxfp4_cache_append(k, v, *place, q=q, rotation=rotation, page=self.page)
        y = rca.mxfp4_cache_attention(q, *place, max_query=most, page=self.page)
        return rca.mxfp4_grouped_matmul(y.view(y.shape[0], -1), self.out, rows, x.shape[1])


class Block:
    """A batch of sequences: their tables, lengths, and the block's ranks."""

    def __init__(self, width, heads, kv_heads, d, ranks, prompts, room, page, device, generator):
        each = -(-(max(prompts) + room) // page)
        pages = each * len(prompts)
        self.ranks = [Rank(width, heads // ranks, kv_heads // ranks, d, pages, page, device, generator)
                      for _ in range(ranks)]
        self.table = torch.randperm(pages, device=device, generator=generator).to(torch.int32).view(len(prompts), each)
        self.lengths = torch.zeros(len(prompts), dtype=torch.int32, device=device)
        self.norm = torch.ones(width, device=device)
        angle = torch.arange(each * page, device=device, dtype=torch.float64)[:, None]
        angle = angle * 10000.0 ** (-torch.arange(d // 2, device=device, dtype=torch.float64) / (d // 2))
        self.rotation = torch.cat([angle.cos(), angle.sin()], 1).float()

    def forward(self, x, residual, offsets, rows, most):
        """One step of rows offsets[s] to offsets[s + 1] of sequence s, whose lengths have grown by them."""
        state = self.table, self.lengths, offsets
        partial = [r.forward(x, self.rotation, state, rows, most) for r in self.ranks]
        y = rca.allreduce_emulate(partial, rca.INT4)[0].view_as(residual)
        return rca.block_norm(y, residual, self.norm)[:2]


def serve(steps=32, prompts=(700, 64, 1500, 200), ranks=2, width=1024, heads=16, kv_heads=4, d=64, page=64, seed=0, log=print):
    """Outputs of the prompts' rows and of every step's."""
    if ranks < 1 or heads % ranks or kv_heads % ranks:
        raise ValueError(f"{heads} heads on {kv_heads} of the cache cannot be shared by {ranks} ranks alike")
    if min(prompts, default=0) < 1:
        raise ValueError("every sequence needs a prompt of one token at least")
    device = torch.device("cuda:0")
    g = torch.Generator(device=device).manual_seed(seed)
    block = Block(width, heads, kv_heads, d, ranks, prompts, max(steps, 1), page, device, g)   # (the first call takes a row)
    randn = lambda n: torch.randn(n, width, device=device, generator=g).to(torch.bfloat16)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731

    new = i32(prompts)
    offsets = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
    block.lengths += new
    x = randn(sum(prompts))
    outputs = [block.forward(x, x, offsets, i32([0, sum(prompts)]), max(prompts))]
    log(f"prompts: {sum(prompts)} rows")

    count = len(prompts)
    x, offsets, rows = randn(count), torch.arange(count + 1, dtype=torch.int32, device=device), i32([0, count])
    block.lengths += 1                                     # a first call outside the capture, of tokens that the
    block.forward(x, x, offsets, rows, 1)                  # first step writes again
    block.lengths -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.lengths += 1
        h, z = block.forward(x, x, offsets, rows, 1)
    start = time.perf_counter()
    for _ in range(steps):
        graph.replay()
        outputs.append((h.clone(), z.clone()))
        x.copy_(z)                                         # stands for the layers in between and the next token
    torch.cuda.synchronize()
    log(f"steps: {(time.perf_counter() - start) / max(steps, 1) * 1e6:.0f} us each, "
        f"{block.lengths.tolist()} tokens in the cache")
    return outputs


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 1500, 200])
    p.add_argument("--ranks", type=int, default=2)
    a = p.parse_args()
    serve(a.steps, a.prompts, a.ranks)
