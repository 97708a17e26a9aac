"""A training step of a tensor-parallel expert block with quantized collectives.

K emulated ranks share one GPU.  Each holds a slice of every expert's MXFP4
weights; a step runs

    partial products of the experts   mxfp4_grouped_matmul       (each rank)
    all-reduce of the partial sums    allreduce_emulate          (INT4 payload)
    post norm, gate, residual, norm   block_norm
    their gradients                   block_norm_backward
    the weights' gradients            grouped_matmul_dw          (each rank)
    the rows' gradients               mxfp4_grouped_matmul_dx    (each rank)
    global norm and clipping          grad_norm_clip

and updates FP32 master weights, which are cast to MXFP4 again for the next
one (the cast is passed straight through, the all-reduce's rounding too).

    python examples/expert_block.py [--steps 20] [--rows 512] [--ranks 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduction_codec_amd as rca  # noqa: E402


def sort_by_expert(expert: torch.Tensor, experts: int):
    """(order of the rows, offsets of the experts' groups)."""
    counts = torch.bincount(expert, minlength=experts)
    return expert.argsort(stable=True), torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


class ExpertBlock:
    """experts x (width x hidden) weights, the hidden dimension split over the ranks."""

    def __init__(self, experts, width, hidden, ranks, device, generator):
        randn = lambda *s: torch.randn(*s, device=device, generator=generator)  # noqa: E731
        self.width, self.ranks = width, ranks
        self.master = [randn(experts, width, hidden // ranks) * hidden ** -0.5 for _ in range(ranks)]
        self.post = torch.ones(width, device=device)
        self.pre = torch.ones(width, device=device)
        self.gate = torch.full((width,), 0.5, device=device)

    def parameters(self):
        return self.master + [self.pre, self.post, self.gate]

    def forward(self, x, residual, offsets):
        """x: one slice of the hidden rows for each rank, sorted by expert."""
        self.packed = [rca.quantize_pack(w, rca.MXFP4) for w in self.master]
        partial = [rca.mxfp4_grouped_matmul(x[r], self.packed[r], offsets, self.width) for r in range(self.ranks)]
        y = rca.allreduce_emulate(partial, rca.INT4)[0].view_as(residual)
        h, z, stats = rca.block_norm(y, residual, self.pre, post_weight=self.post, gate=self.gate, stats=True)
        self.saved = x, offsets, y, h, stats
        return h, z

    def backward(self, dz):
        """(gradients in the order of parameters(), gradients of x)."""
        x, offsets, y, h, stats = self.saved
        dy, _, dpre, dpost, dgate = rca.block_norm_backward(dz, None, h, stats, y, self.pre, post_weight=self.post,
                                                            gate=self.gate)
        dw = [rca.grouped_matmul_dw(dy, x[r], offsets) for r in range(self.ranks)]
        dx = [rca.mxfp4_grouped_matmul_dx(dy, self.packed[r], offsets, x[r].shape[1]) for r in range(self.ranks)]
        return dw + [dpre, dpost, dgate], dx


def train(steps=20, rows=512, ranks=2, experts=8, width=512, hidden=1024, lr=2.0, max_norm=1.0, device="cuda:0", log=print):
    """Fits the block to another one's outputs; the losses of the steps."""
    g = torch.Generator(device=device).manual_seed(1)
    block = ExpertBlock(experts, width, hidden, ranks, device, g)
    goal = ExpertBlock(experts, width, hidden, ranks, device, g)
    x = torch.randn(rows, hidden, device=device, generator=g)
    order, offsets = sort_by_expert(torch.randint(0, experts, (rows,), device=device, generator=g), experts)
    x = [s.contiguous().to(torch.bfloat16) for s in x[order].chunk(ranks, 1)]
    residual = torch.randn(rows, width, device=device, generator=g).to(torch.bfloat16)
    _, target = goal.forward(x, residual, offsets)
    losses = []
    for step in range(steps):
        _, z = block.forward(x, residual, offsets)
        off = z.float() - target.float()
        losses.append(float(off.square().mean()))
        grads, _ = block.backward((off * (2.0 / rows)).to(torch.bfloat16))
        norm = rca.grad_norm_clip(grads, max_norm)
        for p, d in zip(block.parameters(), grads):
            p.sub_(d, alpha=lr)
        log(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.3f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--ranks", type=int, default=2)
    args = ap.parse_args()
    train(args.steps, args.rows, args.ranks)
