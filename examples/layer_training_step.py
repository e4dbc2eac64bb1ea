"""Training one sequence-parallel layer on the logical ranks of one GPU, then serving it a token.

    python examples/layer_training_step.py [--steps 20] [--world 4] [--rows 256] [--features 1024] [--outputs 1536]

Every rank owns `rows` rows of the input and `outputs / world` rows of the weight.  A step is what such a rank does:

    all_gather        the ranks' input rows, into every region of the symmetric heap
    linear            its columns of the layer on all rows: act(x w^T + b), the pre-activation kept
    linear_backward   dw and db of its shard, from the loss's gradient
    AdamW.step        its shard, with master weights and 8-bit states rounded stochastically

The target is another layer's output, so the loss has to fall.  Device memory and streams are torch's.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gemm_all_gather_amd import binding as ag  # noqa: E402

ACT = "gelu_tanh"


class Rank:
    """One logical rank: its input rows, its rows of the weight, and its optimizer."""

    def __init__(self, view, index, world, rows, features, outputs, gen):
        self.view, self.index = view, index
        self.M, self.N, self.K = world * rows, outputs // world, features
        dev = dict(device="cuda")
        self.input = torch.randn(rows, features, generator=gen, **dev).bfloat16()
        self.master = torch.randn(self.N, features, generator=gen, **dev) / features ** 0.5
        self.w = self.master.bfloat16()
        self.master_b, self.b = torch.zeros(self.N, **dev), torch.zeros(self.N, dtype=torch.bfloat16, **dev)
        self.dw, self.db = torch.zeros_like(self.w), torch.zeros_like(self.b)
        blocks = [-(-t.numel() // ag.AG_ADAMW_BLOCK) for t in (self.w, self.b)]
        zeros = lambda n, t: torch.zeros(n, dtype=t, **dev)  # noqa: E731
        self.optimizer = ag.AdamW(
            [self.w, self.b], [self.dw, self.db],
            [zeros(t.numel(), torch.int8) for t in (self.w, self.b)],
            [zeros(t.numel(), torch.uint8) for t in (self.w, self.b)],
            masters=[self.master, self.master_b],
            exp_avg_scales=[zeros(n, torch.float32) for n in blocks],
            exp_avg_sq_scales=[zeros(n, torch.float32) for n in blocks])
        self.y = torch.empty(self.M, self.N, dtype=torch.bfloat16, **dev)
        self.z, self.dy = torch.empty_like(self.y), torch.empty_like(self.y)
        self.target = None

    def x(self, offset):
        """Address of the gathered input in this rank's region."""
        return self.view.rank_ptr(self.index, offset)

    def layer(self, x, M, y, z, workspace, stream, w=None, b=None):
        ag.linear(x, self.w if w is None else w, y, M, self.N, self.K, "bf16", act=ACT,
                  bias=self.b if b is None else b, z=z, workspace=workspace, stream=stream)


def train(steps=20, world=4, rows=256, features=1024, outputs=1536, lr=3e-3, seed=0):
    """The loss of every step, and the served token's output with its expected one."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    nbytes = world * rows * features * 2
    region = ag.heap_region_bytes(nbytes + 4096)
    slab = torch.empty(world * region, dtype=torch.uint8, device="cuda")
    heap = ag.Heap.wrap(slab, world, region)
    offset = heap.alloc(nbytes)
    ranks = [Rank(heap.view(r), r, world, rows, features, outputs, gen) for r in range(world)]
    M, N, K = ranks[0].M, ranks[0].N, features
    x0 = ranks[0].x(offset)
    forward = ag.plan_linear(x0, ranks[0].w, ranks[0].y, M, N, K, "bf16", act=ACT, bias=ranks[0].b, z=ranks[0].z)
    grads = dict(act=ACT, z=ranks[0].z, dw=ranks[0].dw, db=ranks[0].db)
    backward = ag.plan_linear_backward(ranks[0].dy, x0, None, M, N, K, "bf16", **grads)
    need = max(1, forward.workspace_bytes, backward.workspace_bytes)
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")     # the ranks run on one stream: shared
    stream = torch.cuda.current_stream()

    def gather():
        for r in ranks:
            ag.all_gather(r.view, world, 0, 1, r.input, offset, rows, K, "bf16", stream=stream)

    gather()
    for r in ranks:     # what another layer of the same shape makes of the input
        w = (torch.randn(N, K, generator=gen, device="cuda") / K ** 0.5).bfloat16()
        b = torch.randn(N, generator=gen, device="cuda").mul_(0.1).bfloat16()
        r.layer(r.x(offset), M, r.y, None, workspace, stream, w, b)
        r.target = r.y.float()
    losses = []
    for step in range(1, steps + 1):
        gather()
        loss = 0.0
        for r in ranks:
            r.layer(r.x(offset), M, r.y, r.z, workspace, stream)
            err = r.y.float() - r.target
            loss = loss + err.square().mean() / world
            r.dy.copy_(err)
            ag.linear_backward(r.dy, r.x(offset), None, M, N, K, "bf16", act=ACT, z=r.z, dw=r.dw, db=r.db,
                               workspace=workspace, stream=stream)
            r.optimizer.step(step, lr, weight_decay=0.0, grad_scale=1.0 / M, seed=step, stream=stream)
        losses.append(float(loss))
    # one token through the trained layer: every rank's columns
    token = ranks[0].input[:1]
    out = torch.empty(world, 1, N, dtype=torch.bfloat16, device="cuda")
    for r in ranks:
        r.layer(token, 1, out[r.index], None, None, stream)
        r.layer(r.x(offset), M, r.y, None, workspace, stream)
    torch.cuda.synchronize()
    want = torch.stack([r.y[:1] for r in ranks])        # the token is the gathered input's first row
    for r in ranks:
        r.optimizer.destroy()
        r.view.destroy()
    heap.destroy()
    return losses, out.float().cpu(), want.float().cpu()


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--world", type=int, default=4)
    p.add_argument("--rows", type=int, default=256)
    p.add_argument("--features", type=int, default=1024)
    p.add_argument("--outputs", type=int, default=1536)
    a = p.parse_args()
    losses, out, want = train(a.steps, a.world, a.rows, a.features, a.outputs)
    for i, loss in enumerate(losses, 1):
        print(f"step {i:3d}  loss {loss:.5f}")
    print(f"one token: largest difference from the batch's row {float((out - want).abs().max()):.2g}")


if __name__ == "__main__":
    main()
