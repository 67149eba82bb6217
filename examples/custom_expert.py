"""A model whose experts are not the fused layer's, trained with clipped gradients and asked token by token.

    python examples/custom_expert.py [--steps 60]

Each block is: norm, router, GELU experts with a bias, weighted sum, residual add. The experts are built
from the operators of expert_ops: the selection's order by expert, the tokens' rows in that order, two
products grouped by expert, the weighted sum back. Between backward and optimizer the gradients of all
parameters are scaled down to a largest norm. The same forward serves one token. The task: the successor
of each token under a fixed permutation.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from moe_ffn_expert_gb300.block_ops import moe_router, residual_norm
from moe_ffn_expert_gb300.expert_ops import expert_combine, expert_dispatch, expert_table, grouped_mm
from moe_ffn_expert_gb300.grad_ops import clip_grad_norm


class Experts(torch.nn.Module):
    """E experts gelu(x W1 + b1) W2, k of them per token."""

    def __init__(self, H, I, E, k):
        super().__init__()
        p = torch.nn.Parameter
        self.k = k
        self.router = p(torch.randn(E, H) / H ** 0.5)
        self.w1 = p((torch.randn(E, H, I) / H ** 0.5).bfloat16())
        self.b1 = p(torch.zeros(E, I))
        self.w2 = p((torch.randn(E, I, H) / I ** 0.5).bfloat16())

    def forward(self, n):
        """n [T,H] bf16 -> ([T,H] bf16, the ids picked)."""
        ids, weights, *_ = moe_router(n.float() @ self.router.t(), self.k)
        table = expert_table(ids, self.router.shape[0])
        expert_of_row = ids.flatten()[table.slot_of_row]
        h = grouped_mm(expert_dispatch(n, table), self.w1, table.offsets, out_dtype=torch.float32)
        h = torch.nn.functional.gelu(h + self.b1[expert_of_row]).bfloat16()
        return expert_combine(grouped_mm(h, self.w2, table.offsets), table, weights), ids


class Model(torch.nn.Module):
    def __init__(self, vocab=256, H=512, I=1024, E=16, k=4, layers=2):
        super().__init__()
        self.embedding = torch.nn.Parameter(torch.randn(vocab, H))
        self.blocks = torch.nn.ModuleList(Experts(H, I, E, k) for _ in range(layers))
        self.norms = torch.nn.ParameterList(torch.ones(H) for _ in range(layers + 1))
        self.head = torch.nn.Parameter(torch.randn(vocab, H) / H ** 0.5)

    def forward(self, tokens):
        x = self.embedding[tokens]
        n = residual_norm(x, pre_weight=self.norms[0], normed_dtype=torch.bfloat16)[1]
        for block, weight in zip(self.blocks, list(self.norms)[1:]):
            x, n = residual_norm(x, block(n)[0], pre_weight=weight)
        return n.float() @ self.head.t()


def train(model, successor, steps, batch=1024, max_norm=1.0, seed=0):
    """(losses, gradient norms before clipping) of the steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=2e-3)
    losses, norms = [], []
    for _ in range(steps):
        tokens = torch.randint(len(successor), (batch,), generator=g, device="cuda")
        loss = torch.nn.functional.cross_entropy(model(tokens), successor[tokens])
        loss.backward()
        norms.append(clip_grad_norm([p.grad for p in model.parameters()], max_norm))
        opt.step()
        opt.zero_grad(set_to_none=True)
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args()
    torch.manual_seed(0)
    with torch.device("cuda"):
        model = Model()
        successor = torch.randperm(256)
    losses, norms = train(model, successor, args.steps)
    print("training loss: first %.3f, last %.3f; gradient norm: first %.2f, last %.2f"
          % (losses[0], losses[-1], norms[0], norms[-1]))
    tokens = torch.arange(64, device="cuda")
    with torch.no_grad():
        one = torch.cat([model(t[None]) for t in tokens])
        right = (one.argmax(1) == successor[tokens]).float().mean()
    print("asked one at a time: %.0f %% of 64 tokens right" % (100 * right))


if __name__ == "__main__":
    main()
