"""A small model of MoE blocks, trained and then served with the same weights.

    python examples/moe_block.py [--steps 60] [--e4m3]

Each block is: norm, router, the fused MoE-FFN layer, norm of its output, channel gate, residual
add. Two calls of residual_norm per model step more than there are blocks: the norm after one block
and the norm before the next are one pass over the stream. Training uses moe_router (with the
statistics for the balancing and z losses) and hyper_mega_moe; serving uses MoEDecoder, in bf16 or
with 8-bit expert weights. The task: the successor of each token under a fixed permutation.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from moe_ffn_expert_gb300.block_ops import (MoEDecoder, moe_router, quantize_expert_weights,
                                            residual_norm)
from moe_ffn_expert_gb300.torch_api import hyper_mega_moe


class MoEBlock(torch.nn.Module):
    def __init__(self, H, I, E, k):
        super().__init__()
        p = torch.nn.Parameter
        self.k = k
        self.pre_weight = p(torch.ones(H))     # of the norm before the block
        self.post_weight = p(torch.ones(H))    # of the norm of its output
        self.gate = p(torch.full((H,), 0.5))   # per channel
        self.router = p(torch.randn(E, H) / H ** 0.5)
        self.up = p((torch.randn(E, H, 2 * I) / H ** 0.5).bfloat16())
        self.down = p((torch.randn(E, I, H) / I ** 0.5).bfloat16())

    def forward(self, x, n, next_weight):
        """The stream after the block, that normed by next_weight, and the router's losses."""
        T, E = n.shape[0], self.router.shape[0]
        ids, weights, prob_sum, lse = moe_router(n.float() @ self.router.t(), self.k, stats=True)
        f = hyper_mega_moe(n, ids, weights, self.up, self.down)
        x, n = residual_norm(x, f, post_weight=self.post_weight, gate=self.gate,
                             pre_weight=next_weight)
        used = torch.bincount(ids.flatten(), minlength=E).float() / (T * self.k)
        balance = E * (used * prob_sum).sum() / T
        return x, n, balance, lse.square().mean()


class Model(torch.nn.Module):
    def __init__(self, vocab=256, H=512, I=256, E=16, k=4, layers=2):
        super().__init__()
        self.embedding = torch.nn.Parameter(torch.randn(vocab, H))
        self.blocks = torch.nn.ModuleList(MoEBlock(H, I, E, k) for _ in range(layers))
        self.last_weight = torch.nn.Parameter(torch.ones(H))
        self.head = torch.nn.Parameter(torch.randn(vocab, H) / H ** 0.5)

    def norm_weights(self):
        """Of the norm behind each block."""
        return [b.pre_weight for b in list(self.blocks)[1:]] + [self.last_weight]

    def forward(self, tokens):
        """Logits and the sums of the blocks' balancing and z losses."""
        x = self.embedding[tokens]
        n = residual_norm(x, pre_weight=self.blocks[0].pre_weight, normed_dtype=torch.bfloat16)[1]
        balance = z = 0.0
        for block, weight in zip(self.blocks, self.norm_weights()):
            x, n, b, s = block(x, n, weight)
            balance, z = balance + b, z + s
        return n.float() @ self.head.t(), balance, z


class Server:
    """The model for up to `max_tokens` tokens a call, without gradients."""

    def __init__(self, model, max_tokens=64, e4m3=False):
        self.model, self.layers = model, []
        for b in model.blocks:
            up, down = b.up.detach(), b.down.detach()
            us = ds = None
            if e4m3:
                (up, us), (down, ds) = quantize_expert_weights(up), quantize_expert_weights(down)
            self.layers.append(MoEDecoder(up, down, k=b.k, up_scale=us, down_scale=ds,
                                          router_weight=b.router.detach(), max_tokens=max_tokens))

    @torch.no_grad()
    def __call__(self, tokens):
        m = self.model
        x = m.embedding[tokens]
        n = residual_norm(x, pre_weight=m.blocks[0].pre_weight, normed_dtype=torch.bfloat16)[1]
        for block, layer, weight in zip(m.blocks, self.layers, m.norm_weights()):
            x, n = residual_norm(x, layer(n), post_weight=block.post_weight, gate=block.gate,
                                 pre_weight=weight)
        return n.float() @ m.head.t()


def train(model, successor, steps, batch=1024, seed=0):
    """The losses of the steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(len(successor), (batch,), generator=g, device="cuda")
        logits, balance, z = model(tokens)
        loss = torch.nn.functional.cross_entropy(logits, successor[tokens])
        (loss + 1e-2 * balance + 1e-3 * z).backward()
        opt.step()
        opt.zero_grad(set_to_none=True)
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--e4m3", action="store_true", help="serve with 8-bit expert weights")
    args = ap.parse_args()
    torch.manual_seed(0)
    with torch.device("cuda"):
        model = Model()
        successor = torch.randperm(256)
    losses = train(model, successor, args.steps)
    print("training loss: first %.3f, last %.3f" % (losses[0], losses[-1]))
    serve = Server(model, e4m3=args.e4m3)
    tokens = torch.arange(64, device="cuda")
    one = torch.cat([serve(t[None]) for t in tokens])
    many = serve(tokens)
    right = (many.argmax(1) == successor[tokens]).float().mean()
    print("served: %.0f %% of 64 tokens right; one at a time and together differ by at most %.3f"
          % (100 * right, (one - many).abs().max()))


if __name__ == "__main__":
    main()
