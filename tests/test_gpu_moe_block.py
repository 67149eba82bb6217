"""The example that trains and serves a model of MoE blocks with the block operators together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def new_model(example, seed=0):
    torch.manual_seed(seed)
    with torch.device("cuda"):
        return example.Model(vocab=64, H=256, I=128, E=8, k=2)


def plain(model, tokens, picks):
    """The model's training pass in 64 bits with the given experts; logits, balance, z and leaves."""
    leaf = {k: p.detach().double().requires_grad_(True) for k, p in model.named_parameters()}

    def norm(x, w):
        return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    L = len(model.blocks)
    x = leaf["embedding"][tokens]
    n, balance, z = norm(x, leaf["blocks.0.pre_weight"]), 0.0, 0.0
    for l in range(L):
        p = {k: leaf[f"blocks.{l}.{k}"] for k in ("post_weight", "gate", "router", "up", "down")}
        logits = n @ p["router"].t()
        ids = picks[l].long()
        w = torch.softmax(logits.gather(1, ids), 1)
        prob = torch.softmax(logits, 1)
        E = prob.shape[1]
        used = torch.bincount(ids.flatten(), minlength=E).double() / ids.numel()
        balance = balance + E * (used * prob.mean(0)).sum()
        z = z + torch.logsumexp(logits, 1).square().mean()
        f = torch.zeros_like(n)
        for e in range(E):
            t, k = (ids == e).nonzero(as_tuple=True)
            a, b = (n[t] @ p["up"][e]).chunk(2, 1)
            f = f.index_add(0, t, w[t, k][:, None] * ((a * torch.sigmoid(a) * b) @ p["down"][e]))
        x = x + p["gate"] * norm(f, p["post_weight"])
        n = norm(x, leaf[f"blocks.{l + 1}.pre_weight"] if l + 1 < L else leaf["last_weight"])
    return n @ leaf["head"].t(), balance, z, leaf


def test_a_step_against_plain_64_bits(example, monkeypatch):
    """bf16 activations (relative rounding 2^-9 each, a few per block, random) move a gradient by
    well under 2 % of its norm; the experts picked are the model's own, so that a tie cannot differ."""
    model = new_model(example)
    picks, route = [], example.moe_router
    monkeypatch.setattr(example, "moe_router",
                        lambda *a, **kw: (lambda r: (picks.append(r[0]), r)[1])(route(*a, **kw)))
    tokens = torch.randint(64, (300,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    target = (tokens * 5 + 3) % 64

    def total(logits, balance, z):
        return torch.nn.functional.cross_entropy(logits, target) + 0.3 * balance + 0.1 * z

    got = model(tokens)
    loss = total(*got)
    loss.backward()
    logits, balance, z, leaf = plain(model, tokens, picks)
    ref = total(logits, balance, z)
    ref.backward()
    loss, ref = float(loss.detach()), float(ref.detach())
    assert abs(loss - ref) <= 1e-2 * ref
    assert (got[0].double() - logits).norm() <= 2e-2 * logits.norm()
    for name, p in model.named_parameters():
        assert (p.grad.double() - leaf[name].grad).norm() <= 2e-2 * leaf[name].grad.norm(), name


def test_it_learns_and_serves_what_it_learned(example):
    model = new_model(example)
    successor = torch.randperm(64, generator=torch.Generator().manual_seed(2)).cuda()
    losses = example.train(model, successor, 60, batch=512)
    assert losses[-1] < 0.2 * losses[0]
    tokens = torch.arange(64, device="cuda")
    with torch.no_grad():
        full = model(tokens)[0]
    for e4m3 in (False, True):
        serve = example.Server(model, e4m3=e4m3)
        got = serve(tokens)
        # 8-bit weights: relative rounding of up to 2^-4 per weight, random over the sums
        assert (got - full).norm() <= (0.1 if e4m3 else 0.02) * full.norm()
        assert (got.argmax(1) == successor).float().mean() > 0.95
        assert all(layer.status() == 0 for layer in serve.layers)
