"""The example whose experts are built from the operators of expert_ops, with clipped gradients."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "custom_expert.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("custom_expert", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def new_model(example, seed=0):
    torch.manual_seed(seed)
    with torch.device("cuda"):
        return example.Model(vocab=64, H=256, I=128, E=8, k=2)


def plain(model, tokens, picks):
    """The logits and leaves in 64 bits with the given experts."""
    leaf = {k: p.detach().double().requires_grad_(True) for k, p in model.named_parameters()}

    def norm(x, w):
        return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    x = leaf["embedding"][tokens]
    n = norm(x, leaf["norms.0"])
    for l, ids in enumerate(picks):
        p = {k: leaf[f"blocks.{l}.{k}"] for k in ("router", "w1", "b1", "w2")}
        w = torch.softmax((n @ p["router"].t()).gather(1, ids.long()), 1)
        f = torch.zeros_like(n)
        for e in range(p["b1"].shape[0]):
            t, k = (ids == e).nonzero(as_tuple=True)
            h = torch.nn.functional.gelu(n[t] @ p["w1"][e] + p["b1"][e])
            f = f.index_add(0, t, w[t, k][:, None] * (h @ p["w2"][e]))
        x = x + f
        n = norm(x, leaf[f"norms.{l + 1}"])
    return n @ leaf["head"].t(), leaf


def test_a_clipped_step_against_plain_64_bits(example, monkeypatch):
    """bf16 activations (relative rounding 2^-8 each, a few per block, random) move a gradient by well
    under 2 % of its norm; the experts picked are the model's own, so that a tie cannot differ."""
    model = new_model(example)
    picks, route = [], example.moe_router
    monkeypatch.setattr(example, "moe_router",
                        lambda *a, **kw: (lambda r: (picks.append(r[0]), r)[1])(route(*a, **kw)))
    tokens = torch.randint(64, (300,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    target = (tokens * 5 + 3) % 64
    logits = model(tokens)
    torch.nn.functional.cross_entropy(logits, target).backward()
    ref, leaf = plain(model, tokens, picks)
    torch.nn.functional.cross_entropy(ref, target).backward()
    assert (logits.double() - ref).norm() <= 2e-2 * ref.norm()
    for name, p in model.named_parameters():
        assert (p.grad.double() - leaf[name].grad).norm() <= 2e-2 * leaf[name].grad.norm(), name
    before = {k: p.grad.clone() for k, p in model.named_parameters()}
    total = math.sqrt(sum(float(g.double().square().sum()) for g in before.values()))
    norm = example.clip_grad_norm([p.grad for p in model.parameters()], total / 3)
    assert abs(float(norm) - total) <= 1e-6 * total
    for name, p in model.named_parameters():
        want = before[name].double() / 3
        assert ((p.grad.double() - want).abs() <= (torch.finfo(p.grad.dtype).eps / 2 + 2e-6) * want.abs() + 1e-40).all()


def test_it_runs_and_one_token_gives_what_many_do(example):
    model = new_model(example)
    successor = torch.randperm(64, generator=torch.Generator().manual_seed(2)).cuda()
    losses, norms = example.train(model, successor, 3, batch=128)
    assert all(math.isfinite(v) for v in losses + norms) and all(v > 0 for v in norms)
    tokens = torch.arange(64, device="cuda")
    with torch.no_grad():
        many = model(tokens)
        one = torch.cat([model(t[None]) for t in tokens])
    # the same numbers in other sums: a few bf16 roundings that may fall the other way
    assert (one - many).norm() <= 2e-2 * many.norm()
