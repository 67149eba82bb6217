"""What clip_grad_norm refuses of tensors that are not dense, before anything is launched or changed: host
logic only, with a library that notes whether it was called."""
import pytest
import torch

from moe_ffn_expert_gb300 import _abi, grad_ops


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def mm_grad_workspace_size(self, n):
            return 256

        def mm_grad_clip(self, *_):
            made.append("mm_grad_clip")
            return 0

    real = torch.empty
    monkeypatch.setattr(_abi, "_lib", lambda: Library())
    monkeypatch.setattr(grad_ops, "_elsewhere", lambda _: False)
    monkeypatch.setattr(grad_ops, "_stream", lambda _: 0)
    monkeypatch.setattr(grad_ops, "_device", lambda op, first: torch.device("cuda", 0))
    monkeypatch.setattr(grad_ops._T, "get_device", lambda t: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))
    return made


def gaps(n=6):
    return torch.arange(2.0 * n).view(n, 2)[:, 0]


def test_the_call_is_reached(calls):
    a, b = torch.ones(5), gaps()
    grad_ops.clip_grad_norm([a, b], 1.0)
    grad_ops.clip_grad_norm([a, b], 1.0, out=[torch.ones(5), gaps()])
    grad_ops.clip_grad_norm([a, b], 1.0, out=[a, b])
    both = torch.zeros(6, 2)
    grad_ops.clip_grad_norm([both[:, 0], both[:, 1]], 1.0)
    grad_ops.clip_grad_norm([both[:, :0], both[:, :0], a], 1.0)
    assert len(calls) == 5


def test_a_tensor_given_twice(calls):
    a, b, c = torch.ones(6), gaps(), gaps()
    wide = torch.zeros(4, 10)
    for src, out in (([b, b], None), ([a, b, b], None), ([wide[:, ::2], wide[:, ::2]], None), ([wide[:, :3], wide], None),
                     ([a, a, b], None), ([a, c], [b, b]), ([b, c], [a, a]), ([b, c], [c, a]), ([a, b], [b, c])):
        with pytest.raises(ValueError, match="twice"):
            grad_ops.clip_grad_norm(src, 1.0, out=out)
    assert not calls


def test_an_expanded_tensor_is_not_written_to(calls):
    """Refused before the others are scaled."""
    a, one = torch.ones(4, 5), torch.ones(5)
    for src, out in (([a, one.expand(4, 5)], None), ([a, torch.ones(()).expand(7)], None), ([a], [one.expand(4, 5)]),
                     ([a, torch.ones(4, 1).expand(4, 5)[:, 1:]], None)):
        with pytest.raises(ValueError, match="several places"):
            grad_ops.clip_grad_norm(src, 1.0, out=out)
    assert not calls
    grad_ops.clip_grad_norm([one.expand(4, 5)], 1.0, out=[a])  # read, it is a tensor as any other
    grad_ops.clip_grad_norm([one[:0].expand(4, 0)], 1.0)
    assert len(calls) == 2
