"""The gradients come from kernels that autograd cannot see into: a derivative of them is refused,
not taken as zero. The kernels' calls are replaced by host stand-ins (f(x) = x^2, or w = z^2)."""
import pytest
import torch

from moe_ffn_expert_gb300 import block_ops, torch_api


def leaf(*shape):
    return torch.arange(1.0, 1.0 + torch.Size(shape).numel()).view(shape).requires_grad_(True)


def norm(monkeypatch, x):
    monkeypatch.setattr(block_ops, "residual_norm_forward", lambda r, *_, **__: (r.detach() ** 2, None))
    monkeypatch.setattr(block_ops, "residual_norm_backward",
                        lambda out, b, d, *_, **__: ((2 * out.detach().sqrt() * d.detach()), None, None, None, None))
    return block_ops.residual_norm(x)[0]


def router(monkeypatch, x):
    ids = torch.zeros(x.shape, dtype=torch.int32)
    monkeypatch.setattr(block_ops, "router_forward", lambda z, *_, **__: (ids, z.detach() ** 2, None, None))
    monkeypatch.setattr(block_ops, "router_backward", lambda z, i, d, *_, **__: 2 * z.detach() * d.detach())
    return block_ops.moe_router(x, 2)[1]


def layer(monkeypatch, x):
    class Space:
        def __init__(self, *_, **__):
            self.dims, self.buf = None, torch.empty(0)

        @classmethod
        def wrap(cls, *_):
            return cls()

    monkeypatch.setattr(torch_api, "Workspace", Space)
    monkeypatch.setattr(torch_api, "check_inputs", lambda *_: (1, 1, 1, 1, 1))
    monkeypatch.setattr(torch_api, "forward", lambda ws, x, *_, **__: x.detach() ** 2)
    monkeypatch.setattr(torch_api, "backward",
                        lambda ws, dy, x, *_, **__: (2 * x.detach() * dy.detach(), torch.zeros(2, 2), None, None))
    other = torch.zeros(2, 2)
    return torch_api.hyper_mega_moe(x, other, other, other, other)


@pytest.mark.parametrize("call", [norm, router, layer])
@pytest.mark.parametrize("strided", [False, True])
def test_a_second_derivative_is_refused(monkeypatch, call, strided):
    x = leaf(2, 2) if call is not layer else leaf(2, 2).detach().bfloat16().requires_grad_(True)
    y = call(monkeypatch, x.t() if strided else x)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    assert torch.equal(g.detach().float(), 2 * x.detach().float())
    with pytest.raises(RuntimeError, match="differentiable once"):
        (g.square().sum() + x.square().sum()).backward()  # the second term alone would have had a gradient
