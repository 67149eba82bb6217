"""Gradients that autograd must not differentiate again.

The backward passes run in libmm.so, out of autograd's sight: under create_graph their results would
be constants, and a loss with a second derivative would silently lose it. (torch's
once_differentiable refuses only what depends on the incoming gradients, not on the saved inputs.)
"""
import torch


class _Refused(torch.autograd.Function):
    @staticmethod
    def forward(ctx, name, grad, *sources):
        ctx.name = name
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} is differentiable once: its gradient has no derivative")


def first_order_only(name, grads, sources):
    """`grads`, which raise when they are differentiated. `sources`: the tensors they depend on."""
    if not torch.is_grad_enabled():  # no create_graph
        return grads
    on = [t for t in sources if t is not None and t.requires_grad]
    return tuple(_Refused.apply(name, g, *on) if g is not None and on else g for g in grads)
