"""Calls of expert_ops and grad_ops whose tensors are on a GPU that is not the current one run with that
GPU as the current one (host logic only, as in test_device_cpu), and what the host refuses before any
CUDA call."""
import pytest
import torch

from moe_ffn_expert_gb300 import expert_ops, grad_ops
from test_device_cpu import Elsewhere, Reached, state  # noqa: F401


def table(t):
    return expert_ops.ExpertTable(t, t, t, 1, 1, 1)


@pytest.mark.parametrize("call", [
    lambda t: expert_ops.expert_table(t, 4),
    lambda t: expert_ops.dispatch_forward(t, table(t)),
    lambda t: expert_ops.combine_forward(t, table(t), t),
    lambda t: expert_ops.combine_backward(t, t, table(t), t),
    lambda t: expert_ops.grouped_mm_forward(t, t, t),
    lambda t: expert_ops.grouped_mm_weight_grad(t, t, t, t),
    lambda t: grad_ops.grad_norm([t]),
    lambda t: grad_ops.clip_grad_norm([t, None], 1.0),
    lambda t: grad_ops.clip_grad_norm([t], 1.0, out=[t])])
def test_operators_make_the_tensors_device_the_current_one(state, call):  # noqa: F811
    with pytest.raises(Reached):
        call(Elsewhere(state))
    assert state["current"] == 0


def test_host_tensors_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    ids, x, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 8), torch.zeros(3, 2)
    off, b = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    rows = torch.zeros(3, 8, dtype=torch.bfloat16)
    order = expert_ops.ExpertTable(off, ids, ids.flatten(), 3, 2, 2)
    for call in (lambda: expert_ops.expert_table(ids, 4), lambda: expert_ops.dispatch_forward(x, order),
                 lambda: expert_ops.combine_forward(torch.zeros(6, 8), order, w),
                 lambda: expert_ops.combine_backward(x, torch.zeros(6, 8), order, w),
                 lambda: expert_ops.grouped_mm_forward(rows, b, off),
                 lambda: expert_ops.grouped_mm_weight_grad(rows, rows, off, b), lambda: grad_ops.grad_norm(x),
                 lambda: grad_ops.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA device only"):
            call()


def test_clipping_refuses_what_it_cannot_mean(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    a, b = torch.ones(4), torch.ones(4)
    for kwargs in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=-1.0),
                   dict(max_norm=1.0, eps=float("inf")), dict(max_norm=1.0, out=[a]), dict(max_norm=1.0, out=[a, None])):
        with pytest.raises(ValueError):
            grad_ops.clip_grad_norm([a, b], **kwargs)


@pytest.mark.parametrize("froms,tos,apart", [
    ([1, 2, 3], [1, 2, 3], True), ([1, 2, 3], [4, 5, 6], True), ([1, 2], [5, 5], False), ([1, 2], [2, 3], False),
    ([1, 2], [3, 1], False), ([0, 0, 1], [0, 0, 2], True), ([0, 1], [0, 1], True), ([1, 0, 0], [1, 0, 0], True),
    ([1, 2], [2, 1], False)])
def test_addresses_given_twice(froms, tos, apart):
    assert grad_ops._apart(froms, tos) == apart
    if len(set(froms) - {0}) != len(froms) - froms.count(0):
        assert not grad_ops._apart(froms, froms)


def test_dense_tensors():
    t = torch.zeros(3, 4, 5)
    for dense in (t, t.permute(2, 0, 1), t.transpose(0, 1), t[1:], t[:, :0], torch.zeros(())):
        assert grad_ops._dense(dense)
    for gaps in (t[:, 1:3], t[..., 0], t.expand(2, 3, 4, 5), t[0, 0].expand(2, 5), t[::2]):
        assert not grad_ops._dense(gaps)
