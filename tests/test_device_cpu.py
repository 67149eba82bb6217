"""Calls whose tensors are on a GPU that is not the current one run with that GPU as the current one.
Host logic only: the current device and the tensors are stand-ins, and nothing is launched."""
import pytest
import torch

from moe_ffn_expert_gb300 import _abi, block_ops, torch_api


class Reached(Exception):
    """The call went on to its tensors."""


class Elsewhere:
    """A tensor on cuda:1; what is asked beyond its device is asked with cuda:1 as the current one."""
    device = torch.device("cuda", 1)

    def __init__(self, state):
        self._state = state

    def get_device(self):
        return 1

    def __getattr__(self, name):
        assert self._state["current"] == 1, f"{name} asked with another device as the current one"
        raise Reached(name)


@pytest.fixture
def state(monkeypatch):
    state = {"current": 0}

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *_):
            state["current"] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    return state


@pytest.mark.parametrize("call", [
    lambda t: block_ops.residual_norm_forward(t, t, post_weight=t),
    lambda t: block_ops.residual_norm_backward(t, t, t, None),
    lambda t: block_ops.router_forward(t, 2, stats=True),
    lambda t: block_ops.router_backward(t, t, t),
    lambda t: block_ops.quantize_expert_weights(t),
    lambda t: object.__new__(block_ops.MoEDecoder)._call(t, t, t)])
def test_operators_make_the_tensors_device_the_current_one(state, call):
    with pytest.raises(Reached):
        call(Elsewhere(state))
    assert state["current"] == 0


def test_a_device_that_is_current_is_not_set_again(state, monkeypatch):
    state["current"] = 1
    monkeypatch.setattr(torch.cuda, "device", None)  # would fail if it were called
    with pytest.raises(Reached):
        block_ops.router_forward(Elsewhere(state), 2)
    assert not block_ops._elsewhere(torch.zeros(1))  # host tensors are refused by the checks


def test_the_layer_makes_the_tensors_device_the_current_one(state, monkeypatch):
    seen = []

    def call(*_):
        seen.append(state["current"])
        return _abi.MM_OK

    monkeypatch.setattr(_abi, "mm_forward_ex", call)
    monkeypatch.setattr(_abi, "mm_backward_ex", call)
    monkeypatch.setattr(torch_api, "_stream", lambda device: 0)
    monkeypatch.setattr(torch_api, "_ptr", lambda t: 0)
    ws = torch_api.Workspace.wrap(_abi.dims(1, 64, 64, 1, 1), torch.empty(0))
    x = Elsewhere(state)
    torch_api.forward(ws, x, x, x, x, x, y=x)
    torch_api.backward(ws, x, x, x, x, x, x, dx=x, d_topk=x, d_up=x, d_down=x)
    assert seen == [1, 1] and state["current"] == 0
