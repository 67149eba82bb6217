"""What the calls of expert_ops hand to the library for tensors of any strides: host logic only, with a
library that notes the numbers at the addresses it is given."""
import ctypes

import pytest
import torch

from moe_ffn_expert_gb300 import _abi, expert_ops

T, K, E, H = 6, 2, 3, 4
ORDER = torch.randperm(T * K, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(T, K)
OFFSETS = torch.tensor([0, 5, 7, 12], dtype=torch.int32)


def read(address, n, kind=ctypes.c_int32):
    return list((kind * n).from_address(address))


@pytest.fixture
def given(monkeypatch):
    """What the last call was given: offsets (None without), row_of_slot."""
    got = {}

    class Library:
        def mm_expert_dispatch(self, d, x, offsets, row_of_slot, rows, stream):
            got.update(offsets=read(offsets, E + 1), row_of_slot=read(row_of_slot, T * K))
            return 0

        def mm_expert_combine(self, d, rows, row_of_slot, weights, y, stream):
            got.update(offsets=None, row_of_slot=read(row_of_slot, T * K))
            return 0

        def mm_expert_combine_backward(self, d, dy, rows, offsets, row_of_slot, *rest):
            got.update(offsets=read(offsets, E + 1), row_of_slot=read(row_of_slot, T * K))
            return 0

    monkeypatch.setattr(_abi, "_lib", lambda: Library())
    monkeypatch.setattr(expert_ops, "_on_gpu", lambda *_: None)
    monkeypatch.setattr(expert_ops, "_elsewhere", lambda _: False)
    monkeypatch.setattr(expert_ops, "_stream", lambda _: 0)
    monkeypatch.setattr(expert_ops, "_row_plans", expert_ops._Plans())
    return got


def strided(t):
    wide = torch.full((*t.shape[:-1], 2 * t.shape[-1]), 1000, dtype=t.dtype)
    wide[..., ::2] = t
    return wide[..., ::2]


ROWS = {"contiguous": ORDER, "strided": strided(ORDER), "transposed": ORDER.t().contiguous().t(),
        "expanded": ORDER[:1].expand(T, K)}
BOUNDS = {"contiguous": OFFSETS, "strided": strided(OFFSETS), "expanded": OFFSETS[1:2].expand(E + 1)}
CALLS = {"dispatch": lambda table: expert_ops.dispatch_forward(torch.zeros(T, H), table),
         "combine": lambda table: expert_ops.combine_forward(torch.zeros(T * K, H), table, torch.ones(T, K)),
         "backward": lambda table: expert_ops.combine_backward(torch.zeros(T, H), torch.zeros(T * K, H), table)}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
@pytest.mark.parametrize("known", [False, True])
def test_tables_of_any_strides(given, call, known):
    """Whether or not a call of the same shapes has been checked before."""
    if known:
        call(expert_ops.ExpertTable(OFFSETS, ORDER, ORDER.flatten(), T, K, E))
    for row_of_slot in ROWS.values():
        for offsets in BOUNDS.values():
            given.clear()
            call(expert_ops.ExpertTable(offsets, row_of_slot, ORDER.flatten(), T, K, E))
            assert given["row_of_slot"] == row_of_slot.flatten().tolist()
            assert given["offsets"] in (None, offsets.tolist())
