"""PyTorch entry points of the step between the backward pass and the optimizer (include/mm_experts.h).

    norm = clip_grad_norm([p.grad for p in model.parameters()], max_norm)   # scales them in place
    norm = grad_norm(grads)                                                 # the norm alone

Both take tensors of bfloat16 and float32, any number and sizes, on one device, and return the norm as
a float32 tensor without waiting for it. Two launches per thousand tensors, on the current stream; in a
captured graph the addresses are those of the capture.
"""
from __future__ import annotations

import struct

import torch

from . import _abi
from .block_ops import _elsewhere, _stream

_TYPE = {torch.bfloat16: _abi.MM_BF16, torch.float32: _abi.MM_FP32}
_REF = struct.Struct("@qqqii")  # mm_tensor_ref


def _dense(t):
    """Whether the elements fill t's memory without gaps or overlaps, in whatever order."""
    if t.is_contiguous():
        return True
    order = sorted(range(t.dim()), key=t.stride, reverse=True)
    return t.permute(order).is_contiguous()


def _packed(src, dst, device):
    """The descriptions of contiguous tensors as mm_tensor_ref[]."""
    buf = bytearray(_REF.size * len(src))
    index = device.index
    for i, (s, d) in enumerate(zip(src, dst)):
        if s.get_device() != index or d.get_device() != index:
            raise ValueError(f"all tensors must be on {device}")
        try:
            _REF.pack_into(buf, i * _REF.size, s.data_ptr(), d.data_ptr(), s.numel(), _TYPE[s.dtype],
                           _TYPE[d.dtype])
        except KeyError:
            raise TypeError("gradients must be bfloat16 or float32") from None
    return buf


def _tensors(tensors):
    return [tensors] if isinstance(tensors, torch.Tensor) else [t for t in tensors if t is not None]


def _call(src, dst, clip, device):
    buf = _packed(src, dst, device)
    at = (_abi.ctypes.c_char * len(buf)).from_buffer(buf) if buf else None
    norm = torch.empty((), dtype=torch.float32, device=device)
    lib = _abi._lib()
    nbytes = int(lib.mm_grad_workspace_size(len(src)))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if clip is None:
        _abi.check(lib.mm_grad_norm(len(src), at, norm.data_ptr(), ws.data_ptr(), nbytes, _stream(norm)),
                   "mm_grad_norm")
    else:
        _abi.check(lib.mm_grad_clip(len(src), at, *clip, norm.data_ptr(), ws.data_ptr(), nbytes, _stream(norm)),
                   "mm_grad_clip")
    return norm


def _device(op, tensors):
    if not tensors[0].is_cuda:
        raise ValueError(f"{op} runs on a CUDA device only (no CPU path)")
    return tensors[0].device


def grad_norm(tensors):
    """The root of the sum of the squares of all elements of all tensors (None entries are left out), a
    float32 scalar. Summed in 64 bits: right for elements of any size."""
    tensors = _tensors(tensors)
    if not tensors:
        return torch.zeros((), device="cuda")
    if _elsewhere(tensors[0]):
        with torch.cuda.device(tensors[0].device):
            return grad_norm(tensors)
    device = _device("grad_norm", tensors)
    src = [t.detach() if _dense(t) else t.detach().contiguous() for t in tensors]
    return _call(src, src, None, device)


def clip_grad_norm(tensors, max_norm, *, eps=1e-6, out=None):
    """Multiplies all tensors by min(1, max_norm / (norm + eps)), norm being grad_norm(tensors), which is
    returned. In place, or into the tensors `out` (of the same shapes, bfloat16 or float32, not
    overlapping `tensors`): for gradients that are accumulated in 32 bits and handed on in 16, or kept.
    None entries are left out. A NaN in one tensor makes all of them NaN, an infinity makes finite
    elements 0."""
    given = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    targets = given if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    if len(targets) != len(given):
        raise ValueError("expected as many tensors in `out`")
    if any(d is None for s, d in zip(given, targets) if s is not None):
        raise ValueError("`out` lacks a tensor")
    pairs = [(s, d) for s, d in zip(given, targets) if s is not None]
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0.0 or not 0.0 <= eps <= 3e38:
        raise ValueError("max_norm and eps must not be negative")
    if not pairs:
        return torch.zeros((), device="cuda")
    if _elsewhere(pairs[0][0]):
        with torch.cuda.device(pairs[0][0].device):
            return clip_grad_norm(tensors, max_norm, eps=eps, out=out)
    device = _device("clip_grad_norm", [s for s, _ in pairs])
    sources = {s.data_ptr(): i for i, (s, _) in enumerate(pairs) if s.numel()}
    src, dst, late, seen = [], [], [], set()
    for i, (s, d) in enumerate(pairs):
        if d.shape != s.shape:
            raise ValueError("`out` must have the tensors' shapes")
        if d.numel():
            at = d.data_ptr()
            if at in seen or sources.get(at, i) != i:
                raise ValueError("a tensor is given twice")
            seen.add(at)
        if not (s.is_contiguous() and d.is_contiguous()) and not (s.stride() == d.stride() and _dense(s)):
            s = s.detach().contiguous()  # elements with gaps, or in two orders
            if out is None or not d.is_contiguous():
                late.append((d, torch.empty_like(s, dtype=d.dtype) if out is not None else s))
                d = late[-1][1]
        src.append(s)
        dst.append(d)
    norm = _call(src, dst, (max_norm, eps), device)
    with torch.no_grad():
        for target, value in late:
            target.copy_(value)
    torch.autograd.graph.increment_version([d for _, d in pairs])
    return norm
