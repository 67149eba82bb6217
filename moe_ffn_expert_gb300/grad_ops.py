"""PyTorch entry points of the step between the backward pass and the optimizer (include/mm_experts.h).

    norm = clip_grad_norm([p.grad for p in model.parameters()], max_norm)   # scales them in place
    norm = grad_norm(grads)                                                 # the norm alone

Both take tensors of bfloat16 and float32, any number and sizes, on one device, and return the norm as
a float32 tensor without waiting for it. Two launches per thousand tensors, on the current stream; in a
captured graph the addresses are those of the capture. Of a call with few elements the host's part is
the larger one: per tensor some 0.6 us (clip_grad_norm into other tensors 1.2), so tensors are asked for
their properties a whole list at a time.
"""
from __future__ import annotations

from array import array

import torch

from . import _abi
from .block_ops import _elsewhere, _stream

_T = torch.Tensor
_TYPE = {torch.bfloat16: _abi.MM_BF16, torch.float32: _abi.MM_FP32}
# the last 8 bytes of mm_tensor_ref: both types, one of them
_TYPES = {(s, d): _TYPE[s] | _TYPE[d] << 32 for s in _TYPE for d in _TYPE}
_ONE_TYPE = {s: _TYPES[s, s] for s in _TYPE}


def _dense(t):
    """Whether the elements fill t's memory without gaps or overlaps, in whatever order."""
    if t.is_contiguous():
        return True
    order = sorted(range(t.dim()), key=t.stride, reverse=True)
    return t.permute(order).is_contiguous()


def _repeats(t):
    """Whether t is an expanded tensor, which cannot be written to."""
    return t.numel() > 0 and any(n > 1 and step == 0 for n, step in zip(t.shape, t.stride()))


def _apart(froms, tos):
    """No address twice among `tos`, and none of them another's of `froms` (empty tensors have none)."""
    once = set(tos)
    if len(once) != len(tos) and len(once - {0}) != len(tos) - tos.count(0):
        return False
    if froms is tos or once.isdisjoint(froms):
        return True
    place = {p: i for i, p in enumerate(froms) if p}
    return all(place.get(p, i) == i for i, p in enumerate(tos))


def _call(src, dst, clip, device):
    """The library's call for tensors whose memory is taken as it lies."""
    n, same = len(src), src is dst
    if set(map(_T.get_device, src)) | set(() if same else map(_T.get_device, dst)) != {device.index}:
        raise ValueError(f"all tensors must be on {device}")
    refs = [0] * (4 * n)  # mm_tensor_ref[n]
    froms = list(map(_T.data_ptr, src))
    refs[0::4], refs[2::4] = froms, map(_T.numel, src)
    refs[1::4] = tos = froms if same else list(map(_T.data_ptr, dst))
    if clip is not None and not _apart(froms, tos):
        raise ValueError("a tensor is given twice")
    types = [t.dtype for t in src]
    to_types = types if same else [t.dtype for t in dst]
    try:
        if types == to_types:
            refs[3::4] = map(_ONE_TYPE.__getitem__, types)
        else:
            refs[3::4] = map(_TYPES.__getitem__, zip(types, to_types))
    except KeyError:
        raise TypeError("gradients must be bfloat16 or float32") from None
    refs = array("q", refs)
    norm = torch.empty((), dtype=torch.float32, device=device)
    lib, at = _abi._lib(), refs.buffer_info()[0]
    nbytes = int(lib.mm_grad_workspace_size(n))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if clip is None:
        _abi.check(lib.mm_grad_norm(n, at, norm.data_ptr(), ws.data_ptr(), nbytes, _stream(norm)), "mm_grad_norm")
    else:
        _abi.check(lib.mm_grad_clip(n, at, *clip, norm.data_ptr(), ws.data_ptr(), nbytes, _stream(norm)),
                   "mm_grad_clip")
    return norm


def _list(tensors):
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


_NONE = type(None)


def _device(op, first):
    if not first.is_cuda:
        raise ValueError(f"{op} runs on a CUDA device only (no CPU path)")
    return first.device


def grad_norm(tensors):
    """The root of the sum of the squares of all elements of all tensors (None entries are left out), a
    float32 scalar. Summed in 64 bits: right for elements of any size."""
    tensors = _list(tensors)
    if _NONE in map(type, tensors):
        tensors = [t for t in tensors if t is not None]
    if not tensors:
        return torch.zeros((), device="cuda")
    if _elsewhere(tensors[0]):
        with torch.cuda.device(tensors[0].device):
            return grad_norm(tensors)
    device = _device("grad_norm", tensors[0])
    if not all(map(_T.is_contiguous, tensors)):
        tensors = [t if _dense(t) else t.detach().contiguous() for t in tensors]
    return _call(tensors, tensors, None, device)


def clip_grad_norm(tensors, max_norm, *, eps=1e-6, out=None):
    """Multiplies all tensors by min(1, max_norm / (norm + eps)), norm being grad_norm(tensors), which is
    returned. In place, or into the tensors `out` (of the same shapes, bfloat16 or float32, not
    overlapping `tensors`): for gradients that are accumulated in 32 bits and handed on in 16, or kept.
    Expanded tensors cannot be scaled and are refused. None entries are left out. A NaN in one tensor makes all of them NaN, an infinity makes finite
    elements 0."""
    src = _list(tensors)
    dst = src if out is None else _list(out)
    if len(dst) != len(src):
        raise ValueError("expected as many tensors in `out`")
    if _NONE in map(type, src):
        pairs = [(s, d) for s, d in zip(src, dst) if s is not None]
        src = [s for s, _ in pairs]
        dst = src if out is None else [d for _, d in pairs]
    if out is not None and _NONE in map(type, dst):
        raise ValueError("`out` lacks a tensor")
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0.0 or not 0.0 <= eps <= 3e38:
        raise ValueError("max_norm and eps must not be negative")
    if not src:
        return torch.zeros((), device="cuda")
    if _elsewhere(src[0]):
        with torch.cuda.device(src[0].device):
            return clip_grad_norm(src, max_norm, eps=eps, out=None if out is None else dst)
    device = _device("clip_grad_norm", src[0])
    if out is not None and list(map(_T.size, src)) != list(map(_T.size, dst)):
        raise ValueError("`out` must have the tensors' shapes")
    given, late = dst, []
    if not all(map(_T.is_contiguous, src)) or (out is not None and not all(map(_T.is_contiguous, dst))):
        froms = list(map(_T.data_ptr, src))  # (stand-ins have addresses of their own)
        if not _apart(froms, froms if out is None else list(map(_T.data_ptr, dst))):
            raise ValueError("a tensor is given twice")
        if any(map(_repeats, dst)):
            raise ValueError("a tensor to write shows one element at several places")
        src, dst, late = _in_order(src, dst, out is None)
    norm = _call(src, dst, (max_norm, eps), device)
    if late:
        with torch.no_grad():
            for target, value in late:
                target.copy_(value)
    torch.autograd.graph.increment_version(given)
    return norm


def _in_order(src, dst, in_place):
    """src and dst with stand-ins where the two do not hold their elements in one order without gaps, and
    the (tensor, stand-in) pairs to copy back."""
    late, froms, tos = [], [], []
    for s, d in zip(src, dst):
        if not (s.is_contiguous() and d.is_contiguous()) and not (s.stride() == d.stride() and _dense(s)):
            s = s.detach().contiguous()
            if in_place or not d.is_contiguous():
                value = s if in_place else torch.empty_like(s, dtype=d.dtype)
                late.append((d, value))
                d = value
        froms.append(s)
        tos.append(d)
    return froms, froms if in_place else tos, late
