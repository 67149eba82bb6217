"""PyTorch entry points of the operators for experts of a caller's own form (include/mm_experts.h).

    out = grouped_mm(rows, weight, offsets)             # each expert's rows times its matrix

`grouped_mm` is differentiable once (a second derivative is refused); the `*_forward` / `*_backward`
functions are the calls it makes. As in block_ops: argument marshalling only, on the current stream of
the tensors' device; non-contiguous tensors are copied to contiguous ones.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._first_order import first_order_only
from .block_ops import _aligned, _contiguous, _elsewhere, _on_gpu, _Plans, _sig, _stream, _type

# ------------------------------------------------------------------------------- grouped products

_grouped_plans = _Plans()


def _index32(t, most):
    """32-bit offsets; numbers that do not fit stay outside [0, most]."""
    if t.dtype == torch.int64:
        t = t.clamp(-1, most + 1).to(torch.int32)
    return _contiguous(t)


def _layout(weight):
    """(whether [E,K,N] is kept as [E,N,K], the contiguous and aligned tensor)."""
    if not weight.is_contiguous() and weight.transpose(1, 2).is_contiguous():
        return True, _aligned(weight.transpose(1, 2))
    return False, _aligned(weight)


def _grouped_plan(rows, weight, offsets, out_type, transposed, flags, key, d_out=None):
    """Checks the inputs; (address of the descriptor, workspace bytes, descriptor)."""
    _on_gpu("grouped_mm", rows, weight, offsets, d_out)
    if weight.dim() != 3 or rows.dim() != 2 or rows.shape[1] != weight.shape[1]:
        raise ValueError("expected rows[R,K] and weight[E,K,N]")
    R, (E, K, N) = rows.shape[0], weight.shape
    for name, t in (("rows", rows), ("weight", weight), ("d_out", d_out)):
        if t is not None and t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16")
    if offsets.shape != (E + 1,) or offsets.dtype not in (torch.int32, torch.int64):
        raise ValueError("expected offsets[E+1] in int32 or int64")
    if d_out is not None and d_out.shape != (R, N):
        raise ValueError("expected d_out[R,N]")
    d = _abi.mm_grouped_desc(R, K, N, E, transposed, out_type, flags)
    at = ctypes.addressof(d)
    ws = int(_abi._lib().mm_grouped_workspace_size(at))
    if ws == 0:
        raise ValueError(f"unsupported sizes R={R} K={K} N={N} E={E}")
    return _grouped_plans.remember(key, (at, ws, d))


def _odd(weight):
    """Zeros that bring K and N to multiples of 8."""
    return (-weight.shape[1] % 8, -weight.shape[2] % 8) if weight.dim() == 3 else (0, 0)


def _widened(t, *pad):
    return torch.nn.functional.pad(t, pad) if any(pad) else t


def grouped_mm_forward(rows, weight, offsets, *, out_dtype=None, flags=0):
    """out [R,N]: out[r] = rows[r] @ weight[e] for offsets[e] <= r < offsets[e+1], zero rows elsewhere.
    rows [R,K] and weight [E,K,N] bf16 (a transposed view of contiguous [E,N,K] is read as it is),
    offsets [E+1] rising from 0 on; offsets that do not rise or end above R make `out` NaN. out_dtype:
    bfloat16 (None) or float32. K and N in multiples of 8 are read in place; others cost padded copies."""
    if _elsewhere(rows):
        with torch.cuda.device(rows.device):
            return grouped_mm_forward(rows, weight, offsets, out_dtype=out_dtype, flags=flags)
    pk, pn = _odd(weight)
    if (pk or pn) and rows.dim() == 2 and rows.shape[1] == weight.shape[1]:
        out = grouped_mm_forward(_widened(rows, 0, pk), _widened(weight, 0, pn, 0, pk), offsets,
                                 out_dtype=out_dtype, flags=flags)
        return out[:, :weight.shape[2]].contiguous()
    transposed, kept = _layout(weight) if weight.dim() == 3 else (False, weight)
    out_dtype = out_dtype or torch.bfloat16
    key = (_sig(rows), _sig(weight), _sig(offsets), out_dtype, transposed, flags)
    at, nbytes, _ = _grouped_plans.get(key) or _grouped_plan(
        rows, weight, offsets, _type("out", torch.empty(0, dtype=out_dtype)), transposed, flags, key)
    rows, offsets = _aligned(rows), _index32(offsets, rows.shape[0])
    out = torch.empty((rows.shape[0], weight.shape[2]), dtype=out_dtype, device=rows.device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=rows.device)
    _abi.check(_abi._lib().mm_grouped_mm(
        at, rows.data_ptr(), kept.data_ptr(), offsets.data_ptr(), out.data_ptr(), ws.data_ptr(), nbytes,
        _stream(rows)), "mm_grouped_mm")
    return out


def grouped_mm_weight_grad(rows, d_out, offsets, weight, *, dtype=None, into=None, flags=0):
    """d_weight [E,K,N], d_weight[e] = rows_e^T d_out_e, laid out as `weight` (of which only shape and
    layout count), bfloat16 (None) or float32. `into`: such a tensor that the sums are added to instead
    (gradients accumulated over micro-batches)."""
    if _elsewhere(rows):
        with torch.cuda.device(rows.device):
            return grouped_mm_weight_grad(rows, d_out, offsets, weight, dtype=dtype, into=into, flags=flags)
    if into is not None:
        if into.shape != weight.shape or into.device != rows.device:
            raise ValueError("expected `into` of the weight's shape on its device")
        if dtype is not None and dtype != into.dtype:
            raise TypeError("dtype is for results of their own: sums have the dtype of `into`")
        dtype = into.dtype
    dtype = dtype or torch.bfloat16
    pk, pn = _odd(weight)
    if (pk or pn) and rows.dim() == 2 and d_out.dim() == 2 and rows.shape[1] == weight.shape[1] \
            and d_out.shape[1] == weight.shape[2]:
        E, K, N = weight.shape
        wide = weight.new_empty(1).expand(E, K + pk, N + pn)  # (its shape is all that counts)
        got = grouped_mm_weight_grad(_widened(rows, 0, pk), _widened(d_out, 0, pn), offsets, wide,
                                     dtype=torch.float32 if into is not None else dtype, flags=flags)
        got = got[:, :K, :N]
        if into is not None:
            return into.add_(got)
        return got.contiguous()
    if weight.dim() != 3:
        raise ValueError("expected weight[E,K,N]")
    E, K, N = weight.shape
    like = weight if into is None else into
    transposed = not like.is_contiguous() and like.transpose(1, 2).is_contiguous()
    if into is not None and not (transposed or into.is_contiguous()):
        raise ValueError("`into` must be contiguous, or a transposed view of a contiguous tensor")
    if into is not None and into.data_ptr() % 16:
        raise ValueError("`into` must start on a 16-byte boundary")
    key = ("weight", _sig(rows), _sig(d_out), (weight.shape, weight.dtype), _sig(offsets), dtype, transposed, flags)
    at, nbytes, _ = _grouped_plans.get(key) or _grouped_plan(
        rows, weight, offsets, _type("the weight gradient", torch.empty(0, dtype=dtype)), transposed,
        flags, key, d_out)
    rows, d_out, offsets = _aligned(rows), _aligned(d_out), _index32(offsets, rows.shape[0])
    if into is not None:
        out = into.transpose(1, 2) if transposed else into
    else:
        out = torch.empty((E, N, K) if transposed else (E, K, N), dtype=dtype, device=rows.device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=rows.device)
    _abi.check(_abi._lib().mm_grouped_mm_weight_grad(
        at, rows.data_ptr(), d_out.data_ptr(), offsets.data_ptr(), out.data_ptr(), into is not None,
        ws.data_ptr(), nbytes, _stream(rows)), "mm_grouped_mm_weight_grad")
    return out.transpose(1, 2) if transposed else out


def grouped_mm_backward(d_out, rows, weight, offsets, *, weight_grad_dtype=None, weight_grad=None, flags=0):
    """(d_rows bf16 [R,K], d_weight [E,K,N]) for d_out bf16 [R,N]. weight_grad_dtype: bfloat16 (None) or
    float32; weight_grad: a tensor that the weight's gradient is added to instead."""
    d_rows = grouped_mm_forward(d_out, weight.transpose(1, 2), offsets, flags=flags)
    return d_rows, grouped_mm_weight_grad(rows, d_out, offsets, weight, dtype=weight_grad_dtype,
                                          into=weight_grad, flags=flags)


class GroupedMMFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weight, offsets, out_dtype):
        ctx.save_for_backward(rows, weight, offsets)
        return grouped_mm_forward(rows, weight, offsets, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, d_out):
        rows, weight, offsets = ctx.saved_tensors
        d = d_out.to(torch.bfloat16)
        d_rows = d_weight = None
        if ctx.needs_input_grad[0]:
            d_rows = grouped_mm_forward(d, weight.transpose(1, 2), offsets)
        if ctx.needs_input_grad[1]:
            d_weight = grouped_mm_weight_grad(rows, d, offsets, weight)
        return (*first_order_only("grouped_mm", (d_rows, d_weight), (rows, weight, d_out)), None, None)


def grouped_mm(rows, weight, offsets, *, out_dtype=None):
    """grouped_mm_forward with gradients for rows and weight (of a float32 result rounded to bfloat16
    first: the products take no wider ones)."""
    return GroupedMMFunction.apply(rows, weight, offsets, out_dtype)
