"""PyTorch entry points of the operators for experts of a caller's own form (include/mm_experts.h).

The fused layer (torch_api) is one SwiGLU expert in bf16. Experts with another activation, a bias,
adapters or results in 32 bits are built from its parts:

    ids, weights, *_ = moe_router(logits, k)                     # block_ops
    table = expert_table(ids, num_experts)                       # the slots' order by expert
    rows  = expert_dispatch(x, table)                            # the tokens' rows in that order
    h     = grouped_mm(rows, w1, table.offsets)                  # each expert's rows times its matrix
    h     = torch.nn.functional.gelu(h)
    o     = grouped_mm(h, w2, table.offsets)
    y     = expert_combine(o, table, weights)                    # each token's weighted sum

Any number of tokens, one included. `expert_dispatch`, `grouped_mm` and `expert_combine` are
differentiable once (a second derivative is refused); the `*_forward` / `*_backward` functions are the
calls they make. As in block_ops: argument marshalling only, on the current stream of the tensors'
device; non-contiguous tensors are copied to contiguous ones.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _abi
from ._first_order import first_order_only
from .block_ops import _aligned, _contiguous, _elsewhere, _on_gpu, _Plans, _ptr, _sig, _stream, _type

# ------------------------------------------------------------------------------- order and rows

_table_plans, _row_plans = _Plans(), _Plans()


class ExpertTable(NamedTuple):
    """The order of a selection's slots s = t k + j by expert, equal ones by s."""
    offsets: torch.Tensor      # int32 [E+1]: where each expert's rows start, and where the last one's end
    row_of_slot: torch.Tensor  # int32 [T,k]: place of a slot, -1 for one without an expert
    slot_of_row: torch.Tensor  # int32 [T k]: slot at a place, -1 behind offsets[E]
    T: int
    K: int
    E: int


def expert_table(topk_ids, num_experts):
    """ExpertTable of topk_ids [T,k] (int32 or int64). A slot whose id is outside [0, num_experts) has no
    expert: nobody computes it, and it adds nothing to its token."""
    if _elsewhere(topk_ids):
        with torch.cuda.device(topk_ids.device):
            return expert_table(topk_ids, num_experts)
    E = int(num_experts)
    key = (_sig(topk_ids), E)
    plan = _table_plans.get(key)
    if plan is None:
        _on_gpu("expert_table", topk_ids)
        if topk_ids.dim() != 2 or topk_ids.dtype not in (torch.int32, torch.int64):
            raise ValueError("expected topk_ids[T,k] in int32 or int64")
        T, K = topk_ids.shape
        d = _abi.mm_expert_desc(T, 0, E, K, 0)
        at = ctypes.addressof(d)
        nbytes = int(_abi._lib().mm_expert_table_workspace_size(at))
        if nbytes == 0:
            raise ValueError(f"unsupported sizes T={T} k={K} num_experts={E}")
        plan = _table_plans.remember(key, (at, nbytes, T, K, d))
    at, nbytes, T, K, _ = plan
    if topk_ids.dtype == torch.int64:  # (a number beyond 32 bits must not become an expert's)
        topk_ids = topk_ids.clamp(-1, E).to(torch.int32)
    ids, dev = _contiguous(topk_ids), topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row = torch.empty((T, K), dtype=torch.int32, device=dev)
    slot = torch.empty(T * K, dtype=torch.int32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if T * K > 2048 else None
    _abi.check(_abi._lib().mm_expert_table(
        at, ids.data_ptr(), offsets.data_ptr(), row.data_ptr(), slot.data_ptr(), _ptr(ws), nbytes,
        _stream(ids)), "mm_expert_table")
    return ExpertTable(offsets, row, slot, T, K, E)


def _row_plan(op, table, tokens, rows, weights, key):
    """Checks the inputs; (address of the descriptor, descriptor). tokens [T,H], rows [T k,H], weights
    [T,k]: those of them that the call has."""
    first = tokens if tokens is not None else rows
    _on_gpu(op, first, tokens, rows, weights, table.offsets, table.row_of_slot)
    T, K, E = table.T, table.K, table.E
    for name, t, shape in (("offsets", table.offsets, (E + 1,)), ("row_of_slot", table.row_of_slot, (T, K))):
        if t.shape != shape or t.dtype != torch.int32:
            raise ValueError(f"expected the table's {name} of shape {shape} in int32")
    if first.dim() != 2:
        raise ValueError("expected rows of shape [n,H]")
    H = first.shape[1]
    for name, t, n in (("tokens", tokens, T), ("rows", rows, T * K)):
        if t is not None and t.shape != (n, H):
            raise ValueError(f"expected the {name}' rows of shape [{n},{H}]")
        if t is not None and t.dtype != first.dtype:
            raise TypeError(f"{op}: all rows must have one dtype")
    if weights is not None and (weights.shape != (T, K) or weights.dtype != torch.float32):
        raise ValueError("expected weights[T,k] in float32")
    d = _abi.mm_expert_desc(T, H, E, K, _type("rows", first))
    return _row_plans.remember(key, (ctypes.addressof(d), d))


def dispatch_forward(x, table):
    """rows [T k,H]: row r is x[t] for the token t of the slot at place r; zeros behind offsets[E]."""
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return dispatch_forward(x, table)
    key = ("dispatch", _sig(x), _sig(table.offsets), _sig(table.row_of_slot), table[3:])
    at, _ = _row_plans.get(key) or _row_plan("expert_dispatch", table, x, None, None, key)
    x, offsets, row_of_slot = _contiguous(x), _contiguous(table.offsets), _contiguous(table.row_of_slot)
    rows = torch.empty((table.T * table.K, x.shape[1]), dtype=x.dtype, device=x.device)
    _abi.check(_abi._lib().mm_expert_dispatch(
        at, x.data_ptr(), offsets.data_ptr(), row_of_slot.data_ptr(), rows.data_ptr(), _stream(x)),
        "mm_expert_dispatch")
    return rows


def combine_forward(rows, table, weights=None):
    """y [T,H]: y[t] = sum_j weights[t,j] rows[place of slot (t, j)], over the slots with an expert
    (weights fp32 [T,k]; None: 1). rows bfloat16 or float32."""
    if _elsewhere(rows):
        with torch.cuda.device(rows.device):
            return combine_forward(rows, table, weights)
    key = ("combine", _sig(rows), _sig(weights), _sig(table.offsets), _sig(table.row_of_slot), table[3:])
    at, _ = _row_plans.get(key) or _row_plan("expert_combine", table, None, rows, weights, key)
    rows, weights, row_of_slot = _contiguous(rows), _contiguous(weights), _contiguous(table.row_of_slot)
    y = torch.empty((table.T, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    _abi.check(_abi._lib().mm_expert_combine(
        at, rows.data_ptr(), row_of_slot.data_ptr(), _ptr(weights), y.data_ptr(), _stream(rows)),
        "mm_expert_combine")
    return y


def combine_backward(dy, rows, table, weights=None, *, weight_grad=True):
    """(d_rows [T k,H], d_weights fp32 [T,k]) for dy [T,H]: d_rows[place] = weight * dy[token] (zeros
    behind offsets[E]), d_weights = <dy[token], rows[place]> (None without weight_grad: `rows` may be
    None then)."""
    if _elsewhere(dy):
        with torch.cuda.device(dy.device):
            return combine_backward(dy, rows, table, weights, weight_grad=weight_grad)
    if not weight_grad:
        rows = None
    key = ("backward", _sig(dy), _sig(rows), _sig(weights), _sig(table.offsets), _sig(table.row_of_slot), table[3:])
    plan = _row_plans.get(key)
    if plan is None:
        if weight_grad and rows is None:
            raise ValueError("the weights' gradient needs the rows")
        plan = _row_plan("expert_combine", table, dy, rows, weights, key)
    dy, rows, weights = _contiguous(dy), _contiguous(rows), _contiguous(weights)
    offsets, row_of_slot = _contiguous(table.offsets), _contiguous(table.row_of_slot)
    d_rows = torch.empty((table.T * table.K, dy.shape[1]), dtype=dy.dtype, device=dy.device)
    d_weights = None
    if weight_grad:
        d_weights = torch.empty((table.T, table.K), dtype=torch.float32, device=dy.device)
    _abi.check(_abi._lib().mm_expert_combine_backward(
        plan[0], dy.data_ptr(), _ptr(rows), offsets.data_ptr(), row_of_slot.data_ptr(), _ptr(weights),
        d_rows.data_ptr(), _ptr(d_weights), _stream(dy)), "mm_expert_combine_backward")
    return d_rows, d_weights


class DispatchFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table):
        ctx.save_for_backward(*table[:3])
        ctx.sizes = table[3:]
        return dispatch_forward(x, table)

    @staticmethod
    def backward(ctx, d_rows):
        table = ExpertTable(*ctx.saved_tensors, *ctx.sizes)
        return (*first_order_only("expert_dispatch", (combine_forward(d_rows, table),), (d_rows,)), None)


def expert_dispatch(x, table):
    """dispatch_forward with a gradient for x."""
    return DispatchFunction.apply(x, table)


class CombineFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, table):
        ctx.save_for_backward(rows, weights, *table[:3])
        ctx.sizes = table[3:]
        return combine_forward(rows, table, weights)

    @staticmethod
    def backward(ctx, dy):
        rows, weights, *order = ctx.saved_tensors
        d_rows, d_weights = combine_backward(dy, rows, ExpertTable(*order, *ctx.sizes), weights,
                                             weight_grad=ctx.needs_input_grad[1])
        return (*first_order_only("expert_combine", (d_rows, d_weights), (rows, weights, dy)), None)


def expert_combine(rows, table, weights=None):
    """combine_forward with gradients for rows and weights (any floating type)."""
    if weights is not None:
        if not weights.is_floating_point():
            raise TypeError("weights must be floating point")
        weights = weights.to(torch.float32)
    return CombineFunction.apply(rows, weights, table)


# ------------------------------------------------------------------------------- grouped products

_grouped_plans = _Plans()


def _index32(t, most):
    """32-bit offsets; numbers that do not fit stay outside [0, most]."""
    if t.dtype == torch.int64:
        t = t.clamp(-1, most + 1).to(torch.int32)
    return _contiguous(t)


def _transposed(weight):
    """Whether [E,K,N] is kept as contiguous [E,N,K]."""
    return not weight.is_contiguous() and weight.dim() == 3 and weight.transpose(1, 2).is_contiguous()


def _grouped_plan(rows, weight, offsets, out_type, transposed, flags, key, d_out=None):
    """Checks the inputs; (address of the descriptor, workspace bytes, zeros that bring K and N to
    multiples of 8, descriptor). With such zeros there is no descriptor."""
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
    pad = (-K % 8, -N % 8)
    if any(pad) and K and N:
        return _grouped_plans.remember(key, (0, 0, pad, None))
    d = _abi.mm_grouped_desc(R, K, N, E, transposed, out_type, flags)
    at = ctypes.addressof(d)
    lib = _abi._lib()
    ws = int((lib.mm_grouped_mm_workspace_size if d_out is None else lib.mm_grouped_weight_grad_workspace_size)(at))
    if ws == 0:
        raise ValueError(f"unsupported sizes R={R} K={K} N={N} E={E}")
    return _grouped_plans.remember(key, (at, ws, None, d))


def grouped_status(device="cuda"):
    """A status for the calls of grouped_mm, which may share it: what check_grouped_status looks at."""
    return torch.zeros(2, dtype=torch.int32, device=device)


#: what a wait that ran out was for
_AWAITED = {1: "a free stage for operands", 2: "a free accumulator", 3: "operands", 4: "the next tile",
            5: "a free place for a tile", 6: "a sum"}


def check_grouped_status(status):
    """Waits for the current stream, and raises MMError (MM_ERR_TIMEOUT) if a wait in a call that was given
    `status` ran out: that call's result is NaN where it is missing, and the device is not to be trusted."""
    code, where = status.tolist()
    _abi.check(code, f"grouped_mm, CTA {where >> 8} awaiting {_AWAITED.get(where & 255, where & 255)}")


def _status_ptr(status, device):
    if status is None:
        return None
    if status.shape != (2,) or status.dtype != torch.int32 or not status.is_contiguous() or status.device != device:
        raise ValueError(f"expected status[2] in int32 on {device}, contiguous")
    return status.data_ptr()


def _widened(t, *pad):
    return torch.nn.functional.pad(t, pad) if any(pad) else t


def grouped_mm_forward(rows, weight, offsets, *, out_dtype=None, flags=0, status=None):
    """out [R,N]: out[r] = rows[r] @ weight[e] for offsets[e] <= r < offsets[e+1], zero rows elsewhere.
    rows [R,K] and weight [E,K,N] bf16 (a transposed view of contiguous [E,N,K] is read as it is),
    offsets [E+1] rising from 0 on; offsets that do not rise or end above R make `out` NaN. out_dtype:
    bfloat16 (None) or float32. K and N in multiples of 8 are read in place; others cost padded copies.
    status: a grouped_status, which a wait that runs out on the device sets (its results are NaN)."""
    if _elsewhere(rows):
        with torch.cuda.device(rows.device):
            return grouped_mm_forward(rows, weight, offsets, out_dtype=out_dtype, flags=flags, status=status)
    transposed = _transposed(weight)
    key = (_sig(rows), _sig(weight), _sig(offsets), out_dtype, transposed, flags)
    plan = _grouped_plans.get(key)
    if plan is None:
        out_type = _type("out", torch.empty(0, dtype=out_dtype or torch.bfloat16))
        plan = _grouped_plan(rows, weight, offsets, out_type, transposed, flags, key)
    at, nbytes, pad, _ = plan
    if pad is not None:
        out = grouped_mm_forward(_widened(rows, 0, pad[0]), _widened(weight, 0, pad[1], 0, pad[0]), offsets,
                                 out_dtype=out_dtype, flags=flags, status=status)
        return out[:, :weight.shape[2]].contiguous()
    rows, offsets = _aligned(rows), _index32(offsets, rows.shape[0])
    kept = _aligned(weight.transpose(1, 2) if transposed else weight)
    out = torch.empty((rows.shape[0], weight.shape[2]), dtype=out_dtype or torch.bfloat16, device=rows.device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=rows.device) if nbytes > 256 else None
    _abi.check(_abi._lib().mm_grouped_mm_ex(
        at, rows.data_ptr(), kept.data_ptr(), offsets.data_ptr(), out.data_ptr(), _ptr(ws), nbytes,
        _status_ptr(status, rows.device), _stream(rows)), "mm_grouped_mm")
    return out


def grouped_mm_weight_grad(rows, d_out, offsets, weight, *, dtype=None, into=None, flags=0, status=None):
    """d_weight [E,K,N], d_weight[e] = rows_e^T d_out_e, laid out as `weight` (of which only shape and
    layout count), bfloat16 (None) or float32. `into`: such a tensor that the sums are added to instead
    (gradients accumulated over micro-batches). status: as in grouped_mm_forward."""
    if _elsewhere(rows):
        with torch.cuda.device(rows.device):
            return grouped_mm_weight_grad(rows, d_out, offsets, weight, dtype=dtype, into=into, flags=flags,
                                          status=status)
    if into is not None:
        if into.shape != weight.shape or into.device != rows.device:
            raise ValueError("expected `into` of the weight's shape on its device")
        if dtype is not None and dtype != into.dtype:
            raise TypeError("dtype is for results of their own: sums have the dtype of `into`")
        dtype = into.dtype
        if not (into.is_contiguous() or _transposed(into)):
            raise ValueError("`into` must be contiguous, or a transposed view of a contiguous tensor")
    dtype = dtype or torch.bfloat16
    transposed = _transposed(weight if into is None else into)
    key = ("weight", _sig(rows), _sig(d_out), (weight.shape, weight.dtype), _sig(offsets), dtype, transposed, flags)
    plan = _grouped_plans.get(key)
    if plan is None:
        out_type = _type("the weight gradient", torch.empty(0, dtype=dtype))
        plan = _grouped_plan(rows, weight, offsets, out_type, transposed, flags, key, d_out)
    at, nbytes, pad, _ = plan
    E, K, N = weight.shape
    if pad is not None:
        wide = weight.new_empty(1).expand(E, K + pad[0], N + pad[1])  # (its shape is all that counts)
        got = grouped_mm_weight_grad(_widened(rows, 0, pad[0]), _widened(d_out, 0, pad[1]), offsets, wide,
                                     dtype=torch.float32 if into is not None else dtype, flags=flags, status=status)
        got = got[:, :K, :N]
        if into is not None:
            return into.add_(got)
        return got.transpose(1, 2).contiguous().transpose(1, 2) if transposed else got.contiguous()
    if into is not None and into.data_ptr() % 16:  # TMA and 16-byte stores want other memory
        return into.add_(grouped_mm_weight_grad(rows, d_out, offsets, weight, dtype=torch.float32, flags=flags,
                                                status=status))
    sign = _status_ptr(status, rows.device)
    rows, d_out, offsets = _aligned(rows), _aligned(d_out), _index32(offsets, rows.shape[0])
    if into is not None:
        torch.autograd.graph.increment_version(into)
        out = into.transpose(1, 2) if transposed else into
    else:
        out = torch.empty((E, N, K) if transposed else (E, K, N), dtype=dtype, device=rows.device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=rows.device)
    _abi.check(_abi._lib().mm_grouped_mm_weight_grad_ex(
        at, rows.data_ptr(), d_out.data_ptr(), offsets.data_ptr(), out.data_ptr(), into is not None,
        ws.data_ptr(), nbytes, sign, _stream(rows)), "mm_grouped_mm_weight_grad")
    return out.transpose(1, 2) if transposed else out


def grouped_mm_backward(d_out, rows, weight, offsets, *, weight_grad_dtype=None, weight_grad=None, flags=0,
                        status=None):
    """(d_rows bf16 [R,K], d_weight [E,K,N]) for d_out bf16 [R,N]. weight_grad_dtype: bfloat16 (None) or
    float32; weight_grad: a tensor that the weight's gradient is added to instead."""
    d_rows = grouped_mm_forward(d_out, weight.transpose(1, 2), offsets, flags=flags, status=status)
    return d_rows, grouped_mm_weight_grad(rows, d_out, offsets, weight, dtype=weight_grad_dtype,
                                          into=weight_grad, flags=flags, status=status)


class GroupedMMFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weight, offsets, out_dtype, status=None):
        ctx.save_for_backward(rows, weight, offsets)
        ctx.status = status
        return grouped_mm_forward(rows, weight, offsets, out_dtype=out_dtype, status=status)

    @staticmethod
    def backward(ctx, d_out):
        rows, weight, offsets = ctx.saved_tensors
        d = d_out.to(torch.bfloat16)
        d_rows = d_weight = None
        if ctx.needs_input_grad[0]:
            d_rows = grouped_mm_forward(d, weight.transpose(1, 2), offsets, status=ctx.status)
        if ctx.needs_input_grad[1]:
            d_weight = grouped_mm_weight_grad(rows, d, offsets, weight, status=ctx.status)
        return (*first_order_only("grouped_mm", (d_rows, d_weight), (rows, weight, d_out)), None, None, None)


def grouped_mm(rows, weight, offsets, *, out_dtype=None, status=None):
    """grouped_mm_forward with gradients for rows and weight (of a float32 result rounded to bfloat16
    first: the products take no wider ones). status: of both directions."""
    return GroupedMMFunction.apply(rows, weight, offsets, out_dtype, status)
