"""PyTorch entry points of the operators beside the fused MoE-FFN layer (include/mm_ops.h).

Training and prompts:

    n            = residual_norm(x, None, pre_weight=w)[1]      # the norm before a block
    logits       = n @ router_weight.T                          # the router's product
    ids, weights, prob_sum, lse = moe_router(logits, k, stats=True)
    f            = hyper_mega_moe(n, ids, weights, up, down)    # torch_api
    x, n         = residual_norm(x, f, post_weight=..., gate=..., pre_weight=...)

A few tokens at a time (inference):

    layer = MoEDecoder(up, down, k=8, router_weight=router_weight)   # once per layer
    f     = layer(n)                                                 # router, experts, sum

`residual_norm` and `moe_router` are differentiable once (a second derivative is refused); the
`*_forward` / `*_backward` functions are the calls they make. Argument marshalling only: shapes and
types are checked, non-contiguous tensors are copied to contiguous ones, and everything else runs in
libmm.so on the current stream of the tensors' device, which becomes the current one for the call if
it is not.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._first_order import first_order_only

_TYPE = {torch.bfloat16: _abi.MM_BF16, torch.float32: _abi.MM_FP32}
_SCORE = {"softmax": _abi.MM_SCORE_SOFTMAX, "sigmoid": _abi.MM_SCORE_SIGMOID}


def _stream(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contiguous(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _aligned(t):
    """A contiguous tensor on a 16-byte boundary, as TMA wants it: `t` itself if it is one."""
    t = _contiguous(t)
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _type(name, t):
    try:
        return _TYPE[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}") from None


def _on_gpu(op, first, *others):
    if not first.is_cuda:
        raise ValueError(f"{op} runs on a CUDA device only (no CPU path)")
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"{op}: all tensors must be on {first.device}")


def _elsewhere(t):
    """Whether t is on a GPU that is not the current one (the library launches on the current one)."""
    device = t.get_device()
    return device >= 0 and device != torch._C._cuda_getDevice()


class _Plans(dict):
    """What a call of some signature (shapes, types, devices, options) needs: checked and described
    once. Small calls cost less than their checks."""

    def remember(self, key, plan):
        if len(self) >= 1024:
            self.clear()
        self[key] = plan
        return plan


def _sig(t):
    return None if t is None else (t.shape, t.dtype, t.get_device())


# ------------------------------------------------------------------------------- residual_norm

_norm_plans = _Plans()


def _norm_plan(residual, branch, post_weight, pre_weight, gate, residual_scale, eps, block_type,
               key):
    """Checks the inputs; (address of the descriptor, backward workspace bytes, descriptor).
    block_type: normed's type where there is no branch."""
    _on_gpu("residual_norm", residual, branch, post_weight, pre_weight, gate)
    if residual.dim() != 2:
        raise ValueError("expected residual[T,H]")
    T, H = residual.shape
    if branch is None:
        if post_weight is not None or gate is not None:
            raise ValueError("post_weight and gate belong to a branch")
    elif branch.shape != residual.shape:
        raise ValueError("expected branch[T,H] of residual's shape")
    params = [t for t in (post_weight, pre_weight, gate) if t is not None]
    for name, t in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if t is not None and t.shape != (H,):
            raise ValueError(f"expected {name}[H]")
    groups = 0
    if gate is not None:
        groups = 1 if gate.dim() == 1 else gate.shape[0]
        if gate.dim() not in (1, 2) or gate.shape[-1] != H or groups < 1 or T % groups:
            raise ValueError("expected gate[H] or gate[G,H] with T a multiple of G")
    if any(p.dtype != params[0].dtype for p in params):
        raise TypeError("post_weight, pre_weight and gate must have one dtype")
    stream = _type("residual", residual)
    block = _type("branch", branch) if branch is not None else stream
    if block > stream:
        raise TypeError("a bfloat16 residual needs a bfloat16 branch")
    if branch is None and block_type is not None:
        block = _TYPE.get(block_type, 2)
        if block > stream:
            raise TypeError("normed must be no wider than the residual")
    elif pre_weight is not None and block_type is not None and _TYPE.get(block_type) != block:
        raise TypeError("normed has the branch's dtype: normed_dtype is for calls without a branch")
    param = _type("parameters", params[0]) if params else stream
    d = _abi.mm_norm_desc(T, H, groups, stream, block, param, residual_scale, eps)
    at = ctypes.addressof(d)
    return _norm_plans.remember(
        key, (at, int(_abi._lib().mm_residual_norm_workspace_size(at)), d))


def residual_norm_forward(residual, branch=None, *, post_weight=None, pre_weight=None, gate=None,
                          residual_scale=1.0, eps=1e-6, normed_dtype=None):
    """(residual_out, normed): r' = residual_scale * r + gate * rmsnorm(branch, post_weight) and
    rmsnorm(r', pre_weight) (None without a pre_weight). `gate` is [H] (per channel) or [G, H],
    row g for the g-th T / G tokens. normed has the branch's type; without a branch
    `normed_dtype` (the residual's if None)."""
    if _elsewhere(residual):
        with torch.cuda.device(residual.device):
            return residual_norm_forward(
                residual, branch, post_weight=post_weight, pre_weight=pre_weight, gate=gate,
                residual_scale=residual_scale, eps=eps, normed_dtype=normed_dtype)
    residual_scale, eps = float(residual_scale), float(eps)
    key = (_sig(residual), _sig(branch), _sig(post_weight), _sig(pre_weight), _sig(gate),
           residual_scale, eps, normed_dtype)
    plan = _norm_plans.get(key) or _norm_plan(residual, branch, post_weight, pre_weight, gate,
                                              residual_scale, eps, normed_dtype, key)
    residual, branch, gate = _contiguous(residual), _contiguous(branch), _contiguous(gate)
    post_weight, pre_weight = _contiguous(post_weight), _contiguous(pre_weight)
    out = torch.empty_like(residual)
    normed = None
    if pre_weight is not None:
        if branch is not None:
            normed = torch.empty_like(branch)
        else:
            normed = torch.empty_like(residual, dtype=normed_dtype or residual.dtype)
    _abi.check(_abi._lib().mm_residual_norm_forward(
        plan[0], residual.data_ptr(), _ptr(branch), _ptr(post_weight), _ptr(pre_weight), _ptr(gate),
        out.data_ptr(), _ptr(normed), _stream(residual)), "mm_residual_norm_forward")
    return out, normed


def residual_norm_backward(residual_out, branch, d_residual_out, d_normed, *, post_weight=None,
                           pre_weight=None, gate=None, residual_scale=1.0, eps=1e-6):
    """(d_residual, d_branch, d_post_weight, d_pre_weight, d_gate) at the forward's residual_out
    and branch; None in the place of what was not given. d_residual_out may be None (zero);
    d_normed is given exactly if pre_weight is."""
    if _elsewhere(residual_out):
        with torch.cuda.device(residual_out.device):
            return residual_norm_backward(
                residual_out, branch, d_residual_out, d_normed, post_weight=post_weight,
                pre_weight=pre_weight, gate=gate, residual_scale=residual_scale, eps=eps)
    residual_scale, eps = float(residual_scale), float(eps)
    key = (_sig(residual_out), _sig(branch), _sig(post_weight), _sig(pre_weight), _sig(gate),
           residual_scale, eps, _sig(d_residual_out), _sig(d_normed))
    plan = _norm_plans.get(key)
    if plan is None:
        if (d_normed is None) != (pre_weight is None):
            raise ValueError("give d_normed exactly if pre_weight is given")
        if d_residual_out is None and d_normed is None:
            raise ValueError("give d_residual_out or d_normed")
        _on_gpu("residual_norm", residual_out, d_residual_out, d_normed)
        if d_residual_out is not None and (d_residual_out.shape != residual_out.shape
                                           or d_residual_out.dtype != residual_out.dtype):
            raise ValueError("d_residual_out must have residual_out's shape and dtype")
        if d_normed is not None:
            _type("d_normed", d_normed)
            if d_normed.shape != residual_out.shape:
                raise ValueError("d_normed must have residual_out's shape")
            if branch is not None and d_normed.dtype != branch.dtype:
                raise TypeError("d_normed must have the branch's dtype")
        plan = _norm_plan(residual_out, branch, post_weight, pre_weight, gate, residual_scale, eps,
                          None if d_normed is None else d_normed.dtype, key)
    residual_out, branch, gate = _contiguous(residual_out), _contiguous(branch), _contiguous(gate)
    d_residual_out, d_normed = _contiguous(d_residual_out), _contiguous(d_normed)
    post_weight, pre_weight = _contiguous(post_weight), _contiguous(pre_weight)
    like = torch.empty_like
    dr = like(residual_out)
    df = None if branch is None else like(branch)
    dpost = None if post_weight is None else like(post_weight)
    dpre = None if pre_weight is None else like(pre_weight)
    dg = None if gate is None else like(gate)
    ws = torch.empty(plan[1], dtype=torch.uint8, device=residual_out.device)
    _abi.check(_abi._lib().mm_residual_norm_backward(
        plan[0], residual_out.data_ptr(), _ptr(branch), _ptr(post_weight), _ptr(pre_weight),
        _ptr(gate), _ptr(d_residual_out), _ptr(d_normed), dr.data_ptr(), _ptr(df), _ptr(dpost),
        _ptr(dpre), _ptr(dg), ws.data_ptr(), plan[1], _stream(residual_out)),
        "mm_residual_norm_backward")
    return dr, df, dpost, dpre, dg


class ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, branch, post_weight, pre_weight, gate, residual_scale, eps, ndt):
        out, normed = residual_norm_forward(
            residual, branch, post_weight=post_weight, pre_weight=pre_weight, gate=gate,
            residual_scale=residual_scale, eps=eps, normed_dtype=ndt)
        ctx.save_for_backward(out, branch, post_weight, pre_weight, gate)
        ctx.scale, ctx.eps = residual_scale, eps
        ctx.set_materialize_grads(False)
        ctx.ndt = None if normed is None else normed.dtype
        return out, normed

    @staticmethod
    def backward(ctx, d_out, d_normed):
        out, branch, post_weight, pre_weight, gate = ctx.saved_tensors
        if pre_weight is not None and d_normed is None:  # the normed output was not used
            d_normed = torch.zeros(out.shape, dtype=ctx.ndt, device=out.device)
        if d_out is None and d_normed is None:
            return (None,) * 8
        dr, df, dpost, dpre, dg = residual_norm_backward(
            out, branch, d_out, d_normed, post_weight=post_weight, pre_weight=pre_weight,
            gate=gate, residual_scale=ctx.scale, eps=ctx.eps)
        return (*first_order_only("residual_norm", (dr, df, dpost, dpre, dg),
                                  (*ctx.saved_tensors, d_out, d_normed)), None, None, None)


def residual_norm(residual, branch=None, *, post_weight=None, pre_weight=None, gate=None,
                  residual_scale=1.0, eps=1e-6, normed_dtype=None):
    """residual_norm_forward with gradients for residual, branch, both weights and the gate."""
    return ResidualNormFunction.apply(residual, branch, post_weight, pre_weight, gate,
                                      residual_scale, eps, normed_dtype)


# ------------------------------------------------------------------------------- router

_router_plans = _Plans()


def _router_plan(logits, k, score, normalize, scale, bias, key):
    """Checks the inputs; (address of the descriptor, workspace bytes, T, E, device, descriptor)."""
    _on_gpu("the router", logits, bias)
    if logits.dim() != 2:
        raise ValueError("expected logits[T,E]")
    if score not in _SCORE:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    T, E = logits.shape
    if not 1 <= k <= E:
        raise ValueError("expected 1 <= k <= E")
    if bias is not None and (bias.shape != (E,) or bias.dtype != torch.float32):
        raise ValueError("expected bias[E] in float32")
    d = _abi.mm_router_desc(T, E, k, _type("logits", logits), _SCORE[score], int(normalize),
                            scale)
    at = ctypes.addressof(d)
    ws = int(_abi._lib().mm_router_workspace_size(at))
    return _router_plans.remember(key, (at, ws, T, E, logits.device, d))


def router_forward(logits, k, *, bias=None, score="softmax", normalize=True, scale=1.0,
                   stats=False):
    """(topk_ids int32 [T,k], topk_weights fp32 [T,k], prob_sum fp32 [E], lse fp32 [T]); the last
    two are None without `stats`. See mm_ops.h for the definitions. `bias` fp32 [E] takes part in
    the selection only."""
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return router_forward(logits, k, bias=bias, score=score, normalize=normalize,
                                  scale=scale, stats=stats)
    k, normalize, scale = int(k), bool(normalize), float(scale)
    key = (_sig(logits), k, score, normalize, scale, _sig(bias))
    at, ws_bytes, T, E, dev, _ = _router_plans.get(key) or _router_plan(
        logits, k, score, normalize, scale, bias, key)
    logits, bias = _contiguous(logits), _contiguous(bias)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    prob_sum = lse = ws = None
    if stats:
        prob_sum = torch.empty(E, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _abi.check(_abi._lib().mm_router_forward(
        at, logits.data_ptr(), _ptr(bias), ids.data_ptr(), weights.data_ptr(), _ptr(prob_sum),
        _ptr(lse), _ptr(ws), ws_bytes if stats else 0, _stream(logits)), "mm_router_forward")
    return ids, weights, prob_sum, lse


def router_backward(logits, topk_ids, d_weights, d_prob_sum=None, d_lse=None, *, score="softmax",
                    normalize=True, scale=1.0):
    """d_logits (the logits' type) from the gradients of topk_weights, prob_sum and lse."""
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return router_backward(logits, topk_ids, d_weights, d_prob_sum, d_lse, score=score,
                                   normalize=normalize, scale=scale)
    normalize, scale = bool(normalize), float(scale)
    key = (_sig(logits), _sig(topk_ids), _sig(d_weights), _sig(d_prob_sum), _sig(d_lse), score,
           normalize, scale)
    plan = _router_plans.get(key)
    if plan is None:
        if topk_ids.dim() != 2 or topk_ids.dtype != torch.int32:
            raise ValueError("expected topk_ids[T,k] in int32")
        _on_gpu("the router", logits, topk_ids, d_weights, d_prob_sum, d_lse)
        T, E = logits.shape if logits.dim() == 2 else (-1, -1)
        for name, t, shape in (("topk_ids", topk_ids, (T, topk_ids.shape[1])),
                               ("d_weights", d_weights, tuple(topk_ids.shape)),
                               ("d_prob_sum", d_prob_sum, (E,)), ("d_lse", d_lse, (T,))):
            if t is not None and tuple(t.shape) != shape:
                raise ValueError(f"expected {name} of shape {shape}")
            if t is not None and t is not topk_ids and t.dtype != torch.float32:
                raise TypeError(f"{name} must be float32")
        plan = _router_plan(logits, topk_ids.shape[1], score, normalize, scale, None, key)
    logits, topk_ids, d_weights = _contiguous(logits), _contiguous(topk_ids), _contiguous(d_weights)
    d_prob_sum, d_lse = _contiguous(d_prob_sum), _contiguous(d_lse)
    dz = torch.empty_like(logits)
    _abi.check(_abi._lib().mm_router_backward(
        plan[0], logits.data_ptr(), topk_ids.data_ptr(), d_weights.data_ptr(), _ptr(d_prob_sum),
        _ptr(d_lse), dz.data_ptr(), _stream(logits)), "mm_router_backward")
    return dz


class RouterFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, score, normalize, scale, stats):
        ids, weights, prob_sum, lse = router_forward(
            logits, k, bias=bias, score=score, normalize=normalize, scale=scale, stats=stats)
        ctx.save_for_backward(logits, ids)
        ctx.how = dict(score=score, normalize=normalize, scale=scale)
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return ids, weights, prob_sum, lse

    @staticmethod
    def backward(ctx, _, d_weights, d_prob_sum, d_lse):
        logits, ids = ctx.saved_tensors
        if d_weights is None and d_prob_sum is None and d_lse is None:
            return (None,) * 7
        if d_weights is None:
            d_weights = torch.zeros(ids.shape, dtype=torch.float32, device=ids.device)
        dz = router_backward(logits, ids, d_weights, d_prob_sum, d_lse, **ctx.how)
        return (*first_order_only("moe_router", (dz,), (logits, d_weights, d_prob_sum, d_lse)),
                *(None,) * 6)


def moe_router(logits, k, *, bias=None, score="softmax", normalize=True, scale=1.0, stats=False):
    """router_forward with a gradient for the logits (through topk_weights, prob_sum and lse)."""
    return RouterFunction.apply(logits, k, bias, score, normalize, scale, stats)


# ------------------------------------------------------------------------------- decode

def quantize_expert_weights(w):
    """(q float8_e4m3fn of w's shape, scale fp32 [..., ceil(R/128), ceil(C/128)]) of bf16 matrices
    w [..., R, C]: one scale per 128 x 128 block (mm_quantize_blocks)."""
    if _elsewhere(w):
        with torch.cuda.device(w.device):
            return quantize_expert_weights(w)
    if w.dim() < 2 or w.dtype != torch.bfloat16 or not w.is_cuda:
        raise ValueError("expected bfloat16 matrices [..., R, C] on a CUDA device")
    w = _aligned(w)
    *lead, R, C = w.shape
    n = w.numel() // (R * C) if R * C else 0
    q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
    scale = torch.empty((*lead, -(-R // 128), -(-C // 128)), dtype=torch.float32, device=w.device)
    _abi.check(_abi._lib().mm_quantize_blocks(n, R, C, w.data_ptr(), q.data_ptr(), scale.data_ptr(),
                                              _stream(w)), "mm_quantize_blocks")
    return q, scale


def _padded(t, rows, cols):
    """A copy of a matrix or matrices with zero rows and columns added (1-byte types as bytes)."""
    as_bytes = t.view(torch.uint8) if t.element_size() == 1 else t
    return torch.nn.functional.pad(as_bytes, (0, cols, 0, rows)).view(t.dtype)


class MoEDecoder:
    """The whole MoE layer for up to `max_tokens` (<= 64) tokens a call, inference only: keeps the
    weights, their description and a workspace between calls.

    up_proj_weight [E,H,2I], down_proj_weight [E,I,H]: bf16, or float8_e4m3fn with up_scale /
    down_scale (quantize_expert_weights). With router_weight [E,H] (bf16 or fp32) a call takes the
    tokens alone and selects k experts as moe_router does (router_bias fp32 [E], score, normalize,
    scale); without one it takes topk_ids and topk_weights [T,k]. `shared`: (up [H,2Is],
    down [Is,H]) of a shared expert, and their two scales for 8-bit weights (or None, None).

    The decoder reads the given tensors in every call, so that updates of the weights take effect in
    the next one. Two kinds it has to copy: tensors that are not contiguous (matrices: from a 16-byte
    boundary on), and, as mm_decode takes H in multiples of 8 (8-bit weights: 16), those of another H,
    with zeros up to the next multiple (x is padded and y cut in every call). A call takes over the
    updates of copied tensors that autograd counts (in-place operations, an optimizer's step); after
    others (through `.data` or a raw pointer, of inference tensors, or before a captured graph's
    replay) call reload().

    Calls run on the current stream and use the one workspace: one decoder serves one stream."""

    def __init__(self, up_proj_weight, down_proj_weight, *, k, up_scale=None, down_scale=None,
                 router_weight=None, router_bias=None, score="softmax", normalize=True, scale=1.0,
                 shared=None, max_tokens=64):
        up, down = up_proj_weight, down_proj_weight
        if up.dim() != 3 or down.dim() != 3:
            raise ValueError("expected up_proj_weight[E,H,2I] and down_proj_weight[E,I,H]")
        E, H, I2 = up.shape
        I = I2 // 2
        if I2 % 2 or down.shape != (E, I, H):
            raise ValueError("expected up_proj_weight[E,H,2I] and down_proj_weight[E,I,H]")
        if up.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or down.dtype != up.dtype:
            raise TypeError("expert weights must be bfloat16 or float8_e4m3fn")
        fp8 = up.dtype == torch.float8_e4m3fn
        if score not in _SCORE:
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        shared = tuple(shared) + (None,) * (4 - len(shared)) if shared is not None else (None,) * 4
        s_up, s_down, s_us, s_ds = shared
        Is = 0
        if (s_up is None) != (s_down is None):
            raise ValueError("give both shared-expert weights or neither")
        if s_up is not None:
            Is = s_down.shape[0]
            if s_up.shape != (H, 2 * Is) or s_down.shape != (Is, H):
                raise ValueError("expected shared weights [H,2Is] and [Is,H]")
            if s_up.dtype != up.dtype or s_down.dtype != up.dtype:
                raise TypeError("shared-expert weights must have the experts' type")

        def blocks(n):
            return -(-n // 128)

        for name, t, shape in (("up_scale", up_scale, (E, blocks(H), blocks(I2))),
                               ("down_scale", down_scale, (E, blocks(I), blocks(H))),
                               ("shared up scale", s_us, (blocks(H), blocks(2 * Is))),
                               ("shared down scale", s_ds, (blocks(Is), blocks(H)))):
            wanted = fp8 and (Is > 0 or not name.startswith("shared"))
            if (t is not None) != wanted:
                raise ValueError(f"{name} goes with float8_e4m3fn weights, and only with them")
            if t is not None and (t.shape != shape or t.dtype != torch.float32):
                raise ValueError(f"expected {name} of shape {shape} in float32")
        if router_weight is not None and router_weight.shape != (E, H):
            raise ValueError("expected router_weight[E,H]")
        if router_bias is not None and (router_weight is None or router_bias.shape != (E,)
                                        or router_bias.dtype != torch.float32):
            raise ValueError("expected router_bias[E] in float32, with a router_weight")
        if not 1 <= k <= E:
            raise ValueError("expected 1 <= k <= E")
        given = [up, down, up_scale, down_scale, s_up, s_down, s_us, s_ds, router_weight, router_bias]
        _on_gpu("MoEDecoder", *given)
        kept = list(given)
        self._pad = -H % (16 if fp8 else 8)
        with torch.inference_mode(False), torch.no_grad():  # copies can be renewed from anywhere
            if self._pad:  # (the blocks of 128 that have scales stay the same)
                for i, (rows, cols) in {0: (self._pad, 0), 1: (0, self._pad), 4: (self._pad, 0),
                                        5: (0, self._pad), 8: (0, self._pad)}.items():
                    if kept[i] is not None:
                        kept[i] = _padded(kept[i], rows, cols)
            kept = [_aligned(t) if i in (0, 1, 4, 5, 8) else _contiguous(t) for i, t in enumerate(kept)]
        self._kept = kept
        self._copies = [(g, t) for g, t in zip(given, kept) if t is not g]
        self._versions = self._count_updates()
        self._weights = _abi.mm_decode_weights(*[_ptr(t) for t in kept])
        self._weights_at = ctypes.addressof(self._weights)
        self.routes = router_weight is not None
        self.k, self.H, self.device, self.max_tokens = int(k), H, up.device, int(max_tokens)
        rt = _type("router_weight", router_weight) if self.routes else _abi.MM_BF16
        self._fields = (Is, _abi.MM_E4M3 if fp8 else _abi.MM_BF16, rt, _SCORE[score], int(normalize),
                        float(scale))
        self._dims = (H + self._pad, I, E)
        self._descs = {}
        nbytes = self._desc(self.max_tokens)[1]
        if nbytes == 0:
            raise ValueError(f"unsupported sizes max_tokens={max_tokens} H={H} I={I} E={E} k={k} Is={Is}")
        self._ws = torch.empty(nbytes, dtype=torch.uint8, device=up.device)

    def _count_updates(self):
        return [0 if g.is_inference() else g._version for g, _ in self._copies]

    @torch.no_grad()
    def reload(self):
        """Takes over the present values of the given tensors that the decoder keeps copies of."""
        self._versions = self._count_updates()
        for given, copy in self._copies:
            if given.element_size() == 1:  # 8-bit types have few operations of their own
                given, copy = given.view(torch.uint8), copy.view(torch.uint8)
            copy[tuple(slice(n) for n in given.shape)].copy_(given)

    def _desc(self, T):
        """(address of the descriptor of a call with T tokens, its workspace bytes)."""
        got = self._descs.get(T)
        if got is None:
            H, I, E = self._dims
            d = _abi.mm_decode_desc(_abi.dims(T, H, I, E, self.k), *self._fields)
            at = ctypes.addressof(d)
            got = self._descs[T] = (at, int(_abi._lib().mm_decode_workspace_size(at)), d)
        return got

    def _call(self, x, ids, weights):
        if _elsewhere(x):
            with torch.cuda.device(x.device):
                return self._call(x, ids, weights)
        if x.dim() != 2 or x.shape[1] != self.H or x.dtype != torch.bfloat16 or x.device != self.device:
            raise ValueError(f"expected x[T,{self.H}] in bfloat16 on {self.device}")
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens in a decoder for {self.max_tokens}")
        if self._copies and self._count_updates() != self._versions:
            self.reload()
        x = torch.nn.functional.pad(x, (0, self._pad)) if self._pad else _aligned(x)
        y = torch.empty_like(x)
        _abi.check(_abi._lib().mm_decode(
            self._desc(T)[0], self._weights_at, x.data_ptr(), _ptr(ids), _ptr(weights), y.data_ptr(),
            self._ws.data_ptr(), self._ws.numel(), _stream(x)), "mm_decode")
        return y[:, :self.H].contiguous() if self._pad else y

    def __call__(self, x, topk_ids=None, topk_weights=None):
        """y [T,H] bf16 for x [T,H] bf16."""
        if self.routes:
            if topk_ids is not None or topk_weights is not None:
                raise ValueError("this decoder routes by itself (it has a router_weight)")
            return self._call(x, None, None)
        if topk_ids is None or topk_weights is None:
            raise ValueError("a decoder without a router_weight needs topk_ids and topk_weights")
        if topk_ids.shape != (x.shape[0], self.k) or topk_weights.shape != topk_ids.shape:
            raise ValueError(f"expected topk_ids and topk_weights [T,{self.k}]")
        if topk_ids.dtype not in (torch.int32, torch.int64):
            raise TypeError("topk_ids must be int32 or int64")
        if topk_ids.device != self.device or topk_weights.device != self.device:
            raise ValueError(f"expected topk_ids and topk_weights on {self.device}")
        if topk_ids.dtype == torch.int64:  # (a number beyond 32 bits must not become another expert's)
            topk_ids = topk_ids.clamp(-1, self._dims[2])
        ids = _contiguous(topk_ids.to(torch.int32))
        return self._call(x, ids, _contiguous(topk_weights.to(torch.float32)))

    def with_routing(self, x):
        """(y, topk_ids int32 [T,k], topk_weights fp32 [T,k]) of a decoder that routes."""
        if not self.routes:
            raise ValueError("this decoder has no router_weight")
        ids = torch.empty((x.shape[0], self.k), dtype=torch.int32, device=self.device)
        weights = torch.empty((x.shape[0], self.k), dtype=torch.float32, device=self.device)
        return self._call(x, ids, weights), ids, weights

    def status(self) -> int:
        """Waits for the current stream and returns the last call's status (MM_OK,
        MM_ERR_BAD_EXPERT_ID or MM_ERR_TIMEOUT)."""
        with torch.cuda.device(self.device):
            return _abi.mm_get_status(self._ws.data_ptr(), _stream(self._ws))
