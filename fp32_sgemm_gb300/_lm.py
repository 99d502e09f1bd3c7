"""Language-model operators on torch tensors: the C ABI of
include/sgemm_gb300_lm.h.

Every function takes float32, float16 or bfloat16 CUDA tensors (the same type
for all matrices of a call; weights in 4 or 8 bits beside them) with any row
pitch (stride(-1) == 1), enqueues its work on torch's current stream (or
`stream`) and returns new tensors unless `out` is given.  A call's workspace comes from torch's allocator and is its
own, so calls on several streams or from several threads need no handles of
their own, and calls can be captured with torch.cuda.graph; a `handle` (the
device's default one otherwise) carries the wait limit and the error word.
The checks and the calls are in csrc/lm_binding.cpp.

grouped_gemm() and linear_cross_entropy() are differentiable in x and w,
route_topk() in the logits, expert_dispatch() in x and expert_combine() in rows
and weights: where gradients are recorded and one of them requires one, the result
carries a graph whose backward pass makes the gradient calls below, on the stream
current there.  (A result in `out` carries neither graph nor tangent, nor do those of
the gradient calls themselves.)  What has no gradient here, the products with 4-bit
and 8-bit weights, int8_quantize() and lse by itself, says so when one is asked for;
so do all of them of an operand with a tangent (forward mode).
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _build
from ._binding import _default_handles, default_handle, load_library


def _load():
    import importlib.machinery
    import importlib.util
    import os

    load_library()
    if not os.path.exists(_build.LM_BINDING_PATH):
        raise RuntimeError(f"{_build.LM_BINDING_PATH} is not built; run fp32_sgemm_gb300.build()")
    loader = importlib.machinery.ExtensionFileLoader("fp32_sgemm_gb300._lm_binding", _build.LM_BINDING_PATH)
    spec = importlib.util.spec_from_file_location("fp32_sgemm_gb300._lm_binding", _build.LM_BINDING_PATH,
                                                  loader=loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    return module


_c = _load()


def _handle(x, handle, name="x"):
    if handle is not None:
        return handle
    try:
        index = x.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _default_handles.get(index) or default_handle(index)


class _GroupedGemm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, group_ends, trans_w, handle, stream):
        y = _c.grouped_gemm(x, w, group_ends, trans_w, None, handle, stream)
        ctx.save_for_backward(x, w, group_ends)
        ctx.trans_w, ctx.handle = trans_w, handle
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, group_ends = ctx.saved_tensors
        dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = _c.grouped_gemm(dy, w, group_ends, not ctx.trans_w, None, ctx.handle, None)
        if ctx.needs_input_grad[1]:
            dw = _c.grouped_gemm_weight_grad(x, dy, group_ends, ctx.trans_w, None, ctx.handle, None)
        return dx, dw, None, None, None, None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, handle, stream):
        loss, lse = _c.linear_cross_entropy(x, w, target, handle, stream)
        ctx.save_for_backward(x, w, target, lse)
        ctx.handle = handle
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dlse):
        if dlse is not None:
            raise NotImplementedError("linear_cross_entropy has no gradient by lse, only by loss")
        if dloss is None:
            return None, None, None, None, None
        dx, dw = _c.linear_cross_entropy_grad(*ctx.saved_tensors, dloss.contiguous(), ctx.handle, None)
        return (dx if ctx.needs_input_grad[0] else None, dw if ctx.needs_input_grad[1] else None, None, None, None)


class _W4Gemm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, q, scales, zeros, handle, stream):
        return _c.w4_gemm(x, q, scales, zeros, None, handle, stream)

    @staticmethod
    def backward(ctx, dy):
        raise NotImplementedError("w4_gemm has no gradient")


class _Int8Quantize(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, handle, stream):
        q, scales = _c.int8_quantize(x, handle, stream)
        ctx.mark_non_differentiable(q)
        return q, scales

    @staticmethod
    def backward(ctx, dq, dscales):
        raise NotImplementedError("int8_quantize has no gradient")


class _Int8Gemm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, scales, x_scales, group_ends, dtype, handle, stream):
        return _c.int8_gemm(x, w, scales, x_scales, group_ends, dtype, None, handle, stream)

    @staticmethod
    def backward(ctx, dy):
        raise NotImplementedError("int8_gemm and int8_grouped_gemm have no gradient")


class _RouteTopK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, normalize, handle, stream):
        weights, experts = _c.route_topk(logits, k, normalize, handle, stream)
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        ctx.normalize, ctx.handle = normalize, handle
        return weights, experts

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, dexperts):
        logits, experts = ctx.saved_tensors
        return (_c.route_topk_grad(logits, experts, dweights.contiguous(), ctx.normalize, ctx.handle, None),
                None, None, None, None)


class _ExpertDispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, experts, num_experts, handle, stream):
        rows, slots, group_ends = _c.expert_dispatch(x, experts, num_experts, handle, stream)
        ctx.save_for_backward(slots)
        ctx.mark_non_differentiable(slots, group_ends)
        ctx.handle = handle
        return rows, slots, group_ends

    @staticmethod
    @once_differentiable
    def backward(ctx, drows, dslots, dends):
        slots, = ctx.saved_tensors
        return _c.expert_combine(drows.contiguous(), slots, None, None, ctx.handle, None), None, None, None, None


class _ExpertCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, slots, weights, handle, stream):
        y = _c.expert_combine(rows, slots, weights, None, handle, stream)
        # (What only the weights' gradient reads is kept for that alone.)
        ctx.save_for_backward(rows if ctx.needs_input_grad[2] else None, slots, weights)
        ctx.handle = handle
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, slots, weights = ctx.saved_tensors
        drows, dweights = _c.expert_combine_grad(dy.contiguous(), rows, slots, weights, ctx.needs_input_grad[0],
                                                 ctx.needs_input_grad[2], ctx.handle, None)
        return drows, None, dweights, None, None


def grouped_gemm(x, w, group_ends, *, trans_w: bool = False, out=None, handle=None, stream=None):
    """y[t] = x[t] @ op(w[g]) for every row t of group g; returns y [T, N].

    x [T, K]: rows sorted by group; w [G, K, N], or [G, N, K] with trans_w
    (op transposes); group_ends [G] int32 on the device: the row at which
    each group ends (a group may be empty).  Rows behind the last end get
    zeros.  The gradient by x is ``grouped_gemm(dy, w, group_ends,
    trans_w=not trans_w)``; that by w, grouped_gemm_weight_grad().
    """
    handle = _handle(x, handle)
    y = _c.grouped_gemm(x, w, group_ends, trans_w, out, handle, stream)
    return _GroupedGemm.apply(x, w, group_ends, trans_w, handle, stream) if y is None else y


def grouped_gemm_weight_grad(x, dy, group_ends, *, trans_w: bool = False, out=None, handle=None,
                             stream=None):
    """Gradient of grouped_gemm() by w: dw[g] = x_g^T @ dy_g, [G, K, N]
    (with trans_w dy_g^T @ x_g, [G, N, K]); zero for an empty group."""
    return _c.grouped_gemm_weight_grad(x, dy, group_ends, trans_w, out, _handle(x, handle), stream)


def linear_cross_entropy(x, w, target, *, handle=None, stream=None):
    """Cross entropy of the logits x @ w.T, which are never kept.

    x [T, D], w [V, D], target [T] int64 (outside [0, V): not counted, loss
    0); returns (loss, lse), float32 [T]: lse[t] = log sum_v exp(x_t . w_v),
    loss[t] = lse[t] - x_t . w_target.
    """
    handle = _handle(x, handle)
    both = _c.linear_cross_entropy(x, w, target, handle, stream)
    return _LinearCrossEntropy.apply(x, w, target, handle, stream) if both is None else both


def linear_cross_entropy_grad(x, w, target, lse, dloss, *, handle=None, stream=None):
    """Gradients (dx, dw) of linear_cross_entropy() for the gradient dloss
    [T] (float32) by each token's loss; lse from the forward call."""
    return _c.linear_cross_entropy_grad(x, w, target, lse, dloss, _handle(x, handle), stream)


def w4_gemm(x, q, scales, zeros=None, *, out=None, handle=None, stream=None):
    """y = x @ W.T for 4-bit weights with group scales; returns y [M, N].

    x [M, K] (a few rows); q [N, K // 2] uint8, column 2 i of W in the low
    four bits of byte i, column 2 i + 1 in the high four; scales [N, groups]
    of x's type and zeros [N, groups] uint8 (0 to 255) or None (8 everywhere), groups of
    K // groups = 32, 64 or 128 columns:
    W[n, k] = scales[n, k // group] * (q[n, k] - zeros[n, k // group]).
    """
    handle = _handle(x, handle)
    y = _c.w4_gemm(x, q, scales, zeros, out, handle, stream)
    return _W4Gemm.apply(x, q, scales, zeros, handle, stream) if y is None else y


def route_topk(logits, k, *, normalize: bool = True, handle=None, stream=None):
    """A router's choice: the k largest of each token's logits [T, E], in
    falling order, the lower index first among equals.

    Returns (weights, experts): float32 [T, k] softmax weights, over the chosen
    alone with normalize (they add up to 1) and over all E without; int64 [T, k].
    A logit of -inf is never chosen: where fewer than k are left the expert is -1
    and its weight 0.  Differentiable in logits; route_topk_grad() by itself.
    """
    handle = _handle(logits, handle, "logits")
    both = _c.route_topk(logits, k, normalize, handle, stream)
    return _RouteTopK.apply(logits, k, normalize, handle, stream) if both is None else both


def route_topk_grad(logits, experts, dweights, *, normalize: bool = True, handle=None, stream=None):
    """Gradient of route_topk() by the logits, [T, E], for its experts and the
    gradient dweights [T, k] (float32) by its weights."""
    return _c.route_topk_grad(logits, experts, dweights, normalize, _handle(logits, handle, "logits"), stream)


def expert_dispatch(x, experts, num_experts, *, handle=None, stream=None):
    """Tokens x [T, D] sorted by expert: experts [T, k] int64, as route_topk()
    gives them (what is outside [0, num_experts) is no expert).

    Returns (rows, slots, group_ends): rows [T * k, D], each expert's in the
    order of the choices, those of no expert behind the last end and zero; slots
    [T, k] int32, the row of each choice (~r for a row r of no expert); group_ends
    [num_experts] int32, as grouped_gemm() takes them.  Differentiable in x; the
    gradient is ``expert_combine(drows, slots)``.
    """
    handle = _handle(x, handle)
    parts = _c.expert_dispatch(x, experts, num_experts, handle, stream)
    return _ExpertDispatch.apply(x, experts, num_experts, handle, stream) if parts is None else parts


def expert_combine(rows, slots, weights=None, *, out=None, handle=None, stream=None):
    """y[t] = sum_j weights[t, j] * rows[slots[t, j]]; returns y [T, D].

    rows [T * k, D] and slots [T, k] as expert_dispatch() lays them out, weights
    [T, k] float32 or None (1).  A slot that names no row (a negative one, as of a
    choice of no expert or one that is dropped, or T * k and more) adds nothing; a
    row is named at most once.  Summed in float32 in the order of j.  Differentiable
    in rows and weights; expert_combine_grad() by itself.
    """
    handle = _handle(rows, handle, "rows")
    y = _c.expert_combine(rows, slots, weights, out, handle, stream)
    return _ExpertCombine.apply(rows, slots, weights, handle, stream) if y is None else y


def expert_combine_grad(dy, rows, slots, weights=None, *, handle=None, stream=None):
    """Gradients (drows [T * k, D], dweights [T, k] float32) of expert_combine()
    for the gradient dy [T, D] by y: drows[slots[t, j]] = weights[t, j] * dy[t], zeros
    for rows that no slot names (of one named twice undefined), dweights[t, j] = dy[t] .
    rows[slots[t, j]], 0 for a slot that names no row."""
    return _c.expert_combine_grad(dy, rows, slots, weights, True, True, _handle(rows, handle, "rows"), stream)


def int8_quantize(x, *, handle=None, stream=None):
    """Rows of x [T, K] as 8-bit integers with a scale each: (q, scales), int8
    [T, K] and float32 [T].

    scales[t] = max |x[t]| / 127, q = x / scales to the nearest integer (ties to
    even).  A row with an infinity or a NaN has scale NaN.  Weights are quantised
    the same way, a row per output channel.
    """
    handle = _handle(x, handle)
    both = _c.int8_quantize(x, handle, stream)
    return _Int8Quantize.apply(x, handle, stream) if both is None else both


def int8_gemm(x, w, scales, *, x_scales=None, dtype=None, out=None, handle=None, stream=None):
    """y = x @ w.T in 8-bit integers with scales for each token and channel;
    returns y [T, N].

    w [N, K] int8 with scales [N] float32; x [T, K] float32, float16 or bfloat16,
    each row of which becomes integers as by int8_quantize(), or int8 with
    x_scales [T] float32 (quantised once for several products).
    y[t, n] = x_scales[t] * scales[n] * (the exact sum of q[t, k] * w[n, k]), in
    dtype (x's if it has one).
    """
    handle = _handle(x, handle)
    y = _c.int8_gemm(x, w, scales, x_scales, None, dtype, out, handle, stream)
    return _Int8Gemm.apply(x, w, scales, x_scales, None, dtype, handle, stream) if y is None else y


def int8_grouped_gemm(x, w, scales, group_ends, *, x_scales=None, dtype=None, out=None, handle=None, stream=None):
    """int8_gemm() by group: w [G, N, K] int8 with scales [G, N], the rows of x
    sorted by group and group_ends [G] as for grouped_gemm().  Rows behind the
    last end get zeros."""
    if group_ends is None:
        raise TypeError("group_ends must be a torch.Tensor")
    handle = _handle(x, handle)
    y = _c.int8_gemm(x, w, scales, x_scales, group_ends, dtype, out, handle, stream)
    return _Int8Gemm.apply(x, w, scales, x_scales, group_ends, dtype, handle, stream) if y is None else y
