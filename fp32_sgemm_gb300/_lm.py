"""Language-model operators on torch tensors: the C ABI of
include/sgemm_gb300_lm.h.

Every function takes float32, float16 or bfloat16 CUDA tensors (the same type
for all matrices of a call) with any row pitch (stride(-1) == 1), enqueues its
work on torch's current stream (or `stream`) and returns new tensors unless
`out` is given.  A call's workspace comes from torch's allocator and is its
own, so calls on several streams or from several threads need no handles of
their own, and calls can be captured with torch.cuda.graph; a `handle` (the
device's default one otherwise) carries the wait limit and the error word.
The checks and the calls are in csrc/lm_binding.cpp.

grouped_gemm() and linear_cross_entropy() are differentiable in x and w: where
gradients are recorded and one of them requires one, the result carries a graph
whose backward pass makes the gradient calls below, on the stream current there.
(A result in `out` carries none.)  What has no gradient here, the products with
4-bit weights and lse by itself, says so when one is asked for.
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


def _handle(x, handle):
    if handle is not None:
        return handle
    try:
        index = x.get_device()
    except AttributeError:
        raise TypeError("x must be a torch.Tensor") from None
    if index < 0:
        raise ValueError("x must be a CUDA tensor")
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
