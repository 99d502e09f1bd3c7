"""Language-model operators on torch tensors: the C ABI of
include/sgemm_gb300_lm.h, argument marshalling only.

Every function takes float32, float16 or bfloat16 CUDA tensors (the same type
for all matrices of a call) with any row pitch (stride(-1) == 1), enqueues its
work on torch's current stream (or `stream`) and returns new tensors unless
`out` is given.
"""

from __future__ import annotations

import ctypes

from ._binding import _check, _stream_ptr, _torch, default_handle


def _type_of(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _mat(t, name, dtype, device, shape=None):
    """(ptr, pitch) of a row-major matrix of the call's type and device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = t.shape
    if rows > 0 and cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row major (stride(1) == 1)")
    pitch = t.stride(0) if rows > 1 else max(cols, 1)
    if rows > 1 and pitch < cols:
        raise ValueError(f"{name} has overlapping rows")
    return t.data_ptr(), max(pitch, 1)


def _stack(t, name, dtype, device, shape):
    """(ptr, pitch, stride) of a stack of row-major matrices."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[0] == 0:
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        return None, max(shape[2], 1), 0
    ptr, pitch = _mat(t[0], name, dtype, device)
    stride = t.stride(0) if t.shape[0] > 1 else 0
    if t.shape[0] > 1 and t[0].numel() and stride < (shape[1] - 1) * pitch + shape[2]:
        raise ValueError(f"{name} must hold one matrix per group (no broadcast)")
    return ptr, pitch, stride


def _ends(t, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError("group_ends must be an int32 tensor")
    if not t.is_cuda or t.device != device or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"group_ends must be a contiguous 1-D tensor on {device}")
    return t.data_ptr()


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _workspace(h, key, query):
    """Attach the workspace a call needs; `query` asks the library once per key."""
    need = h._ws_sizes.get(key)
    if need is None:
        n = ctypes.c_size_t()
        query(ctypes.byref(n))
        if len(h._ws_sizes) > 256:
            h._ws_sizes.clear()
        need = h._ws_sizes[key] = n.value
    h._ensure_workspace(need)


def grouped_gemm(x, w, group_ends, *, trans_w: bool = False, out=None, handle=None, stream=None):
    """y[t] = x[t] @ op(w[g]) for every row t of group g; returns y [T, N].

    x [T, K]: rows sorted by group; w [G, K, N], or [G, N, K] with trans_w
    (op transposes); group_ends [G] int32 on the device: the row at which
    each group ends (a group may be empty).  Rows behind the last end get
    zeros.  The gradient by x is ``grouped_gemm(dy, w, group_ends,
    trans_w=not trans_w)``; that by w, grouped_gemm_weight_grad().
    """
    torch = _torch()
    ty = _type_of(x, "x")
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", x.dtype, dev)
    T, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a 3-D tensor [groups, rows, cols]")
    G, N = w.shape[0], w.shape[1 if trans_w else 2]
    wp, ldw, sw = _stack(w, "w", x.dtype, dev, (G, N, K) if trans_w else (G, K, N))
    ends = _ends(group_ends, dev)
    if group_ends.shape[0] != G:
        raise ValueError(f"group_ends has {group_ends.shape[0]} entries for {G} groups")
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=dev)
    yp, ldy = _mat(out, "out", x.dtype, dev, (T, N))
    h = handle or default_handle(dev)
    op = int(bool(trans_w))
    if T and N and K and G:
        key = ("grouped", ty, op, T, N, K, G, xp & 15, ldx, wp & 15, ldw, sw)
        _workspace(h, key, lambda n: _check(h._lib.sgemmGroupedWorkspaceSize(
            h.ptr, ty, op, T, N, K, G, xp, ldx, wp, ldw, sw, n), "sgemmGroupedWorkspaceSize"))
    _check(h._lib.sgemmGrouped(h.ptr, ty, op, T, N, K, G, xp, ldx, wp, ldw, sw, ends, yp, ldy,
                               _stream_ptr(stream, dev.index)), "sgemmGrouped")
    return out


def grouped_gemm_weight_grad(x, dy, group_ends, *, trans_w: bool = False, out=None, handle=None,
                             stream=None):
    """Gradient of grouped_gemm() by w: dw[g] = x_g^T @ dy_g, [G, K, N]
    (with trans_w dy_g^T @ x_g, [G, N, K]); zero for an empty group."""
    torch = _torch()
    ty = _type_of(x, "x")
    dev = _device(x, "x")
    T = x.shape[0] if x.dim() == 2 else -1
    a, b = (dy, x) if trans_w else (x, dy)
    ap, lda = _mat(a, "dy" if trans_w else "x", x.dtype, dev)
    bp, ldb = _mat(b, "x" if trans_w else "dy", x.dtype, dev)
    if a.shape[0] != T or b.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, dy has {dy.shape[0]}")
    M, N = a.shape[1], b.shape[1]
    ends = _ends(group_ends, dev)
    G = group_ends.shape[0]
    if out is None:
        out = torch.empty((G, M, N), dtype=x.dtype, device=dev)
    cp, ldc, sc = _stack(out, "out", x.dtype, dev, (G, M, N))
    h = handle or default_handle(dev)
    if T and M and N and G:
        key = ("wgrad", ty, T, M, N, G, ap & 15, lda, bp & 15, ldb)
        _workspace(h, key, lambda n: _check(h._lib.sgemmGroupedWeightGradWorkspaceSize(
            h.ptr, ty, T, M, N, G, ap, lda, bp, ldb, n), "sgemmGroupedWeightGradWorkspaceSize"))
    _check(h._lib.sgemmGroupedWeightGrad(h.ptr, ty, T, M, N, G, ap, lda, bp, ldb, ends, cp, ldc, sc,
                                         _stream_ptr(stream, dev.index)), "sgemmGroupedWeightGrad")
    return out


def _vector(t, name, dtype, device, n):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if not t.is_cuda or t.device != device or tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} on {device}")
    return t.data_ptr()


def _loss_operands(x, w, target):
    torch = _torch()
    ty = _type_of(x, "x")
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", x.dtype, dev)
    wp, ldw = _mat(w, "w", x.dtype, dev)
    T, D = x.shape
    V = w.shape[0]
    if w.shape[1] != D:
        raise ValueError(f"x has {D} columns, w {w.shape[1]}")
    return ty, dev, T, V, D, xp, ldx, wp, ldw, _vector(target, "target", torch.int64, dev, T)


def linear_cross_entropy(x, w, target, *, handle=None, stream=None):
    """Cross entropy of the logits x @ w.T, which are never kept.

    x [T, D], w [V, D], target [T] int64 (outside [0, V): not counted, loss
    0); returns (loss, lse), float32 [T]: lse[t] = log sum_v exp(x_t . w_v),
    loss[t] = lse[t] - x_t . w_target.
    """
    torch = _torch()
    ty, dev, T, V, D, xp, ldx, wp, ldw, tp = _loss_operands(x, w, target)
    loss, lse = (torch.empty(T, dtype=torch.float32, device=dev) for _ in range(2))
    h = handle or default_handle(dev)
    if T:
        key = ("xent", ty, T, V, D, xp & 15, ldx, wp & 15, ldw)
        _workspace(h, key, lambda n: _check(h._lib.sgemmCrossEntropyWorkspaceSize(
            h.ptr, ty, T, V, D, xp, ldx, wp, ldw, n), "sgemmCrossEntropyWorkspaceSize"))
    _check(h._lib.sgemmCrossEntropy(h.ptr, ty, T, V, D, xp, ldx, wp, ldw, tp, loss.data_ptr(), lse.data_ptr(),
                                    _stream_ptr(stream, dev.index)), "sgemmCrossEntropy")
    return loss, lse


def linear_cross_entropy_grad(x, w, target, lse, dloss, *, handle=None, stream=None):
    """Gradients (dx, dw) of linear_cross_entropy() for the gradient dloss
    [T] (float32) by each token's loss; lse from the forward call."""
    torch = _torch()
    ty, dev, T, V, D, xp, ldx, wp, ldw, tp = _loss_operands(x, w, target)
    lp = _vector(lse, "lse", torch.float32, dev, T)
    gp = _vector(dloss, "dloss", torch.float32, dev, T)
    dx = torch.empty((T, D), dtype=x.dtype, device=dev)
    dw = torch.empty((V, D), dtype=x.dtype, device=dev)
    h = handle or default_handle(dev)
    if T:
        key = ("xent_grad", ty, T, V, D, xp & 15, ldx, wp & 15, ldw)
        _workspace(h, key, lambda n: _check(h._lib.sgemmCrossEntropyGradWorkspaceSize(
            h.ptr, ty, T, V, D, xp, ldx, wp, ldw, n), "sgemmCrossEntropyGradWorkspaceSize"))
    _check(h._lib.sgemmCrossEntropyGrad(h.ptr, ty, T, V, D, xp, ldx, wp, ldw, tp, lp, gp, dx.data_ptr(),
                                        max(D, 1), dw.data_ptr(), max(D, 1),
                                        _stream_ptr(stream, dev.index)), "sgemmCrossEntropyGrad")
    return dx, dw


def w4_gemm(x, q, scales, zeros=None, *, out=None, handle=None, stream=None):
    """y = x @ W.T for 4-bit weights with group scales; returns y [M, N].

    x [M, K] (a few rows); q [N, K // 2] uint8, column 2 i of W in the low
    four bits of byte i, column 2 i + 1 in the high four; scales [N, groups]
    of x's type and zeros [N, groups] uint8 or None (8 everywhere), groups of
    K // groups = 32, 64 or 128 columns:
    W[n, k] = scales[n, k // group] * (q[n, k] - zeros[n, k // group]).
    """
    torch = _torch()
    ty = _type_of(x, "x")
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", x.dtype, dev)
    M, K = x.shape
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError("q must be a 2-D tensor")
    N = q.shape[0]
    qp, ldq = _mat(q, "q", torch.uint8, dev, (N, K // 2))
    sp, lds = _mat(scales, "scales", x.dtype, dev)
    groups = scales.shape[1]
    if scales.shape[0] != N:
        raise ValueError(f"scales has {scales.shape[0]} rows, q {N}")
    if K == 0 or groups == 0 or K % groups:
        if K or groups:
            raise ValueError(f"{groups} groups do not divide {K} columns")
        group = 32
    else:
        group = K // groups
    zp, ldz = (None, 0) if zeros is None else _mat(zeros, "zeros", torch.uint8, dev, (N, groups))
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=dev)
    yp, ldy = _mat(out, "out", x.dtype, dev, (M, N))
    h = handle or default_handle(dev)
    if M and N and K:
        key = ("w4", ty, M, N, K, group)
        _workspace(h, key, lambda n: _check(h._lib.sgemmW4WorkspaceSize(h.ptr, ty, M, N, K, group, n),
                                            "sgemmW4WorkspaceSize"))
    _check(h._lib.sgemmW4(h.ptr, ty, M, N, K, group, xp, ldx, qp, ldq, sp, lds, zp, ldz, yp, ldy,
                          _stream_ptr(stream, dev.index)), "sgemmW4")
    return out
