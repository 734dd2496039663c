"""Tokens in the order of their experts, and back, on the GPU, through libtilegemm.

Argument checks and marshalling only: the operators are the HIP kernels behind
tg_moe_sort, tg_moe_gather, tg_moe_combine and tg_moe_combine_grad
(include/tilegemm.h).  With moe_route before them and moe_gemm_fp8 between them
they make the experts of a layer for any number of tokens.  Everything runs on
the current stream of the tensors' device; workspaces and outputs come from
PyTorch's allocator.
"""
from __future__ import annotations

from typing import NamedTuple

from . import _native
from ._native import BF16, F32
from .experts import _call, _int32
from .fp8 import F8, _f8


class MoeOrder(NamedTuple):
    """(token, choice) pairs sorted by expert.

    position: int32 [T, k], the row of each pair, -1 without one; source: int32
    [T k], the pair t k + j of each row, -1 for rows behind the last; offsets:
    int32 [E + 1], expert e has rows offsets[e] .. offsets[e + 1] - 1, in the
    order of their pairs.  Any tuple of these three serves where a MoeOrder is
    asked for.
    """
    position: "torch.Tensor"                           # noqa: F821
    source: "torch.Tensor"                             # noqa: F821
    offsets: "torch.Tensor"                            # noqa: F821


def moe_sort(ids, E):
    """Sorts the pairs of a token and one of its choices by expert.

    ids: [T, k] int32, as moe_route gives them; an id outside [0, E) has no
    row.  The order is stable.  At most 1024 experts and 16 choices.  Returns a
    MoeOrder.
    """
    import torch
    if ids.dim() != 2 or ids.dtype != torch.int32:
        raise TypeError("ids must be an int32 [T, k] tensor")
    if not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous tensor on the GPU")
    T, k = ids.shape
    _int32(E, "E")
    need = _native.moe_sort_workspace_bytes(T, E, k)
    dev = ids.device
    position = torch.empty((T, k), dtype=torch.int32, device=dev)
    source = torch.empty((T * k,), dtype=torch.int32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(_native.moe_sort_ptr, dev, T, E, k, ids.data_ptr(), position.data_ptr(), source.data_ptr(),
          offsets.data_ptr(), ws.data_ptr() if need else None, need)
    return MoeOrder(position, source, offsets)


def _position(order, T, device):
    import torch
    if order is None or isinstance(order, torch.Tensor) or len(order) != 3:
        raise TypeError("order must be a MoeOrder: position, source, offsets")
    position = order[0]
    if position.dtype != torch.int32 or position.dim() != 2 or not position.is_contiguous() or \
            position.device != device:
        raise ValueError("order.position must be a contiguous int32 [T, k] tensor on the rows' device")
    if T is not None and position.shape[0] != T:
        raise ValueError(f"order is of {position.shape[0]} tokens, not {T}")
    return position, position.shape[0], position.shape[1]


def _rows(x, name):
    import torch
    if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name} must be a float32 or bfloat16 [rows, H] tensor")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the GPU")
    return x.shape


def moe_gather(x, order, out=None):
    """Rows in the order of the experts: out[position[t, j]] = x[t].

    x: [T, H] bfloat16 or float32, or an F8 of T x H, block 1 (quantised rows,
    moved with their scales).  Returns [T k, H], an F8 for an F8.  Rows that no
    pair has are left as they were in `out`, and hold anything in a new tensor.
    The gradient of x is moe_combine(gradient of the rows, order).
    """
    import torch
    if isinstance(x, torch.Tensor):
        T, H = _rows(x, "x")
        position, T, k = _position(order, T, x.device)
        n = out.shape[0] if out is not None and out.dim() == 2 else T * k
        if out is None:
            out = torch.empty((n, H), dtype=x.dtype, device=x.device)
        elif out.shape != (n, H) or out.dtype != x.dtype or not out.is_contiguous() or out.device != x.device:
            raise ValueError("out must be a contiguous [rows, H] tensor of x's dtype on x's device")
        size = H * x.element_size()
        if size:
            _call(_native.moe_gather_ptr, x.device, T, k, n, position.data_ptr(), size, x.data_ptr(), out.data_ptr(),
                  0, None, None)
        return out
    a, T = _f8(x, 0, None, None, "x", (1,))
    K, dev = x[2], x[0].device
    position, T, k = _position(order, T, dev)
    width, chunks = x[0].shape[1], x[1].shape[1]
    if out is None:
        n = T * k
        out = F8(torch.empty((n, width), dtype=torch.float8_e4m3fn, device=dev),
                 torch.empty((n, chunks), dtype=torch.float32, device=dev), K, 1)
    b, n = _f8(out, 0, K, dev, "out", (1,))
    _call(_native.moe_gather_ptr, dev, T, k, n, position.data_ptr(), width, a.codes, b.codes, 4 * chunks, a.scales,
          b.scales)
    return F8(*out)


def moe_combine(x, order, weights=None, out=None):
    """Rows back to their tokens: y[t] = sum_j weights[t, j] * x[position[t, j]].

    x: [rows, H] bfloat16 or float32; weights: [T, k] float32, or None (all 1:
    the gradient of moe_gather).  fp32 sums, rounded once; a token without rows
    gets zeros.  Returns y [T, H], like x.
    """
    import torch
    n, H = _rows(x, "x")
    position, T, k = _position(order, None, x.device)
    if weights is not None:
        _pair_weights(weights, T, k, x.device)
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    elif out.shape != (T, H) or out.dtype != x.dtype or not out.is_contiguous() or out.device != x.device:
        raise ValueError("out must be a contiguous [T, H] tensor of x's dtype on x's device")
    if H:
        _call(_native.moe_combine_ptr, x.device, T, k, n, H, x.data_ptr(), F32 if x.dtype == torch.float32 else BF16,
              position.data_ptr(), weights.data_ptr() if weights is not None else None, out.data_ptr())
    return out


def _pair_weights(weights, T, k, device):
    import torch
    if weights.dtype != torch.float32 or weights.shape != (T, k) or not weights.is_contiguous() or \
            weights.device != device:
        raise ValueError("weights must be a contiguous float32 [T, k] tensor on the rows' device")


def moe_combine_grad(dy, x, order, weights, out=None):
    """Gradients of moe_combine(x, order, weights) for the gradient dy of its result.

    Returns (dx, dweights): dx[position[t, j]] = weights[t, j] * dy[t], like x
    (rows that no pair has are left as they were in `out`, and hold anything in
    a new tensor); dweights[t, j] = <dy[t], x[position[t, j]]>, float32 [T, k],
    0 for pairs without a row.  weights has to be given: without it the gradient
    of x is moe_gather(dy, order).
    """
    import torch
    if weights is None:
        raise TypeError("weights must be given; without weights the gradient of x is moe_gather(dy, order)")
    T, Hy = _rows(dy, "dy")
    n, H = _rows(x, "x")
    if Hy != H or dy.dtype != x.dtype or dy.device != x.device:
        raise ValueError("dy must be [T, H] of x's dtype, on x's device")
    position, T, k = _position(order, T, x.device)
    _pair_weights(weights, T, k, x.device)
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous() or out.device != x.device:
        raise ValueError("out must be a contiguous tensor like x")
    if H == 0:
        return out, torch.zeros((T, k), dtype=torch.float32, device=x.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _call(_native.moe_combine_grad_ptr, x.device, T, k, n, H, dy.data_ptr(), x.data_ptr(),
          F32 if x.dtype == torch.float32 else BF16, position.data_ptr(), weights.data_ptr(), out.data_ptr(),
          dw.data_ptr())
    return out, dw
