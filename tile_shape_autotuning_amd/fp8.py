"""8-bit matrices and their products on the GPU, through libtilegemm.

Argument checks and marshalling only: the operators are the HIP kernels behind
tg_fp8_quantize, tg_gemm_fp8 and tg_moe_gemm_fp8 (include/tilegemm.h).
Everything runs on the current stream of the tensors' device; workspaces and
outputs come from PyTorch's allocator, so calls on different streams, and
captured graphs, never share any.
"""
from __future__ import annotations

from typing import NamedTuple

from . import _native
from ._native import ACT, BF16, BF16_F32OUT, F32, FAST_SUMS, F8Matrix
from .experts import _call, _int32


class F8(NamedTuple):
    """A stack of R x K matrices in 8 bits (K: the index that products sum over).

    codes: float8_e4m3fn [.., R, 128 ceil(K / 128)], zero past K; scales:
    float32, block = 1: [.., R, ceil(K / 128)], one for 128 elements of a row;
    block = 128: [.., ceil(R / 128), ceil(K / 128)], one for a block of 128 x
    128.  An element is code * scale.  Any tuple of these four serves where an
    F8 is asked for.
    """
    codes: "torch.Tensor"                              # noqa: F821
    scales: "torch.Tensor"                             # noqa: F821
    K: int
    block: int


def _f8(m, lead, K, device, name, blocks=(1, 128)):
    """(tg_f8, R) of an F8 with `lead` leading dimensions, or the reason it is none (K, device None: as it says)."""
    import torch
    if m is None or isinstance(m, torch.Tensor) or len(m) != 4:
        raise TypeError(f"{name} must be an F8: codes, scales, K, block")
    codes, scales, mk, block = m
    if block not in blocks:
        raise ValueError(f"{name}: block must be {' or '.join(str(b) for b in blocks)}")
    if K is not None and mk != K:
        raise ValueError(f"{name} has K = {mk}, not {K}")
    if mk < 1:
        raise ValueError(f"{name}: K must be at least 1")
    if codes.dtype != torch.float8_e4m3fn or codes.dim() != lead + 2 or codes.shape[-1] != -(-mk // 128) * 128:
        raise ValueError(f"{name}: codes must be float8_e4m3fn with {lead + 2} dimensions, the last {-(-mk // 128) * 128}")
    R = codes.shape[-2]
    shape = (*codes.shape[:-2], -(-R // block), -(-mk // 128))
    if scales.dtype != torch.float32 or scales.shape != shape:
        raise ValueError(f"{name}: scales must be float32 {shape}")
    if not codes.is_cuda or device is not None and codes.device != device or scales.device != codes.device:
        raise ValueError(f"{name}: codes and scales must be on the GPU, on the other arguments' device")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")
    return F8Matrix(codes.data_ptr(), scales.data_ptr(), block, 0), R


def _output(out, out_dtype, shape, device):
    import torch
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    if out is None:
        return torch.empty(shape, dtype=out_dtype, device=device)
    if out.shape != shape or out.dtype != out_dtype or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous {tuple(shape)} tensor of the output dtype on A's device")
    return out


def _c_type(out, fast_sums):
    return (BF16 if out.element_size() == 2 else BF16_F32OUT) | (FAST_SUMS if fast_sums else 0)


def fp8_quantize(x, block=1, values=False):
    """Quantises matrices [.., R, K] to 8 bits, with a scale for each 128
    elements of a row (block=1: activations) or for each block of 128 x 128
    (block=128: weights).

    x: float32 or bfloat16, contiguous, or the transpose of its last two
    dimensions of a contiguous tensor (the operands of gradients: W.transpose(-1,
    -2), x.transpose(-1, -2)).  scale = max|x| / 448 over the block, code = the
    e4m3 nearest to x / scale; a block with an infinity or NaN is NaN.  Returns
    an F8; with values=True also the values that the codes stand for, in x's
    shape, order and dtype.
    """
    import torch
    if block not in (1, 128):
        raise ValueError("block must be 1 or 128")
    if x.dim() < 2:
        raise ValueError("x must have at least two dimensions")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError("x must be on the GPU")
    rows_first = x.is_contiguous()
    if not rows_first and not x.transpose(-1, -2).is_contiguous():
        raise ValueError("x, or the transpose of its last two dimensions, must be contiguous")
    lead, (R, K) = x.shape[:-2], x.shape[-2:]
    if K < 1:
        raise ValueError("K must be at least 1")
    C, dev = -(-K // 128), x.device
    codes = torch.empty((*lead, R, C * 128), dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((*lead, -(-R // block), C), dtype=torch.float32, device=dev)
    out = torch.empty_like(x) if values else None      # keeps x's order
    _call(_native.fp8_quantize_ptr, dev, lead.numel(), R, K, block, x.data_ptr(),
          F32 if x.dtype == torch.float32 else BF16, rows_first, codes.data_ptr(), scales.data_ptr(),
          out.data_ptr() if values else None)
    q = F8(codes, scales, K, block)
    return (q, out) if values else q


def gemm_fp8(A, B, bias=None, act="none", out=None, out_dtype=None, fast_sums=False):
    """C = act(A @ B^T + bias) of two 8-bit matrices.

    A: an F8 of M x K, block 1; B: an F8 of N x K (a layer's output rows x input
    columns), block 1 or 128; bias: [N] float32 or None; act: "none" | "relu" |
    "gelu"; out_dtype: torch.bfloat16 (default) or torch.float32.  All sums are
    fp32; fast_sums=True lets the matrix cores' 8-bit form add up the products of
    more than 64 rows, at up to twice the rate, which loses small products beside
    large ones (tilegemm.h).  Runs on the current stream and returns C [M, N].

    A layer and its gradients, x [T, K], W [N, K], dy [T, N]:
      y  = gemm_fp8(fp8_quantize(x), fp8_quantize(W, 128))
      dx = gemm_fp8(fp8_quantize(dy), fp8_quantize(W.transpose(0, 1), 128))
      dW = gemm_fp8(fp8_quantize(dy.transpose(0, 1)), fp8_quantize(x.transpose(0, 1)), out_dtype=torch.float32)
    """
    import torch
    a, M = _f8(A, 0, None, None, "A", (1,))
    K, dev = A[2], A[0].device
    b, N = _f8(B, 0, K, dev, "B")
    out = _output(out, out_dtype, (M, N), dev)
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (N,) or not bias.is_contiguous()
                             or bias.device != dev):
        raise ValueError("bias must be a contiguous float32 [N] tensor on A's device")
    need = _native.gemm_fp8_workspace_bytes(M, N, K) if M > 64 else 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(_native.gemm_fp8_ptr, dev, M, N, K, a, b, bias.data_ptr() if bias is not None else None, out.data_ptr(),
          _c_type(out, fast_sums),
          ACT[act] if isinstance(act, str) else _int32(int(act), "act"), ws.data_ptr() if need else None, need)
    return out


def moe_gemm_fp8(A, B, offsets, out=None, out_dtype=None, fast_sums=False):
    """gemm_fp8 for each expert on its own rows: C[r] = A[r] @ B[e]^T for the
    rows r in offsets[e] .. offsets[e + 1] - 1.

    A: an F8 of n x K, block 1, rows in the order of moe_gather; B: an F8 [E, N,
    K], block 1 or 128; offsets: [E + 1] int32 (MoeOrder.offsets); out_dtype:
    torch.bfloat16 (default) or torch.float32; fast_sums: as in gemm_fp8, for more
    than 32 rows an expert on average.  Rows that no expert has are left as they
    were in `out`, and hold anything in a new tensor.  Returns C [n, N].
    """
    import torch
    a, n = _f8(A, 0, None, None, "A", (1,))
    K, dev = A[2], A[0].device
    b, N = _f8(B, 1, K, dev, "B")
    E = B[0].shape[0]
    if offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or not offsets.is_contiguous() or \
            offsets.device != dev:
        raise ValueError("offsets must be a contiguous int32 [E + 1] tensor on A's device")
    out = _output(out, out_dtype, (n, N), dev)
    _call(_native.moe_gemm_fp8_ptr, dev, n, E, N, K, a, b, offsets.data_ptr(), out.data_ptr(),
          _c_type(out, fast_sums))
    return out
