"""4-bit weights and mixture-of-experts layers on the GPU, through libtilegemm.

Argument checks and marshalling only, like the rest of the package: the
operators are the HIP kernels behind tg_w4_quantize, tg_gemm_w4, tg_moe_route,
tg_moe_mlp and tg_moe_layer (include/tilegemm.h).  Everything runs on the
current stream of the tensors' device; workspaces and outputs come from
PyTorch's allocator, so calls on different streams, and captured graphs, never
share any.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from . import _native
from ._native import ACT, BF16, BF16_F32OUT, F32, GATE, W_BF16, W_W4, Weight


class W4(NamedTuple):
    """A stack of K x N weight matrices in 4 bits (K: the reduction index).

    words: int32 [.., ceil(N/16), ceil(K/128), 64, 4]; scales: bfloat16 or
    float32 [.., ceil(N/16), ceil(K/group), 16]; zeros: uint8 like scales, or
    None (8 everywhere).  Element (k, n) is scale * (code - zero).  Word
    [n // 16, k // 128, 16 * (k % 32 // 8) + n % 16, k % 128 // 32] holds it in
    nibble k % 8 // 2 + 4 * (k % 2).  Any tuple of these six serves where a W4
    is asked for.
    """
    words: "torch.Tensor"                              # noqa: F821
    scales: "torch.Tensor"                             # noqa: F821
    zeros: Optional["torch.Tensor"]                    # noqa: F821
    K: int
    N: int
    group: int


def _call(entry, device, *args):
    """Calls an entry point of the library on `device` and its current stream; raises what the library refuses."""
    import torch
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(entry, device, *args)
    _native.lib().tg_set_stream(torch._C._cuda_getCurrentRawStream(index))
    st = entry(*args)
    if st:
        _native.check(st)


def _group(group, name):
    # the library takes 32 bits, and ctypes cuts what is longer without a word
    if group not in (32, 64) and (group < 128 or group % 128 or group >= 2 ** 31):
        raise ValueError(f"{name}group must be 32, 64 or a multiple of 128 below 2^31")


def _int32(v, name):
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} = {v} is out of range")
    return v


def _w4(w, lead, K, N, device, name):
    """tg_weight of a W4 with the leading dimensions `lead`, or the reason it is none (N None: as it says)."""
    import torch
    if w is None or isinstance(w, torch.Tensor) or len(w) != 6:
        raise TypeError(f"{name} must be a W4: words, scales, zeros, K, N, group")
    words, scales, zeros, wk, wn, group = w
    N = wn if N is None else N
    if (wk, wn) != (K, N):
        raise ValueError(f"{name}: weights are {wk} x {wn}, not {K} x {N}")
    _group(group, f"{name}: ")
    P, C, G = -(-N // 16), -(-K // 128), -(-K // group)
    if words.dtype != torch.int32 or words.shape != (*lead, P, C, 64, 4):
        raise ValueError(f"{name}: words must be int32 {(*lead, P, C, 64, 4)}")
    if scales.dtype not in (torch.bfloat16, torch.float32) or scales.shape != (*lead, P, G, 16):
        raise ValueError(f"{name}: scales must be bfloat16 or float32 {(*lead, P, G, 16)}")
    if not (words.is_contiguous() and scales.is_contiguous()) or words.device != device or scales.device != device:
        raise ValueError(f"{name}: words and scales must be contiguous, on the input's device")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape or not zeros.is_contiguous()
                              or zeros.device != device):
        raise ValueError(f"{name}: zeros must be a contiguous uint8 tensor shaped like scales, on the input's device")
    return Weight(W_W4, group, F32 if scales.dtype == torch.float32 else BF16, 0, words.data_ptr(), scales.data_ptr(),
                  zeros.data_ptr() if zeros is not None else None)


def _weight(w, lead, K, N, device, name):
    """tg_weight of a bf16 tensor [*lead, N, K] or of a W4."""
    import torch
    if not isinstance(w, torch.Tensor):
        return _w4(w, lead, K, N, device, name)
    if w.dtype != torch.bfloat16 or w.shape != (*lead, N, K) or not w.is_contiguous() or w.device != device:
        raise ValueError(f"{name} must be a contiguous bfloat16 {(*lead, N, K)} tensor on x's device, or a W4")
    return Weight(W_BF16, 0, 0, 0, w.data_ptr(), None, None)


def w4_quantize(W, group=128, zero_point=False, scale_dtype=None, values=False):
    """Quantises weights [.., K, N] to 4 bits, a scale for each `group` rows of
    a column (and a zero point with zero_point=True).

    W: float32 or bfloat16, contiguous, or the transpose of its last two
    dimensions of a contiguous tensor (a layer's [.., N, K] as W.transpose(-1,
    -2)).  group: 32, 64 or a multiple of 128; scale_dtype: torch.bfloat16
    (default) or torch.float32.  Returns a W4; with values=True also the values
    that the codes stand for, in W's shape, order and dtype.
    """
    import torch
    _group(group, "")
    if W.dim() < 2:
        raise ValueError("W must have at least two dimensions")
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("W must be float32 or bfloat16")
    if not W.is_cuda:
        raise ValueError("W must be on the GPU")
    scale_dtype = scale_dtype or torch.bfloat16
    if scale_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("scale_dtype must be float32 or bfloat16")
    rows_first = W.is_contiguous()
    if not rows_first and not W.transpose(-1, -2).is_contiguous():
        raise ValueError("W, or the transpose of its last two dimensions, must be contiguous")
    lead, (K, N) = W.shape[:-2], W.shape[-2:]
    if K < 1 or N < 1:
        raise ValueError("K and N must be at least 1")
    P, C, G = -(-N // 16), -(-K // 128), -(-K // group)
    dev = W.device
    words = torch.empty((*lead, P, C, 64, 4), dtype=torch.int32, device=dev)
    scales = torch.empty((*lead, P, G, 16), dtype=scale_dtype, device=dev)
    zeros = torch.empty((*lead, P, G, 16), dtype=torch.uint8, device=dev) if zero_point else None
    out = torch.empty_like(W) if values else None      # keeps W's order
    _call(_native.w4_quantize_ptr, dev, lead.numel(), K, N, group, W.data_ptr(),
          F32 if W.dtype == torch.float32 else BF16, rows_first, F32 if scale_dtype == torch.float32 else BF16,
          words.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zero_point else None, out.data_ptr() if values else None)
    q = W4(words, scales, zeros, K, N, group)
    return (q, out) if values else q


def gemm_w4(A, B, bias=None, act="none", out=None, out_dtype=None):
    """C = act(A @ B + bias) with B in 4 bits.

    A: [M, K] bfloat16, contiguous; B: a W4 without leading dimensions; bias:
    [N] float32 or None; act: "none" | "relu" | "gelu"; out_dtype:
    torch.bfloat16 (default) or torch.float32.  Runs on the current stream and
    returns C.  Rows of A whose elements stay below 8e34 never overflow on the
    way; what larger ones give is in tilegemm.h.
    """
    import torch
    if A.dim() != 2 or A.dtype != torch.bfloat16:
        raise TypeError("A must be a bfloat16 [M, K] tensor")
    if not A.is_cuda or not A.is_contiguous():
        raise ValueError("A must be a contiguous tensor on the GPU")
    M, K = A.shape
    dev = A.device
    w = _w4(B, (), K, None, dev, "B")
    N = B[4]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous [M, N] tensor of the output dtype on A's device")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (N,) or not bias.is_contiguous()
                             or bias.device != dev):
        raise ValueError("bias must be a contiguous float32 [N] tensor on A's device")
    _call(_native.gemm_w4_ptr, dev, M, N, K, A.data_ptr(), w, bias.data_ptr() if bias is not None else None,
          out.data_ptr(), BF16 if out_dtype == torch.bfloat16 else BF16_F32OUT,
          ACT[act] if isinstance(act, str) else _int32(int(act), "act"))
    return out


def _logits(logits, k):
    import torch
    _int32(k, "k")
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be a float32 or bfloat16 [T, E] tensor")
    if not logits.is_cuda or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous tensor on the GPU")
    T = logits.shape[0]
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    return ids, torch.empty((T, k), dtype=torch.float32, device=logits.device)


def moe_route(logits, k, renorm=True):
    """The k largest of each token's logits [T, E] (float32 or bfloat16).

    Returns (ids, weights): int32 [T, k] in falling order of the logits, ties
    to the lowest index, and float32 [T, k], the softmax over all E at those
    experts, with renorm divided by its sum over the k.  At most 1024 experts
    and 16 choices.
    """
    import torch
    ids, weights = _logits(logits, k)
    T, E = logits.shape
    _call(_native.moe_route_ptr, logits.device, T, E, k, logits.data_ptr(),
          F32 if logits.dtype == torch.float32 else BF16, renorm, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def _experts(x, gate_up, down, E, k, gate, out):
    import torch
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise TypeError("x must be a bfloat16 [T, H] tensor")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous tensor on the GPU")
    T, H = x.shape
    if isinstance(gate_up, torch.Tensor):
        if gate_up.dim() != 4:
            raise ValueError("gate_up must be [E, 2, I, H]")
        n, inter = gate_up.shape[0], gate_up.shape[2]
    else:
        if gate_up is None or len(gate_up) != 6 or gate_up[0].dim() != 6:
            raise TypeError("gate_up must be a bfloat16 [E, 2, I, H] tensor or a W4 with leading dimensions (E, 2)")
        n, inter = gate_up[0].shape[0], gate_up[4]
    if E is not None and n != E:
        raise ValueError(f"gate_up holds {n} experts, logits are for {E}")
    up = _weight(gate_up, (n, 2), H, inter, x.device, "gate_up")
    dn = _weight(down, (n,), inter, H, x.device, "down")
    if gate not in GATE:
        raise ValueError(f"gate must be one of {sorted(GATE)}")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous() or out.device != x.device:
        raise ValueError("out must be a contiguous bfloat16 tensor shaped like x")
    ws = torch.empty(_native.moe_workspace_bytes(T, H, inter, k), dtype=torch.uint8, device=x.device)
    return T, H, inter, n, up, dn, out, ws


def moe_mlp(x, ids, weights, gate_up, down, gate="silu", out=None):
    """The experts of a gated feed-forward layer, for a few tokens.

    y[t] = sum_j weights[t, j] * Down_e (gate(Gate_e x[t]) * (Up_e x[t])), e =
    ids[t, j].  x: [T, H] bfloat16; ids: [T, k] int32, weights: [T, k] float32;
    gate_up: bfloat16 [E, 2, I, H] (gate, up) or a W4 with leading dimensions
    (E, 2), K = H, N = I; down: bfloat16 [E, H, I] or a W4 with leading
    dimension (E,), K = I, N = H; gate: "silu" | "gelu".  ids outside [0, E)
    add nothing.  Tokens are taken in passes of up to 64; a pass of n reads an
    expert's weights once for each 16 of its tokens that chose the expert (for
    each 32 where n > 16 and n k > 8 E).  Returns y [T, H] bfloat16.
    """
    import torch
    if ids.dim() != 2 or ids.dtype != torch.int32 or weights.dtype != torch.float32 or weights.shape != ids.shape:
        raise TypeError("ids must be int32 [T, k] and weights float32 of that shape")
    if ids.shape[0] != x.shape[0] or ids.device != x.device or weights.device != x.device or \
            not (ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError("ids and weights must be contiguous, one row for each of x's, on x's device")
    k = _int32(ids.shape[1], "k")
    T, H, inter, n, up, dn, out, ws = _experts(x, gate_up, down, None, k, gate, out)
    _call(_native.moe_mlp_ptr, x.device, T, H, inter, n, k, x.data_ptr(), ids.data_ptr(), weights.data_ptr(), up, dn,
          out.data_ptr(), GATE[gate], ws.data_ptr(), ws.numel())
    return out


def moe_layer(x, logits, gate_up, down, k, renorm=True, gate="silu", out=None):
    """moe_route and moe_mlp in one call: returns (y, ids, weights)."""
    import torch
    ids, weights = _logits(logits, k)
    if logits.shape[0] != x.shape[0] or logits.device != x.device:
        raise ValueError("logits must have one row for each of x's, on x's device")
    T, H, inter, n, up, dn, out, ws = _experts(x, gate_up, down, logits.shape[1], k, gate, out)
    _call(_native.moe_layer_ptr, x.device, T, H, inter, n, k, x.data_ptr(), logits.data_ptr(),
          F32 if logits.dtype == torch.float32 else BF16, renorm, up, dn, out.data_ptr(), ids.data_ptr(),
          weights.data_ptr(), GATE[gate], ws.data_ptr(), ws.numel())
    return out, ids, weights
