"""8-bit matrices, their products, and rows in the order of their experts: the
plain fp64 definitions (test infrastructure only; the library never calls this
module).

    element      code * scale; code e4m3, scale shared by 128 elements of a row
                 (block 1) or by a block of 128 x 128 (block 128)
    quantise     scale = fp32(max |x| / 448), code = e4m3 nearest to x / scale
    product      act(A . B^T + bias)
    order        pairs t k + j by expert, in order within one
    combine      y[t] = sum_j w[t, j] x[position[t, j]], and its gradients

Arrays are numpy; codes are uint8, rows padded with zeros to whole 128.
"""
from __future__ import annotations

import numpy as np

from oracle.experts_ref import round_bf16   # noqa: F401  (callers round with it)


def code_value(c: int) -> float:
    """Value of one e4m3 code, from its bit fields."""
    sign, e, m = -1.0 if c & 128 else 1.0, c >> 3 & 15, c & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


VALUES = np.array([code_value(c) for c in range(256)])


def nearest(q):
    """Codes nearest to finite q, ties to even codes, magnitudes above 448 to 448."""
    q = np.asarray(q, np.float64)
    table = VALUES[:127]
    a = np.abs(q)
    hi = np.clip(np.searchsorted(table, a, side="left"), 1, 126)
    lo = hi - 1
    up, down = table[hi] - a, a - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * np.signbit(q)).astype(np.uint8)


def quantise(x, block):
    """x [R, K] fp64 (of fp32 or bf16 values) -> (codes [R, Kp], scales [P, C] fp32)."""
    R, K = x.shape
    C, P = -(-K // 128), -(-R // block)
    codes, scales = np.zeros((R, C * 128), np.uint8), np.zeros((P, C), np.float32)
    for p in range(P):
        for c in range(C):
            at = np.s_[p * block:(p + 1) * block, c * 128:min(K, (c + 1) * 128)]
            b = x[at]
            if not np.isfinite(b).all():
                scales[p, c] = np.nan
                codes[at] = 0x7F
                continue
            s = np.float32(np.abs(b).max() / 448.0)
            scales[p, c] = s
            if s > 0:
                codes[at] = nearest(b / np.float64(s))
    return codes, scales


def dense(codes, scales, K, block):
    """Elements [R, K] in fp64."""
    r, k = np.meshgrid(np.arange(codes.shape[0]), np.arange(K), indexing="ij")
    return VALUES[codes[:, :K]] * scales[r // block, k // 128].astype(np.float64)


def order(ids, E):
    """(position [T, k], source [T k], offsets [E + 1]) pair by pair."""
    flat = ids.reshape(-1)
    position, source = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    offsets, row = np.zeros(E + 1, np.int32), 0
    for e in range(E):
        offsets[e] = row
        for i in np.flatnonzero(flat == e):
            position[i], source[row] = row, i
            row += 1
    offsets[E] = row
    return position.reshape(ids.shape), source, offsets


def gather(x, position, out):
    out = out.copy()
    for t in range(position.shape[0]):
        for r in position[t]:
            if 0 <= r < out.shape[0]:
                out[r] = x[t]
    return out


def combine(x, position, weights):
    y = np.zeros((position.shape[0], x.shape[1]))
    for t in range(position.shape[0]):
        for j, r in enumerate(position[t]):
            if 0 <= r < x.shape[0]:
                y[t] += weights[t, j] * x[r]
    return y


def combine_grad(dy, x, position, weights, dx):
    dx, dw = dx.copy(), np.zeros(weights.shape)
    for t in range(position.shape[0]):
        for j, r in enumerate(position[t]):
            if 0 <= r < x.shape[0]:
                dx[r] = weights[t, j] * dy[t]
                dw[t, j] = float(np.dot(dy[t], x[r]))
    return dx, dw
