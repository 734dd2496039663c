"""4-bit weights, expert routing and expert layers: the plain fp64 definitions
(test infrastructure only; the library never calls this module).

    w4 element   scale * (code - zero), scale and zero shared by `group` rows of a column
    quantise     symmetric: scale = max|w| / 7, zero 8; else scale = (hi - lo) / 15,
                 zero = rint(-lo / scale); code = clamp(rint(w / scale) + zero, 0, 15)
    route        the k largest logits (ties: lowest index), softmax weights
    mlp          y[t] = sum_j w[t, j] Down_e (gate(Gate_e x[t]) * (Up_e x[t]))

Arrays are numpy; bf16 values come and go as fp64 (exact).
"""
from __future__ import annotations

import math

import numpy as np

from tile_shape_autotuning_amd import workloads as wl


def round_bf16(v):
    """To fp32, then to bf16, as fp64."""
    return wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(np.asarray(v, np.float32))).astype(np.float64)


def pack(codes):
    """Codes [K, N] -> words [P, C, 64, 4] uint32, one element at a time."""
    K, N = codes.shape
    words = np.zeros((-(-N // 16), -(-K // 128), 64, 4), np.uint32)
    for k in range(K):
        lane, t, r = 16 * (k % 32 // 8), k % 128 // 32, k % 8
        nibble = r // 2 + (4 if r % 2 else 0)
        for n in range(N):
            words[n // 16, k // 128, lane + n % 16, t] |= np.uint32(int(codes[k, n]) << (4 * nibble))
    return words


def unpack(words, K, N):
    """Words -> codes [K, N]."""
    k, n = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    w = words[n // 16, k // 128, 16 * (k % 32 // 8) + n % 16, k % 128 // 32].astype(np.uint64)
    return ((w >> (4 * (k % 8 // 2 + 4 * (k % 2))).astype(np.uint64)) & np.uint64(15)).astype(np.int64)


def panels(t):
    """Per-group values [G, N] -> storage [P, G, 16], zeros past N."""
    G, N = t.shape
    P = -(-N // 16)
    out = np.zeros((G, P * 16), t.dtype)
    out[:, :N] = t
    return np.ascontiguousarray(out.reshape(G, P, 16).transpose(1, 0, 2))


def dense(words, scales, zeros, K, N, group):
    """Storage -> weights [K, N] in fp64; scales, zeros [P, G, 16]."""
    k, n = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    at = (n // 16, k // group, n % 16)
    z = 8.0 if zeros is None else zeros[at].astype(np.float64)
    return scales[at].astype(np.float64) * (unpack(words, K, N) - z)


def quantize(W, group, zero_point, scale_bf16):
    """(codes [K, N], scales [G, N], zeros [G, N], values [K, N]) of finite W [K, N] (fp32 values)."""
    W = np.asarray(W, np.float64)
    K, N = W.shape
    G = -(-K // group)
    codes, values = np.zeros((K, N), np.int64), np.zeros((K, N))
    scales, zeros = np.zeros((G, N)), np.full((G, N), 8)
    for g in range(G):
        w = W[g * group:(g + 1) * group]
        lo, hi = np.minimum(w.min(0), 0.0), np.maximum(w.max(0), 0.0)
        if zero_point:
            s = (hi - lo).astype(np.float32).astype(np.float64) / 15.0
        else:
            s = np.maximum(hi, -lo) / 7.0
        s = round_bf16(s) if scale_bf16 else s.astype(np.float32).astype(np.float64)
        unit = np.where(s > 0, s, 1.0)
        z = np.clip(np.rint(-lo / unit), 0, 15) if zero_point else np.full(N, 8.0)
        q = np.clip(np.rint(w / unit) + z, 0, 15)
        q = np.where(s > 0, q, z)
        codes[g * group:(g + 1) * group] = q
        values[g * group:(g + 1) * group] = (q - z) * s
        scales[g], zeros[g] = s, z
    return codes, scales, zeros, values


def act(v, name):
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "gelu":
        return 0.5 * v * np.vectorize(math.erfc, otypes=[float])(-v / math.sqrt(2.0))
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    return v


def route(logits, k, renorm):
    """ids [T, k], weights [T, k]; finite or -inf logits."""
    v = np.asarray(logits, np.float64)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k]
    weights = np.zeros(ids.shape)
    for t in range(v.shape[0]):
        top = v[t].max()
        if top == -np.inf:
            continue
        p = np.exp(v[t] - top)
        weights[t] = p[ids[t]] / (p[ids[t]].sum() if renorm else p.sum())
    return ids.astype(np.int32), weights


def mlp(x, ids, weights, gate, up, down, kind):
    """y [T, H], and the sums of |products| of the last product that bound its rounding.
    x [T, H], gate, up [E, H, I], down [E, I, H]."""
    T, H = x.shape
    y, size = np.zeros((T, H)), np.zeros((T, H))
    E = gate.shape[0]
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            h = weights[t, j] * act(x[t] @ gate[e], kind) * (x[t] @ up[e])
            y[t] += h @ down[e]
            size[t] += np.abs(h) @ np.abs(down[e])
    return y, size
