"""CPU oracle of the block around the layer: the norms before and after it, the
8-bit activation checkpoints and the experts on 4-bit weights.

TEST INFRASTRUCTURE ONLY: plain NumPy in float64 (the two quantizers state their
fp32 and bf16 steps explicitly), sharing no code with the CUDA path. Results are
the values before the tensors' own bf16 rounding.
"""
from __future__ import annotations

import numpy as np

__all__ = ["norm_in", "norm_in_backward", "norm_out", "norm_out_backward", "scale_bf16_up",
           "ckpt8_pack", "ckpt8_restore", "ckpt8_swiglu", "w4_quantize", "w4_values",
           "grouped_ffn_w4"]


# ---------------------------------------------------------------- norms
def norm_in(x, gain, eps):
    r = 1.0 / np.sqrt(np.mean(x ** 2, axis=1) + eps)
    return x * r[:, None] * gain, r


def norm_in_backward(dxn, x, gain, r, dres=None):
    """(dx, dgain): the derivative of x r(x) gain, written over the saved r."""
    xh = x * r[:, None]
    u = dxn * gain
    dx = r[:, None] * (u - xh * np.mean(u * xh, axis=1, keepdims=True))
    return dx if dres is None else dx + dres, (dxn * xh).sum(0)


def _gate_rows(gate, span, T):
    return np.ones((T, 1)) if gate is None else gate[np.arange(T) // span]


def norm_out(y, resid, gain, w, inv_perm, K, shared, gate, span, scale, eps):
    """(out, z, r or None)."""
    T = resid.shape[0]
    z = np.zeros_like(resid)
    for j in range(K):
        a = np.arange(T) * K + j
        rows = y[a if inv_perm is None else inv_perm[a]]
        z = z + (rows if w is None else w[:, j:j + 1] * rows)
    if shared is not None:
        z = z + shared
    n, r = z, None
    if gain is not None:
        n, r = norm_in(z, gain, eps)
    return resid + scale * _gate_rows(gate, span, T) * n, z, r


def norm_out_backward(dout, z, r, gain, gate, span, scale):
    """(dz, dgain or None, dgate or None)."""
    T = dout.shape[0]
    dn = scale * _gate_rows(gate, span, T) * dout
    n, dz, dgain, dgate = z, dn, None, None
    if gain is not None:
        dz, dgain = norm_in_backward(dn, z, gain, r)
        n = z * r[:, None] * gain
    if gate is not None:
        dgate = np.zeros_like(gate)
        t = scale * dout * n
        np.add.at(dgate, np.arange(T) // span,
                  t.sum(1, keepdims=True) if gate.shape[1] == 1 else t)
    return dz, dgain, dgate


# ---------------------------------------------------------------- 8-bit checkpoints
def scale_bf16_up(amax, steps):
    """max(amax / steps in fp32, 2^-110) rounded up to bf16, as float64."""
    t = np.maximum(np.float32(amax) / np.float32(steps), np.float32(2.0 ** -110))
    b = t.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0xffff) & 0xffff0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def ckpt8_pack(x):
    """(q int64 [M, N], s float64 [M, ceil(N / 32)])."""
    M, N = x.shape
    nb = -(-N // 32)
    q = np.zeros((M, N), dtype=np.int64)
    s = np.zeros((M, nb))
    for b in range(nb):
        v = x[:, 32 * b:32 * b + 32].astype(np.float32)
        fine = np.isfinite(v)
        s[:, b] = scale_bf16_up(np.where(fine, np.abs(v), 0).max(1), 127)
        r = np.float32(1.0) / s[:, b].astype(np.float32)
        code = np.rint(np.where(fine, v, 0) * r[:, None])      # an fp32 product, ties to even
        q[:, 32 * b:32 * b + 32] = np.where(fine, code, -128)
    return q, s


def ckpt8_restore(q, s):
    v = q * np.repeat(s, 32, axis=1)[:, :q.shape[1]]
    return np.where(q == -128, np.nan, v)


def ckpt8_swiglu(q, s):
    """(gu, h) of a checkpointed [G | U]."""
    v = ckpt8_restore(q, s)
    G, U = np.split(v, 2, axis=1)
    with np.errstate(over="ignore"):
        return v, G / (1.0 + np.exp(-G)) * U


# ---------------------------------------------------------------- 4-bit weights
def w4_quantize(w, group):
    """w [E, K, N] -> codes [E, N, K] in 0 .. 15 and scales [E, N, K / group]."""
    E, K, N = w.shape
    v = np.swapaxes(w, 1, 2).astype(np.float32).reshape(E, N, K // group, group)
    s = scale_bf16_up(np.abs(v).max(3).reshape(-1), 7).reshape(E, N, K // group)
    r = np.float32(1.0) / s.astype(np.float32)
    q = np.clip(np.rint(v * r[..., None]), -7, 7) + 8
    return q.reshape(E, N, K).astype(np.int64), s


def w4_values(codes, s):
    """The weights [E, N, K] that codes [E, N, K] and scales [E, N, groups] stand for."""
    return (codes - 8) * np.repeat(s, codes.shape[2] // s.shape[2], axis=2)


def grouped_ffn_w4(xp, offsets, gate, up, down, h=None):
    """(y, h) of rows xp in expert order; gate, up [E, I, d] and down [E, d, I] values. With
    h given (as stored), y is its product and the returned h is still the one before rounding."""
    M = xp.shape[0]
    ref_h = np.zeros((M, gate.shape[1]))
    y = np.zeros((M, down.shape[1]))
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        G, U = xp[a:b] @ gate[e].T, xp[a:b] @ up[e].T
        with np.errstate(over="ignore"):
            ref_h[a:b] = G / (1.0 + np.exp(-G)) * U
        y[a:b] = (ref_h if h is None else h)[a:b] @ down[e].T
    return y, ref_h
