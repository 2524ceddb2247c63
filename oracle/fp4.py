"""CPU oracle of the microscaled 4-bit floats and of the products grouped by expert.

TEST INFRASTRUCTURE ONLY: plain NumPy in float64, sharing no code with the CUDA path.
Quotients that lie on a rounding border are exact in float64 (a bf16 value has 8
significant bits, a block scale 4, a border times a scale at most 7), so every code is
decided as the definition says. Results are the values before a tensor's own rounding.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E2M1", "e2m1", "e4m3", "row_factor", "quantize_rows", "restore", "swiglu",
           "grouped_product", "grouped_ffn_fp4", "atoms_of_rows", "atoms_of_weights"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1(v):
    """Codes 0 .. 15 of the nearest E2M1 values, ties to the even code, at most 6."""
    a = np.minimum(np.abs(v), 6.0)
    lo = np.clip(np.searchsorted(E2M1, a, side="right") - 1, 0, 6)
    dl, dh = a - E2M1[lo], E2M1[lo + 1] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, lo + 1)
    return c + 8 * (np.signbit(v) & (c > 0))


def e4m3(v):
    """Nearest E4M3 value of v >= 0, ties to even, at most 448: (byte, value)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(v, 2.0 ** -40))
    e = np.maximum(e - 1, -6)
    m = np.rint(np.ldexp(v, 3 - e))                  # 8 .. 16 for normals, below 8 for subnormals
    val = np.minimum(np.ldexp(m, e - 3), 448.0)
    _, e2 = np.frexp(np.maximum(val, 2.0 ** -40))
    e2 = np.maximum(e2 - 1, -6)
    mant = np.ldexp(val, 3 - e2).astype(np.int64)
    byte = np.where(mant >= 8, (e2 + 7) * 8 + mant - 8, mant)
    return byte, val


def row_factor(top):
    """The smallest 2^n, n >= -100, with top <= 2688 * 2^n."""
    m, e = np.frexp(np.asarray(top, dtype=np.float64) / 2688.0)
    n = np.where(m == 0.5, e - 1, e)
    return np.ldexp(1.0, np.maximum(np.where(np.asarray(top) > 0, n, -100), -100))


def quantize_rows(v, block, factor=None):
    """(codes, block scale bytes, row factor or None) of rows v; `factor` [rows] fixes the factors."""
    rows, K = v.shape
    b = v.reshape(rows, K // block, block)
    finite = np.isfinite(b)
    clean = np.where(finite, b, 0.0)
    top = np.abs(clean).max(2)
    if block == 16:
        ok = finite.all((1, 2))
        g = row_factor(np.where(ok, top.max(1), 0.0)) if factor is None else factor
        byte, s = e4m3(top / (6.0 * g[:, None]))
        unit = s * g[:, None]
        keep = ok[:, None] & (unit > 0)
        if factor is None:
            byte = np.where(ok[:, None], byte, 0)
            g = np.where(ok, g, np.nan)
        else:
            byte = np.where(finite.all(2), byte, 0x7f)
            keep = finite.all(2) & (unit > 0)
    else:
        ok = finite.all(2)
        _, e = np.frexp(np.where(ok & (top > 0), top, 1.0))
        X = np.clip(np.where(ok & (top > 0), e - 3, -126), -126, 125)
        unit, byte, g, keep = np.ldexp(1.0, X), np.where(ok, X + 127, 255), None, ok
    q = e2m1(np.where(keep[:, :, None], clean / np.where(keep, unit, 1.0)[:, :, None], 0.0))
    return q.reshape(rows, K), byte, g


def restore(codes, byte, g, block):
    """Values of codes [.., K], scale bytes [.., K/block] and factors broadcast over rows."""
    val = np.where(codes > 7, -1.0, 1.0) * E2M1[codes & 7]
    if block == 16:
        mant, ex = byte & 7, byte >> 3
        s = np.where(ex > 0, np.ldexp(8.0 + mant, ex - 10), np.ldexp(1.0 * mant, -9))
        s = np.where(byte == 0x7f, np.nan, s) * np.asarray(g)[..., None]
    else:
        s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return val * np.repeat(s, block, axis=-1)


def swiglu(G, U):
    with np.errstate(over="ignore"):
        return G / (1.0 + np.exp(-G)) * U


def grouped_product(x, offsets, w):
    """x rows times w[e] [K, N] of their expert."""
    y = np.zeros((x.shape[0], w.shape[2]))
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e]
    return y


def grouped_ffn_fp4(x, offsets, wg, wu, wd, block, h_scale=None, round_h=None):
    """(y, restored H): x and the weights [E, N, K] restored values. round_h: H's rounding before
    its rows are scaled by their own maximum."""
    t = lambda w: np.swapaxes(w, 1, 2)   # noqa: E731
    h = swiglu(grouped_product(x, offsets, t(wg)), grouped_product(x, offsets, t(wu)))
    factor = None
    if h_scale is not None:
        factor = np.repeat(h_scale, np.diff(offsets))
    elif round_h is not None:
        h = round_h(h)
    hv = restore(*quantize_rows(h, block, factor), block)
    return grouped_product(hv, offsets, t(wd)), hv


def _atom(tile_rows, K, block):
    """Scale bytes of up to 128 rows as atoms [KA, 512]."""
    ka = -(-K // (4 * block))
    out = np.zeros((ka, 512), dtype=np.int64)
    for r in range(tile_rows.shape[0]):
        for j in range(K // block):
            out[j // 4, (r % 32) * 16 + (r // 32) * 4 + j % 4] = tile_rows[r, j]
    return out


def atoms_of_rows(byte, offsets, K, block):
    """{tile: atoms} of expert-ordered rows, and which bytes of each are defined."""
    out, first = {}, 0
    for e in range(len(offsets) - 1):
        n = offsets[e + 1] - offsets[e]
        for i in range(-(-n // 128)):
            a = offsets[e] + 128 * i
            rows = byte[a:min(a + 128, offsets[e + 1])]
            out[first + i] = (_atom(rows, K, block), _atom(np.ones_like(rows), K, block) > 0)
        first += 2 * ((-(-n // 128) + 1) // 2)
    return out


def atoms_of_weights(a, K, block, b=None):
    """sf [E, tiles, KA, 512] of scale bytes [E, N, K/block]."""
    E, N, _ = a.shape
    out = []
    for e in range(E):
        if b is None:
            tiles = [a[e, i:i + 128] for i in range(0, N, 128)]
        elif N % 128 == 0:
            tiles = [m[e, i:i + 128] for i in range(0, N, 128) for m in (a, b)]
        else:
            tiles = [np.concatenate((a[e, i:i + 64], b[e, i:i + 64])) for i in range(0, N, 64)]
        out.append([_atom(t, K, block) for t in tiles])
    return np.array(out)
