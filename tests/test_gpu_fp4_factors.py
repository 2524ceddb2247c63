"""The 32-bit factors of 4-bit products far from one: each in fp32's range, their product not.

y is the sum of exact terms times the factors of the row and the matrix (and H's), whatever the
order of the factors: a representable result may not be lost because two factors alone leave the
range, and a sum of zero is zero. Tolerance: half an ulp of the stored bf16 value plus 1e-3 of the
row's RMS, as the other products (the results are normal numbers)."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, rounding_excess, to_dev

pytestmark = pytest.mark.gpu

F32, BF, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _matrix(rng, E, N, K, g, zero=()):
    """Codes, scales and factors g [E] of E matrices [N, K] (rows in `zero` of zeros), the product's
    form on the device and the values."""
    codes = rng.integers(0, 16, size=(E, N, K))
    codes[:, list(zero)] = 0
    byte = rng.integers(104, 120, size=(E, N, K // 16))    # 2^6 to 2^8
    g = np.asarray(g, dtype=np.float32)
    val = F.restore(codes, byte, g.astype(np.float64)[:, None] * np.ones((E, N)), 16)
    packed = to_dev((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8), U8)
    return val, packed, to_dev(byte, U8), to_dev(g, F32)


def _unit_rows(y, want):
    """Both in units of each row's size, a power of two."""
    size = np.exp2(np.round(np.log2(np.sqrt(np.mean(want ** 2, axis=1, keepdims=True)))))
    return y / size, want / size


def _product(rng, ex, g, zero=(), N=136, K=192):
    """Rows of size 2^ex times matrices of factors g: (y, float64 result: the factor times the sum)."""
    E, n = len(g), 40
    offsets = np.arange(E + 1) * n
    x = O.round_bf16(rng.normal(size=(E * n, K)) * np.exp2(ex))
    val, codes, byte, _ = _matrix(rng, E, N, K, np.ones(E), zero)
    off, g = to_dev(offsets, I32), np.asarray(g, dtype=np.float32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off)
    y = f64(B.moe_grouped_gemm_fp4(rows, off, (codes, B.moe_fp4_pack_scales(byte), to_dev(g, F32))))
    xv = F.restore(*F.quantize_rows(x, 16), 16)
    sums = F.grouped_product(xv, offsets, np.swapaxes(val, 1, 2))
    with np.errstate(invalid="ignore"):
        return y, np.repeat(g.astype(np.float64), n)[:, None] * sums


@pytest.mark.parametrize("N,K", [(136, 192), (72, 192), (136, 1152)])     # every instance of the product
@pytest.mark.parametrize("ex,g", [
    (-70, 1.36 * 2.0 ** -64),    # factors 2^-80 2^-64: a subnormal product of five bits, sums of 2^21
    (-90, 1.36 * 2.0 ** -44),    # the same, rows smaller
    (-88, 1.9 * 2.0 ** -100),    # the result is zero
    (60, 1.1 * 2.0 ** -70), (-60, 1.1 * 2.0 ** 60), (-80, 1.7 * 2.0 ** 100), (100, 1.7 * 2.0 ** -100),
])
def test_product(ex, g, N, K):
    y, want = _product(np.random.default_rng([ex + 200, 1]), ex, [g, g * 1.7, g * 2.5], N=N, K=K)
    if np.abs(want).max() < 2.0 ** -135:      # below half the smallest bf16
        assert (y == 0).all()
        return
    assert_bf16_close(*_unit_rows(y, want), "y")


def test_zero_sums_stay_zero():
    """Factors whose product is beyond fp32: outputs with a row of zeros are zero, the others
    overflow."""
    zero = (3, 100, 135)
    y, want = _product(np.random.default_rng(7), 118, [1.5 * 2.0 ** 40, 2.0 ** 21, 1.0], zero)
    assert (y[:, list(zero)] == 0).all()
    top = float(torch.finfo(BF).max)
    big = np.abs(want) > 1.01 * top
    assert big.any() and np.array_equal(np.isinf(y), np.isinf(y) & (np.abs(want) > 0.99 * top))
    assert np.isinf(y[big]).all() and np.array_equal(np.sign(y[big]), np.sign(want[big]))
    assert not np.isnan(y).any()


@pytest.mark.parametrize("hidden", ["fixed", "row"])
@pytest.mark.parametrize("I", [128, 192])
def test_experts(I, hidden):
    """Gate factors so small that silu(G) = G / 2, up factors as large; H's and the down
    projection's far from one the other way."""
    rng = np.random.default_rng([I, len(hidden)])
    E, d, n = 3, 192, 70
    offsets = np.arange(E + 1) * n
    x = O.round_bf16(rng.normal(size=(E * n, d)) * 2.0 ** -79)     # rows' factors near 2^-90
    unit = np.array([1.3, 0.9, 1.6], dtype=np.float32)
    wg, gq, gs, gg = _matrix(rng, E, I, d, unit * 2.0 ** -56)      # 2^-89 2^-56: subnormal
    wu, uq, us, ug = _matrix(rng, E, I, d, unit * 2.0 ** 110)
    # G of 2^-122, U of 2^44, H = G U / 2 of 2^-79
    wd, dq, ds, dg = _matrix(rng, E, d, I, unit * 2.0 ** 70)
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off)
    xv = F.restore(*F.quantize_rows(x, 16), 16)
    t = lambda w: np.swapaxes(w, 1, 2)   # noqa: E731
    h = F.swiglu(F.grouped_product(xv, offsets, t(wg)), F.grouped_product(xv, offsets, t(wu)))
    hs = None
    if hidden == "fixed":
        hs = (np.abs(h).reshape(E, -1).max(1) / 2688).astype(np.float32)
        assert (hs > 2.0 ** -100).all()
    y = f64(B.moe_grouped_ffn_fp4(rows, off, (gq, uq, B.moe_fp4_pack_scales(gs, us), gg, ug),
                                  (dq, B.moe_fp4_pack_scales(ds), dg),
                                  h_scale=None if hs is None else to_dev(hs, F32)))
    want, _ = F.grouped_ffn_fp4(xv, offsets, wg, wu, wd, 16,
                                h_scale=None if hs is None else hs.astype(np.float64),
                                round_h=O.round_bf16 if hidden == "row" else None)
    y, want = _unit_rows(y, want)
    assert np.isfinite(y).all()
    off_rows = (rounding_excess(y, want) > 1e-3 * np.sqrt(np.mean(want ** 2))).any(1)
    # a code of H next to a border may be the neighbour (chance 2^-17 a value, see the tests of many
    # tiles): E n I 2^-17 = 0.3 rows
    assert off_rows.sum() <= 3, off_rows.sum()


def test_factors_that_are_not_finite_or_zero():
    """A matrix factor of zero gives zeros, of Inf Inf by the sum's sign, of NaN NaN."""
    rng = np.random.default_rng(5)
    y, want = _product(rng, 0, [0.0, np.inf, np.nan, 1.0])
    assert (y[:40] == 0).all() and np.isnan(y[80:120]).all()
    assert np.array_equal(y[40:80], want[40:80], equal_nan=True)
    assert np.isfinite(y[120:]).all()


@pytest.mark.parametrize("ex", [-92, 0, 105, 121])
def test_hidden_factors_at_their_ends(ex):
    """H of size 2^ex under a fixed factor of 2^-99 to 2^115."""
    rng = np.random.default_rng([ex + 200, 3])
    E, d, I, n = 3, 192, 192, 70
    offsets = np.arange(E + 1) * n
    x = O.round_bf16(rng.normal(size=(E * n, d)))
    unit = np.array([1.3, 0.9, 1.6], dtype=np.float32)
    wg, gq, gs, gg = _matrix(rng, E, I, d, unit * 2.0 ** -12)
    wu, uq, us, ug = _matrix(rng, E, I, d, unit * 2.0 ** (ex - 12))
    wd, dq, ds, dg = _matrix(rng, E, d, I, unit * 2.0 ** -ex)
    xv = F.restore(*F.quantize_rows(x, 16), 16)
    t = lambda w: np.swapaxes(w, 1, 2)   # noqa: E731
    h = F.swiglu(F.grouped_product(xv, offsets, t(wg)), F.grouped_product(xv, offsets, t(wu)))
    hs = (np.abs(h).reshape(E, -1).max(1) / 2688).astype(np.float32)
    assert (hs >= 2.0 ** -100).all() and (hs <= 2.0 ** 117).all()
    off = to_dev(offsets, I32)
    y = f64(B.moe_grouped_ffn_fp4(B.moe_fp4_quantize_rows(to_dev(x, BF), off), off,
                                  (gq, uq, B.moe_fp4_pack_scales(gs, us), gg, ug),
                                  (dq, B.moe_fp4_pack_scales(ds), dg), h_scale=to_dev(hs, F32)))
    want, _ = F.grouped_ffn_fp4(xv, offsets, wg, wu, wd, 16, h_scale=hs.astype(np.float64))
    off_rows = (rounding_excess(y, want) > 1e-3 * np.sqrt(np.mean(want ** 2))).any(1)
    assert off_rows.sum() <= 3, off_rows.sum()      # E n I 2^-16 = 0.6 rows with a changed code
