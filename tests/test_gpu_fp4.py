"""GPU parity of the microscaled 4-bit floats with the CPU oracle.

Codes, scale bytes and row factors are compared bit for bit (a code of zero has one sign).
Products: every term is exact and sums are fp32, then one bf16 rounding: within half an ulp
of the stored value plus 1e-3 of the tensor's RMS, as the other products of this library are
held to. The experts' hidden rows are quantized from fp32 values, so a value next to a
rounding border may take the neighbouring code: y is compared with the product of the
oracle's H, where a changed code of H moves a row of y by at most its step (half the value,
at most 2 units of its block) times a weight; such rows are counted and have to be few.
"""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, i64, rounding_excess, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _nibbles(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def _bits(codes):
    """Codes with one zero."""
    return np.where(codes & 7, codes, 0)


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def _rows(rng, M, d):
    """Rows with blocks and rows of very different sizes, zeros, ties and exact powers of two."""
    x = rng.normal(size=(M, d)) * np.exp2(rng.integers(-12, 12, size=(M, 1)))
    x *= np.exp2(rng.integers(-9, 3, size=(M, d // 16))).repeat(16, axis=1)
    x[:, :16] = 0.0
    if M > 1:
        x[1] = 0.0
    if M > 2:
        x[2] = rng.integers(-24, 25, size=d) * 0.25          # borders of power-of-two scales
    if M > 3:
        x[3] = rng.integers(-96, 97, size=d) * 2.0 ** -130   # below every scale
    if M > 4:
        x[4] = rng.normal(size=d) * 2.0 ** 124
    return O.round_bf16(x)


def _check_rows(rows, x, offsets, block):
    q, sf, rs = rows
    codes, byte, g = F.quantize_rows(x, block)
    assert np.array_equal(_bits(_nibbles(i64(q))), _bits(codes))
    if block == 16:
        assert np.array_equal(f64(rs), g, equal_nan=True)
    got = i64(sf)
    for t, (want, known) in F.atoms_of_rows(byte, offsets, x.shape[1], block).items():
        assert np.array_equal(got[t][known], want[known]), t
    return codes, byte, g


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("d,counts", [
    (64, [1]), (128, [0, 3]), (192, [5, 0, 129, 1]), (1024, [130, 2]), (2048, [9, 260, 0]),
    (2112, [7, 7]), (4096, [3, 40]), (4160, [6]), (8192, [2, 5]), (16384, [5]),
])
def test_rows(block, d, counts):
    offsets = np.concatenate([[0], np.cumsum(counts)])
    x = _rows(np.random.default_rng([d, block]), offsets[-1], d)
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    codes, byte, g = _check_rows(rows, x, offsets, block)
    back = B.moe_fp4_dequantize_rows(rows, off, block)
    want = F.restore(codes, byte, g, block)
    assert np.array_equal(f64(back), O.round_bf16(want))   # q s has 5 bits: exact in bf16 but at its ends


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,E,K,d", [(1, 8, 8, 128), (37, 5, 3, 320), (300, 16, 6, 2048), (64, 4, 1, 64)])
def test_dispatched_rows(block, T, E, K, d):
    rng = np.random.default_rng([T, d])
    x = _rows(rng, T, d)
    idx = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    counts, off, perm, inv = B.moe_build_permutation(to_dev(idx, I32), E)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block, inv_perm=inv, K=K)
    _check_rows(rows, x[i64(perm) // K], i64(off), block)


@pytest.mark.parametrize("block", [16, 32])
def test_rows_that_are_not_finite(block):
    x = _rows(np.random.default_rng(5), 6, 256)
    x[0, 20], x[5, 200], x[5, 3] = np.inf, np.nan, -np.inf
    off = to_dev(np.array([0, 6]), I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    codes, byte, g = _check_rows(rows, x, [0, 6], block)
    back = f64(B.moe_fp4_dequantize_rows(rows, off, block))
    bad = np.zeros((6, 256), dtype=bool)
    if block == 16:
        bad[[0, 5]] = True
    else:
        bad[0, 0:32] = bad[5, 192:224] = bad[5, 0:32] = True
    assert np.array_equal(np.isnan(back), bad)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("E,K,N", [(1, 64, 8), (3, 192, 136), (2, 1024, 256), (2, 320, 72)])
def test_weights(block, E, K, N):
    rng = np.random.default_rng([E, K, N])
    w = np.swapaxes(_rows(rng, E * N, K).reshape(E, N, K), 1, 2)
    w = O.round_bf16(np.clip(w, -2.0 ** 60, 2.0 ** 60))
    codes, scales, scale = B.moe_fp4_quantize_weights(to_dev(w, BF), block)
    t = np.swapaxes(w, 1, 2).reshape(E * N, K)
    factor = None
    if block == 16:
        g = F.row_factor(np.abs(w).max((1, 2)))
        assert np.array_equal(f64(scale), g)
        factor = np.repeat(g, N)
    want, byte, _ = F.quantize_rows(t, block, factor)
    assert np.array_equal(i64(scales).reshape(E * N, -1), byte)
    assert np.array_equal(_bits(_nibbles(i64(codes)).reshape(E * N, K)), _bits(want))
    sf = B.moe_fp4_pack_scales(scales, block=block)
    assert np.array_equal(i64(sf), F.atoms_of_weights(i64(scales), K, block))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("I,K", [(64, 64), (192, 128), (128, 320), (384, 64)])
def test_gate_and_up_scales(block, I, K):
    rng = np.random.default_rng([I, K])
    a, b = (rng.integers(0, 127, size=(2, I, K // block)) for _ in range(2))
    sf = B.moe_fp4_pack_scales(to_dev(a, U8), to_dev(b, U8), block)
    assert np.array_equal(i64(sf), F.atoms_of_weights(a, K, block, b))


def _matrix(rng, E, N, K, block):
    """A plain 4-bit checkpoint [E, N, K] with every code: (codes, bytes, factors), on the device the
    same, and its values."""
    codes = rng.integers(0, 16, size=(E, N, K))
    if block == 16:
        byte = rng.integers(1, 126, size=(E, N, K // 16))
        byte = np.where(rng.random(byte.shape) < 0.9, rng.integers(40, 72, size=byte.shape), byte)
        g = (0.5 + rng.random(E)).astype(np.float32).astype(np.float64) * 2.0 ** -5
        val = F.restore(codes, byte, g[:, None] * np.ones((E, N)), block)
    else:
        byte, g = rng.integers(118, 124, size=(E, N, K // 32)), None
        val = F.restore(codes, byte, None, block)
    on = (to_dev(_pack(codes), U8), to_dev(byte, U8), None if g is None else to_dev(g, F32))
    return val, on


COUNTS = [
    (1, [1]), (1, [128]), (2, [0, 3]), (3, [129, 0, 256]), (4, [257, 1, 127, 30]), (5, [0, 0, 5, 0, 0]),
    (2, [300, 513]),
]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K,N", [(64, 8), (128, 128), (192, 200), (256, 256), (320, 392), (768, 512), (1408, 72)])
@pytest.mark.parametrize("E,counts", COUNTS)
def test_product(block, K, N, E, counts):
    rng = np.random.default_rng([K, N, E, block])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    x = O.round_bf16(rng.normal(size=(M, K)) * np.exp2(rng.integers(-3, 4, size=(M, 1))))
    val, (codes, byte, g) = _matrix(rng, E, N, K, block)
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    out = torch.full((M + 3, N), 7.0, dtype=BF, device=dev())
    y = B.moe_grouped_gemm_fp4(rows, off, (codes, B.moe_fp4_pack_scales(byte, block=block), g), block,
                               out=out[:M])
    xv = F.restore(*F.quantize_rows(x, block), block)
    want = F.grouped_product(xv, offsets, np.swapaxes(val, 1, 2))
    # each row by its own size: the rows' factors differ
    size = np.sqrt(np.mean(want ** 2, axis=1, keepdims=True)) + 1e-30
    assert_bf16_close(f64(y) / np.exp2(np.round(np.log2(size))), want / np.exp2(np.round(np.log2(size))), "y")
    assert (f64(out[M:]) == 7.0).all()


def test_rows_behind_the_last_expert_are_left():
    rng = np.random.default_rng(3)
    x = to_dev(O.round_bf16(rng.normal(size=(40, 128))), BF)
    off = to_dev(np.array([0, 7, 33]), I32)
    _, (codes, byte, g) = _matrix(rng, 2, 64, 128, 16)
    rows = B.moe_fp4_quantize_rows(x, off, 16)
    y = torch.full((40, 64), 7.0, dtype=BF, device=dev())
    B.moe_grouped_gemm_fp4(rows, off, (codes, B.moe_fp4_pack_scales(byte), g), out=y)
    assert (f64(y)[33:] == 7.0).all() and (f64(y)[:33] != 7.0).any(1).all()
    back = torch.full((40, 128), 7.0, dtype=BF, device=dev())
    B.moe_fp4_dequantize_rows(rows, off, out=back)
    assert (f64(back)[33:] == 7.0).all()


@pytest.mark.parametrize("block", [16, 32])
def test_a_row_that_is_not_finite_stays_alone(block):
    rng = np.random.default_rng(9)
    x = O.round_bf16(rng.normal(size=(200, 256)))
    x[3, 100], x[150, 7] = np.nan, np.inf
    off = to_dev(np.array([0, 100, 200]), I32)
    _, (codes, byte, g) = _matrix(rng, 2, 96, 256, block)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    y = f64(B.moe_grouped_gemm_fp4(rows, off, (codes, B.moe_fp4_pack_scales(byte, block=block), g), block))
    bad = np.zeros(200, dtype=bool)
    bad[[3, 150]] = True
    assert np.array_equal(np.isnan(y).all(1), bad) and np.isfinite(y[~bad]).all()


def _experts(rng, E, d, I, block):
    vals, on = zip(*[_matrix(rng, E, *s, block) for s in ((I, d), (I, d), (d, I))])
    (gq, gs, g1), (uq, us, u1), (dq, ds, d1) = on
    wgu = (gq, uq, B.moe_fp4_pack_scales(gs, us, block), g1, u1)
    return vals, wgu, (dq, B.moe_fp4_pack_scales(ds, block=block), d1)


@pytest.mark.parametrize("block,hidden", [(16, "fixed"), (16, "row"), (32, "block")])
@pytest.mark.parametrize("d,I,E,counts", [
    (64, 64, 1, [1]), (128, 128, 2, [0, 130]), (256, 192, 3, [31, 257, 4]), (192, 384, 2, [300, 5]),
    (2048, 768, 3, [2, 129, 0]), (320, 1408, 2, [17, 33]),
])
def test_experts(block, hidden, d, I, E, counts):
    rng = np.random.default_rng([d, I, E, block])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    (wg, wu, wd), wgu, wdown = _experts(rng, E, d, I, block)
    size = np.sqrt(np.mean(wg ** 2) * d)
    x = O.round_bf16(rng.normal(size=(M, d)) / size)     # G and U of size one
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    xv = F.restore(*F.quantize_rows(x, block), block)
    hs = (0.5 + rng.random(E)).astype(np.float32) * np.float32(4e-3) if hidden == "fixed" else None
    y = B.moe_grouped_ffn_fp4(rows, off, wgu, wdown, block,
                              h_scale=None if hs is None else to_dev(hs, F32))
    want, hv = F.grouped_ffn_fp4(xv, offsets, wg, wu, wd, block,
                                 h_scale=None if hs is None else hs.astype(np.float64),
                                 round_h=O.round_bf16 if hidden == "row" else None)
    rms = np.sqrt(np.mean(want ** 2))
    off_rows = (rounding_excess(f64(y), want) > 1e-3 * rms).any(1)
    # fp32 sums move H by about 2^-22 of its size; borders lie 1/8 of a value apart at least, so a
    # value meets one with a chance below 2^-18 (rounded to bf16 first: below 2^-12, where a bf16
    # step meets a border): a row of I values with I 2^-18 (I 2^-12)
    chance = I * (2.0 ** -12 if hidden == "row" else 2.0 ** -18)
    assert off_rows.sum() <= 3 + 3 * chance * M, off_rows.sum()
    assert np.sqrt(np.mean((f64(y) - want) ** 2)) <= 5e-3 * rms


@pytest.mark.parametrize("block,fixed", [(16, True), (16, False), (32, False)])
def test_experts_with_a_row_that_is_not_finite(block, fixed):
    rng = np.random.default_rng(11)
    _, wgu, wd = _experts(rng, 2, 128, 192, block)
    x = O.round_bf16(rng.normal(size=(150, 128)))
    x[0, 5], x[149, 100] = np.inf, np.nan
    off = to_dev(np.array([0, 20, 150]), I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    hs = torch.full((2,), 0.01, device=dev()) if fixed else None
    y = f64(B.moe_grouped_ffn_fp4(rows, off, wgu, wd, block, h_scale=hs))
    bad = np.zeros(150, dtype=bool)
    bad[[0, 149]] = True
    assert np.array_equal(np.isnan(y).all(1), bad) and np.isfinite(y[~bad]).all()


def test_empty_batches():
    off = torch.zeros(4, dtype=I32, device=dev())
    rows = B.moe_fp4_quantize_rows(torch.empty(0, 128, dtype=BF, device=dev()), off)
    _, wgu, wd = _experts(np.random.default_rng(1), 3, 128, 64, 16)
    assert B.moe_fp4_dequantize_rows(rows, off).shape == (0, 128)
    assert B.moe_grouped_ffn_fp4(rows, off, wgu, wd).shape == (0, 128)
    w = (wd[0], wd[1], wd[2])
    rows = B.moe_fp4_quantize_rows(torch.empty(0, 64, dtype=BF, device=dev()), off)
    assert B.moe_grouped_gemm_fp4(rows, off, w).shape == (0, 128)
