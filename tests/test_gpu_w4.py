"""GPU parity of the 4-bit experts with the CPU oracle.

Codes and scales are bit-exact. h and y are bf16 roundings of fp32 sums of exact
products: within half a bf16 ulp of the oracle plus 1e-3 of the tensor's RMS (y
against the product of the stored h)."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import block as K
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, i64, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _nibbles(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def _matrix(rng, E, N, Kd, group):
    """(codes 0 .. 15, scales) with every code and scales of different sizes."""
    codes = rng.integers(0, 16, size=(E, N, Kd))
    s = O.round_bf16((0.2 + rng.random((E, N, Kd // group))) * 0.02)
    return codes, s


def _plain(m):
    return to_dev(_nibbles(m[0]), torch.uint8), to_dev(m[1], BF)


def _experts(seed, E, d, I, g_gu, g_d):
    rng = np.random.default_rng(seed)
    mats = [_matrix(rng, E, I, d, g_gu), _matrix(rng, E, I, d, g_gu), _matrix(rng, E, d, I, g_d)]
    wgu = B.moe_w4_pack_weights(*_plain(mats[0]), *_plain(mats[1]))
    wd = B.moe_w4_pack_weights(*_plain(mats[2]))
    return [K.w4_values(*m) for m in mats], wgu, wd


def _check(x, offsets, vals, wgu, wd):
    y, h = B.moe_grouped_ffn_w4(to_dev(x, BF), to_dev(offsets, I32), wgu, wd)
    ry, rh = K.grouped_ffn_w4(x, offsets, *vals, h=f64(h))
    assert_bf16_close(f64(h), rh, "h")
    assert_bf16_close(f64(y), ry, "y")
    return y, h


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("E,Kd,N", [(1, 128, 8), (3, 256, 40), (5, 640, 136)])
def test_quantize(E, Kd, N, group):
    w = O.round_bf16(np.random.default_rng([E, Kd, N]).normal(size=(E, Kd, N)) * 0.02)
    w[0, :group, 0] = 0.0
    codes, s = B.moe_w4_quantize_weights(to_dev(w, BF), group)
    rq, rs = K.w4_quantize(w, group)
    assert np.array_equal(f64(s), rs)
    c = i64(codes)
    assert np.array_equal(np.stack([c & 15, c >> 4], -1).reshape(rq.shape), rq)


@pytest.mark.parametrize("E,d,I,g_gu,g_d,counts", [
    (1, 64, 64, 64, 64, [1]),
    (1, 64, 64, 32, 32, [8]),
    (2, 128, 64, 128, 64, [0, 3]),
    (4, 256, 320, 64, 32, [7, 0, 8, 9]),
    (3, 2048, 768, 128, 128, [1, 1, 1]),
    (3, 768, 1408, 32, 128, [16, 17, 31]),
    (2, 192, 704, 64, 64, [32, 33]),
    (3, 512, 256, 128, 32, [65, 0, 100]),
    (40, 128, 128, 32, 64, [0] * 17 + [2] + [0] * 15 + [1] + [0] * 6),   # slots past a ballot
    (2, 4096, 128, 128, 128, [5, 12]),
    # the persistent kernel: rows past a pass of 8, empty experts between, uneven k-tiles
    (16, 1024, 704, 64, 64, [1, 0, 9, 8, 0, 3, 17, 0, 0, 2, 8, 1, 7, 0, 0, 16]),
    (96, 512, 192, 32, 64, [i * 7 % 11 for i in range(96)]),
    (24, 2048, 768, 128, 32, [8] * 24),
    (300, 1152, 128, 64, 32, [i % 3 for i in range(300)]),
    (12, 4096, 1024, 128, 128, [5, 0, 7, 8, 1, 1, 9, 0, 2, 3, 4, 6]),
    (40, 1024, 1408, 64, 64, [i * 5 % 9 for i in range(39)] + [17]),
    (32, 1024, 1408, 64, 32, [i * 7 % 19 for i in range(32)]),            # up to 16 rows an entry
    (24, 1152, 1472, 128, 32, [16, 17, 8, 0] * 5 + [33, 1, 15, 9]),
])
def test_ffn(E, d, I, g_gu, g_d, counts):
    vals, wgu, wd = _experts([E, d, I], E, d, I, g_gu, g_d)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    x = O.round_bf16(np.random.default_rng(d).normal(size=(offsets[-1], d)))
    _check(x, offsets, vals, wgu, wd)


@pytest.mark.parametrize("E,d,I,rows", [(2, 256, 128, 5), (24, 2048, 768, 8), (40, 1024, 1408, 3)])
def test_large_elements_under_codes_of_eight(E, d, I, rows):
    """Elements 2^12 times the others whose weights are zero leave nothing in the sums."""
    rng = np.random.default_rng([E, d])
    at = np.arange(7, d, 256)
    mats = [_matrix(rng, E, I, d, 64), _matrix(rng, E, I, d, 64), _matrix(rng, E, d, I, 64)]
    for codes, _ in mats[:2]:
        codes[:, :, at] = 8
    wgu = B.moe_w4_pack_weights(*_plain(mats[0]), *_plain(mats[1]))
    wd = B.moe_w4_pack_weights(*_plain(mats[2]))
    x = rng.normal(size=(E * rows, d))
    x[:, at] *= 4096.0
    _check(O.round_bf16(x), np.arange(E + 1) * rows, [K.w4_values(*m) for m in mats], wgu, wd)


@pytest.mark.parametrize("E,d,I,rows", [(2, 256, 128, 5), (24, 2048, 768, 8), (2, 256, 128, 20)])
def test_rows_that_are_not_finite_stay_apart(E, d, I, rows):
    """A row with an infinity and one with a NaN: not finite themselves, the others' bits kept."""
    _, wgu, wd = _experts([E, d, 1], E, d, I, 64, 64)
    x = O.round_bf16(np.random.default_rng(d).normal(size=(E * rows, d)))
    offsets = to_dev(np.arange(E + 1) * rows, I32)
    y, h = B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd)
    bad = [1, rows + 2]
    x[bad[0], 3], x[bad[1], d - 1] = np.inf, np.nan
    y2, h2 = B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd)
    rest = torch.ones(E * rows, dtype=torch.bool, device=y.device)
    rest[bad] = False
    assert torch.equal(y[rest], y2[rest]) and torch.equal(h[rest], h2[rest])
    assert not torch.isfinite(y2[bad].float()).any()


@pytest.mark.parametrize("T,k,E", [(1, 1, 4), (1, 4, 4), (3, 2, 16), (16, 6, 8), (64, 2, 8)])
def test_rows_through_the_permutation(T, k, E):
    """Tokens read through moe_build_permutation's perm: the dispatched call's bits."""
    d, I = 256, 128
    vals, wgu, wd = _experts([T, k], E, d, I, 64, 32)
    rng = np.random.default_rng(T)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    x = to_dev(O.round_bf16(rng.normal(size=(T, d))), BF)
    _, offsets, perm, _ = B.moe_build_permutation(to_dev(idx, I32), E)
    y, h = B.moe_grouped_ffn_w4(x, offsets, wgu, wd, perm=perm, K=k)
    xp = B.moe_dispatch(x, perm, k)
    y2, h2 = _check(f64(xp), i64(offsets), vals, wgu, wd)
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_a_row_does_not_depend_on_the_batch_it_is_in():
    """Rows of one expert in a batch of 40 against batches of the same size class."""
    vals, wgu, wd = _experts(3, 1, 512, 256, 64, 64)
    x = O.round_bf16(np.random.default_rng(3).normal(size=(40, 512)))
    y, _ = _check(x, np.array([0, 40]), vals, wgu, wd)
    x2 = x.copy()
    x2[1:] = 0.0
    y2, _ = B.moe_grouped_ffn_w4(to_dev(x2, BF), to_dev(np.array([0, 40]), I32), wgu, wd)
    assert torch.equal(y[0], y2[0]) and (y2[1:] == 0).all()


def test_quantized_bf16_weights_end_to_end():
    """bf16 weights quantized and laid out here, against the oracle's own quantization of them."""
    E, d, I = 2, 256, 192
    rng = np.random.default_rng(0)
    w = [O.round_bf16(rng.normal(size=(E, a, b)) * 0.05) for a, b in ((d, I), (d, I), (I, d))]
    plain = [B.moe_w4_quantize_weights(to_dev(m, BF), 32) for m in w]
    wgu = B.moe_w4_pack_weights(*plain[0], *plain[1])
    wd = B.moe_w4_pack_weights(*plain[2])
    vals = [K.w4_values(*K.w4_quantize(m, 32)) for m in w]
    _check(O.round_bf16(rng.normal(size=(24, d))), np.array([0, 10, 24]), vals, wgu, wd)


def test_weights_past_two_to_the_31_bytes():
    """The last of many experts, whose weights lie past 4 GB."""
    E, d, I, g = 272, 4096, 4096, 128
    dv = dev()
    codes = [torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device=dv)
             for n, k in ((I, d), (I, d), (d, I))]
    scales = [((torch.rand(E, n, k // g, device=dv) + 0.2) * 0.004).to(BF)
              for n, k in ((I, d), (I, d), (d, I))]
    wgu = B.moe_w4_pack_weights(codes[0], scales[0], codes[1], scales[1])
    wd = B.moe_w4_pack_weights(codes[2], scales[2])
    assert wgu[0].numel() > 1 << 32 and wd[0].numel() > 1 << 31
    x = O.round_bf16(np.random.default_rng(7).normal(size=(5, d)))
    counts = np.zeros(E, dtype=np.int64)
    counts[0], counts[-1] = 2, 3
    offsets = np.concatenate([[0], np.cumsum(counts)])
    y, h = B.moe_grouped_ffn_w4(to_dev(x, BF), to_dev(offsets, I32), wgu, wd)
    vals = []
    for c, s in zip(codes, scales):
        c = i64(c[[0, -1]])
        q = np.stack([c & 15, c >> 4], -1).reshape(2, c.shape[1], -1)
        vals.append(K.w4_values(q, f64(s[[0, -1]])))
    ry, rh = K.grouped_ffn_w4(x, np.array([0, 2, 5]), *vals, h=f64(h))
    assert_bf16_close(f64(h), rh, "h")
    assert_bf16_close(f64(y), ry, "y")


def test_not_finite_rows_stay_apart():
    vals, wgu, wd = _experts(4, 2, 128, 128, 32, 32)
    x = O.round_bf16(np.random.default_rng(4).normal(size=(12, 128)))
    offsets = np.array([0, 5, 12])
    y, _ = _check(x, offsets, vals, wgu, wd)
    x[2, 3] = np.nan
    x[9, 100] = np.inf
    y2, _ = B.moe_grouped_ffn_w4(to_dev(x, BF), to_dev(offsets, I32), wgu, wd)
    keep = [i for i in range(12) if i not in (2, 9)]
    assert torch.equal(y[keep], y2[keep]) and y2[2].isnan().all()


def test_no_rows():
    _, wgu, wd = _experts(5, 3, 64, 64, 32, 32)
    x = torch.empty(0, 64, dtype=BF, device=dev())
    y, h = B.moe_grouped_ffn_w4(x, torch.zeros(4, dtype=I32, device=dev()), wgu, wd)
    assert y.shape == (0, 64) and h.shape == (0, 64)


def test_refusals():
    _, wgu, wd = _experts(6, 2, 128, 64, 64, 64)
    x = torch.zeros(4, 128, dtype=BF, device=dev())
    off = torch.tensor([0, 2, 4], dtype=I32, device=dev())
    with pytest.raises(ValueError):
        B.moe_w4_quantize_weights(torch.zeros(1, 96, 8, dtype=BF, device=dev()), 32)   # K % 64
    with pytest.raises(ValueError):
        B.moe_w4_quantize_weights(torch.zeros(1, 128, 8, dtype=BF, device=dev()), 48)
    codes = torch.zeros(1, 12, 64, dtype=torch.uint8, device=dev())
    with pytest.raises(ValueError):
        B.moe_w4_pack_weights(codes, torch.ones(1, 12, 2, dtype=BF, device=dev()))     # N % 32
    with pytest.raises(ValueError):
        B.moe_w4_pack_weights(codes, torch.ones(1, 12, 2, dtype=BF, device=dev()), codes, None)
    with pytest.raises(ValueError):
        B.moe_grouped_ffn_w4(x, off, wd, wgu)
    with pytest.raises(ValueError):
        B.moe_grouped_ffn_w4(x[:, :64].contiguous(), off, wgu, wd)
    with pytest.raises(ValueError):
        B.moe_grouped_ffn_w4(x, off[:2], wgu, wd)
    with pytest.raises(ValueError):
        B.moe_grouped_ffn_w4(x, off, wgu, wd, perm=torch.zeros(4, dtype=I32, device=dev()), K=2)
    with pytest.raises(TypeError):
        B.moe_grouped_ffn_w4(x.float(), off, wgu, wd)
    with pytest.raises(B.MoEError) as e:
        B.moe_grouped_ffn_w4(x, off, wgu, wd, ws=torch.zeros(16, dtype=torch.uint8, device=dev()))
    assert e.value.status == B.MOE_ERR_WORKSPACE
