"""GPU parity of the products grouped by expert and their weight gradient with float64.

Products: fp32 sums of exact bf16 products, then one bf16 rounding: within half an ulp of the
stored value plus 1e-3 of the tensor's RMS. Weight gradients stay in fp32: a sum of n products
of size one, each addition rounded to 2^-24 of the running sum (the tensor cores may truncate:
2^-23), is off by at most n 2^-23 times the largest partial sum, in the mean far less; 1e-5 of
the RMS times the square root of the longest segment covers both."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


COUNTS = [[1], [0, 3], [129, 0, 256], [257, 1, 127, 30], [0, 0, 5, 0, 0], [16, 15, 17, 64]]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (200, 256), (520, 392), (2048, 16)])
@pytest.mark.parametrize("counts", COUNTS)
def test_product(trans, K, N, counts):
    rng = np.random.default_rng([K, N, len(counts)])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M, E = int(offsets[-1]), len(counts)
    x = O.round_bf16(rng.normal(size=(M, K)))
    w = O.round_bf16(rng.normal(size=(E, K, N)))
    out = torch.full((M + 5, N), 7.0, dtype=BF, device=dev())
    off = to_dev(offsets, I32)
    y = B.moe_grouped_gemm(to_dev(x, BF), off, to_dev(np.swapaxes(w, 1, 2) if trans else w, BF), trans,
                           out=out[:M])
    assert_bf16_close(f64(y), F.grouped_product(x, offsets, w), "y")
    assert (f64(out[M:]) == 7.0).all()


def _wgrad(x, dy, offsets):
    return np.stack([x[a:b].T @ dy[a:b] for a, b in zip(offsets[:-1], offsets[1:])])


def _dw_close(got, want, counts):
    tol = 1e-5 * np.sqrt(max(counts)) * np.sqrt(np.mean(want ** 2))
    assert np.abs(got - want).max() <= tol


@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (264, 264), (520, 40)])
@pytest.mark.parametrize("counts", COUNTS)
def test_weight_gradient(K, N, counts):
    rng = np.random.default_rng([K, N, len(counts), 1])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M, E = int(offsets[-1]), len(counts)
    x, dy = O.round_bf16(rng.normal(size=(M, K))), O.round_bf16(rng.normal(size=(M, N)))
    x2, dy2 = O.round_bf16(rng.normal(size=(M, K))), O.round_bf16(rng.normal(size=(M, N)))
    off = to_dev(offsets, I32)
    dw = B.moe_grouped_gemm_wgrad(to_dev(x, BF), to_dev(dy, BF), off)
    one = _wgrad(x, dy, offsets)
    _dw_close(f64(dw), one, counts)
    assert (f64(dw)[np.array(counts) == 0] == 0).all()
    again = B.moe_grouped_gemm_wgrad(to_dev(x2, BF), to_dev(dy2, BF), off, accumulate=True, out=dw)
    assert again is dw
    _dw_close(f64(dw), one + _wgrad(x2, dy2, offsets), counts)


def test_many_experts():
    """Past the expert counts up to which the deeper rings' tables fit."""
    rng = np.random.default_rng(600)
    counts = rng.integers(0, 4, size=600)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    x, dy = O.round_bf16(rng.normal(size=(M, 72))), O.round_bf16(rng.normal(size=(M, 40)))
    w = O.round_bf16(rng.normal(size=(600, 72, 40)))
    off = to_dev(offsets, I32)
    assert_bf16_close(f64(B.moe_grouped_gemm(to_dev(x, BF), off, to_dev(w, BF))),
                      F.grouped_product(x, offsets, w), "y")
    _dw_close(f64(B.moe_grouped_gemm_wgrad(to_dev(x, BF), to_dev(dy, BF), off)), _wgrad(x, dy, offsets),
              [4])


def test_gradients_by_differences():
    """loss = sum(y r): central differences of the float64 product against the three calls."""
    rng = np.random.default_rng(2)
    offsets = np.array([0, 5, 5, 12])
    x, w = O.round_bf16(rng.normal(size=(12, 16))), O.round_bf16(rng.normal(size=(3, 16, 24)))
    r = O.round_bf16(rng.normal(size=(12, 24)))
    off = to_dev(offsets, I32)
    dx = f64(B.moe_grouped_gemm(to_dev(r, BF), off, to_dev(w, BF), trans=True))
    dw = f64(B.moe_grouped_gemm_wgrad(to_dev(x, BF), to_dev(r, BF), off))
    loss = lambda a, b: (F.grouped_product(a, offsets, b) * r).sum()   # noqa: E731
    for _ in range(20):
        i = (rng.integers(12), rng.integers(16))
        e = np.zeros_like(x)
        e[i] = 1e-3
        d = (loss(x + e, w) - loss(x - e, w)) / 2e-3
        assert abs(dx[i] - d) <= 2.0 ** -8 * abs(d) + 1e-6
        i = (rng.integers(3), rng.integers(16), rng.integers(24))
        e = np.zeros_like(w)
        e[i] = 1e-3
        d = (loss(x, w + e) - loss(x, w - e)) / 2e-3
        assert abs(dw[i] - d) <= 1e-5 * max(1.0, abs(d))


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_rows_that_are_not_finite_stay_with_their_expert(value):
    rng = np.random.default_rng(4)
    counts = [13, 0, 21, 70, 3]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    x, dy = rng.normal(size=(107, 72)), rng.normal(size=(107, 40))
    x[offsets[2]:offsets[3]] = value          # all rows of experts 2 and 4
    dy[offsets[4]:] = value
    x, dy = O.round_bf16(x), O.round_bf16(dy)
    dw = f64(B.moe_grouped_gemm_wgrad(to_dev(x, BF), to_dev(dy, BF), to_dev(offsets, I32)))
    fine = [0, 1, 3]
    assert np.isfinite(dw[fine]).all() and not np.isfinite(dw[[2, 4]]).any()
    clean = _wgrad(np.nan_to_num(x, nan=0, posinf=0), np.nan_to_num(dy, nan=0, posinf=0), offsets)
    _dw_close(dw[fine], clean[fine], counts)
    w = to_dev(O.round_bf16(rng.normal(size=(5, 72, 40))), BF)
    y = f64(B.moe_grouped_gemm(to_dev(x, BF), to_dev(offsets, I32), w))
    bad = np.zeros(107, dtype=bool)
    bad[offsets[2]:offsets[3]] = True
    assert np.array_equal(~np.isfinite(y).any(1), bad) and np.isfinite(y[~bad]).all()


def test_rows_behind_the_last_expert():
    """They are not written, and what they hold reaches no gradient."""
    rng = np.random.default_rng(6)
    x, dy = rng.normal(size=(60, 64)), rng.normal(size=(60, 72))
    x[41:], dy[41:] = np.nan, np.nan
    x, dy = O.round_bf16(x), O.round_bf16(dy)
    offsets = np.array([0, 20, 41])
    off = to_dev(offsets, I32)
    y = torch.full((60, 72), 7.0, dtype=BF, device=dev())
    B.moe_grouped_gemm(to_dev(x, BF), off, to_dev(O.round_bf16(rng.normal(size=(2, 64, 72))), BF), out=y)
    assert (f64(y)[41:] == 7.0).all() and np.isfinite(f64(y)).all()
    _dw_close(f64(B.moe_grouped_gemm_wgrad(to_dev(x, BF), to_dev(dy, BF), off)), _wgrad(x, dy, offsets), [20])


def test_empty_batches():
    off = torch.zeros(3, dtype=I32, device=dev())
    x, dy = torch.empty(0, 64, dtype=BF, device=dev()), torch.empty(0, 72, dtype=BF, device=dev())
    assert B.moe_grouped_gemm(x, off, torch.ones(2, 64, 72, dtype=BF, device=dev())).shape == (0, 72)
    dw = torch.ones(2, 64, 72, device=dev())
    assert (f64(B.moe_grouped_gemm_wgrad(x, dy, off, accumulate=True, out=dw)) == 1).all()
    assert (f64(B.moe_grouped_gemm_wgrad(x, dy, off, out=dw)) == 0).all()
