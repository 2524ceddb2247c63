"""GPU parity of the 8-bit activation checkpoints with the CPU oracle.

Codes, scales and restored rows are bit-exact (each step of the definition is
one correctly rounded fp32 operation, and code times scale is exact); h is
within half a bf16 ulp plus 1e-3 of its RMS; dtopk_w, an fp32 sum of d products
in some order, within (d + 16) 2^-24 of the sum of their magnitudes."""
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


def _rows(seed, M, N):
    """Rows of very different sizes, with zero blocks, ties and tiny values among them."""
    rng = np.random.default_rng([seed, M, N])
    x = rng.normal(size=(M, N)) * 10.0 ** rng.integers(-5, 5, size=(M, 1))
    x[rng.random((M, N)) < 0.05] = 0.0
    x[M // 2, :32] = 0.0
    x[M // 3] = rng.integers(-254, 255, size=N) / 2.0      # halves of a step of 1
    x[M // 3, 0::32] = 127.0
    x[M - 1] *= 1e-36
    return O.round_bf16(x)


SHAPES = [(1, 8), (1, 2048), (3, 40), (5, 24), (64, 136), (257, 1536), (1000, 2048), (33, 8200)]


@pytest.mark.parametrize("M,N", SHAPES)
def test_pack_and_restore(M, N):
    x = _rows(1, M, N)
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    rq, rs = K.ckpt8_pack(x)
    assert np.array_equal(f64(s), rs)
    assert np.array_equal(i64(q), rq)
    back = B.moe_ckpt8_dispatch(q, s)
    assert np.array_equal(f64(back), O.round_bf16(K.ckpt8_restore(rq, rs)))


def test_values_that_are_not_finite():
    x = _rows(2, 8, 72)
    x[2, 5], x[2, 70], x[3, 33], x[4, :32] = np.inf, -np.inf, np.nan, np.inf
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    rq, rs = K.ckpt8_pack(x)
    assert np.array_equal(i64(q), rq) and np.array_equal(f64(s), rs)
    back = f64(B.moe_ckpt8_dispatch(q, s))
    assert np.array_equal(np.isnan(back), ~np.isfinite(x))


def test_largest_and_smallest_values():
    big = float(torch.finfo(BF).max)
    x = np.zeros((3, 32))
    x[0, :3] = [big, -big, big / 4]
    x[1, :3] = [2.0 ** -133, -2.0 ** -126, 2.0 ** -120]     # below the smallest scale's step
    x[2, 0] = 2.0 ** -100
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    rq, rs = K.ckpt8_pack(x)
    assert np.array_equal(i64(q), rq) and np.array_equal(f64(s), rs)


@pytest.mark.parametrize("T,d,E,k", [(1, 8, 4, 4), (100, 136, 16, 3), (513, 2048, 64, 8),
                                     (64, 520, 64, 16), (40, 72, 40, 32), (77, 264, 8, 1)])
def test_dispatch(T, d, E, k):
    x = _rows(3, T, d)
    rng = np.random.default_rng(T)
    inv = rng.permutation(T * k)
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    xp = B.moe_ckpt8_dispatch(q, s, to_dev(inv, I32), k)
    want = O.round_bf16(K.ckpt8_restore(*K.ckpt8_pack(x)))
    assert np.array_equal(f64(xp)[inv], np.repeat(want, k, axis=0))


@pytest.mark.parametrize("M,I", [(1, 8), (3, 24), (70, 136), (333, 768), (64, 1408), (1000, 200)])
def test_swiglu(M, I):
    x = O.round_bf16(np.random.default_rng([M, I]).normal(size=(M, 2 * I)) * 4.0)
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    gu, h = B.moe_ckpt8_swiglu(q, s)
    rgu, rh = K.ckpt8_swiglu(i64(q), f64(s))
    assert np.array_equal(f64(gu), O.round_bf16(rgu))
    assert_bf16_close(f64(h), rh, "h")


def test_swiglu_of_large_gates():
    x = np.zeros((2, 64))
    x[0, :3], x[0, 32:35] = [200.0, -200.0, 100.0], [1.0, 1.0, -2.0]
    x[1, :2], x[1, 32:34] = [3e38, -3e38], [1.0, 1.0]
    q, s = B.moe_ckpt8_pack(to_dev(x, BF))
    _, h = B.moe_ckpt8_swiglu(q, s)
    _, rh = K.ckpt8_swiglu(i64(q), f64(s))
    got = f64(h)
    assert np.isfinite(got).all()
    assert (np.abs(got - rh) <= 2.0 ** -8 * np.abs(rh) + 1e-30).all()


@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (33, 136, 3), (257, 2048, 8), (50, 4104, 6),
                                   (20, 72, 32)])
def test_combine_backward(T, d, k):
    rng = np.random.default_rng([T, d, k])
    dout, y = O.round_bf16(rng.normal(size=(T, d))), _rows(4, T * k, d)
    w, inv = rng.random((T, k)).astype(np.float32), rng.permutation(T * k)
    q, s = B.moe_ckpt8_pack(to_dev(y, BF))
    dy, dw = B.moe_ckpt8_combine_backward(to_dev(dout, BF), q, s, to_dev(w, F32), to_dev(inv, I32))
    yr = K.ckpt8_restore(*K.ckpt8_pack(y))
    at = inv.reshape(T, k)
    terms = dout[:, None, :] * yr[at]
    assert (np.abs(f64(dw) - terms.sum(2)) <= (d + 16) * 2.0 ** -24 * np.abs(terms).sum(2)).all()
    want = O.round_bf16(w.astype(np.float64)[:, :, None] * dout[:, None, :])
    assert np.array_equal(f64(dy)[at], want)
    # the bf16 call on the restored rows gives the same dy bits
    back = B.moe_ckpt8_dispatch(q, s)
    assert torch.equal(dy, B.moe_combine_backward(to_dev(dout, BF), back, to_dev(w, F32),
                                                  to_dev(inv, I32))[0])


@pytest.mark.parametrize("N", [8192, 8208])
def test_past_two_to_the_31_elements(N):
    """Rows whose offsets pass 32 bits: the last rows as in a call of their own."""
    M = 262400
    x = torch.zeros(M, N, dtype=BF, device=dev())
    tail = torch.randn(40, N, device=dev()).to(BF)
    x[-40:] = tail
    q, s = B.moe_ckpt8_pack(x)
    qt, st = B.moe_ckpt8_pack(tail)
    assert torch.equal(q[-40:], qt) and torch.equal(s[-40:], st)
    assert not q[:-40].any()
    back = B.moe_ckpt8_dispatch(q, s, out=x)
    assert torch.equal(back[-40:], B.moe_ckpt8_dispatch(qt, st))
    _, h = B.moe_ckpt8_swiglu(q, s, out=(x, torch.empty(M, N // 2, dtype=BF, device=dev())))
    assert torch.equal(h[-40:], B.moe_ckpt8_swiglu(qt, st)[1])


def test_a_mark_reaches_the_gradients():
    T, d, k = 4, 64, 2
    rng = np.random.default_rng(8)
    y = rng.normal(size=(T * k, d))
    inv = np.arange(T * k)
    y[3, 9] = np.inf
    q, s = B.moe_ckpt8_pack(to_dev(y, BF))
    _, dw = B.moe_ckpt8_combine_backward(to_dev(rng.normal(size=(T, d)), BF), q, s,
                                         to_dev(rng.random((T, k)), F32), to_dev(inv, I32))
    assert np.array_equal(np.isnan(f64(dw)).reshape(-1), inv == 3)


def test_gradients_that_are_not_finite():
    """Infinities and NaN of dout go into their own elements of dy, and into their token's dw."""
    T, d, k = 6, 72, 3
    rng = np.random.default_rng(9)
    dout, w, inv = O.round_bf16(rng.normal(size=(T, d))), rng.random((T, k)) + 0.1, rng.permutation(T * k)
    dout[1, 4], dout[1, 9], dout[4, 70] = np.inf, -np.inf, np.nan
    q, s = B.moe_ckpt8_pack(to_dev(O.round_bf16(rng.normal(size=(T * k, d))), BF))
    dy, dw = B.moe_ckpt8_combine_backward(to_dev(dout, BF), q, s, to_dev(w, F32), to_dev(inv, I32))
    got = f64(dy)[inv.reshape(T, k)]
    want = w.astype(np.float32).astype(np.float64)[:, :, None] * dout[:, None, :]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    assert np.array_equal(np.sign(got[np.isinf(got)]), np.sign(want[np.isinf(want)]))
    rows = np.isfinite(dout).all(1)
    assert np.array_equal(np.isfinite(f64(dw)).all(1), rows)


def test_no_rows():
    none = torch.empty(0, 64, dtype=BF, device=dev())
    q, s = B.moe_ckpt8_pack(none)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    assert B.moe_ckpt8_dispatch(q, s).shape == (0, 64)
    gu, h = B.moe_ckpt8_swiglu(q, s)
    assert gu.shape == (0, 64) and h.shape == (0, 32)


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF, device=dev())
    q, s = B.moe_ckpt8_pack(x)
    with pytest.raises(B.MoEError) as e:
        B.moe_ckpt8_pack(torch.zeros(4, 12, dtype=BF, device=dev()))
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        B.moe_ckpt8_pack(x.float())
    with pytest.raises(ValueError):
        B.moe_ckpt8_pack(x[:, :32])
    with pytest.raises(ValueError):
        B.moe_ckpt8_dispatch(q, s[:, :1].contiguous())
    with pytest.raises(ValueError):
        B.moe_ckpt8_dispatch(q, s, torch.zeros(4, dtype=I32, device=dev()), 2)
    with pytest.raises(B.MoEError):
        B.moe_ckpt8_dispatch(q, s, K=33)
    with pytest.raises(B.MoEError) as e:       # I = 4
        B.moe_ckpt8_swiglu(torch.zeros(2, 8, dtype=torch.int8, device=dev()),
                           torch.ones(2, 1, dtype=BF, device=dev()))
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        B.moe_ckpt8_combine_backward(x, q, s, torch.ones(4, 2, device=dev()),
                                     torch.zeros(8, dtype=I32, device=dev()))
