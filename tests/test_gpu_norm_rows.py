"""GPU parity of the block's norms where one row group takes many rows: the rings in
shared memory wrap, look-ups run ahead of their row, gate rows change within a group
and the gradients' sums are joined from many groups. The largest row counts too.

Tolerances as in test_gpu_norm.py (u = 2^-24): bf16 results half an ulp of the stored
value plus 1e-3 of the tensor's RMS; rstd (d + 16) u, relative; fp32 sums of n
products (n + 16) u of the sum of the products' magnitudes."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import block as K
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def test_the_most_rows_an_int_holds():
    """T = 2^31 - 1: the first and last rows of norm_in and norm_out against the oracle."""
    T, d, n = 2 ** 31 - 1, 8, 64
    x = torch.zeros(T, d, dtype=BF, device=dev())
    ends = torch.randn(2 * n, d, device=dev()).to(BF)
    x[:n], x[-n:] = ends[:n], ends[n:]
    gain = torch.rand(d, device=dev()) + 0.5
    xn, r = B.moe_norm_in(x, gain)
    want, rw = K.norm_in(f64(ends), f64(gain), EPS)
    assert_bf16_close(f64(torch.cat([xn[:n], xn[-n:]])), want, "xn")
    assert (np.abs(f64(torch.cat([r[:n], r[-n:]])) - rw) <= (d + 16) * U * rw).all()
    del r
    normed = torch.cat([xn[:n], xn[-n:]])
    B.moe_norm_out(xn, x, gain, out=(x, None, None))     # in place on the residual stream
    want, _, _ = K.norm_out(f64(normed), f64(ends), f64(gain), None, None, 1, None, None, 1, 1.0, EPS)
    assert_bf16_close(f64(torch.cat([x[:n], x[-n:]])), want, "out")


@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("cols", [1, 64])
def test_an_empty_batch_keeps_its_shapes(rows, cols):
    """No tokens, K = 8: what a batch that routed nothing passes on, with a gate per channel or
    one for the model (one row) or per token (no row); its sums are zero."""
    d, k = 64, 8
    none = torch.empty(0, d, dtype=BF, device=dev())
    gain, gate = torch.ones(d, device=dev()), torch.ones(rows, cols, device=dev())
    w, inv = torch.empty(0, k, device=dev()), torch.empty(0, dtype=I32, device=dev())
    out, z, r = B.moe_norm_out(none, none, gain, w, inv, none, gate)
    assert out.shape == (0, d) and z.shape == (0, d) and r.shape == (0,)
    dgate = torch.full_like(gate, 7.0)
    dgain = torch.full_like(gain, 7.0)
    B.moe_norm_out_backward(none, none, r, gain, gate, out=(none, dgain, dgate))
    assert (dgate == 0).all() and (dgain == 0).all()
    _, _, dgate = B.moe_norm_out_backward(none, none, None, None, gate)
    assert (dgate == 0).all()
    with pytest.raises(ValueError):
        B.moe_norm_out(none, none, gain, gate=torch.ones(2, cols, device=dev()))


def _bf(rng, *shape, scale=1.0):
    return O.round_bf16(rng.normal(size=shape) * scale)


def _f32(rng, *shape):
    return (0.5 + rng.random(shape)).astype(np.float32).astype(np.float64)


def _rows_sum(terms, span):
    """Sums over rows of `span` terms each, the last perhaps shorter: (sums, bounds)."""
    at = np.arange(0, terms.shape[0], span)
    n = np.minimum(span, terms.shape[0] - at)[:, None]
    return np.add.reduceat(terms, at), (n + 16) * U * np.add.reduceat(np.abs(terms), at) + 1e-35


def assert_sums(got, terms, span, cols, name):
    """fp32 sums over rows of `span` terms, over the columns too with one column."""
    want, bound = _rows_sum(terms, span)
    if cols == 1:
        n = np.minimum(span, terms.shape[0] - np.arange(0, terms.shape[0], span)) * terms.shape[1]
        mag = _rows_sum(np.abs(terms), span)[0].sum(1, keepdims=True)
        want, bound = want.sum(1, keepdims=True), (n[:, None] + 16) * U * mag + 1e-35
    err = np.abs(f64(got).reshape(want.shape) - want)
    assert (err <= bound).all(), f"{name}: {(err / bound).max():.2f} of the bound"


# 1, 2 and 4 vectors a thread; on 152 SMs 7, 5, 7, 15 and 14 rows a group, the last rows short
@pytest.mark.parametrize("T,d", [(30001, 136), (12001, 264), (15001, 512), (9000, 2048),
                                 (2000, 8200)])
def test_norm_in(T, d):
    rng = np.random.default_rng([T, d])
    x, gain = _bf(rng, T, d, scale=3.0), _f32(rng, d)
    xn, r = B.moe_norm_in(to_dev(x, BF), to_dev(gain, F32), EPS)
    ref, rr = K.norm_in(x, gain, EPS)
    assert (np.abs(f64(r) - rr) <= (d + 16) * U * rr).all()
    assert_bf16_close(f64(xn), ref, "xn")


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("T,d", [(30001, 136), (5003, 2056), (2001, 8200)])
def test_norm_in_backward(T, d, with_res):
    rng = np.random.default_rng([T, d, 1])
    x, gain, dxn = _bf(rng, T, d, scale=3.0), _f32(rng, d), _bf(rng, T, d)
    dres = _bf(rng, T, d) if with_res else None
    r = K.norm_in(x, gain, EPS)[1].astype(np.float32).astype(np.float64)
    dx, dgain = B.moe_norm_in_backward(to_dev(dxn, BF), to_dev(x, BF), to_dev(gain, F32),
                                       to_dev(r, F32), to_dev(dres, BF) if with_res else None)
    assert_bf16_close(f64(dx), K.norm_in_backward(dxn, x, gain, r, dres)[0], "dx")
    assert_sums(dgain, dxn * x * r[:, None], T, d, "dgain")


# rings of two stages (10 and 9 arrays) and of four (2 to 4 arrays), with 10, 7, 14 and 7 rows a
# group or more; gates whose row changes within a group
@pytest.mark.parametrize("T,d,k,shared,with_gain,rows,span", [
    (3001, 2048, 8, True, True, "vector", 7),
    (3001, 2048, 8, False, True, "vector", 700),
    (3001, 2048, 8, False, False, "one", 3),
    (5003, 1032, 2, True, True, "one", 1),
    (5003, 1032, 2, False, True, None, 1),
    (5003, 1032, 3, False, False, "vector", 2),
    (40001, 64, 1, False, True, "one", 40001),
    (40001, 64, 1, True, True, "vector", 5),
    (2003, 7168, 3, False, True, "vector", 11),
    (1501, 264, 31, True, True, "one", 400),
])
def test_norm_out(T, d, k, shared, with_gain, rows, span):
    rng = np.random.default_rng([T, d, k])
    y, resid = _bf(rng, T * k, d), _bf(rng, T, d, scale=3.0)
    sh = _bf(rng, T, d) if shared else None
    w, inv, gain = _f32(rng, T, k), rng.permutation(T * k), _f32(rng, d) if with_gain else None
    gate = None if rows is None else _f32(rng, -(-T // span), d if rows == "vector" else 1)
    out, z, r = B.moe_norm_out(
        to_dev(y, BF), to_dev(resid, BF), None if gain is None else to_dev(gain, F32),
        to_dev(w, F32), to_dev(inv, I32), None if sh is None else to_dev(sh, BF),
        None if gate is None else to_dev(gate, F32), span, 0.625, EPS)
    ro, rz, rr = K.norm_out(y, resid, gain, w, inv, k, sh, gate, span, 0.625, EPS)
    assert_bf16_close(f64(out), ro, "out")
    assert_bf16_close(f64(z), rz, "z")
    if with_gain:
        assert (np.abs(f64(r) - rr) <= (d + 2 * k + 16) * 4 * U * rr).all()


# more than 1024 groups (their sums joined by the wide join, short spans apart from it), groups
# with several whole spans, groups within one span, several rows a group at d > 8192
@pytest.mark.parametrize("with_gain", [True, False])
@pytest.mark.parametrize("T,d,rows,span", [
    (5001, 64, "vector", 1), (5001, 64, "vector", 3), (5001, 64, "vector", 4000),
    (5001, 64, "one", 5001),
    (20000, 136, "vector", 1), (20000, 136, "vector", 3), (20000, 136, "vector", 7000),
    (20000, 136, "one", 1), (20000, 136, "one", 7),
    (5003, 2056, "vector", 2), (5003, 2056, "vector", 5), (5003, 2056, "vector", 1000),
    (5003, 2056, None, 1),
    (2001, 8200, "vector", 3), (2001, 8200, "vector", 2001), (2001, 8200, "one", 500),
    (700, 16384, "vector", 100),
])
def test_norm_out_backward(T, d, rows, span, with_gain):
    rng = np.random.default_rng([T, d, span])
    gate = None if rows is None else _f32(rng, -(-T // span), d if rows == "vector" else 1)
    dout, z = _bf(rng, T, d), _bf(rng, T, d)
    gain = _f32(rng, d) if with_gain else None
    r = K.norm_in(z, np.ones(d), EPS)[1].astype(np.float32).astype(np.float64)
    dz, dgain, dgate = B.moe_norm_out_backward(
        to_dev(dout, BF), to_dev(z, BF), to_dev(r, F32), to_dev(gain, F32) if with_gain else None,
        None if gate is None else to_dev(gate, F32), span, 0.625)
    at = gate[np.arange(T) // span] if gate is not None else np.ones((T, 1))
    dn = 0.625 * at * dout
    n, want = z, dn
    if with_gain:
        want, _ = K.norm_in_backward(dn, z, gain, r)
        n = z * r[:, None] * gain
        assert_sums(dgain, dn * z * r[:, None], T, d, "dgain")
    assert_bf16_close(f64(dz), want, "dz")
    if gate is not None:
        assert_sums(dgate, 0.625 * dout * n, span, gate.shape[1], "dgate")
