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

from _parity import assert_bf16_close, dev, ensure_built, f64

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
