"""Pins of the block oracle (oracle/block.py) on the CPU: the norms' gradients
against central differences, the norm's scale invariance, checkpoint codes in
closed form, error bounds of both quantizers, and the 4-bit experts against the
bf16 oracle on exactly representable weights."""
import numpy as np
import pytest

from oracle import block as K
from oracle import moe_oracle as O


def _numeric(f, a, h=1e-5):
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = a[i]
        a[i] = old + h
        up = f()
        a[i] = old - h
        dn = f()
        a[i] = old
        g[i] = (up - dn) / (2 * h)
    return g


def test_norm_in_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, gain, v = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8))
    f = lambda: (K.norm_in(x, gain, 1e-3)[0] * v).sum()   # noqa: E731
    dx, dgain = K.norm_in_backward(v, x, gain, K.norm_in(x, gain, 1e-3)[1])
    # central differences of an O(1) function: h^2 and 1e-16 / h both near 1e-10
    assert np.allclose(dx, _numeric(f, x), atol=1e-8)
    assert np.allclose(dgain, _numeric(f, gain), atol=1e-8)


@pytest.mark.parametrize("with_gain", [True, False])
@pytest.mark.parametrize("gate_shape,span", [(None, 1), ((5, 1), 1), ((1, 8), 5), ((3, 8), 2),
                                             ((2, 1), 3)])
def test_norm_out_gradient_against_differences(with_gain, gate_shape, span):
    rng = np.random.default_rng(1)
    T, d, k = 5, 8, 2
    y, resid = rng.normal(size=(T * k, d)), rng.normal(size=(T, d))
    w, inv = rng.random((T, k)), rng.permutation(T * k)
    gain = rng.normal(size=d) if with_gain else None
    gate = rng.normal(size=gate_shape) if gate_shape else None
    v = rng.normal(size=(T, d))
    run = lambda: K.norm_out(y, resid, gain, w, inv, k, None, gate, span, 0.7, 1e-3)   # noqa: E731
    f = lambda: (run()[0] * v).sum()   # noqa: E731
    _, z, r = run()
    dz, dgain, dgate = K.norm_out_backward(v, z, r, gain, gate, span, 0.7)
    dy = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            dy[inv[t * k + j]] = w[t, j] * dz[t]
    assert np.allclose(dy, _numeric(f, y), atol=1e-8)
    if with_gain:
        assert np.allclose(dgain, _numeric(f, gain), atol=1e-8)
    if gate is not None:
        assert np.allclose(dgate, _numeric(f, gate), atol=1e-8)


def test_norm_is_invariant_under_scaling_and_has_unit_rms():
    x = np.random.default_rng(2).normal(size=(4, 64))
    a, _ = K.norm_in(x, np.ones(64), 0.0)
    b, _ = K.norm_in(1000 * x, np.ones(64), 0.0)
    assert np.allclose(a, b)
    assert np.allclose(np.mean(a ** 2, axis=1), 1.0)


def test_checkpoint_codes_in_closed_form():
    x = np.zeros((2, 40))
    x[0, :4] = [127.0, -127.0, 0.5, 1.5]     # s = 1: rint ties to even
    x[0, 32:35] = [np.inf, 254.0, np.nan]     # s = 2 from the finite value alone
    q, s = K.ckpt8_pack(x)
    assert s.shape == (2, 2) and s[0, 0] == 1.0 and s[0, 1] == 2.0
    assert q[0, :4].tolist() == [127, -127, 0, 2] and q[0, 32:35].tolist() == [-128, 127, -128]
    assert (q[1] == 0).all() and (s[1] == 2.0 ** -110).all()
    v = K.ckpt8_restore(q, s)
    assert np.isnan(v[0, 32]) and v[0, 33] == 254.0 and (v[1] == 0).all()


def test_checkpoint_error_is_half_a_step():
    x = O.round_bf16(np.random.default_rng(3).normal(size=(16, 96)) * 10.0 **
                     np.random.default_rng(4).integers(-6, 6, size=(16, 1)))
    q, s = K.ckpt8_pack(x)
    assert np.abs(q).max() <= 127
    step = np.repeat(s, 32, axis=1)
    assert (np.abs(K.ckpt8_restore(q, s) - x) <= step * (0.5 + 1e-6)).all()
    top = np.abs(x).reshape(16, 3, 32).max(2)
    assert (s >= top / 127).all() and (s <= top / 127 * (1 + 2.0 ** -7)).all()


def test_w4_quantizer_error_and_codes():
    w = O.round_bf16(np.random.default_rng(5).normal(size=(2, 128, 24)) * 0.02)
    q, s = K.w4_quantize(w, 32)
    assert q.shape == (2, 24, 128) and q.min() >= 1 and q.max() <= 15
    err = np.abs(K.w4_values(q, s) - np.swapaxes(w, 1, 2))
    assert (err <= np.repeat(s, 32, axis=2) * (0.5 + 1e-6)).all()


def test_w4_experts_equal_the_bf16_oracle_on_representable_weights():
    rng = np.random.default_rng(6)
    E, d, I, M = 3, 64, 64, 10
    codes = [rng.integers(0, 16, size=(E, n, k)) for n, k in ((I, d), (I, d), (d, I))]
    scales = [np.full((E, c.shape[1], c.shape[2] // 32), 2.0 ** -6) for c in codes]
    vals = [K.w4_values(c, s) for c, s in zip(codes, scales)]
    x, offsets = O.round_bf16(rng.normal(size=(M, d))), np.array([0, 4, 4, 10])
    y, h = K.grouped_ffn_w4(x, offsets, *vals)
    ref = O.grouped_ffn(x, offsets, *[np.swapaxes(v, 1, 2) for v in vals], exact=True)
    assert np.allclose(y, ref[0]) and np.allclose(h, ref[2])
