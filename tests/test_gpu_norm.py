"""GPU parity of the block's norms and their gradients with the CPU oracle.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
* bf16 results: half an ulp of the stored value plus 1e-3 of the tensor's RMS
  (the shared bound of element-wise bf16 results);
* rstd: a sum of d squares, a division, an inverse root: (d + 16) u, relative;
* fp32 sums of n products (dgain, dgate): any order of n additions is within
  (n + 16) u of the sum of the products' magnitudes.
"""
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


def _rng(*seed):
    return np.random.default_rng(list(seed))


def _bf(rng, *shape, scale=1.0):
    return O.round_bf16(rng.normal(size=shape) * scale)


def _f32(rng, *shape):
    return (0.5 + rng.random(shape)).astype(np.float32).astype(np.float64)


def assert_sum_close(got, terms, axis, name):
    """fp32 sums of ``terms`` over ``axis``."""
    n = np.prod([terms.shape[a] for a in np.atleast_1d(axis)])
    bound = (n + 16) * U * np.abs(terms).sum(axis) + 1e-35
    err = np.abs(f64(got) - terms.sum(axis))
    assert (err <= bound).all(), f"{name}: {(err / bound).max():.2f} of the bound"


def assert_gate_sums(got, terms, rows, span, cols, name):
    for s in range(rows):
        t = terms[s * span:(s + 1) * span]
        assert_sum_close(got[s] if cols > 1 else got[s, 0], t, 0 if cols > 1 else (0, 1), name)


# d below a warp's row, off the powers of two, at one and two vectors a thread
SHAPES = [(1, 8), (1, 4096), (2, 264), (7, 128), (33, 2056), (1000, 136), (515, 768), (640, 2048),
          (300, 4096), (37, 8192), (19, 8200), (5, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_in(T, d):
    rng = _rng(T, d)
    x, gain = _bf(rng, T, d, scale=3.0), _f32(rng, d)
    xn, r = B.moe_norm_in(to_dev(x, BF), to_dev(gain, F32), EPS)
    ref, rr = K.norm_in(x, gain, EPS)
    assert (np.abs(f64(r) - rr) <= (d + 16) * U * rr).all()
    assert_bf16_close(f64(xn), ref, "xn")


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_in_backward(T, d, with_res):
    rng = _rng(T, d, 1)
    x, gain, dxn = _bf(rng, T, d, scale=3.0), _f32(rng, d), _bf(rng, T, d)
    dres = _bf(rng, T, d) if with_res else None
    r = K.norm_in(x, gain, EPS)[1].astype(np.float32).astype(np.float64)
    dx, dgain = B.moe_norm_in_backward(to_dev(dxn, BF), to_dev(x, BF), to_dev(gain, F32),
                                       to_dev(r, F32), to_dev(dres, BF) if with_res else None)
    assert_bf16_close(f64(dx), K.norm_in_backward(dxn, x, gain, r, dres)[0], "dx")
    assert_sum_close(dgain, dxn * x * r[:, None], 0, "dgain")


def test_norm_in_gradient_against_differences():
    """The gradient kernel against central differences of the oracle's forward."""
    rng = _rng(5)
    x, gain, v = _bf(rng, 3, 16), _f32(rng, 16), _bf(rng, 3, 16)
    r = K.norm_in(x, gain, EPS)[1]
    dx, _ = B.moe_norm_in_backward(to_dev(v, BF), to_dev(x, BF), to_dev(gain, F32), to_dev(r, F32))
    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        p, m = x.copy(), x.copy()
        p[i] += 1e-5
        m[i] -= 1e-5
        num[i] = ((K.norm_in(p, gain, EPS)[0] - K.norm_in(m, gain, EPS)[0]) * v).sum() / 2e-5
    assert_bf16_close(f64(dx), num, "dx")


GATES = [(None, None), ("token", 1), ("one", None), ("channel", None), ("sequence", 3),
         ("sequence", 64), ("sequence1", 50)]


def _gate(rng, kind, span, T, d):
    """(gate or None, span): one column for token, one and sequence1, d otherwise."""
    if kind is None:
        return None, 1
    span = {"token": 1, "one": T, "channel": T}.get(kind, span)
    return _f32(rng, -(-T // span), 1 if kind in ("token", "one", "sequence1") else d), span


@pytest.mark.parametrize("kind,span", GATES)
@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (1, 2048, 8), (13, 136, 3), (130, 520, 6),
                                   (257, 2048, 8), (50, 4096, 16), (9, 8200, 32), (70, 64, 2)])
def test_norm_out(T, d, k, kind, span):
    rng = _rng(T, d, k)
    gate, span = _gate(rng, kind, span, T, d)
    y, resid, shared = _bf(rng, T * k, d), _bf(rng, T, d, scale=3.0), _bf(rng, T, d)
    w, inv, gain = _f32(rng, T, k), rng.permutation(T * k), _f32(rng, d)
    for g, sh in ((gain, shared), (gain, None), (None, shared)):
        out, z, r = B.moe_norm_out(
            to_dev(y, BF), to_dev(resid, BF), None if g is None else to_dev(g, F32),
            to_dev(w, F32), to_dev(inv, I32), None if sh is None else to_dev(sh, BF),
            None if gate is None else to_dev(gate, F32), span, 0.625, EPS)
        ro, rz, rr = K.norm_out(y, resid, g, w, inv, k, sh, gate, span, 0.625, EPS)
        assert_bf16_close(f64(out), ro, "out")
        assert_bf16_close(f64(z), rz, "z")
        assert (r is None) == (g is None)
        if r is not None:
            assert (np.abs(f64(r) - rr) <= (d + 2 * k + 16) * 4 * U * rr).all()


def test_norm_out_of_a_plain_input_and_its_inference_form():
    rng = _rng(9)
    T, d = 21, 264
    y, resid, gain = _bf(rng, T, d), _bf(rng, T, d), _f32(rng, d)
    args = (to_dev(y, BF), to_dev(resid, BF), to_dev(gain, F32))
    out, z, r = B.moe_norm_out(*args)
    assert_bf16_close(f64(out), K.norm_out(y, resid, gain, None, None, 1, None, None, 1, 1.0, EPS)[0],
                      "out")
    assert np.array_equal(f64(z), y)
    bare, no_z, no_r = B.moe_norm_out(*args, save=False)
    assert torch.equal(out, bare) and no_z is None and no_r is None
    same = args[1].clone()      # in place on the residual stream
    B.moe_norm_out(args[0], same, args[2], out=(same, None, None))
    assert torch.equal(out, same)


def test_norm_out_combines_like_the_combine():
    rng = _rng(10)
    T, d, k = 77, 520, 6
    y, w, inv = to_dev(_bf(rng, T * k, d), BF), to_dev(_f32(rng, T, k), F32), \
        to_dev(rng.permutation(T * k), I32)
    _, z, _ = B.moe_norm_out(y, torch.zeros(T, d, dtype=BF, device=dev()), None, w, inv)
    assert torch.equal(z, B.moe_combine(y, w, inv))


@pytest.mark.parametrize("kind,span", GATES + [("sequence", 7), ("sequence1", 1000)])
@pytest.mark.parametrize("with_gain", [True, False])
@pytest.mark.parametrize("T,d", [(1, 8), (65, 136), (700, 64), (901, 520), (1300, 2056),
                                 (640, 4096), (21, 8200)])
def test_norm_out_backward(T, d, with_gain, kind, span):
    rng = _rng(T, d, 2)
    gate, span = _gate(rng, kind, span, T, d)
    dout, z = _bf(rng, T, d), _bf(rng, T, d)
    gain = _f32(rng, d) if with_gain else None
    r = K.norm_in(z, np.ones(d), EPS)[1].astype(np.float32).astype(np.float64)
    dz, dgain, dgate = B.moe_norm_out_backward(
        to_dev(dout, BF), to_dev(z, BF), to_dev(r, F32), to_dev(gain, F32) if with_gain else None,
        None if gate is None else to_dev(gate, F32), span, 0.625)
    rz, _, _ = K.norm_out_backward(dout, z, r, gain, gate, span, 0.625)
    assert_bf16_close(f64(dz), rz, "dz")
    n = z * r[:, None] * gain if with_gain else z
    if gate is not None:
        assert_gate_sums(dgate, 0.625 * dout * n, gate.shape[0], span, gate.shape[1], "dgate")
    if with_gain:
        rows = np.ones((T, 1)) if gate is None else gate[np.arange(T) // span]
        assert_sum_close(dgain, 0.625 * rows * dout * z * r[:, None], 0, "dgain")


def test_sums_are_the_same_bits_every_run():
    rng = _rng(11)
    T, d = 3000, 1032
    a = (to_dev(_bf(rng, T, d), BF), to_dev(_bf(rng, T, d), BF), to_dev(_f32(rng, T), F32),
         to_dev(_f32(rng, d), F32), to_dev(_f32(rng, -(-T // 100), d), F32), 100)
    first = B.moe_norm_out_backward(*a)
    for _ in range(3):
        for p, q in zip(first, B.moe_norm_out_backward(*a)):
            assert torch.equal(p, q)


def test_values_that_are_not_finite_stay_in_their_row():
    rng = _rng(12)
    x = to_dev(_bf(rng, 40, 520), BF)
    gain = to_dev(_f32(rng, 520), F32)
    good, _ = B.moe_norm_in(x, gain)
    x[3, 7] = float("nan")
    x[11, 0] = float("inf")
    bad, r = B.moe_norm_in(x, gain)
    keep = torch.ones(40, dtype=torch.bool, device=x.device)
    keep[[3, 11]] = False
    assert torch.equal(good[keep], bad[keep])
    assert bad[3].isnan().all() and bad[11, 0].isnan() and (bad[11, 1:] == 0).all() and r[11] == 0


def test_zero_rows_and_zero_input():
    gain = torch.ones(64, device=dev())
    none = torch.empty(0, 64, dtype=BF, device=dev())
    xn, r = B.moe_norm_in(none, gain)
    assert xn.shape == (0, 64) and r.shape == (0,)
    dgain = torch.full((64,), 7.0, device=dev())
    B.moe_norm_in_backward(none, none, gain, r, out=(none, dgain))
    assert (dgain == 0).all()
    dgain.fill_(7.0)
    B.moe_norm_out_backward(none, none, r, gain, out=(none, dgain, None))
    assert (dgain == 0).all()
    zero = torch.zeros(3, 64, dtype=BF, device=dev())
    xn, r = B.moe_norm_in(zero, gain, 1e-6)
    assert (xn == 0).all() and torch.allclose(r, torch.full_like(r, 1e3))


def test_past_two_to_the_31_elements():
    """Rows whose offsets pass 32 bits: the last rows as in a call of their own."""
    T, d = 262400, 8192
    x = torch.zeros(T, d, dtype=BF, device=dev())
    tail = torch.randn(64, d, device=dev()).to(BF)
    x[-64:] = tail
    gain = torch.rand(d, device=dev()) + 0.5
    xn, r = B.moe_norm_in(x, gain)
    want, rw = K.norm_in(f64(tail), f64(gain), EPS)
    assert_bf16_close(f64(xn[-64:]), want, "xn")
    assert (np.abs(f64(r[-64:]) - rw) <= (d + 16) * U * rw).all()
    out, z, _ = B.moe_norm_out(xn, x, gain)
    ow, zw, _ = B.moe_norm_out(xn[-64:].clone(), tail, gain)
    assert torch.equal(out[-64:], ow) and torch.equal(z[-64:], zw)
    del out, z
    dx, dgain = B.moe_norm_in_backward(xn, x, gain, r, x)
    dw, gw = B.moe_norm_in_backward(xn[-64:].clone(), tail, gain, r[-64:].clone(), tail)
    assert torch.equal(dx[-64:], dw)
    assert_sum_close(dgain, f64(xn[-64:]) * f64(tail) * f64(r[-64:])[:, None], 0, "dgain")


def test_on_another_stream():
    rng = _rng(13)
    x, gain = to_dev(_bf(rng, 5000, 2048), BF), to_dev(_f32(rng, 2048), F32)
    want, _ = B.moe_norm_in(x, gain)
    side = torch.cuda.Stream()
    late = torch.zeros_like(x)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late.copy_(x)
        got, _ = B.moe_norm_in(late, gain)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF, device=dev())
    g = torch.ones(64, device=dev())
    r = torch.ones(4, device=dev())
    with pytest.raises(TypeError):
        B.moe_norm_in(x.float(), g)
    with pytest.raises(ValueError):
        B.moe_norm_in(x, g[:32])
    with pytest.raises(ValueError):
        B.moe_norm_in(x.t(), g)
    with pytest.raises(ValueError):
        B.moe_norm_in(x, g.cpu())
    with pytest.raises(B.MoEError) as e:
        B.moe_norm_in(torch.zeros(4, 12, dtype=BF, device=dev()), g[:12].clone())
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoEError) as e:
        B.moe_norm_in(torch.zeros(1, 16392, dtype=BF, device=dev()), torch.ones(16392, device=dev()))
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        B.moe_norm_out(x, x, g, gate=torch.ones(3, 64, device=dev()), span=2)
    with pytest.raises(ValueError):
        B.moe_norm_out(x, x, g, gate=torch.ones(2, 32, device=dev()), span=2)
    with pytest.raises(ValueError):
        B.moe_norm_out(torch.zeros(6, 64, dtype=BF, device=dev()), x, g)
    with pytest.raises(ValueError):
        B.moe_norm_out_backward(x, x, None, g)
    with pytest.raises(B.MoEError) as e:
        B.moe_norm_in_backward(x, x, g, r, ws=B.new_workspace(256, dev()))
    assert e.value.status == B.MOE_ERR_WORKSPACE
