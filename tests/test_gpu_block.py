"""The whole block: a layer with 8-bit checkpoints against the oracle fed with the
values the codes stand for, layers sharing one scratch, a training step of the
block and the decoding block against the oracle's composition. bf16 results:
the stated 2e-2 of RMS beyond half an ulp of the stored value; fp32 gradients:
2e-2 of RMS."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import block as BL
from grouped_gemm_moe_gb300 import layer as L
from grouped_gemm_moe_gb300 import workloads as W
from oracle import block as K
from oracle import moe_oracle as O

from _parity import (assert_bf16_close, assert_out_close, assert_rms_close, dev, ensure_built, f64,
                     i64, to_dev)

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
CASES = [
    W.small_config("plain", T=300, d=128, E=8, K=2, I=128, R=2),
    W.small_config("shared", T=384, d=128, E=8, K=2, I=128, R=2, shared_I=256),
    W.small_config("odd", T=600, d=136, E=12, K=3, I=200, R=4, shared_I=72),
]
IDS = [c.name for c in CASES]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _drawn(cfg):
    inp = W.make_inputs(cfg, with_backward=True)
    return inp, {k: W.to_f64(v) for k, v in inp.items()}


def _restored(pair):
    return K.ckpt8_restore(i64(pair[0]), f64(pair[1]))


@pytest.mark.parametrize("cfg", CASES, ids=IDS)
def test_layer_with_checkpoints(cfg):
    inp, np_inp = _drawn(cfg)
    plain = L.layer_from_config(cfg, inp, dev())
    layer = L.layer_from_config(cfg, inp, dev(), ckpt8=True)
    logits, x, dout = (inp[k].to(dev()) for k in ("logits", "x", "dout"))
    assert torch.equal(plain.forward(logits, x), layer.forward(logits, x))
    dx = layer.backward(dout)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    # the oracle's backward on what the codes stand for
    fwd = O.layer_forward(np_inp, cfg.K, cfg.R, cfg.renorm)
    x8 = O.round_bf16(_restored(layer.x8))
    gu, h = K.ckpt8_swiglu(i64(layer.gu8[0]), f64(layer.gu8[1]))
    fwd.update(y=_restored(layer.y8), xp=O.dispatch(x8, fwd["perm"], cfg.K), gu=O.round_bf16(gu),
               h=O.round_bf16(h))
    if cfg.shared_I:
        gus, hs = K.ckpt8_swiglu(i64(layer.gus8[0]), f64(layer.gus8[1]))
        fwd.update(gus=O.round_bf16(gus), hs=O.round_bf16(hs))
    rb = O.layer_backward({**np_inp, "x": x8}, fwd, np_inp["dout"], cfg.K, cfg.renorm, pre=True)
    assert_out_close(f64(dx), rb["dx_pre"], name="dx")
    for k in ("dw_gate", "dw_up", "dw_down", "dlogits"):
        assert_rms_close(f64(getattr(layer, k)), rb[k], name=k)
    if cfg.shared_I:
        for k in ("dws_gate", "dws_up", "dws_down"):
            assert_rms_close(f64(getattr(layer, k))[0], rb[k], name=k)


def test_layers_share_a_scratch():
    cfg = CASES[1]
    scratch = L.LayerScratch(cfg.T, cfg.d, cfg.E, cfg.K, cfg.I, cfg.shared_I, dev())
    drawn = [W.make_inputs(cfg, seed=s, with_backward=True) for s in (1, 2)]
    args = [tuple(d[k].to(dev()) for k in ("logits", "x", "dout")) for d in drawn]
    alone = []
    for d, (logits, x, dout) in zip(drawn, args):
        layer = L.layer_from_config(cfg, d, dev(), ckpt8=True)
        layer.forward(logits, x)
        layer.backward(dout)
        alone.append([layer.dx.clone(), layer.dw_gate.clone(), layer.dws_down.clone(),
                      layer.dlogits.clone()])
    both = [L.layer_from_config(cfg, d, dev(), ckpt8=True, scratch=scratch) for d in drawn]
    for layer, (logits, x, _) in zip(both, args):
        layer.forward(logits, x)
    for layer, (_, _, dout), want in reversed(list(zip(both, args, alone))):
        layer.backward(dout)
        for a, b in zip((layer.dx, layer.dw_gate, layer.dws_down, layer.dlogits), want):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        L.layer_from_config(cfg, drawn[0], dev(), scratch=scratch)
    with pytest.raises(ValueError):
        L.layer_from_config(CASES[0], W.make_inputs(CASES[0]), dev(), ckpt8=True, scratch=scratch)


@pytest.mark.parametrize("gate,span", [(None, None), ("channel", None), ("sequence", 100)])
@pytest.mark.parametrize("with_gain", [True, False])
@pytest.mark.parametrize("cfg", CASES, ids=IDS)
def test_block_training_step(cfg, with_gain, gate, span):
    inp, np_inp = _drawn(cfg)
    rng = np.random.default_rng(cfg.T)
    f = lambda *s: (0.5 + rng.random(s)).astype(np.float32).astype(np.float64)  # noqa: E731
    gain_in, gain_out = f(cfg.d), f(cfg.d) if with_gain else None
    rows = {None: 0, "channel": 1, "sequence": -(-cfg.T // (span or 1))}[gate]
    g = f(rows, cfg.d) if gate else None
    block = BL.MoEBlock(L.layer_from_config(cfg, inp, dev()), to_dev(gain_in, F32),
                        to_dev(gain_out, F32) if with_gain else None,
                        to_dev(g, F32) if gate else None, span, 0.5)
    x, logits, dout = (inp[k].to(dev()) for k in ("x", "logits", "dout"))
    xn = f64(block.norm(x))
    out = block.forward(logits)
    dxn, dlogits = block.backward(dout)
    dx = block.backward_norm(dxn)

    xr, r_in = K.norm_in(np_inp["x"], gain_in, 1e-6)
    assert_bf16_close(xn, xr, "xn")
    lay = {**np_inp, "x": xn}
    fwd = O.layer_forward(lay, cfg.K, cfg.R, cfg.renorm, pre=True)
    z, n, r = fwd["out_pre"], fwd["out_pre"], None
    if with_gain:
        n, r = K.norm_in(z, gain_out, 1e-6)
    t_span = {None: 1, "channel": cfg.T, "sequence": span}[gate]
    at = np.arange(cfg.T) // t_span
    ref = np_inp["x"] + 0.5 * (g[at] if gate else 1.0) * n
    assert_out_close(f64(out), ref, name="out")
    dz, dg, dgt = K.norm_out_backward(np_inp["dout"], O.round_bf16(z), r, gain_out, g, t_span, 0.5)
    rb = O.layer_backward(lay, fwd, O.round_bf16(dz), cfg.K, cfg.renorm, pre=True)
    assert_out_close(f64(dxn), rb["dx_pre"], name="dxn")
    assert_rms_close(f64(dlogits), rb["dlogits"], name="dlogits")
    assert_rms_close(f64(block.layer.dw_down), rb["dw_down"], name="dw_down")
    if with_gain:
        assert_rms_close(f64(block.dgain_out), dg, name="dgain_out")
    if gate:
        assert_rms_close(f64(block.dgate), dgt, name="dgate")
    rx, rg = K.norm_in_backward(rb["dx"], np_inp["x"], gain_in, r_in, np_inp["dout"])
    assert_out_close(f64(dx), rx, name="dx")
    assert_rms_close(f64(block.dgain_in), rg, name="dgain_in")


@pytest.mark.parametrize("T", [1, 5, 33])
@pytest.mark.parametrize("shared_I,group", [(0, 32), (128, 64)])
def test_decode_block(T, shared_I, group):
    cfg = W.small_config("decode", T=T, d=256, E=8, K=3, I=192, R=1, shared_I=shared_I)
    inp, np_inp = _drawn(cfg)
    weights = {k: v.to(dev()) for k, v in inp.items() if k.startswith("w")}
    rng = np.random.default_rng(T)
    gain_in, gain_out = (0.5 + rng.random((2, cfg.d))).astype(np.float32).astype(np.float64)
    block = BL.MoEDecodeBlock(T, cfg.K, BL.w4_weights(weights, group), to_dev(gain_in, F32),
                              to_dev(gain_out, F32), scale=0.75)
    xn = f64(block.norm(inp["x"].to(dev())))
    out = block.forward(inp["logits"].to(dev()))
    idx, w = O.route_topk(np_inp["logits"], cfg.K, cfg.renorm)
    _, offsets = O.expert_counts_offsets(idx, cfg.E)
    perm, inv = O.stable_permutation(idx, cfg.E)
    q = lambda k: K.w4_values(*K.w4_quantize(np_inp[k], group))  # noqa: E731
    y, _ = K.grouped_ffn_w4(O.dispatch(xn, perm, cfg.K), offsets, q("w_gate"), q("w_up"), q("w_down"))
    ys = None
    if shared_I:
        s = [K.w4_values(*K.w4_quantize(np_inp[k][None], group))
             for k in ("ws_gate", "ws_up", "ws_down")]
        ys, _ = K.grouped_ffn_w4(xn, np.array([0, T]), *s)
    ref, _, _ = K.norm_out(y, np_inp["x"], gain_out, w, inv, cfg.K, ys, None, 1, 0.75, 1e-6)
    assert_out_close(f64(out), ref, name="out")
