"""The persistent kernel of the 4-bit experts, as decoding calls it: rows through the
permutation, every group size in both products, odd numbers of k-tiles, panels that take a
block's rows in several turns, and the whole decoding block on it, alone and in a CUDA graph.

Every size here passes the launch rule's k-tiles (36 000 for gate and up, 20 000 for down) at
16 rows per expert or fewer; ``_persistent`` asserts it. Tolerances as in test_gpu_w4.py."""
import multiprocessing as mp
import os
import sys

import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL
from grouped_gemm_moe_gb300 import workloads as W
from oracle import block as K
from oracle import moe_oracle as O

from _parity import assert_bf16_close, assert_out_close, dev, ensure_built, f64, i64, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _persistent(E, M, d, I, most):
    slots = min(E, M)
    assert min(most, (M - 1) // E + 1) <= 16
    assert slots * (I // 16) * (d // 64) >= 36000 and slots * (d // 32) * (I // 64) >= 20000


def _experts(seed, E, d, I, g_gu, g_d):
    """(the three matrices' values, laid-out gate and up, laid-out down)."""
    rng = np.random.default_rng(seed)
    vals, plain = [], []
    for n, k, g in ((I, d, g_gu), (I, d, g_gu), (d, I, g_d)):
        codes = rng.integers(0, 16, size=(E, n, k), dtype=np.uint8)
        s = O.round_bf16((0.2 + rng.random((E, n, k // g))) * 0.02)
        vals.append(((codes.astype(np.float32) - 8) * np.repeat(s, g, axis=2).astype(np.float32)))
        plain.append((to_dev(codes[..., 0::2] | codes[..., 1::2] << 4, torch.uint8), to_dev(s, BF)))
    return vals, B.moe_w4_pack_weights(*plain[0], *plain[1]), B.moe_w4_pack_weights(*plain[2])


def _reference(x, offsets, vals, h):
    """The oracle one expert at a time: the values of all of them in 64 bits would not fit."""
    y, rh = np.zeros((x.shape[0], x.shape[1])), np.zeros_like(h)
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            one = [v[e:e + 1].astype(np.float64) for v in vals]     # exact: codes times bf16
            y[a:b], rh[a:b] = K.grouped_ffn_w4(x[a:b], np.array([0, b - a]), *one, h=h[a:b])
    return y, rh


def _top_k(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)])


@pytest.mark.parametrize("T,E,k,d,I,g_gu,g_d", [
    (16, 40, 5, 1024, 1024, 32, 128),
    (16, 40, 5, 1024, 1024, 64, 32),
    (64, 40, 5, 1024, 1024, 128, 64),
    (128, 40, 5, 1024, 1024, 32, 32),        # 16 rows per expert
    (9, 40, 5, 1088, 1088, 32, 64),          # 17 k-tiles in both products
    (33, 40, 5, 1088, 1088, 64, 32),
    (13, 12, 3, 4096, 1024, 128, 128),       # room for 13 rows of X in a block
    (1000, 500, 8, 1024, 128, 64, 64),       # more rows in a block than its panel takes
    (16, 128, 8, 2048, 768, 128, 128),
])
def test_rows_through_the_permutation(T, E, k, d, I, g_gu, g_d):
    _persistent(E, T * k, d, I, T)
    vals, wgu, wd = _experts([T, d, I], E, d, I, g_gu, g_d)
    rng = np.random.default_rng([T, E])
    x = O.round_bf16(rng.normal(size=(T, d)))
    _, offsets, perm, _ = B.moe_build_permutation(to_dev(_top_k(rng, T, E, k), I32), E)
    y, h = B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd, perm=perm, K=k)
    rows = x[i64(perm) // k]
    ry, rh = _reference(rows, i64(offsets), vals, f64(h))
    assert_bf16_close(f64(h), rh, "h")
    assert_bf16_close(f64(y), ry, "y")
    y2, h2 = B.moe_grouped_ffn_w4(to_dev(rows, BF), offsets, wgu, wd)     # the dispatched rows
    assert torch.equal(y, y2) and torch.equal(h, h2)
    y3, h3 = (torch.full_like(t, float("nan")) for t in (y, h))
    B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd, perm=perm, K=k, out=(y3, h3))
    assert torch.equal(y, y3) and torch.equal(h, h3)


def test_a_token_that_is_not_finite_stays_apart():
    T, E, k, d, I = 16, 40, 5, 1024, 1024
    _, wgu, wd = _experts([3], E, d, I, 64, 64)
    rng = np.random.default_rng(3)
    x = O.round_bf16(rng.normal(size=(T, d)))
    _, offsets, perm, _ = B.moe_build_permutation(to_dev(_top_k(rng, T, E, k), I32), E)
    y, _ = B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd, perm=perm, K=k)
    x[7, 3], x[9, d - 1] = np.inf, np.nan
    y2, _ = B.moe_grouped_ffn_w4(to_dev(x, BF), offsets, wgu, wd, perm=perm, K=k)
    bad = torch.isin(perm // k, torch.tensor([7, 9], device=perm.device))
    assert bad.sum() == 2 * k
    assert torch.equal(y[~bad], y2[~bad]) and not torch.isfinite(y2[bad].float()).any()


@pytest.mark.parametrize("shared_I", [0, 256])
def test_the_decoding_block_alone_and_in_a_graph(shared_I):
    """The block against the oracle's composition, then captured once and replayed on other
    tokens: the bits of a call on those."""
    T, group = 16, 64
    cfg = W.small_config("decode", T=T, d=1024, E=40, K=5, I=1024, R=1, shared_I=shared_I)
    _persistent(cfg.E, T * cfg.K, cfg.d, cfg.I, T)
    inp = W.make_inputs(cfg)
    np_inp = {k: W.to_f64(v) for k, v in inp.items()}
    weights = {k: v.to(dev()) for k, v in inp.items() if k.startswith("w")}
    rng = np.random.default_rng(T)
    gain_in, gain_out = (0.5 + rng.random((2, cfg.d))).astype(np.float32).astype(np.float64)
    block = BL.MoEDecodeBlock(T, cfg.K, BL.w4_weights(weights, group), to_dev(gain_in, F32),
                              to_dev(gain_out, F32), scale=0.75)
    x, logits = inp["x"].to(dev()), inp["logits"].to(dev())
    xn = f64(block.norm(x))
    out = block.forward(logits).clone()
    idx, w = O.route_topk(np_inp["logits"], cfg.K, cfg.renorm)
    _, offsets = O.expert_counts_offsets(idx, cfg.E)
    perm, inv = O.stable_permutation(idx, cfg.E)
    rows = O.dispatch(xn, perm, cfg.K)
    y = np.zeros_like(rows)
    for e in range(cfg.E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            q = [K.w4_values(*K.w4_quantize(np_inp[k][e:e + 1], group)) for k in ("w_gate", "w_up", "w_down")]
            y[a:b], _ = K.grouped_ffn_w4(rows[a:b], np.array([0, b - a]), *q)
    ys = None
    if shared_I:
        s = [K.w4_values(*K.w4_quantize(np_inp[k][None], group)) for k in ("ws_gate", "ws_up", "ws_down")]
        ys, _ = K.grouped_ffn_w4(xn, np.array([0, T]), *s)
    ref, _, _ = K.norm_out(y, np_inp["x"], gain_out, w, inv, cfg.K, ys, None, 1, 0.75, 1e-6)
    assert_out_close(f64(out), ref, name="out")

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        block.norm(x)
        got = block.forward(logits)
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        new_x = torch.randn(T, cfg.d, generator=g).to(BF).to(dev())
        new_l = torch.randn(T, cfg.E, generator=g).to(dev())
        block.norm(new_x)
        want = block.forward(new_l).clone()
        x.copy_(new_x)
        logits.copy_(new_l)
        block.out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(got, want)


T_, K_, E_, D_, I_ = 16, 5, 40, 1024, 1024


def _outputs(bad=False):
    g = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).to(dev())  # noqa: E731
    scale = lambda *s: (0.01 * (0.2 + torch.rand(*s, generator=g))).to(BF).to(dev())  # noqa: E731
    wgu = B.moe_w4_pack_weights(ints(E_, I_, D_ // 2), scale(E_, I_, D_ // 64),
                                ints(E_, I_, D_ // 2), scale(E_, I_, D_ // 64))
    wd = B.moe_w4_pack_weights(ints(E_, D_, I_ // 2), scale(E_, D_, I_ // 64))
    x = torch.randn(T_, D_, generator=g).to(BF).to(dev())
    idx = torch.stack([torch.randperm(E_, generator=g)[:K_] for _ in range(T_)]).to(I32).to(dev())
    _, offsets, perm, _ = B.moe_build_permutation(idx, E_)
    if bad:
        perm[11], perm[40] = -4 * K_, T_ * K_ + 5
    y, h = B.moe_grouped_ffn_w4(x, offsets, wgu, wd, perm=perm, K=K_)
    status = B.moe_debug_check_status() if bad is not None else 0
    return y.float().cpu().numpy(), h.float().cpu().numpy(), status


def _child(q):
    sys.path.insert(0, ROOT)
    try:
        from grouped_gemm_moe_gb300 import build as build_mod
        B.load(build_mod.build(debug=True))
        q.put((_outputs(), _outputs(bad=True), B.MOE_ERR_DEVICE_CHECK, None))
    except Exception:  # pragma: no cover - reported by the parent
        import traceback
        q.put((None, None, None, traceback.format_exc()))


def test_debug_build_matches_release_and_flags_bad_indexes():
    """In a child process, as test_gpu_debug_block.py: the debug build reads a bad entry of perm
    as row 0 and records it; the other rows keep their bits."""
    _persistent(E_, T_ * K_, D_, I_, T_)
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=_child, args=(q,))
    p.start()
    clean, flagged, code, err = q.get(timeout=600)
    p.join(60)
    assert err is None, err
    y, h, _ = _outputs(bad=None)
    assert clean[2] == 0 and np.array_equal(clean[0], y) and np.array_equal(clean[1], h)
    keep = [i for i in range(T_ * K_) if i not in (11, 40)]
    assert flagged[2] == code
    assert np.array_equal(flagged[0][keep], y[keep]) and np.array_equal(flagged[1][keep], h[keep])
