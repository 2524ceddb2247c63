"""The 4-bit floats and grouped products as a model calls them: the block on them, alone and in
a CUDA graph; experts that are not gated, forward and backward from grouped products; other
streams; sizes past 32 bits; odd alignments; the debug build. Tolerances as in test_gpu_fp4.py."""
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
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, i64, rounding_excess, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _restored(w, block):
    """Oracle values [E, N, K] of bf16 weights w [E, K, N] in 4 bits."""
    E, k, n = w.shape
    t = np.swapaxes(w, 1, 2).reshape(E * n, k)
    factor = np.repeat(F.row_factor(np.abs(w).max((1, 2))), n) if block == 16 else None
    q, byte, _ = F.quantize_rows(t, block, factor)
    return F.restore(q, byte, factor, block).reshape(E, n, k)


@pytest.mark.parametrize("block,fixed,shared_I", [(16, False, 0), (16, True, 128), (32, False, 192)])
def test_the_block_alone_and_in_a_graph(block, fixed, shared_I):
    """The block against the oracle's composition, then captured once and replayed on other
    tokens: the bits of a call on those."""
    T = 70
    cfg = W.small_config("fp4", T=T, d=256, E=12, K=3, I=320, R=1, shared_I=shared_I)
    inp = W.make_inputs(cfg)
    np_inp = {k: W.to_f64(v) for k, v in inp.items()}
    weights = {k: v.to(dev()) for k, v in inp.items() if k.startswith("w")}
    rng = np.random.default_rng(T)
    gain_in, gain_out = (0.5 + rng.random((2, cfg.d))).astype(np.float32).astype(np.float64)
    x, logits = inp["x"].to(dev()), inp["logits"].to(dev())
    h_scale = sh_scale = None
    if fixed:    # from a pass of the bf16 experts on the block's own rows
        xn, _ = B.moe_norm_in(x, to_dev(gain_in, F32))
        idx, _ = B.moe_route_topk(logits, cfg.K, cfg.renorm)
        _, off, perm, _ = B.moe_build_permutation(idx, cfg.E)
        _, h, _ = B.moe_grouped_ffn(B.moe_dispatch(xn, perm, cfg.K), off, weights["w_gate"],
                                    weights["w_up"], weights["w_down"], save_gu=False)
        h_scale = BL.fp4_h_scale(h, off)
        tops = np.array([np.abs(f64(h))[a:b].max() if b > a else 0.0
                         for a, b in zip(i64(off)[:-1], i64(off)[1:])])
        assert np.allclose(f64(h_scale), np.where(tops > 0, tops, tops.max()) / 2688, rtol=1e-6)
        if shared_I:
            s_off = torch.tensor([0, T], dtype=I32, device=dev())
            _, h, _ = B.moe_grouped_ffn(xn, s_off, *(weights[k].unsqueeze(0) for k in
                                                     ("ws_gate", "ws_up", "ws_down")), save_gu=False)
            sh_scale = BL.fp4_h_scale(h, s_off)
    blk = BL.MoEFp4Block(T, cfg.K, BL.fp4_weights(weights, block), to_dev(gain_in, F32),
                         to_dev(gain_out, F32), scale=0.75, block=block, h_scale=h_scale,
                         sh_scale=sh_scale)
    xn = f64(blk.norm(x))
    out = blk.forward(logits).clone()
    idx, w = O.route_topk(np_inp["logits"], cfg.K, cfg.renorm)
    _, offsets = O.expert_counts_offsets(idx, cfg.E)
    perm, inv = O.stable_permutation(idx, cfg.E)

    def experts(rows, offs, names, hs):
        v = F.restore(*F.quantize_rows(rows, block), block)
        y, _ = F.grouped_ffn_fp4(v, offs, *(_restored(np_inp[n].reshape(-1, *np_inp[n].shape[-2:]), block)
                                            for n in names), block,
                                 h_scale=None if hs is None else f64(hs),
                                 round_h=O.round_bf16 if block == 16 and hs is None else None)
        return y
    y = experts(O.dispatch(xn, perm, cfg.K), offsets, ("w_gate", "w_up", "w_down"), h_scale)
    ys = experts(xn, np.array([0, T]), ("ws_gate", "ws_up", "ws_down"), sh_scale) if shared_I else None
    ref, _, _ = K.norm_out(y, np_inp["x"], gain_out, w, inv, cfg.K, ys, None, 1, 0.75, 1e-6)
    # a token with a changed code of H (see test_gpu_fp4.py) may be off: I K 2^-12 of them at most
    size = np.sqrt(np.mean((ref - np_inp["x"]) ** 2))
    off = (rounding_excess(f64(out), ref) > 2e-2 * size).any(1)
    assert off.sum() <= 3 + 3 * T * cfg.K * cfg.I * 2.0 ** -12, off.sum()
    assert np.sqrt(np.mean((f64(out) - ref) ** 2)) <= 2e-2 * size
    assert B.moe_read_device_status(blk.ws_ffn) == 0

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        blk.norm(x)
        got = blk.forward(logits)
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        new_x = torch.randn(T, cfg.d, generator=g).to(BF).to(dev())
        new_l = torch.randn(T, cfg.E, generator=g).to(dev())
        blk.norm(new_x)
        want = blk.forward(new_l).clone()
        x.copy_(new_x)
        logits.copy_(new_l)
        blk.out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(got, want)


def test_experts_that_are_not_gated():
    """y = relu(x W1)^2 W2 with its gradients from grouped products, over two microbatches and in
    a graph, against float64 on the stored intermediates."""
    rng = np.random.default_rng(8)
    E, d, I, T, k = 9, 136, 200, 83, 2
    w1 = O.round_bf16(rng.normal(size=(E, d, I)) / np.sqrt(d))
    w2 = O.round_bf16(rng.normal(size=(E, I, d)) / np.sqrt(I))
    W1, W2 = to_dev(w1, BF), to_dev(w2, BF)
    dw1, dw2 = torch.zeros(E, d, I, device=dev()), torch.zeros(E, I, d, device=dev())
    ws1 = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_GEMM_WGRAD, T * k, E, 1, 1, d, I), dev())
    ws2 = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_GEMM_WGRAD, T * k, E, 1, 1, I, d), dev())
    idx = to_dev(np.stack([rng.permutation(E)[:k] for _ in range(T)]), I32)
    _, off, perm, _ = B.moe_build_permutation(idx, E)
    offsets = i64(off)
    x = [torch.empty(T * k, d, dtype=BF, device=dev()) for _ in range(2)]
    dy = [torch.empty(T * k, d, dtype=BF, device=dev()) for _ in range(2)]

    def step():
        kept = []
        for i in range(2):
            u = B.moe_grouped_gemm(x[i], off, W1, ws=ws1)
            h = torch.relu(u.float()).square().to(BF)
            y = B.moe_grouped_gemm(h, off, W2, ws=ws1)
            dh = B.moe_grouped_gemm(dy[i], off, W2, trans=True, ws=ws1)
            du = (dh.float() * 2.0 * torch.relu(u.float())).to(BF)
            dx = B.moe_grouped_gemm(du, off, W1, trans=True, ws=ws1)
            B.moe_grouped_gemm_wgrad(h, dy[i], off, accumulate=i > 0, ws=ws2, out=dw2)
            B.moe_grouped_gemm_wgrad(x[i], du, off, accumulate=i > 0, ws=ws1, out=dw1)
            kept.append((u, h, y, dh, du, dx))
        return kept

    def fill(seed):
        r = np.random.default_rng(seed)
        for t in (*x, *dy):
            t.copy_(to_dev(O.round_bf16(r.normal(size=(T * k, d))), BF))

    fill(1)
    kept = step()
    want1, want2 = np.zeros((E, d, I)), np.zeros((E, I, d))
    t = lambda w: np.swapaxes(w, 1, 2)   # noqa: E731
    for i, (u, h, y, dh, du, dx) in enumerate(kept):
        for got, rows, w in ((u, x[i], w1), (y, h, w2), (dh, dy[i], t(w2)), (dx, du, t(w1))):
            assert_bf16_close(f64(got), F.grouped_product(f64(rows), offsets, w), "product")
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            want1[e] += f64(x[i])[a:b].T @ f64(du)[a:b]
            want2[e] += f64(h)[a:b].T @ f64(dy[i])[a:b]
    for got, want in ((dw1, want1), (dw2, want2)):
        assert np.abs(f64(got) - want).max() <= 1e-5 * np.sqrt(T) * np.sqrt(np.mean(want ** 2))

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step()
    fill(2)
    want = [[v.clone() for v in r] for r in step()], dw1.clone(), dw2.clone()
    dw1.fill_(float("nan"))
    dw2.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r, s in zip(held, want[0]) for a, b in zip(r, s))
    assert torch.equal(dw1, want[1]) and torch.equal(dw2, want[2])


def _fp4_matrix(g, E, n, k):
    codes = torch.randint(0, 256, (E, n, k // 2), generator=g, dtype=U8, device=dev())
    scales = torch.randint(48, 72, (E, n, k // 16), generator=g, dtype=U8, device=dev())
    return codes, B.moe_fp4_pack_scales(scales), torch.full((E,), 0.01, device=dev())


def test_two_streams_with_their_own_workspaces():
    g = torch.Generator(device=dev()).manual_seed(5)
    E, d, I, M = 6, 256, 192, 500
    off = torch.tensor([0, 100, 130, 130, 300, 499, 500], dtype=I32, device=dev())
    wgu = [_fp4_matrix(g, E, I, d)[0] for _ in range(2)]
    sf = torch.randint(48, 72, (E, I, d // 16), generator=g, dtype=U8, device=dev())
    one = torch.full((E,), 0.01, device=dev())
    gu = (*wgu, B.moe_fp4_pack_scales(sf, sf), one, one)
    wd = _fp4_matrix(g, E, d, I)
    xs = [torch.randn(M, d, generator=g, device=dev()).to(BF) for _ in range(2)]
    run = lambda x, ws: B.moe_grouped_ffn_fp4(B.moe_fp4_quantize_rows(x, off), off, gu, wd, ws=ws)  # noqa: E731
    size = B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, M, E, 1, 1, d, I)
    wss = [B.new_workspace(size, dev()) for _ in range(2)]
    want = [run(x, wss[0]).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(xs[i], wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(v, want[i]) for v in got[i])
        assert B.moe_read_device_status(wss[i]) == 0


@pytest.mark.parametrize("E", [449, 1024])
def test_many_experts(E):
    """Past the expert count up to which the deeper ring's tables fit."""
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 3, size=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M, k, n = int(offsets[-1]), 1152, 136
    x = O.round_bf16(rng.normal(size=(M, k)))
    codes = rng.integers(0, 16, size=(E, n, k))
    byte = rng.integers(40, 72, size=(E, n, k // 16))
    g = np.full(E, 2.0 ** -5)
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off)
    packed = to_dev((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8), U8)
    y = B.moe_grouped_gemm_fp4(rows, off, (packed, B.moe_fp4_pack_scales(to_dev(byte, U8)), to_dev(g, F32)))
    xv = F.restore(*F.quantize_rows(x, 16), 16)
    want = np.zeros((M, n))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            want[a:b] = xv[a:b] @ F.restore(codes[e], byte[e], np.full(n, g[e]), 16).T
    assert_bf16_close(f64(y), want, "y")


@pytest.mark.parametrize("block", [16, 32])
def test_bases_that_are_not_32_byte_aligned(block):
    g = torch.Generator(device=dev()).manual_seed(3)
    off = torch.tensor([0, 40, 90], dtype=I32, device=dev())
    for d in (192, 2048, 4160):
        x = torch.randn(90, d, generator=g, device=dev()).to(BF)
        flat = torch.empty(90 * d + 8, dtype=BF, device=dev())
        odd = flat[8:].view(90, d)
        odd.copy_(x)
        assert odd.data_ptr() % 32 == 16
        a, b = (B.moe_fp4_quantize_rows(t, off, block) for t in (x, odd))
        assert torch.equal(a[0], b[0]) and (block == 32 or torch.equal(a[2], b[2]))
        want = B.moe_fp4_dequantize_rows(a, off, block)
        got = flat.zero_()[8:].view(90, d)
        B.moe_fp4_dequantize_rows(b, off, block, out=got)
        assert torch.equal(got, want) and (flat[:8] == 0).all()


def test_offsets_past_32_bits():
    """Codes, outputs and weights past 2^31 bytes: the last rows as when they are alone."""
    T, k, d, n = 140_000, 8, 4096, 1024
    M = T * k                                   # 2.3 GB of codes, 9.2 GB restored
    g = torch.Generator(device=dev()).manual_seed(7)
    x = torch.randn(T, d, generator=g, device=dev(), dtype=torch.float16).to(BF)
    inv = torch.randperm(M, generator=g, device=dev()).to(I32)
    off = torch.tensor([0, 1000, M - 300, M], dtype=I32, device=dev())
    rows = B.moe_fp4_quantize_rows(x, off, inv_perm=inv, K=k)
    back = B.moe_fp4_dequantize_rows(rows, off)
    w = _fp4_matrix(g, 3, n, d)
    y = B.moe_grouped_gemm_fp4(rows, off, w)
    perm = torch.argsort(inv.long())
    for a, b in ((M - 300, M), (M // 2, M // 2 + 200)):
        xs = x[perm[a:b] // k]
        e = 2 if a == M - 300 else 1
        few = torch.tensor([0] * (e + 1) + [b - a] * (3 - e), dtype=I32, device=dev())
        alone = B.moe_fp4_quantize_rows(xs.contiguous(), few)
        assert torch.equal(rows[0][a:b], alone[0]) and torch.equal(rows[2][a:b], alone[2])
        assert torch.equal(back[a:b], B.moe_fp4_dequantize_rows(alone, few))
        assert torch.equal(y[a:b], B.moe_grouped_gemm_fp4(alone, few, w))
    del back, rows, y
    wide = torch.randn(M, 2048, generator=g, device=dev(), dtype=torch.float16).to(BF)   # 4.6 GB
    wb = torch.randn(3, 2048, 256, generator=g, device=dev()).to(BF)
    y = B.moe_grouped_gemm(wide, off, wb)
    few = torch.tensor([0, 0, 0, 300], dtype=I32, device=dev())
    assert torch.equal(y[M - 300:], B.moe_grouped_gemm(wide[M - 300:], few, wb))
    dw = B.moe_grouped_gemm_wgrad(wide, y, off)
    alone = B.moe_grouped_gemm_wgrad(wide[M - 300:], y[M - 300:], few)
    assert torch.equal(dw[2], alone[2])


def test_same_bits_on_every_run():
    g = torch.Generator(device=dev()).manual_seed(9)
    off = torch.tensor([0, 700, 701, 1500], dtype=I32, device=dev())
    x = torch.randn(1500, 1024, generator=g, device=dev()).to(BF)
    dy = torch.randn(1500, 264, generator=g, device=dev()).to(BF)
    wb = torch.randn(3, 1024, 264, generator=g, device=dev()).to(BF)
    w = _fp4_matrix(g, 3, 264, 1024)

    def all_of():
        dw = B.moe_grouped_gemm_wgrad(x, dy, off)
        B.moe_grouped_gemm_wgrad(x, dy, off, accumulate=True, out=dw)
        return (B.moe_grouped_gemm(x, off, wb), dw,
                B.moe_grouped_gemm_fp4(B.moe_fp4_quantize_rows(x, off), off, w))
    first = all_of()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, all_of()))


def _outputs(bad=False):
    g = torch.Generator().manual_seed(1)
    T, k, d, E = 40, 3, 128, 4
    x = torch.randn(T, d, generator=g).to(BF).to(dev())
    dy = torch.randn(T * k, 72, generator=g).to(BF).to(dev())
    inv = torch.randperm(T * k, generator=g).to(I32).to(dev())
    off = torch.tensor([0, 30, 31, 31, T * k], dtype=I32, device=dev())
    w = torch.randn(E, d, 72, generator=g).to(BF).to(dev())
    codes, scales, scale = B.moe_fp4_quantize_weights(w)
    w4 = (codes, B.moe_fp4_pack_scales(scales), scale)
    rows = B.moe_fp4_quantize_rows(x, off, inv_perm=inv, K=k)
    xp = B.moe_dispatch_scatter(x, inv, k)
    broken = torch.tensor([0, 30, 20, 31, T * k], dtype=I32, device=dev()) if bad else off
    zeros = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=dev())  # noqa: E731
    if bad:
        inv = inv.clone()
        inv[7] = T * k + 5
    status = lambda: B.moe_debug_check_status() if bad is not None else 0  # noqa: E731
    calls = {
        "rows": lambda: B.moe_fp4_quantize_rows(x, off, inv_perm=inv, K=k, out=(
            zeros(T * k, d // 2, dt=U8), torch.zeros_like(rows[1]), zeros(T * k, dt=F32))),
        "gemm_fp4": lambda: [B.moe_grouped_gemm_fp4(rows, broken, w4, out=zeros(T * k, 72))],
        "gemm": lambda: [B.moe_grouped_gemm(xp, broken, w, out=zeros(T * k, 72))],
        "wgrad": lambda: [B.moe_grouped_gemm_wgrad(xp, dy, broken, out=zeros(E, d, 72, dt=F32))],
    }
    return {n: ([t.float().cpu().numpy() for t in f()], status()) for n, f in calls.items()}


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
    """In a child process, as test_gpu_debug_block.py: a bad entry of inv_perm is recorded and its
    copy skipped, offsets that decrease are recorded and nothing is computed."""
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=_child, args=(q,))
    p.start()
    clean, flagged, code, err = q.get(timeout=600)
    p.join(60)
    assert err is None, err
    release = _outputs(bad=None)
    for name, (out, status) in clean.items():
        assert status == 0, name
        assert all(np.array_equal(a, b) for a, b in zip(out, release[name][0])), name
    for name, (out, status) in flagged.items():
        assert status == code, name
        if name != "rows":
            assert not out[0].any(), name
    q0, q1 = clean["rows"][0][0], flagged["rows"][0][0]
    same = (q0 == q1).all(1)
    assert (~same).sum() == 1 and not q1[~same].any()
