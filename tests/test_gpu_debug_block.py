"""The debug-checks build on the operators around the layer, in a child process: on
valid inputs it records no failed check and gives the release library's bits; an
index past its array is recorded and read as row 0 or skipped."""
import multiprocessing as mp
import os
import sys

import numpy as np
import pytest
import torch

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, K, D, I, E = 40, 3, 64, 64, 4


def _outputs(bad=False):
    from grouped_gemm_moe_gb300 import binding as B
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev())  # noqa: E731
    y, resid, x, dout = r(T * K, D), r(T, D), r(T, D), r(T, D)
    w = torch.rand(T, K, generator=g).to(dev())
    gain = torch.ones(D, device=dev())
    inv = torch.randperm(T * K, generator=g).to(torch.int32).to(dev())
    perm = torch.randperm(T * K, generator=g).to(torch.int32).to(dev())
    if bad:
        inv[7] = T * K + 5
        perm[11] = -4
    offsets = torch.tensor([0, 30, 31, 31, T * K], dtype=torch.int32, device=dev())
    weights = [r(E, a, b) for a, b in ((D, I), (D, I), (I, D))]
    plain = [B.moe_w4_quantize_weights(m, 32) for m in weights]
    wgu, wd = B.moe_w4_pack_weights(*plain[0], *plain[1]), B.moe_w4_pack_weights(*plain[2])
    calls = {
        "norm_out": lambda: B.moe_norm_out(y, resid, gain, w, inv)[:2],
        "dispatch": lambda: [B.moe_ckpt8_dispatch(*B.moe_ckpt8_pack(x), inv, K,
                                                  out=torch.zeros_like(y))],
        "combine": lambda: B.moe_ckpt8_combine_backward(dout, *B.moe_ckpt8_pack(y), w, inv,
                                                        out=(torch.zeros_like(y), w.clone())),
        "w4": lambda: B.moe_grouped_ffn_w4(x, offsets, wgu, wd, perm=perm, K=K),
    }
    res = {}
    for name, f in calls.items():
        out = [t.float().cpu().numpy() for t in f()]
        res[name] = (out, B.moe_debug_check_status() if bad is not None else 0)
    return res


def _child(q):
    sys.path.insert(0, ROOT)
    try:
        from grouped_gemm_moe_gb300 import binding as B
        from grouped_gemm_moe_gb300 import build as build_mod
        B.load(build_mod.build(debug=True))
        q.put((_outputs(), _outputs(bad=True), B.MOE_ERR_DEVICE_CHECK, None))
    except Exception:  # pragma: no cover - reported by the parent
        import traceback
        q.put((None, None, None, traceback.format_exc()))


def test_debug_build_matches_release_and_flags_bad_indexes():
    ensure_built()
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
        for a, b in zip(out, release[name][0]):
            assert np.array_equal(a, b), name
    for name, (out, status) in flagged.items():
        assert status == code, name
    # the other tokens keep their results (token 2 holds the bad entry, 7 = 2 K + 1)
    keep = [t for t in range(T) if t != 2]
    assert np.array_equal(flagged["norm_out"][0][0][keep], clean["norm_out"][0][0][keep])
