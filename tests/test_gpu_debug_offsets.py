"""The debug build's quantizers on expert offsets that are out of order: where a row's scales lie follows
from the offsets, so nothing is computed and the check is recorded. In a child process, as
test_gpu_debug_block.py; on offsets in order its results are the release build's, bit for bit."""
import multiprocessing as mp
import os
import sys

import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, K, E = 60, 2, 4
M = T * K
GOOD = [0, 30, 31, 31, M]
BROKEN = ([0, 30, 20, 31, M], [0, 30, 31, 31, M + 8], [5, 30, 31, 31, M])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _outputs(ends, status):
    """What each call leaves in buffers of zeros, and the recorded check."""
    g = torch.Generator().manual_seed(1)
    off = torch.tensor(ends, dtype=I32, device=dev())
    inv = torch.randperm(M, generator=g).to(I32).to(dev())
    out = {}
    for d, block in ((128, 16), (128, 32), (4096, 16), (4096, 32), (8192, 16)):
        x = torch.randn(T, d, generator=g).to(BF).to(dev())
        good = torch.tensor(GOOD, dtype=I32, device=dev())
        rows = B.moe_fp4_quantize_rows(x, good, block, inv, K)
        zeros = tuple(None if t is None else torch.zeros_like(t) for t in rows)
        back = torch.zeros(M, d, dtype=BF, device=dev())
        status()
        B.moe_fp4_quantize_rows(x, off, block, inv, K, out=zeros)
        out[f"rows {d} {block}"] = [t for t in zeros if t is not None], status()
        B.moe_fp4_dequantize_rows(rows, off, block, out=back)
        out[f"back {d} {block}"] = [back], status()
    xp = torch.randn(M, 256, generator=g).to(BF).to(dev())
    q, sf = B.moe_mxfp8_quantize_rows(xp, torch.tensor(GOOD, dtype=I32, device=dev()))
    q, sf = torch.zeros_like(q), torch.zeros_like(sf)
    B.moe_mxfp8_quantize_rows(xp, off, out=(q, sf))
    out["mxfp8 rows"] = [q.view(U8), sf], status()
    return {n: ([t.float().cpu().numpy() for t in ts], s) for n, (ts, s) in out.items()}


def _child(q):
    sys.path.insert(0, ROOT)
    try:
        from grouped_gemm_moe_gb300 import build as build_mod
        B.load(build_mod.build(debug=True))
        q.put(([_outputs(e, B.moe_debug_check_status) for e in (GOOD, *BROKEN)], None))
    except Exception:  # pragma: no cover - reported by the parent
        import traceback
        q.put((None, traceback.format_exc()))


def test_offsets_out_of_order():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=_child, args=(q,))
    p.start()
    got, err = q.get(timeout=600)
    p.join(60)
    assert err is None, err
    release = _outputs(GOOD, lambda: 0)
    for name, (out, status) in got[0].items():
        assert status == 0, name
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(out, release[name][0])), name
    for flagged in got[1:]:
        for name, (out, status) in flagged.items():
            assert status == B.MOE_ERR_DEVICE_CHECK, name
            assert not any(t.any() for t in out), name
