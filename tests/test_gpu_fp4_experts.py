"""The experts on 4-bit floats at small sizes, with a bound on the rows that may hold a changed code of
H from the chance of one (2^-16 a value, derived in test_gpu_fp4_tiles.py): 2 + 3 M I 2^-16 rows, never
more than an eighth of them, so none where there are fewer than eight."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import dev, ensure_built, f64, rounding_excess, to_dev
from test_gpu_fp4_tiles import _matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("block,hidden", [(16, "fixed"), (16, "row"), (32, "block")])
@pytest.mark.parametrize("d,I,E,counts", [
    (64, 64, 1, [1]), (128, 128, 2, [0, 130]), (256, 192, 3, [31, 257, 4]), (192, 384, 2, [300, 5]),
    (2048, 768, 3, [2, 129, 0]), (320, 1408, 2, [17, 33]), (576, 320, 4, [1, 2, 0, 3]),
])
def test_experts(block, hidden, d, I, E, counts):
    rng = np.random.default_rng([d, I, E, block, len(hidden)])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    (wg, gq, gs, gg), (wu, uq, us, ug), (wd, dq, ds, dg) = (
        _matrix(rng, E, *s, block) for s in ((I, d), (I, d), (d, I)))
    x = O.round_bf16(rng.normal(size=(M, d)) / np.sqrt(np.mean(wg ** 2) * d))    # G and U of size one
    hs = ((0.5 + rng.random(E)) * 4e-3).astype(np.float32) if hidden == "fixed" else None
    off = to_dev(offsets, torch.int32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, torch.bfloat16), off, block)
    y = f64(B.moe_grouped_ffn_fp4(rows, off, (gq, uq, B.moe_fp4_pack_scales(gs, us, block), gg, ug),
                                  (dq, B.moe_fp4_pack_scales(ds, block=block), dg), block,
                                  None if hs is None else to_dev(hs, torch.float32)))
    want, _ = F.grouped_ffn_fp4(F.restore(*F.quantize_rows(x, block), block), offsets, wg, wu, wd, block,
                                h_scale=None if hs is None else hs.astype(np.float64),
                                round_h=O.round_bf16 if hidden == "row" else None)
    off_rows = (rounding_excess(y, want) > 1e-3 * np.sqrt(np.mean(want ** 2))).any(1)
    assert off_rows.sum() <= min(2 + 3 * M * I * 2.0 ** -16, M // 8), (off_rows.sum(), M)
