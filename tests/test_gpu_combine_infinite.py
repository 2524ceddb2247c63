"""dy = bf16(w dout) of an infinite gradient is infinite, in the combine's backward, its form for
a slice of the experts and its form on 8-bit checkpoints: a step's overflow check sees it, and
the rest of the row keeps its values."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import moe_oracle as O

from _parity import dev, ensure_built, f64, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("form", ["whole", "slice", "checkpoint"])
@pytest.mark.parametrize("T,d,k", [(5, 72, 3), (40, 2048, 8)])
def test_infinite_gradients(T, d, k, form):
    ensure_built()
    rng = np.random.default_rng([T, d])
    dout = O.round_bf16(rng.normal(size=(T, d)))
    dout[1, 4], dout[1, d - 1], dout[3, 0] = np.inf, -np.inf, np.nan
    dout[2, 5] = float(torch.finfo(BF).max)
    w = (0.1 + rng.random((T, k))).astype(np.float32)
    w[2] += 1.0                                      # 2, 5: past the largest value
    w[4, 0] = 0.0
    inv = rng.permutation(T * k)
    y = to_dev(np.zeros((T * k, d)), BF)
    args = (to_dev(dout, BF), y, to_dev(w, F32), to_dev(inv, I32))
    if form == "whole":
        dy, _ = B.moe_combine_backward(*args)
    elif form == "slice":
        offsets = torch.tensor([0, T * k], dtype=I32, device=dev())
        dy, _ = B.moe_combine_backward_slice(*args, offsets, 0, 1,
                                             out=(torch.empty_like(y), torch.empty_like(args[2])))
    else:
        dy, _ = B.moe_ckpt8_combine_backward(args[0], *B.moe_ckpt8_pack(y), *args[2:])
    with np.errstate(invalid="ignore", over="ignore"):
        exact = torch.from_numpy(w.astype(np.float64)[:, :, None] * dout[:, None, :])
        want = exact.to(F32).to(BF).double().numpy()     # only for what is not finite
    got = f64(dy)[inv].reshape(T, k, d)
    assert np.isinf(want).sum() == 3 * k
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    fine = np.isfinite(want)
    assert np.array_equal(got[fine], O.round_bf16(exact.numpy()[fine]))
