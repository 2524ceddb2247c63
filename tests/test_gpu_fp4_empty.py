"""Batches without a token, and hidden rows of none, through the block on 4-bit floats and its calls
with their usual arguments."""
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
E, d, I, K = 8, 128, 192, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _weights():
    g = torch.Generator(device=dev()).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev()).to(BF) * 0.1   # noqa: E731
    return {"w_gate": rnd(E, d, I), "w_up": rnd(E, d, I), "w_down": rnd(E, I, d),
            "ws_gate": rnd(d, I), "ws_up": rnd(d, I), "ws_down": rnd(I, d)}


@pytest.mark.parametrize("block", [16, 32])
def test_dispatched_rows(block):
    off = torch.zeros(E + 1, dtype=I32, device=dev())
    q, sf, rs = B.moe_fp4_quantize_rows(torch.empty(0, d, dtype=BF, device=dev()), off, block,
                                        inv_perm=torch.empty(0, dtype=I32, device=dev()), K=K)
    assert q.shape == (0, d // 2) and (rs is None) == (block == 32)


@pytest.mark.parametrize("block,fixed", [(16, False), (16, True), (32, False)])
def test_the_block(block, fixed):
    h = [torch.full((n,), 0.01, device=dev()) if fixed else None for n in (E, 1)]
    blk = BL.MoEFp4Block(0, K, BL.fp4_weights(_weights(), block), torch.ones(d, device=dev()),
                         block=block, h_scale=h[0], sh_scale=h[1])
    xn = blk.norm(torch.empty(0, d, dtype=BF, device=dev()))
    out = blk.forward(torch.empty(0, E, device=dev()))
    torch.cuda.synchronize()
    assert xn.shape == out.shape == (0, d)


def test_calibration_on_no_rows():
    off = torch.zeros(E + 1, dtype=I32, device=dev())
    h = BL.fp4_h_scale(torch.empty(0, I, dtype=BF, device=dev()), off)
    assert h.shape == (E,) and (h == 2.0 ** -100).all()
