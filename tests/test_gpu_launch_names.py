"""The names of the grouped products' and 4-bit floats' launches in a profile: none is the layer's, so
that a model which runs both can tell them apart."""
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
E, d, I, M = 2, 128, 192, 40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _names(call):
    B.moe_profile_start(64)
    call()
    torch.cuda.synchronize()
    return [n for n, _ in B.moe_profile_stop()]


def test_names():
    g = torch.Generator(device=dev()).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev()).to(BF)   # noqa: E731
    w = {"w_gate": rnd(E, d, I), "w_up": rnd(E, d, I), "w_down": rnd(E, I, d)}
    x, h = rnd(M, d), rnd(M, I)
    off = torch.tensor([0, 15, M], dtype=I32, device=dev())
    w4 = BL.fp4_weights(w)
    rows, hrows = B.moe_fp4_quantize_rows(x, off), B.moe_fp4_quantize_rows(h, off)
    hs = torch.full((E,), 0.01, device=dev())
    layer = _names(lambda: B.moe_grouped_ffn_backward(
        rnd(M, d), x, B.moe_grouped_ffn(x, off, w["w_gate"], w["w_up"], w["w_down"])[2], h, off,
        w["w_gate"], w["w_up"], w["w_down"]))
    assert layer == ["gemm_gate_up", "gemm_down", "gemm_dh", "gemm_dx", "gemm_wgrad_gate_up", "gemm_wgrad_down"]
    calls = {
        "product": (lambda: B.moe_grouped_gemm(h, off, w["w_down"]), ["gemm"]),
        "input gradient": (lambda: B.moe_grouped_gemm(x, off, w["w_down"], trans=True), ["gemm_trans"]),
        "weight gradient": (lambda: B.moe_grouped_gemm_wgrad(h, x, off), ["gemm_pad_steps", "gemm_wgrad"]),
        "rows": (lambda: B.moe_fp4_quantize_rows(x, off), ["fp4_quantize_rows"]),
        "4-bit product": (lambda: B.moe_grouped_gemm_fp4(hrows, off, w4["wd"]), ["gemm_fp4"]),
        "4-bit experts": (lambda: B.moe_grouped_ffn_fp4(rows, off, w4["wgu"], w4["wd"], h_scale=hs),
                          ["gemm_gate_up_fp4", "gemm_down_fp4"]),
        "4-bit experts, rows": (lambda: B.moe_grouped_ffn_fp4(rows, off, w4["wgu"], w4["wd"]),
                                ["gemm_gate_up_fp4", "fp4_quantize_h", "gemm_down_fp4"]),
    }
    for what, (call, want) in calls.items():
        got = _names(call)
        assert got == want, what
        assert not set(got) & set(layer), what
