"""The 4-bit experts in a workspace of exactly their size, with what lies behind it left as it was; the
block against its calls one by one, bit for bit."""
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL
from grouped_gemm_moe_gb300 import workloads as W

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
KINDS = [(16, True), (16, False), (32, False)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("block,fixed", KINDS)
@pytest.mark.parametrize("I,counts", [(192, [130, 0, 7]), (128, [1]), (320, [257, 300])])
def test_exact_size(block, fixed, I, counts):
    g = torch.Generator(device=dev()).manual_seed(I)
    E, d, M = len(counts), 256, sum(counts)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev()).to(BF)   # noqa: E731
    w = BL.fp4_weights({"w_gate": rnd(E, d, I) * 0.1, "w_up": rnd(E, d, I) * 0.1,
                        "w_down": rnd(E, I, d) * 0.1}, block)
    off = torch.zeros(E + 1, dtype=I32, device=dev())
    off[1:] = torch.cumsum(torch.tensor(counts, device=dev()), 0)
    rows = B.moe_fp4_quantize_rows(rnd(M, d), off, block)
    hs = torch.full((E,), 0.01, device=dev()) if fixed else None
    size = B.workspace_size(B.fp4_ffn_op(block, hs), M, E, 1, 1, d, I)
    buf = torch.full((size + 4096,), 0xab, dtype=U8, device=dev())
    buf[:B.WORKSPACE_HEADER] = 0
    y = B.moe_grouped_ffn_fp4(rows, off, w["wgu"], w["wd"], block, hs, ws=buf[:size])
    assert B.moe_read_device_status(buf[:size]) == 0
    assert (buf[size:] == 0xab).all()
    roomy = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, M, E, 1, 1, d, I), dev())
    assert torch.equal(y, B.moe_grouped_ffn_fp4(rows, off, w["wgu"], w["wd"], block, hs, ws=roomy))
    assert torch.equal(y, B.moe_grouped_ffn_fp4(rows, off, w["wgu"], w["wd"], block, hs))


@pytest.mark.parametrize("block,fixed", KINDS)
@pytest.mark.parametrize("shared_I", [0, 192])
def test_the_block_is_its_calls(block, fixed, shared_I):
    cfg = W.small_config("fp4calls", T=133, d=320, E=10, K=3, I=192, R=1, shared_I=shared_I)
    inp = W.make_inputs(cfg)
    weights = {k: v.to(dev()) for k, v in inp.items() if k.startswith("w")}
    x, logits = inp["x"].to(dev()), inp["logits"].to(dev())
    g = torch.Generator(device=dev()).manual_seed(4)
    gains = 0.5 + torch.rand(2, cfg.d, generator=g, device=dev())
    w4 = BL.fp4_weights(weights, block)
    hs = 0.01 * (0.5 + torch.rand(cfg.E, generator=g, device=dev())) if fixed else None
    sh = torch.full((1,), 0.02, device=dev()) if fixed else None
    blk = BL.MoEFp4Block(cfg.T, cfg.K, w4, gains[0].contiguous(), gains[1].contiguous(), scale=0.75,
                         block=block, h_scale=hs, sh_scale=sh)
    assert blk.ws_ffn.numel() == B.workspace_size(B.fp4_ffn_op(block, hs), cfg.T * cfg.K, cfg.E, 1, 1,
                                                  cfg.d, cfg.I)
    blk.norm(x)
    got = blk.forward(logits)
    xn, _ = B.moe_norm_in(x, gains[0].contiguous())
    _, tw, _, off, _, inv, *_ = B.moe_route_permute_ep(logits, cfg.K, 1, 1, host_splits=False)
    rows = B.moe_fp4_quantize_rows(xn, off, block, inv, cfg.K)
    y = B.moe_grouped_ffn_fp4(rows, off, w4["wgu"], w4["wd"], block, hs)
    ys = None
    if shared_I:
        s_off = torch.tensor([0, cfg.T], dtype=I32, device=dev())
        ys = B.moe_grouped_ffn_fp4(B.moe_fp4_quantize_rows(xn, s_off, block), s_off, w4["sgu"], w4["sd"],
                                   block, sh)
    want, _, _ = B.moe_norm_out(y, x, gains[1].contiguous(), tw, inv, ys, scale=0.75, save=False)
    assert torch.equal(got, want)
