"""What runs on a workspace between the two parts of the experts' backward: an operation that
writes into the workspace past its header ends the data part's record, so that the weight part
reports MOE_ERR_DEVICE_CHECK and writes nothing instead of reading what was overwritten; one that
uses the header alone leaves the weight part's results as they are, bit for bit."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import block as BL

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
COUNTS, d, I = [19, 0, 130, 7], 128, 256      # MXFP8 experts take multiples of 128
E, M = len(COUNTS), sum(COUNTS)
T, K = M // 2, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


class Problem:
    def __init__(self):
        g = torch.Generator(device=dev()).manual_seed(3)
        rnd = lambda *s, sc=1.0: (torch.randn(*s, generator=g, device=dev()) * sc).to(BF)  # noqa: E731
        self.dy, self.xp, self.gu, self.h = rnd(M, d, sc=0.1), rnd(M, d), rnd(M, 2 * I), rnd(M, I, sc=0.5)
        self.wg, self.wu = rnd(E, d, I, sc=0.1), rnd(E, d, I, sc=0.1)
        self.wd = rnd(E, I, d, sc=0.1)
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(COUNTS)]), dtype=I32, device=dev())
        self.logits = torch.randn(T, E, generator=g, device=dev())
        self.logits_wide = torch.randn(T, 512, generator=g, device=dev())
        self.idx = torch.topk(self.logits, K, dim=1)[1].to(I32)
        self.counts = torch.bincount(self.idx.flatten().long(), minlength=E).to(I32)
        self.gain, self.rstd = torch.ones(d, device=dev()), torch.ones(M, device=dev())
        self.rows = {b: B.moe_fp4_quantize_rows(self.xp, self.off, b) for b in (16, 32)}
        w = {"w_gate": self.wg, "w_up": self.wu, "w_down": self.wd}
        self.w4 = {b: BL.fp4_weights(w, b) for b in (16, 32)}
        self.int4 = BL.w4_weights(w, 32)
        self.fp8 = B.moe_mxfp8_quantize_weights(self.wg, self.wu), B.moe_mxfp8_quantize_weights(self.wd)
        self.h_scale = torch.full((E,), 0.01, device=dev())
        self.ws = B.new_workspace(16 << 20, dev())    # more than any of these operations asks for

    def data(self):
        return B.moe_grouped_ffn_backward_data(self.dy, self.xp, self.gu, self.h, self.off, self.wg,
                                               self.wu, self.wd, ws=self.ws)

    def weights(self):
        out = tuple(torch.full(s, 7.0, device=dev()) for s in ((E, d, I), (E, d, I), (E, I, d)))
        B.moe_grouped_ffn_backward_weights(self.dy, self.xp, self.h, self.off, E, I, ws=self.ws, out=out)
        return out, B.moe_read_device_status(self.ws)


def _ffn_fp4(p, block, h_scale=None):
    w = p.w4[block]
    return B.moe_grouped_ffn_fp4(p.rows[block], p.off, w["wgu"], w["wd"], block, h_scale, ws=p.ws)


WRITES = {
    "wgrad": lambda p: B.moe_grouped_gemm_wgrad(p.h, p.dy, p.off, ws=p.ws),
    "ffn_fp4_fixed": lambda p: _ffn_fp4(p, 16, p.h_scale),
    "ffn_fp4_row": lambda p: _ffn_fp4(p, 16),
    "ffn_fp4_block32": lambda p: _ffn_fp4(p, 32),
    "ffn_fp8": lambda p: B.moe_grouped_ffn_fp8(p.xp, p.off, *p.fp8, ws=p.ws),
    "norm_in_backward": lambda p: B.moe_norm_in_backward(p.dy, p.xp, p.gain, p.rstd, ws=p.ws),
    "norm_out_backward": lambda p: B.moe_norm_out_backward(p.dy, p.xp, p.rstd, p.gain, ws=p.ws),
    "norm_out_backward_gate": lambda p: B.moe_norm_out_backward(
        p.dy, p.xp, None, gate=torch.ones(1, 1, device=dev()), ws=p.ws),
    "load_balance": lambda p: B.moe_load_balance(p.logits, p.counts, K, ws=p.ws),
    "build_permutation": lambda p: B.moe_build_permutation(p.idx, E, ws=p.ws),
    "ep_layout": lambda p: B.moe_ep_layout(p.idx, E, 2, host_splits=False, ws=p.ws),
    "build_permutation_ep": lambda p: B.moe_build_permutation_ep(p.idx, E, 2, host_splits=False, ws=p.ws),
    "route_permute_ep": lambda p: B.moe_route_permute_ep(p.logits, K, 2, host_splits=False, ws=p.ws),
    "route_permute_ep_wide": lambda p: B.moe_route_permute_ep(p.logits_wide, K, 2, host_splits=False,
                                                              ws=p.ws),
}

LEAVES = {
    "grouped_gemm": lambda p: B.moe_grouped_gemm(p.h, p.off, p.wd, ws=p.ws),
    "grouped_gemm_trans": lambda p: B.moe_grouped_gemm(p.dy, p.off, p.wd, trans=True, ws=p.ws),
    "grouped_gemm_fp4": lambda p: B.moe_grouped_gemm_fp4(B.moe_fp4_quantize_rows(p.h, p.off), p.off,
                                                         p.w4[16]["wd"], ws=p.ws),
    "grouped_ffn": lambda p: B.moe_grouped_ffn(p.xp, p.off, p.wg, p.wu, p.wd, ws=p.ws),
    "ffn_w4": lambda p: B.moe_grouped_ffn_w4(p.xp, p.off, p.int4["wgu"], p.int4["wd"], ws=p.ws),
    "ep_recv_layout": lambda p: B.moe_ep_recv_layout(p.counts, p.counts, 1, M, host_splits=False, ws=p.ws),
    "empty_wgrad": lambda p: B.moe_grouped_gemm_wgrad(p.h[:0], p.dy[:0], torch.zeros_like(p.off), ws=p.ws),
    "empty_ffn_fp4": lambda p: B.moe_grouped_ffn_fp4(
        B.moe_fp4_quantize_rows(p.xp[:0], torch.zeros_like(p.off)), torch.zeros_like(p.off),
        p.w4[16]["wgu"], p.w4[16]["wd"], ws=p.ws),
}


@pytest.mark.parametrize("name", sorted(WRITES))
def test_a_written_workspace_holds_no_data_part(name):
    p = Problem()
    p.data()
    WRITES[name](p)
    out, status = p.weights()
    assert status == B.MOE_ERR_DEVICE_CHECK
    assert all((t == 7.0).all() for t in out)
    p.data()                                   # another data part, and the weight part runs
    out, status = p.weights()
    assert status == 0
    whole = B.moe_grouped_ffn_backward(p.dy, p.xp, p.gu, p.h, p.off, p.wg, p.wu, p.wd)
    assert all(torch.equal(a, b) for a, b in zip(out, whole[1:]))


@pytest.mark.parametrize("name", sorted(LEAVES))
def test_the_header_alone_leaves_the_data_part(name):
    p = Problem()
    p.data()
    LEAVES[name](p)
    out, status = p.weights()
    assert status == 0
    whole = B.moe_grouped_ffn_backward(p.dy, p.xp, p.gu, p.h, p.off, p.wg, p.wu, p.wd)
    assert all(torch.equal(a, b) for a, b in zip(out, whole[1:]))


def test_in_a_graph():
    """Captured: data part, weight gradient of an adapter on the same workspace, weight part."""
    p = Problem()
    dw = torch.zeros(E, I, d, device=dev())
    out = tuple(torch.full(s, 7.0, device=dev()) for s in ((E, d, I), (E, d, I), (E, I, d)))
    p.data()                                   # kernels load outside the capture
    B.moe_grouped_gemm_wgrad(p.h, p.dy, p.off, ws=p.ws, out=dw)
    dxp = torch.empty_like(p.xp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_grouped_ffn_backward_data(p.dy, p.xp, p.gu, p.h, p.off, p.wg, p.wu, p.wd, ws=p.ws, out=dxp)
        B.moe_grouped_gemm_wgrad(p.h, p.dy, p.off, ws=p.ws, out=dw)
        B.moe_grouped_ffn_backward_weights(p.dy, p.xp, p.h, p.off, E, I, ws=p.ws, out=out)
    for _ in range(2):
        graph.replay()
        assert B.moe_read_device_status(p.ws) == B.MOE_ERR_DEVICE_CHECK
        assert all((t == 7.0).all() for t in out)
