"""Host-side refusals of the grouped products and 4-bit floats (no GPU): bad arguments are
refused before anything is enqueued, by the C entry points and by the bindings."""
import ctypes

import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import build as build_mod
from oracle import fp4 as F

OK = ctypes.c_void_p(0x10000)            # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)
BAD, ALIGN, WS, UNSUP = (B.MOE_ERR_INVALID_ARG, B.MOE_ERR_MISALIGNED, B.MOE_ERR_WORKSPACE,
                         B.MOE_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_grouped_gemm(lib):
    def call(x=OK, off=OK, E=2, M=8, K=16, N=24, w=OK, y=OK, ws=OK, n=256):
        return lib.moe_grouped_gemm(x, off, E, M, K, N, w, 0, y, ws, n, None)
    assert call(E=0) == BAD and call(E=1025) == BAD and call(M=-1) == BAD
    assert call(K=12) == BAD and call(N=12) == BAD and call(K=0) == BAD and call(N=0) == BAD
    assert call(x=None) == BAD and call(off=None) == BAD and call(w=None) == BAD and call(y=None) == BAD
    assert call(x=MIS) == ALIGN and call(w=MIS) == ALIGN and call(y=MIS) == ALIGN
    assert call(ws=None) == WS and call(n=255) == WS and call(ws=MIS) == WS
    assert call(M=0, x=None, y=None, w=None) == B.MOE_OK


def test_grouped_gemm_wgrad(lib):
    size = B.workspace_size(B.MOE_OP_GROUPED_GEMM_WGRAD, 8, 2, 1, 1, 16, 24)
    assert size == 256 + 2 * 16 * (16 + 24) * 2
    assert B.workspace_size(B.MOE_OP_GROUPED_GEMM_WGRAD, 8, 2, 1, 1, 12, 24) == 0

    def call(x=OK, dy=OK, off=OK, E=2, M=8, K=16, N=24, dw=OK, ws=OK, n=size, acc=0):
        return lib.moe_grouped_gemm_wgrad(x, dy, off, E, M, K, N, acc, dw, ws, n, None)
    assert call(E=0) == BAD and call(K=4) == BAD and call(N=4) == BAD and call(M=-1) == BAD
    assert call(x=None) == BAD and call(dy=None) == BAD and call(dw=None) == BAD
    assert call(dw=MIS) == ALIGN and call(dy=MIS) == ALIGN
    assert call(ws=None) == WS and call(n=size - 1) == WS
    # an empty accumulation enqueues nothing (where a device is there to enqueue on)
    assert call(M=0, x=None, dy=None, acc=1) in (B.MOE_OK, UNSUP)


def test_rows(lib):
    def call(x=OK, inv=OK, T=4, K=2, off=OK, E=2, d=64, block=16, q=OK, sf=OK, rs=OK):
        return lib.moe_fp4_quantize_rows(x, inv, T, K, off, E, d, block, q, sf, rs, None)
    assert call(d=32) == BAD and call(d=96) == BAD and call(block=8) == BAD and call(block=64) == BAD
    assert call(K=0) == BAD and call(K=33) == BAD and call(inv=None) == BAD and call(T=-1) == BAD
    assert call(E=0) == BAD and call(E=1025) == BAD and call(d=16448) == UNSUP
    assert call(T=1 << 30, K=2) == UNSUP
    assert call(rs=None) == BAD and call(q=None) == BAD and call(sf=None) == BAD
    assert call(x=MIS) == ALIGN and call(q=MIS) == ALIGN and call(rs=MIS) == ALIGN
    assert call(T=0, x=None, q=None) == B.MOE_OK

    def back(q=OK, sf=OK, rs=OK, off=OK, E=2, M=8, d=64, block=16, out=OK):
        return lib.moe_fp4_dequantize_rows(q, sf, rs, off, E, M, d, block, out, None)
    assert back(d=96) == BAD and back(block=24) == BAD and back(rs=None) == BAD and back(out=None) == BAD
    assert back(out=MIS) == ALIGN and back(d=16448) == UNSUP and back(M=0, q=None) == B.MOE_OK


def test_weights(lib):
    def call(w=OK, E=2, K=64, N=16, block=16, c=OK, s=OK, g=OK):
        return lib.moe_fp4_quantize_weights(w, E, K, N, block, c, s, g, None)
    assert call(K=96) == BAD and call(N=12) == BAD and call(E=0) == BAD and call(g=None) == BAD
    assert call(c=MIS) == ALIGN and call(E=65536) == UNSUP

    def pack(a=OK, b=None, E=2, N=64, K=64, block=16, sf=OK):
        return lib.moe_fp4_pack_scales(a, b, E, N, K, block, sf, None)
    assert pack(K=32) == BAD and pack(N=4) == BAD and pack(b=OK, N=96) == BAD and pack(a=None) == BAD
    assert pack(sf=MIS) == ALIGN and pack(block=0) == BAD


def test_products(lib):
    def call(xq=OK, xsf=OK, rs=OK, off=OK, E=2, M=8, K=64, N=16, block=16, w=OK, wsf=OK, g=OK, y=OK,
             ws=OK, n=256):
        return lib.moe_grouped_gemm_fp4(xq, xsf, rs, off, E, M, K, N, block, w, wsf, g, y, ws, n, None)
    assert call(K=96) == BAD and call(N=12) == BAD and call(E=1025) == BAD and call(block=17) == BAD
    assert call(rs=None) == BAD and call(g=None) == BAD and call(xq=None) == BAD and call(y=None) == BAD
    assert call(xsf=MIS) == ALIGN and call(g=MIS) == ALIGN
    assert call(ws=None) == WS and call(n=0) == WS and call(M=0, xq=None) == B.MOE_OK

    size = B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, 8, 2, 1, 1, 64, 64)
    assert size > 256 and B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, 8, 2, 1, 1, 64, 96) == 0

    def ffn(xq=OK, rs=OK, off=OK, E=2, M=8, d=64, I=64, block=16, gate=OK, g=OK, dg=OK, hs=None, y=OK,
            ws=OK, n=size):
        return lib.moe_grouped_ffn_fp4(xq, OK, rs, off, E, M, d, I, block, gate, OK, OK, g, OK, OK, OK,
                                       dg, hs, y, ws, n, None)
    assert ffn(d=96) == BAD and ffn(I=96) == BAD and ffn(block=32, hs=OK) == BAD and ffn(E=0) == BAD
    assert ffn(g=None) == BAD and ffn(dg=None) == BAD and ffn(gate=None) == BAD and ffn(rs=None) == BAD
    assert ffn(hs=MIS) == ALIGN and ffn(y=MIS) == ALIGN and ffn(I=16448) == UNSUP
    assert ffn(ws=None) == WS and ffn(n=size - 1) == WS and ffn(M=0, xq=None) == B.MOE_OK


class _OnGpu(torch.Tensor):
    """A tensor without storage that says it is on a GPU."""
    is_cuda = True


def _t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(_OnGpu)


U8, F32, I32 = torch.uint8, torch.float32, torch.int32


def test_binding_refusals():
    x, off = _t(8, 64), _t(3, dtype=I32)
    w = _t(2, 64, 24)
    for call, what in (
            (lambda: B.moe_grouped_gemm(x, off, _t(2, 32, 24)), "shape"),
            (lambda: B.moe_grouped_gemm(x, off, w, trans=True), "shape"),
            (lambda: B.moe_grouped_gemm(x, off, _t(3, 64, 24)), "shape"),
            (lambda: B.moe_grouped_gemm(_t(64, 8).t(), off, w), "contiguous"),
            (lambda: B.moe_grouped_gemm(x, _t(1, dtype=I32), w), "offsets"),
            (lambda: B.moe_grouped_gemm_wgrad(x, _t(9, 24), off), "shape"),
            (lambda: B.moe_grouped_gemm_wgrad(x, _t(8, 24), off, accumulate=True,
                                              ws=_t(1 << 20, dtype=U8)), "give it|contiguous"),
            (lambda: B.moe_fp4_quantize_rows(x, off, block=8), "16 or 32"),
            (lambda: B.moe_fp4_quantize_rows(_t(8, 96), off), "multiple of 64"),
            (lambda: B.moe_fp4_quantize_rows(x, off, K=2), "inv_perm"),
            (lambda: B.moe_fp4_quantize_rows(x, off, inv_perm=_t(8, dtype=I32), K=2), "shape"),
            (lambda: B.moe_fp4_quantize_weights(_t(2, 96, 16)), "multiple of 64"),
            (lambda: B.moe_fp4_pack_scales(_t(2, 12, 4, dtype=U8)), "multiple of 8"),
            (lambda: B.moe_fp4_pack_scales(_t(2, 96, 4, dtype=U8), _t(2, 96, 4, dtype=U8)),
             "multiple of 64"),
            (lambda: B.moe_grouped_gemm(_t(2 ** 31, 8), off, _t(2, 8, 8)), "31 bits")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        B.moe_grouped_gemm(_t(8, 64, dtype=F32), off, w)
    with pytest.raises(TypeError):
        B.moe_fp4_quantize_rows(_t(8, 64, dtype=torch.float16), off)


def _fp4_args(M=8, d=64, I=64, E=2):
    rows = (_t(M, d // 2, dtype=U8), _t(-(-M // 128) + 2 * E, 1, 512, dtype=U8), _t(M, dtype=F32))
    gu = [_t(E, I, d // 2, dtype=U8), _t(E, I, d // 2, dtype=U8), _t(E, I // 64, 1, 512, dtype=U8),
          _t(E, dtype=F32), _t(E, dtype=F32)]
    wd = [_t(E, d, I // 2, dtype=U8), _t(E, 1, 1, 512, dtype=U8), _t(E, dtype=F32)]
    return rows, _t(E + 1, dtype=I32), gu, wd


def test_binding_refusals_of_the_products():
    rows, off, gu, wd = _fp4_args()
    bad = [
        lambda: B.moe_grouped_ffn_fp4((rows[0], rows[1], None), off, gu, wd),
        lambda: B.moe_grouped_ffn_fp4((rows[0], rows[1][:4], rows[2]), off, gu, wd),
        lambda: B.moe_grouped_ffn_fp4(rows, _t(4, dtype=I32), gu, wd),
        lambda: B.moe_grouped_ffn_fp4(rows, off, gu[:4] + [None], wd),
        lambda: B.moe_grouped_ffn_fp4(rows, off, [gu[0], _t(2, 128, 32, dtype=U8)] + gu[2:], wd),
        lambda: B.moe_grouped_ffn_fp4(rows, off, gu, [wd[0], None, wd[2]]),
        lambda: B.moe_grouped_ffn_fp4(rows, off, gu, wd, h_scale=_t(3, dtype=F32)),
        lambda: B.moe_grouped_ffn_fp4(rows, off, gu, wd, block=32, h_scale=_t(2, dtype=F32)),
        lambda: B.moe_grouped_gemm_fp4(rows, off, [_t(2, 16, 64, dtype=U8), wd[1], wd[2]]),
        lambda: B.moe_grouped_gemm_fp4(rows, off, [wd[0], wd[1], None]),
        lambda: B.moe_fp4_dequantize_rows((rows[0], rows[1], None), off),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_the_oracle_against_torch():
    """The oracle's E4M3 rounding against torch's over its whole range, and E2M1's ties."""
    rng = np.random.default_rng(0)
    grid = np.arange(0, 127).astype(np.uint8)
    val = torch.from_numpy(grid).view(torch.float8_e4m3fn).double().numpy()
    mid = (val[1:] + val[:-1]) / 2
    v = np.concatenate([val, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), rng.random(20000) * 448,
                        np.ldexp(rng.random(5000), -6)])
    v = v.astype(np.float32).astype(np.float64)
    byte, got = F.e4m3(v)
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn)
    assert np.array_equal(byte, want.view(torch.uint8).numpy()) and np.array_equal(got, want.double().numpy())
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 7.0, -0.25, 0.26, 4.9])
    assert list(F.e2m1(ties)) == [0, 2, 2, 4, 4, 6, 6, 14, 7, 0, 1, 6]
    assert list(F.row_factor(np.array([2688.0, 2688.5, 1344.0, 0.0, 3e38]))) == [
        1.0, 2.0, 0.5, 2.0 ** -100, 2.0 ** np.ceil(np.log2(3e38 / 2688))]
