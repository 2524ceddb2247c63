"""Host-side argument checks of the block's entry points (no GPU): bad arguments
are refused before anything is enqueued."""
import ctypes

import pytest

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import build as build_mod

OK = ctypes.c_void_p(0x10000)            # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)
BAD, ALIGN, WS, UNSUP = (B.MOE_ERR_INVALID_ARG, B.MOE_ERR_MISALIGNED, B.MOE_ERR_WORKSPACE,
                         B.MOE_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_norm_in(lib):
    f = lib.moe_norm_in
    assert f(OK, OK, 4, 12, 1e-6, OK, OK, None) == BAD
    assert f(OK, OK, -1, 16, 1e-6, OK, OK, None) == BAD
    assert f(OK, OK, 4, 16, -1.0, OK, OK, None) == BAD
    assert f(OK, OK, 4, 16, float("nan"), OK, OK, None) == BAD
    assert f(OK, OK, 4, 16392, 1e-6, OK, OK, None) == UNSUP
    assert f(OK, None, 4, 16, 1e-6, OK, OK, None) == BAD
    assert f(MIS, OK, 4, 16, 1e-6, OK, OK, None) == ALIGN
    assert f(None, None, 0, 16, 1e-6, None, None, None) == B.MOE_OK
    g = lib.moe_norm_in_backward
    assert g(OK, OK, OK, OK, None, 4, 16, OK, OK, OK, 256, None) == WS
    assert g(OK, OK, OK, OK, None, 4, 16, OK, OK, None, 1 << 30, None) == WS
    assert g(OK, OK, OK, OK, MIS, 4, 16, OK, OK, OK, 1 << 30, None) == ALIGN
    assert g(OK, OK, OK, None, None, 4, 16, OK, OK, OK, 1 << 30, None) == BAD
    assert g(OK, OK, OK, OK, None, 4, 16, OK, None, OK, 1 << 30, None) == BAD


def test_norm_out(lib):
    f = lib.moe_norm_out

    def call(y=OK, K=2, resid=OK, gate=None, span=1, cols=1, eps=1e-6, T=4, d=16, out=OK,
             shared=None):
        return f(y, OK, OK, K, shared, resid, OK, gate, span, cols, 1.0, eps, T, d, out, None, None,
                 None)
    assert call(K=0) == BAD and call(K=33) == BAD and call(d=20) == BAD and call(eps=-1.0) == BAD
    assert call(gate=OK, span=0) == BAD and call(gate=OK, cols=8) == BAD
    assert call(y=None) == BAD and call(resid=None) == BAD and call(out=None) == BAD
    assert call(shared=MIS) == ALIGN and call(d=16392) == UNSUP
    assert call(T=1 << 30, K=2) == UNSUP
    assert call(T=0, y=None, resid=None, out=None) == B.MOE_OK
    g = lib.moe_norm_out_backward
    assert g(OK, OK, OK, OK, None, 1, 1, 1.0, 4, 16, OK, None, None, OK, 1 << 30, None) == BAD
    assert g(OK, OK, OK, None, OK, 1, 1, 1.0, 4, 16, OK, None, None, OK, 1 << 30, None) == BAD
    assert g(OK, OK, None, OK, None, 1, 1, 1.0, 4, 16, OK, OK, None, OK, 1 << 30, None) == BAD
    assert g(OK, OK, OK, OK, OK, 1, 5, 1.0, 4, 16, OK, OK, OK, OK, 1 << 30, None) == BAD
    assert g(OK, OK, OK, OK, None, 1, 1, 1.0, 4, 16, OK, OK, None, OK, 0, None) == WS


def test_norm_gradients_end_at_two_to_the_30_rows(lib):
    T = (1 << 30) + 1
    n = 1 << 60
    assert lib.moe_norm_in_backward(OK, OK, OK, OK, None, T, 8, OK, OK, OK, n, None) == UNSUP
    assert lib.moe_norm_out_backward(OK, OK, OK, OK, None, 1, 1, 1.0, T, 8, OK, OK, None, OK, n,
                                     None) == UNSUP
    assert B.workspace_size(B.MOE_OP_NORM_BACKWARD, T, 1, 1, 1, 8) == 0
    assert B.workspace_size(B.MOE_OP_NORM_BACKWARD, T - 1, 1, 1, 1, 8) > 0


def test_ckpt8(lib):
    assert lib.moe_ckpt8_pack(OK, 4, 12, OK, OK, None) == BAD
    assert lib.moe_ckpt8_pack(OK, 4, 0, OK, OK, None) == BAD
    assert lib.moe_ckpt8_pack(OK, 4, 16, None, OK, None) == BAD
    assert lib.moe_ckpt8_pack(OK, 4, 16, OK, MIS, None) == ALIGN
    assert lib.moe_ckpt8_pack(None, 0, 16, None, None, None) == B.MOE_OK
    assert lib.moe_ckpt8_dispatch(OK, OK, OK, 4, 33, 16, OK, None) == BAD
    assert lib.moe_ckpt8_dispatch(OK, OK, MIS, 4, 2, 16, OK, None) == ALIGN
    assert lib.moe_ckpt8_swiglu(OK, OK, 4, 12, OK, OK, None) == BAD
    assert lib.moe_ckpt8_swiglu(OK, OK, 4, 16, OK, None, None) == BAD
    assert lib.moe_ckpt8_combine_backward(OK, OK, OK, OK, None, 4, 2, 16, OK, OK, None) == BAD
    assert lib.moe_ckpt8_combine_backward(OK, OK, OK, OK, OK, 1 << 30, 2, 16, OK, OK, None) == UNSUP


def test_w4(lib):
    q = lib.moe_w4_quantize_weights
    assert q(OK, 1, 96, 16, 32, OK, OK, None) == BAD          # K % 64
    assert q(OK, 1, 128, 16, 48, OK, OK, None) == BAD         # group
    assert q(OK, 1, 64, 16, 128, OK, OK, None) == BAD         # K % group
    assert q(OK, 1, 64, 16, 32, MIS, OK, None) == ALIGN
    p = lib.moe_w4_pack_weights
    assert p(OK, OK, OK, None, 1, 16, 64, 32, OK, OK, None) == BAD
    assert p(OK, OK, None, None, 1, 24, 64, 32, OK, OK, None) == BAD     # N % 32
    assert p(OK, OK, OK, OK, 1, 12, 64, 32, OK, OK, None) == BAD         # N % 16
    f = lib.moe_grouped_ffn_w4

    def call(x=OK, perm=None, T=8, K=1, E=2, M=8, d=128, I=64, gg=64, gd=64, ws=OK, n=1 << 30,
             off=OK):
        return f(x, perm, T, K, off, E, M, d, I, gg, gd, OK, OK, OK, OK, OK, OK, ws, n, None)
    assert call(d=96) == BAD and call(I=32) == BAD and call(gg=16) == BAD and call(gd=128) == BAD
    assert call(E=0) == BAD and call(E=1025) == BAD and call(M=9) == BAD
    assert call(perm=OK, K=2) == BAD                          # M is T K
    assert call(x=None) == BAD and call(x=MIS) == ALIGN and call(off=None) == BAD
    assert call(ws=None) == WS and call(n=0) == WS
    assert call(T=0, M=0, x=None) == B.MOE_OK


def test_workspace_sizes(lib):
    assert B.workspace_size(B.MOE_OP_NORM_BACKWARD, 64, 1, 1, 1, 12) == 0
    assert B.workspace_size(B.MOE_OP_NORM_BACKWARD, 64, 1, 1, 1, 128) >= B.WORKSPACE_HEADER
    assert B.workspace_size(B.MOE_OP_GROUPED_FFN_W4, 64, 8, 2, 1, 100, 64) == 0
    assert B.workspace_size(B.MOE_OP_GROUPED_FFN_W4, 64, 8, 2, 1, 128, 64) >= B.WORKSPACE_HEADER
