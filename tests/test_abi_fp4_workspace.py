"""The 4-bit experts' workspace without a bf16 H (no GPU): its size and who may come with it."""
import ctypes

import pytest

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import build as build_mod

OK = ctypes.c_void_p(0x10000)            # aligned, never dereferenced
M, E, d, I = 1000, 3, 128, 192


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_sizes(lib):
    size = lambda op, I=I: B.workspace_size(op, M, E, 1, 1, d, I)   # noqa: E731
    whole, fused = size(B.MOE_OP_GROUPED_FFN_FP4), size(B.MOE_OP_GROUPED_FFN_FP4_FUSED)
    up = lambda n: -(-n // 1024) * 1024                             # noqa: E731
    assert fused == 256 + up(M * I // 2) + up((-(-M // 128) + 2 * E) * -(-I // 64) * 512)
    assert whole == fused + up(2 * M * I) + up(4 * M)
    assert size(B.MOE_OP_GROUPED_FFN_FP4_FUSED, 96) == 0


def test_refusals(lib):
    fused = B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4_FUSED, M, E, 1, 1, d, I)

    def call(n, block, hs, ws=OK):
        f = OK if block == 16 else None
        return lib.moe_grouped_ffn_fp4(OK, OK, f, OK, E, M, d, I, block, OK, OK, OK, f, f, OK, OK, f, hs,
                                       OK, ws, n, None)
    assert call(fused, 16, None) == B.MOE_ERR_WORKSPACE        # rows by their own maximum: bf16 H
    assert call(fused - 1, 16, OK) == B.MOE_ERR_WORKSPACE
    assert call(fused - 1, 32, None) == B.MOE_ERR_WORKSPACE
    assert call(fused, 16, OK, None) == B.MOE_ERR_WORKSPACE
    assert B.fp4_ffn_op(16, None) == B.MOE_OP_GROUPED_FFN_FP4
    assert B.fp4_ffn_op(16, OK) == B.fp4_ffn_op(32, None) == B.MOE_OP_GROUPED_FFN_FP4_FUSED
