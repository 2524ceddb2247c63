"""Rows of an empty batch (no GPU): an empty inv_perm has no address."""
import ctypes

import pytest

from grouped_gemm_moe_gb300 import binding as B
from grouped_gemm_moe_gb300 import build as build_mod

OK = ctypes.c_void_p(0x10000)            # aligned, never dereferenced


@pytest.mark.parametrize("block", [16, 32])
def test_rows(block):
    build_mod.build()
    lib = B.load()
    call = lambda T, inv: lib.moe_fp4_quantize_rows(  # noqa: E731
        OK, inv, T, 2, OK, 2, 64, block, OK, OK, OK, None)
    assert call(0, None) == B.MOE_OK and call(1, None) == B.MOE_ERR_INVALID_ARG
