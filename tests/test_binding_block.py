"""Argument checks of the block's bindings that need no GPU: sizes that do not fit the
C interface's 32-bit integers are refused or brought into range before the call."""
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B


@pytest.mark.parametrize("cols", [1, 64])
@pytest.mark.parametrize("span", [100, 101, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 40])
def test_a_span_past_the_tokens_means_one_gate_row(monkeypatch, span, cols):
    """A span of more than 31 bits would arrive as another number (2^32 + 1 as 1: one gate
    row per token, read and written past the only one)."""
    monkeypatch.setattr(B, "_need", lambda *a: None)
    T, d = 100, 64
    got, got_cols = B._gate_args(torch.ones(1, cols), span, T, d, torch.device("cpu"))
    assert got_cols == cols
    assert T <= got < 2 ** 31      # token T - 1 is in row 0, and the number fits an int


class _OnGpu(torch.Tensor):
    """A tensor without storage that says it is on a GPU."""
    is_cuda = True


def _large(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(_OnGpu)


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 5])
def test_more_rows_than_31_bits_are_refused(rows):
    """Cut to 32 bits, 2^32 rows would be none and 2^32 + 5 five: a call that returns without
    error and without having written its outputs."""
    x = _large(rows, 8)
    gain = _large(8, dtype=torch.float32)
    q, s = _large(rows, 8, dtype=torch.int8), _large(rows, 1)
    for call in (lambda: B.moe_norm_in(x, gain),
                 lambda: B.moe_norm_in_backward(x, x, gain, gain),
                 lambda: B.moe_norm_out(x, x, gain),
                 lambda: B.moe_norm_out_backward(x, x, gain, gain),
                 lambda: B.moe_ckpt8_pack(x),
                 lambda: B.moe_ckpt8_dispatch(q, s),
                 lambda: B.moe_ckpt8_swiglu(q, s),
                 lambda: B.moe_dispatch(x, gain, 1)):
        with pytest.raises(ValueError, match="31 bits"):
            call()
