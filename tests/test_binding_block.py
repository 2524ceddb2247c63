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
