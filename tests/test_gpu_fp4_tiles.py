"""Products and experts on 4-bit floats with several tiles for every cluster: the accumulator handed
back, scale slots and stages carried from tile to tile, for every instance of the kernel.

Tolerances. A product's y: half an ulp of the stored bf16 value plus 1e-3 of the RMS. The experts'
H is quantized from fp32 values that miss the exact ones by about 2^-21 of their size (sums of up to
832 terms and the fast sigmoid); an element's code can differ only where a border between two codes,
or between two scales of its block, lies within that distance. In units of a block's scale its values
spread over [0, 6] with a density of 0.3 at the most near the seven borders, and are off by 2^-19 of
such a unit: a chance of 7 * 0.3 * 2 * 2^-19 < 2^-16 an element. Rounding H to bf16 first moves the
borders by half a bf16 step and adds none (a border is a bf16 value itself, so of two neighbours in
bf16 with different codes one lies on it): the same chance. Each changed code moves one row of y, so M
rows of I values hold off = M I 2^-16 such rows on average; at most 2 + 3 off are accepted, and this
has to be fewer than an eighth of the rows. All other rows are held to the product's tolerance."""
import numpy as np
import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B
from oracle import fp4 as F
from oracle import moe_oracle as O

from _parity import assert_bf16_close, dev, ensure_built, f64, rounding_excess, to_dev

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _matrix(rng, E, N, K, block):
    codes = rng.integers(0, 16, size=(E, N, K))
    if block == 16:
        byte = rng.integers(40, 72, size=(E, N, K // 16))
        g = ((0.5 + rng.random(E)) * 2.0 ** -5).astype(np.float32)
        val = F.restore(codes, byte, g.astype(np.float64)[:, None] * np.ones((E, N)), block)
    else:
        byte, g = rng.integers(118, 124, size=(E, N, K // 32)), None
        val = F.restore(codes, byte, None, block)
    packed = to_dev((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8), U8)
    return val, packed, to_dev(byte, U8), None if g is None else to_dev(g, F32)


def _counts(rng, E):
    """A few rows for most experts; none, a full pair and more than one pair of tiles for others."""
    counts = rng.integers(1, 8, size=E)
    counts[rng.permutation(E)[:8]] = [0, 0, 256, 129, 300, 128, 513, 31]
    return counts


def _clusters():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


@pytest.mark.parametrize("block,hidden", [(16, "fixed"), (16, "row"), (32, "block")])
@pytest.mark.parametrize("d,I", [(320, 768), (832, 448), (576, 192)])
def test_experts(block, hidden, d, I):
    """d of 2, 4 and 3 k-blocks (the last one partial): stages (five) and scale slots (three) stand
    elsewhere at each tile's start. I = 768 on tiles of 128 + 128 columns, 448 and 192 on 64 + 64."""
    rng = np.random.default_rng([d, I, block, len(hidden)])
    E = 64
    counts = _counts(rng, E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    pairs = sum(-(-c // 256) for c in counts)
    assert pairs * (I // (128 if I % 128 == 0 else 64)) > 2 * _clusters()
    (wg, gq, gs, gg), (wu, uq, us, ug), (wd, dq, ds, dg) = (
        _matrix(rng, E, *s, block) for s in ((I, d), (I, d), (d, I)))
    x = O.round_bf16(rng.normal(size=(M, d)) / np.sqrt(np.mean(wg ** 2) * d))    # G and U of size one
    off = to_dev(offsets, I32)
    hs = ((0.5 + rng.random(E)) * 4e-3).astype(np.float32) if hidden == "fixed" else None
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    ws = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, M, E, 1, 1, d, I), dev())
    ws[B.WORKSPACE_HEADER:] = 0xff             # NaN in every format: nothing may be read before it is written
    y = B.moe_grouped_ffn_fp4(rows, off, (gq, uq, B.moe_fp4_pack_scales(gs, us, block), gg, ug),
                              (dq, B.moe_fp4_pack_scales(ds, block=block), dg), block,
                              None if hs is None else to_dev(hs, F32), ws=ws)
    assert B.moe_read_device_status(ws) == 0
    xv = F.restore(*F.quantize_rows(x, block), block)
    want, _ = F.grouped_ffn_fp4(xv, offsets, wg, wu, wd, block,
                                h_scale=None if hs is None else hs.astype(np.float64),
                                round_h=O.round_bf16 if hidden == "row" else None)
    rms = np.sqrt(np.mean(want ** 2))
    off_rows = (rounding_excess(f64(y), want) > 1e-3 * rms).any(1)
    most = 2 + 3 * M * I * 2.0 ** -16
    assert most < M / 8
    assert off_rows.sum() <= most, (off_rows.sum(), most)
    # a changed code of H: at most two units of its block's scale, times a weight
    assert np.sqrt(np.mean((f64(y) - want) ** 2)) <= 5e-3 * rms


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K,N", [(320, 1032), (1344, 1032), (832, 1672)])
def test_product(block, K, N):
    """Five stages (K > 1024) and four."""
    rng = np.random.default_rng([K, N, block])
    E = 64
    counts = _counts(rng, E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    assert sum(-(-c // 256) for c in counts) * -(-N // 256) > 4 * _clusters()
    x = O.round_bf16(rng.normal(size=(M, K)))
    val, codes, byte, g = _matrix(rng, E, N, K, block)
    off = to_dev(offsets, I32)
    rows = B.moe_fp4_quantize_rows(to_dev(x, BF), off, block)
    y = B.moe_grouped_gemm_fp4(rows, off, (codes, B.moe_fp4_pack_scales(byte, block=block), g), block)
    xv = F.restore(*F.quantize_rows(x, block), block)
    assert_bf16_close(f64(y), F.grouped_product(xv, offsets, np.swapaxes(val, 1, 2)), "y")


def test_same_bits_on_every_run_of_the_experts():
    """With other garbage in the workspace and the rows' unwritten scales each time."""
    g = torch.Generator(device=dev()).manual_seed(2)
    E, d, I = 48, 832, 832
    counts = torch.randint(0, 300, (E,), generator=g, device=dev())
    off = torch.zeros(E + 1, dtype=I32, device=dev())
    off[1:] = torch.cumsum(counts, 0)
    M = int(off[-1])
    x = torch.randn(M, d, generator=g, device=dev()).to(BF)
    u8 = lambda *s: torch.randint(0, 256, s, generator=g, dtype=U8, device=dev())   # noqa: E731
    for block in (16, 32):
        lo, hi = (48, 72) if block == 16 else (116, 124)
        sc = lambda n, k: torch.randint(lo, hi, (E, n, k // block), generator=g, dtype=U8, device=dev())  # noqa: E731
        one = torch.full((E,), 0.01, device=dev()) if block == 16 else None
        gu = (u8(E, I, d // 2), u8(E, I, d // 2), B.moe_fp4_pack_scales(sc(I, d), sc(I, d), block), one, one)
        wd = (u8(E, d, I // 2), B.moe_fp4_pack_scales(sc(d, I), block=block), one)
        size = B.workspace_size(B.MOE_OP_GROUPED_FFN_FP4, M, E, 1, 1, d, I)
        for hs in (None, torch.full((E,), 0.02, device=dev())) if block == 16 else (None,):
            first = None
            for fill in (0xff, 0x00, 0x7f, 0xff):
                rows = tuple(None if t is None else torch.empty_like(t)
                             for t in B.moe_fp4_quantize_rows(x, off, block))
                for t in rows:
                    if t is not None:
                        t.view(U8).fill_(fill)
                B.moe_fp4_quantize_rows(x, off, block, out=rows)
                ws = B.new_workspace(size, dev())
                ws[B.WORKSPACE_HEADER:] = fill
                y = B.moe_grouped_ffn_fp4(rows, off, gu, wd, block, hs, ws=ws)
                assert torch.isfinite(y.float()).all()
                first = y if first is None else first
                assert torch.equal(y, first)
