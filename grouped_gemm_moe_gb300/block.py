"""One MoE block of a model around the layer, in training and in decoding.

A block is norm -> router -> experts -> combine, norm, gate and residual add:

    xn  = RMSNorm(x) * gain_in
    out = x + scale * gate * (RMSNorm(combine(experts(xn))) * gain_out)

The router's product xn -> logits is the caller's (a plain matrix product, here
as in the layer), so each pass comes in two calls with the router between them.

Training (``MoEBlock`` around a ``MoELayer``):
    xn = block.norm(x);  logits = router(xn);  out = block.forward(logits)
    dxn, dlogits = block.backward(dout);  dxn += the router's share
    dx = block.backward_norm(dxn)
Tensors that later calls read again are the caller's to leave unchanged until then:
x from ``norm`` until ``backward_norm``, dout from ``backward`` until ``backward_norm``.

With a layer that keeps 8-bit checkpoints and takes a ``BlockScratch`` as its
scratch, a block holds, between its passes, its input (the caller's, or the block
before's out), out, the combined rows and the layer's codes; what it needs while it
is at work it shares with the model's other blocks.

Decoding (``MoEDecodeBlock``, experts on 4-bit weights) and prefill (``MoEFp4Block``, experts
on microscaled 4-bit floats, activations included):
    xn = block.norm(x);  logits = router(xn);  out = block.forward(logits)

This module only allocates tensors and orders the calls; each step is a kernel
of libmoe_gb300.so.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import binding as B
from .layer import LayerScratch, MoELayer


class BlockScratch(LayerScratch):
    """A LayerScratch for the layers of a model's blocks that holds the blocks' own passing
    buffers too. Blocks of one shape on one stream share it and then run one after the
    other, each in the forward from norm to forward, in the backward from backward to
    backward_norm:

    * xn is a block's from its norm until another's, and again (made from x once more, the
      same bits) when its backward returns, for the gradient of the router's product;
    * dxn, what backward returns, lasts until another block's backward;
    * dx, what backward_norm returns, is the next block's dout and is overwritten by that
      block's backward_norm."""

    def __init__(self, T: int, d: int, E: int, K: int, I: int, shared_I: int = 0, device=None):
        super().__init__(T, d, E, K, I, shared_I, device)
        e = lambda: torch.empty(T, d, dtype=torch.bfloat16, device=device)  # noqa: E731
        self.xn, self.dz, self.dxn, self.dx = e(), e(), e(), e()
        self.ws_norm = B.new_workspace(B.workspace_size(B.MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d),
                                       device)
        self.xn_of = None    # the mark of the block whose xn it holds


class MoEBlock:
    """``gain_in`` [d] fp32; ``gain_out`` [d] fp32 or None (no norm after the experts); ``gate``
    fp32 [ceil(T / span), 1 or d] or None; ``scale`` the residual scale. Gradients of the
    vectors are left in dgain_in, dgain_out and dgate. With a BlockScratch as the layer's
    scratch the block works in that."""

    def __init__(self, layer: MoELayer, gain_in: torch.Tensor,
                 gain_out: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 span: Optional[int] = None, scale: float = 1.0, eps: float = 1e-6):
        self.layer = layer
        self.gain_in, self.gain_out, self.gate, self.span = gain_in, gain_out, gate, span
        self.scale, self.eps = float(scale), float(eps)
        T, d, dev = layer.T, layer.d, layer.device
        bf, f32 = torch.bfloat16, torch.float32
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.out, self.z = e(T, d, dt=bf), e(T, d, dt=bf)
        self.rstd_in = e(T, dt=f32)
        self.rstd_out = e(T, dt=f32) if gain_out is not None else None
        s = self.scratch = layer.scratch if isinstance(layer.scratch, BlockScratch) else None
        layer.out = None     # the block ends in moe_norm_out, not in the layer's combine
        if s is not None:
            self.xn, self.dz, self.dx, self.ws, layer.dx = s.xn, s.dz, s.dx, s.ws_norm, s.dxn
        else:
            self.xn, self.dz, self.dx = e(T, d, dt=bf), e(T, d, dt=bf), e(T, d, dt=bf)
            self.ws = B.new_workspace(B.workspace_size(B.MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d), dev)
        self.dgain_in = torch.empty_like(gain_in)
        self.dgain_out = torch.empty_like(gain_out) if gain_out is not None else None
        self.dgate = torch.empty_like(gate) if gate is not None else None
        self.x = self.dout = None
        self._mark = object()

    def norm(self, x: torch.Tensor) -> torch.Tensor:
        """xn, the router's input. x is read again by the passes that follow, backward_norm
        included: leave it unchanged until then."""
        self.x = x
        B.moe_norm_in(x, self.gain_in, self.eps, out=(self.xn, self.rstd_in))
        if self.scratch is not None:
            self.scratch.xn_of = self._mark
        return self.xn

    def forward(self, logits: torch.Tensor, copy_splits: bool = False) -> torch.Tensor:
        if self.scratch is not None and self.scratch.xn_of is not self._mark:
            raise RuntimeError("the shared scratch holds another block's xn: with a BlockScratch "
                               "norm and forward run block by block")
        y, topk_w, inv_perm, shared_y = self.layer.experts(logits, self.xn, copy_splits)
        B.moe_norm_out(y, self.x, self.gain_out, topk_w, inv_perm, shared_y, self.gate, self.span,
                       self.scale, self.eps, out=(self.out, self.z, self.rstd_out))
        return self.out

    def backward(self, dout: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """(dxn, dlogits): the gradients at the experts' input and at the logits. The caller
        adds to dxn what the router's product sends back to xn. dout is read again by
        backward_norm (it is the residual's gradient): leave it unchanged until then."""
        self.dout = dout
        B.moe_norm_out_backward(dout, self.z, self.rstd_out, self.gain_out, self.gate, self.span,
                                self.scale, ws=self.ws, out=(self.dz, self.dgain_out, self.dgate))
        dxn = self.layer.backward(self.dz)
        if self.scratch is not None and self.scratch.xn_of is not self._mark:
            self.norm(self.x)     # for the gradient of the router's product
        return dxn, self.layer.dlogits

    def backward_norm(self, dxn: torch.Tensor) -> torch.Tensor:
        """dx, the residual's share (backward's dout) included."""
        B.moe_norm_in_backward(dxn, self.x, self.gain_in, self.rstd_in, self.dout, ws=self.ws,
                               out=(self.dx, self.dgain_in))
        return self.dx


def w4_weights(weights: Dict[str, torch.Tensor], group: int = 128):
    """A layer's bf16 weights (w_gate, w_up [E,d,I], w_down [E,I,d], and the shared experts'
    ws_* when present) quantized to 4 bits and laid out: {"wgu", "wd"[, "sgu", "sd"]}."""
    def pack(gate, up, down):
        plain = [B.moe_w4_quantize_weights(w.contiguous(), group) for w in (gate, up, down)]
        return (B.moe_w4_pack_weights(*plain[0], *plain[1]), B.moe_w4_pack_weights(*plain[2]))

    out = dict(zip(("wgu", "wd"), pack(weights["w_gate"], weights["w_up"], weights["w_down"])))
    if "ws_gate" in weights:
        shared = [weights[k].unsqueeze(0) for k in ("ws_gate", "ws_up", "ws_down")]
        out.update(zip(("sgu", "sd"), pack(*shared)))
    return out


class MoEDecodeBlock:
    """The block's forward for T tokens on 4-bit experts (``w4`` from ``w4_weights``). Saves
    nothing for a backward pass."""

    def __init__(self, T: int, K: int, w4, gain_in: torch.Tensor,
                 gain_out: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 span: Optional[int] = None, scale: float = 1.0, eps: float = 1e-6,
                 renorm: int = 1):
        self.w4, self.K, self.renorm = w4, K, renorm
        self.gain_in, self.gain_out, self.gate, self.span = gain_in, gain_out, gate, span
        self.scale, self.eps = float(scale), float(eps)
        dev = gain_in.device
        E, d = w4["wgu"][0].shape[0], gain_in.numel()
        I = 16 * w4["wgu"][0].shape[1]
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        TK, n = T * K, E + 1
        self.xn, self.rstd = e(T, d, dt=bf), e(T, dt=f32)
        self.topk_idx, self.topk_w = e(T, K, dt=i32), e(T, K, dt=f32)
        self.counts, self.offsets = e(E, dt=i32), e(E + 1, dt=i32)
        self.perm, self.inv_perm = e(TK, dt=i32), e(TK, dt=i32)
        self.splits, self.send, self.a2a, self.regroup = (e(n, dt=i32), e(TK, dt=i32),
                                                          e(TK, dt=i32), e(TK, dt=i32))
        self.y, self.h, self.out = e(TK, d, dt=bf), e(TK, I, dt=bf), e(T, d, dt=bf)
        self.ws_route = B.new_workspace(B.workspace_size(B.MOE_OP_ROUTE_PERMUTE_EP, T, E, K, 1), dev)
        self.ws_ffn = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_FFN_W4, T, E, K, 1, d, I), dev)
        self.shared = "sgu" in w4
        if self.shared:
            Is = 16 * w4["sgu"][0].shape[1]
            self.s_offsets = torch.tensor([0, T], dtype=i32, device=dev)
            self.ys, self.hs = e(T, d, dt=bf), e(T, Is, dt=bf)
        self.x = None

    def norm(self, x: torch.Tensor) -> torch.Tensor:
        self.x = x
        B.moe_norm_in(x, self.gain_in, self.eps, out=(self.xn, self.rstd))
        return self.xn

    def forward(self, logits: torch.Tensor) -> torch.Tensor:
        B.moe_route_permute_ep(logits, self.K, 1, self.renorm, host_splits=False, ws=self.ws_route,
                               out=(self.topk_idx, self.topk_w, self.counts, self.offsets,
                                    self.perm, self.inv_perm, self.splits, self.send, self.a2a,
                                    self.regroup))
        B.moe_grouped_ffn_w4(self.xn, self.offsets, self.w4["wgu"], self.w4["wd"], perm=self.perm,
                             K=self.K, ws=self.ws_ffn, out=(self.y, self.h))
        shared_y = None
        if self.shared:
            B.moe_grouped_ffn_w4(self.xn, self.s_offsets, self.w4["sgu"], self.w4["sd"],
                                 ws=self.ws_ffn, out=(self.ys, self.hs))
            shared_y = self.ys
        B.moe_norm_out(self.y, self.x, self.gain_out, self.topk_w, self.inv_perm, shared_y,
                       self.gate, self.span, self.scale, self.eps, out=(self.out, None, None))
        return self.out


def fp4_weights(weights: Dict[str, torch.Tensor], block: int = 16):
    """A layer's bf16 weights (as w4_weights takes them) as microscaled 4-bit floats in the form
    moe_grouped_ffn_fp4 takes: {"wgu", "wd"[, "sgu", "sd"]}."""
    def pack(gate, up, down):
        (gq, gs, g), (uq, us, u), (dq, ds, d) = (B.moe_fp4_quantize_weights(w.contiguous(), block)
                                                 for w in (gate, up, down))
        return ((gq, uq, B.moe_fp4_pack_scales(gs, us, block), g, u),
                (dq, B.moe_fp4_pack_scales(ds, block=block), d))

    out = dict(zip(("wgu", "wd"), pack(weights["w_gate"], weights["w_up"], weights["w_down"])))
    if "ws_gate" in weights:
        shared = [weights[k].unsqueeze(0) for k in ("ws_gate", "ws_up", "ws_down")]
        out.update(zip(("sgu", "sd"), pack(*shared)))
    return out


def fp4_h_scale(h: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """h_scale [E] fp32 for moe_grouped_ffn_fp4 from a calibration pass's hidden rows h [M,I] (as
    moe_grouped_ffn leaves them) and offsets: each expert's largest finite |H| / 2688, at least
    2^-100; experts without a row (or whose rows are all zero) take the largest of all."""
    E = offsets.numel() - 1
    rows = torch.arange(h.shape[0], device=h.device)
    e = torch.searchsorted(offsets[1:].long(), rows, right=True)
    size = torch.nan_to_num(h.float(), 0.0, 0.0, 0.0).abs().amax(1)
    top = torch.zeros(E + 1, device=h.device).scatter_reduce_(0, e, size, "amax")[:E]
    return torch.where(top > 0, top, top.amax()).clamp(min=2688 * 2.0 ** -100) / 2688.0


class MoEFp4Block:
    """The block's forward for T tokens on experts in microscaled 4-bit floats (``w4`` from
    ``fp4_weights``): the norm's rows are quantized while they are dispatched and both products
    take 4-bit operands. ``h_scale`` [E] and ``sh_scale`` [1] (shared experts; ``fp4_h_scale``)
    fix the hidden rows' scales, which saves a pass; without them, with block 16, each hidden row
    takes its own. Saves nothing for a backward pass."""

    def __init__(self, T: int, K: int, w4, gain_in: torch.Tensor,
                 gain_out: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 span: Optional[int] = None, scale: float = 1.0, eps: float = 1e-6,
                 renorm: int = 1, block: int = 16, h_scale: Optional[torch.Tensor] = None,
                 sh_scale: Optional[torch.Tensor] = None):
        self.w4, self.K, self.renorm, self.block = w4, K, renorm, block
        self.gain_in, self.gain_out, self.gate, self.span = gain_in, gain_out, gate, span
        self.scale, self.eps = float(scale), float(eps)
        self.h_scale, self.sh_scale = h_scale, sh_scale
        dev = gain_in.device
        d = gain_in.numel()
        E, I, _ = w4["wgu"][0].shape
        bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        TK, n = T * K, E + 1
        self.xn, self.rstd = e(T, d, dt=bf), e(T, dt=f32)
        self.topk_idx, self.topk_w = e(T, K, dt=i32), e(T, K, dt=f32)
        self.counts, self.offsets = e(E, dt=i32), e(E + 1, dt=i32)
        self.perm, self.inv_perm = e(TK, dt=i32), e(TK, dt=i32)
        self.splits, self.send, self.a2a, self.regroup = (e(n, dt=i32), e(TK, dt=i32),
                                                          e(TK, dt=i32), e(TK, dt=i32))

        def rows(M, E):
            shapes = B._fp4_rows_shapes(M, d, E, block)
            return (e(*shapes[0], dt=u8), e(*shapes[1], dt=u8),
                    e(*shapes[2], dt=f32) if block == 16 else None)
        self.rows = rows(TK, E)
        self.y, self.out = e(TK, d, dt=bf), e(T, d, dt=bf)
        self.ws_route = B.new_workspace(B.workspace_size(B.MOE_OP_ROUTE_PERMUTE_EP, T, E, K, 1), dev)
        self.ws_ffn = B.new_workspace(
            B.workspace_size(B.fp4_ffn_op(block, h_scale), TK, E, 1, 1, d, I), dev)
        self.shared = "sgu" in w4
        if self.shared:
            Is = w4["sgu"][0].shape[1]
            self.s_offsets = torch.tensor([0, T], dtype=i32, device=dev)
            self.s_rows, self.ys = rows(T, 1), e(T, d, dt=bf)
            self.ws_sffn = B.new_workspace(
                B.workspace_size(B.fp4_ffn_op(block, sh_scale), T, 1, 1, 1, d, Is), dev)
        self.x = None

    def norm(self, x: torch.Tensor) -> torch.Tensor:
        self.x = x
        B.moe_norm_in(x, self.gain_in, self.eps, out=(self.xn, self.rstd))
        return self.xn

    def forward(self, logits: torch.Tensor) -> torch.Tensor:
        B.moe_route_permute_ep(logits, self.K, 1, self.renorm, host_splits=False, ws=self.ws_route,
                               out=(self.topk_idx, self.topk_w, self.counts, self.offsets,
                                    self.perm, self.inv_perm, self.splits, self.send, self.a2a,
                                    self.regroup))
        B.moe_fp4_quantize_rows(self.xn, self.offsets, self.block, self.inv_perm, self.K,
                                out=self.rows)
        B.moe_grouped_ffn_fp4(self.rows, self.offsets, self.w4["wgu"], self.w4["wd"], self.block,
                              self.h_scale, ws=self.ws_ffn, out=self.y)
        shared_y = None
        if self.shared:
            B.moe_fp4_quantize_rows(self.xn, self.s_offsets, self.block, out=self.s_rows)
            B.moe_grouped_ffn_fp4(self.s_rows, self.s_offsets, self.w4["sgu"], self.w4["sd"],
                                  self.block, self.sh_scale, ws=self.ws_sffn, out=self.ys)
            shared_y = self.ys
        B.moe_norm_out(self.y, self.x, self.gain_out, self.topk_w, self.inv_perm, shared_y,
                       self.gate, self.span, self.scale, self.eps, out=(self.out, None, None))
        return self.out
