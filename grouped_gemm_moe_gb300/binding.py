"""Thin Python binding of libmoe_gb300.so (ctypes).

Every function here has the name of the C entry point it calls and only
marshals arguments: it checks dtypes, shapes and devices, allocates outputs
with ``torch.empty`` on the input's device, and passes raw pointers plus the
current CUDA stream. All arithmetic runs in the library's CUDA kernels; there
is no fallback of any kind. If the shared library has not been built, or the
tensors are not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

# moe_status codes (include/moe_gb300.h)
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_MISALIGNED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_UNSUPPORTED = 4
MOE_ERR_CUDA = 5
MOE_ERR_DEVICE_TIMEOUT = 6
MOE_ERR_DEVICE_CHECK = 7

MOE_OP_BUILD_PERMUTATION = 1
MOE_OP_EP_LAYOUT = 2
MOE_OP_GROUPED_FFN = 3
MOE_OP_GROUPED_FFN_BACKWARD = 4
MOE_OP_LOAD_BALANCE = 5
MOE_OP_EP_RECV_LAYOUT = 6
MOE_OP_GROUPED_FFN_FP8 = 7
MOE_OP_ROUTE_PERMUTE_EP = 8
MOE_OP_NORM_BACKWARD = 9
MOE_OP_GROUPED_FFN_W4 = 10
MOE_OP_GROUPED_FFN_FP4 = 11
MOE_OP_GROUPED_GEMM_WGRAD = 12
MOE_OP_GROUPED_FFN_FP4_FUSED = 13

WORKSPACE_HEADER = 256

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t

# exported symbol -> (restype, argtypes); the single source for the loader and the tests
SIGNATURES = {
    "moe_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_route_topk": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "moe_route_topk_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_load_balance": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_load_balance_backward": (_I, [_P, _P, _I, _I, ctypes.c_float, _I, _P, _P]),
    "moe_build_permutation": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_build_permutation_static": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_ep_layout": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_build_permutation_ep": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _SZ, _P]),
    "moe_route_permute_ep": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                  _P, _P, _SZ, _P]),
    "moe_dispatch": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_dispatch_scatter": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_grouped_ffn": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                                      _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_backward_data": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P,
                                           _P, _SZ, _P]),
    "moe_grouped_ffn_backward_weights": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P,
                                              _SZ, _P]),
    "moe_combine": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_combine_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_dispatch_backward": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_ep_recv_layout": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_dispatch_slice": (_I, [_P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_combine_slice": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "moe_combine_backward_slice": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "moe_dispatch_backward_slice": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "moe_reduce_finish": (_I, [_P, _P, _I, _I, _P, _P]),
    "moe_mxfp8_quantize_rows": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_mxfp8_quantize_weights": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_grouped_ffn_fp8": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_norm_in": (_I, [_P, _P, _I, _I, _F, _P, _P, _P]),
    "moe_norm_in_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_norm_out": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _F, _F, _I, _I, _P, _P, _P, _P]),
    "moe_norm_out_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _F, _I, _I, _P, _P, _P, _P, _SZ,
                                   _P]),
    "moe_ckpt8_pack": (_I, [_P, _I, _I, _P, _P, _P]),
    "moe_ckpt8_dispatch": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_ckpt8_swiglu": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "moe_ckpt8_combine_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_w4_quantize_weights": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "moe_w4_pack_weights": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P]),
    "moe_grouped_ffn_w4": (_I, [_P, _P, _I, _I, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                                _P, _SZ, _P]),
    "moe_grouped_gemm": (_I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _SZ, _P]),
    "moe_grouped_gemm_wgrad": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_fp4_quantize_rows": (_I, [_P, _P, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P]),
    "moe_fp4_dequantize_rows": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_fp4_quantize_weights": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_fp4_pack_scales": (_I, [_P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_grouped_gemm_fp4": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_fp4": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _P, _P, _SZ, _P]),
    "moe_debug_check_status": (_I, [ctypes.POINTER(ctypes.c_int)]),
    "moe_read_device_status": (_I, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
    "moe_debug_wait_timeout": (_I, [_P, _I, _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_cuda_error": (_I, []),
    "moe_version": (_I, []),
    "moe_profile_start": (_I, [_I]),
    "moe_profile_stop": (_I, []),
    "moe_profile_record": (_I, [_I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)]),
}

_lib = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} failed: status {status}"
        if _lib is not None:
            msg += f" ({_lib.moe_status_string(status).decode()})"
            if status == MOE_ERR_CUDA:
                msg += f", cudaError {_lib.moe_last_cuda_error()}"
        super().__init__(msg)


def load(path: str = LIB_PATH):
    """Loads the shared library (once) and declares every exported signature."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with grouped_gemm_moe_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()   # the signatures convert integers


def _stream(dev: torch.device):
    # the current stream's handle without building a Stream object around it
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _check(name: str, rc: int):
    if rc != MOE_OK:
        raise MoEError(name, rc)


def _need(t: torch.Tensor, dtype, ndim: int, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    # ctypes would cut a larger size to its low 32 bits; the cheap test comes first
    if t.numel() > 0x7fffffff and max(t.shape) > 0x7fffffff:
        raise ValueError(f"{name}: sizes are 31 bits at most, got {tuple(t.shape)}")


def workspace_size(op: int, T: int, E: int, K: int, R: int = 1, d: int = 0, I: int = 0) -> int:
    return int(load().moe_workspace_size(op, T, E, K, R, d, I))


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace with its status header zeroed (the rest is scratch)."""
    ws = torch.empty(max(int(nbytes), WORKSPACE_HEADER), dtype=torch.uint8, device=device)
    ws[:WORKSPACE_HEADER].zero_()
    return ws


def moe_workspace_size(op: int, T: int, E: int, K: int, R: int = 1, d: int = 0, I: int = 0) -> int:
    return workspace_size(op, T, E, K, R, d, I)


def moe_route_topk(logits: torch.Tensor, K: int, renorm: int = 1,
                   out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    _need(logits, torch.float32, 2, "logits")
    T, E = logits.shape
    if out is None:
        idx = torch.empty(T, K, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, K, dtype=torch.float32, device=logits.device)
    else:
        idx, w = out
    _check("moe_route_topk", load().moe_route_topk(_ptr(logits), T, E, K, int(renorm), _ptr(idx),
                                                   _ptr(w), _stream(logits.device)))
    return idx, w


def moe_route_topk_backward(logits: Optional[torch.Tensor], topk_idx: torch.Tensor,
                            topk_w: torch.Tensor, dtopk_w: torch.Tensor, E: int, renorm: int = 1,
                            out: Optional[torch.Tensor] = None):
    _need(topk_idx, torch.int32, 2, "topk_idx")
    _need(topk_w, torch.float32, 2, "topk_w")
    _need(dtopk_w, torch.float32, 2, "dtopk_w")
    if logits is not None:
        _need(logits, torch.float32, 2, "logits")
    T, K = topk_idx.shape
    dl = out if out is not None else torch.empty(T, E, dtype=torch.float32, device=topk_idx.device)
    _check("moe_route_topk_backward", load().moe_route_topk_backward(
        _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(dtopk_w), T, E, K, int(renorm), _ptr(dl),
        _stream(topk_idx.device)))
    return dl


def moe_load_balance(logits: torch.Tensor, counts: torch.Tensor, K: int,
                     ws: Optional[torch.Tensor] = None, out=None):
    """Load-balance metrics and loss: returns (load_frac [E], prob_mean [E], stats [4]) with
    stats = (loss, E * max load_frac, empty experts, sum load_frac), all fp32 on device."""
    _need(logits, torch.float32, 2, "logits")
    _need(counts, torch.int32, 1, "counts")
    T, E = logits.shape
    dev = logits.device
    if ws is None:
        ws = new_workspace(workspace_size(MOE_OP_LOAD_BALANCE, T, E, K), dev)
    if out is None:
        out = (torch.empty(E, dtype=torch.float32, device=dev),
               torch.empty(E, dtype=torch.float32, device=dev),
               torch.empty(4, dtype=torch.float32, device=dev))
    frac, pmean, stats = out
    _check("moe_load_balance", load().moe_load_balance(
        _ptr(logits), _ptr(counts), T, E, int(K), _ptr(frac), _ptr(pmean), _ptr(stats), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return frac, pmean, stats


def moe_load_balance_backward(logits: torch.Tensor, load_frac: torch.Tensor, scale: float,
                              dlogits: Optional[torch.Tensor] = None, accumulate: bool = True):
    """scale * d(load-balance loss)/d(logits), added into dlogits (or written if accumulate is
    False or dlogits is None)."""
    _need(logits, torch.float32, 2, "logits")
    _need(load_frac, torch.float32, 1, "load_frac")
    T, E = logits.shape
    if dlogits is None:
        dlogits = torch.empty(T, E, dtype=torch.float32, device=logits.device)
        accumulate = False
    _check("moe_load_balance_backward", load().moe_load_balance_backward(
        _ptr(logits), _ptr(load_frac), T, E, float(scale), 1 if accumulate else 0, _ptr(dlogits),
        _stream(logits.device)))
    return dlogits


def moe_build_permutation(topk_idx: torch.Tensor, E: int, ws: Optional[torch.Tensor] = None,
                          out=None):
    _need(topk_idx, torch.int32, 2, "topk_idx")
    T, K = topk_idx.shape
    dev = topk_idx.device
    nbytes = workspace_size(MOE_OP_BUILD_PERMUTATION, T, E, K)
    if ws is None:
        ws = new_workspace(nbytes, dev)
    if out is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * K, dtype=torch.int32, device=dev)
        inv = torch.empty(T * K, dtype=torch.int32, device=dev)
    else:
        counts, offsets, perm, inv = out
    _check("moe_build_permutation", load().moe_build_permutation(
        _ptr(topk_idx), T, E, K, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(ws),
        ws.numel(), _stream(dev)))
    return counts, offsets, perm, inv


def moe_build_permutation_static(topk_idx: torch.Tensor, E: int, out=None):
    """moe_build_permutation without a workspace: the library's fixed device
    scratch holds the chunk histogram (for callers that cannot allocate)."""
    _need(topk_idx, torch.int32, 2, "topk_idx")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if out is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * K, dtype=torch.int32, device=dev)
        inv = torch.empty(T * K, dtype=torch.int32, device=dev)
    else:
        counts, offsets, perm, inv = out
    _check("moe_build_permutation_static", load().moe_build_permutation_static(
        _ptr(topk_idx), T, E, K, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _stream(dev)))
    return counts, offsets, perm, inv


def moe_ep_layout(topk_idx: torch.Tensor, E: int, R: int, host_splits: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, out=None):
    """Returns (ep_splits [R*E+R*R], send_index, a2a_index, regroup_index, host_splits).
    ``host_splits`` (pinned CPU int32 [R*E+R*R]) receives the one device-to-host copy;
    pass ``False`` to skip the copy."""
    _need(topk_idx, torch.int32, 2, "topk_idx")
    T, K = topk_idx.shape
    dev = topk_idx.device
    n = R * E + R * R
    if host_splits is None:
        host_splits = torch.empty(n, dtype=torch.int32, pin_memory=True)
    elif host_splits is False:
        host_splits = None
    if host_splits is not None:
        if host_splits.is_cuda or host_splits.dtype != torch.int32 or host_splits.numel() < n:
            raise ValueError("host_splits must be a pinned CPU int32 tensor of R*E+R*R elements")
    nbytes = workspace_size(MOE_OP_EP_LAYOUT, T, E, K, R)
    if nbytes == 0:
        raise ValueError("R must divide E and T")
    if ws is None:
        ws = new_workspace(nbytes, dev)
    if out is None:
        splits = torch.empty(n, dtype=torch.int32, device=dev)
        send = torch.empty(T * K, dtype=torch.int32, device=dev)
        a2a = torch.empty(T * K, dtype=torch.int32, device=dev)
        reg = torch.empty(T * K, dtype=torch.int32, device=dev)
    else:
        splits, send, a2a, reg = out
    _check("moe_ep_layout", load().moe_ep_layout(
        _ptr(topk_idx), T, E, K, R, _ptr(splits), _ptr(send), _ptr(a2a), _ptr(reg),
        _ptr(host_splits), _ptr(ws), ws.numel(), _stream(dev)))
    return splits, send, a2a, reg, host_splits


def moe_build_permutation_ep(topk_idx: torch.Tensor, E: int, R: int,
                             host_splits: Optional[torch.Tensor] = None,
                             ws: Optional[torch.Tensor] = None, out=None):
    """Both moe_build_permutation and moe_ep_layout from one pass. Returns
    (counts, offsets, perm, inv_perm, ep_splits, send_index, a2a_index, regroup_index,
    host_splits); ``host_splits=False`` skips the device-to-host copy."""
    _need(topk_idx, torch.int32, 2, "topk_idx")
    T, K = topk_idx.shape
    dev = topk_idx.device
    n = R * E + R * R
    if host_splits is None:
        host_splits = torch.empty(n, dtype=torch.int32, pin_memory=True)
    elif host_splits is False:
        host_splits = None
    nbytes = workspace_size(MOE_OP_EP_LAYOUT, T, E, K, R)
    if nbytes == 0:
        raise ValueError("R must divide E and T")
    if ws is None:
        ws = new_workspace(nbytes, dev)
    if out is None:
        e = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        out = (e(E), e(E + 1), e(T * K), e(T * K), e(n), e(T * K), e(T * K), e(T * K))
    counts, offsets, perm, inv, splits, send, a2a, reg = out
    _check("moe_build_permutation_ep", load().moe_build_permutation_ep(
        _ptr(topk_idx), T, E, K, R, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
        _ptr(splits), _ptr(send), _ptr(a2a), _ptr(reg), _ptr(host_splits), _ptr(ws), ws.numel(),
        _stream(dev)))
    return counts, offsets, perm, inv, splits, send, a2a, reg, host_splits


def moe_route_permute_ep(logits: torch.Tensor, K: int, R: int, renorm: int = 1,
                         host_splits: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, out=None):
    """moe_route_topk and moe_build_permutation_ep in one launch. Returns
    (topk_idx, topk_w, counts, offsets, perm, inv_perm, ep_splits, send_index,
    a2a_index, regroup_index, host_splits); ``host_splits=False`` skips the
    device-to-host copy."""
    _need(logits, torch.float32, 2, "logits")
    T, E = logits.shape
    dev = logits.device
    n = R * E + R * R
    if host_splits is None:
        host_splits = torch.empty(n, dtype=torch.int32, pin_memory=True)
    elif host_splits is False:
        host_splits = None
    nbytes = workspace_size(MOE_OP_ROUTE_PERMUTE_EP, T, E, K, R)
    if nbytes == 0:
        raise ValueError("R must divide E and T")
    if ws is None:
        ws = new_workspace(nbytes, dev)
    if out is None:
        e = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        out = (e(T, K), torch.empty(T, K, dtype=torch.float32, device=dev), e(E), e(E + 1),
               e(T * K), e(T * K), e(n), e(T * K), e(T * K), e(T * K))
    idx, w, counts, offsets, perm, inv, splits, send, a2a, reg = out
    _check("moe_route_permute_ep", load().moe_route_permute_ep(
        _ptr(logits), T, E, K, int(renorm), R, _ptr(idx), _ptr(w), _ptr(counts), _ptr(offsets),
        _ptr(perm), _ptr(inv), _ptr(splits), _ptr(send), _ptr(a2a), _ptr(reg), _ptr(host_splits),
        _ptr(ws), ws.numel(), _stream(dev)))
    return idx, w, counts, offsets, perm, inv, splits, send, a2a, reg, host_splits


def moe_dispatch(x: torch.Tensor, perm: torch.Tensor, K: int, out: Optional[torch.Tensor] = None):
    _need(x, torch.bfloat16, 2, "x")
    _need(perm, torch.int32, 1, "perm")
    T, d = x.shape
    xp = out if out is not None else torch.empty(T * K, d, dtype=torch.bfloat16, device=x.device)
    _check("moe_dispatch", load().moe_dispatch(_ptr(x), T, d, K, _ptr(perm), _ptr(xp),
                                               _stream(x.device)))
    return xp


def moe_dispatch_scatter(x: torch.Tensor, inv_perm: torch.Tensor, K: int,
                         out: Optional[torch.Tensor] = None):
    """The same xp as moe_dispatch, token-major through inv_perm."""
    _need(x, torch.bfloat16, 2, "x")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    T, d = x.shape
    xp = out if out is not None else torch.empty(T * K, d, dtype=torch.bfloat16, device=x.device)
    _check("moe_dispatch_scatter", load().moe_dispatch_scatter(_ptr(x), T, d, K, _ptr(inv_perm),
                                                               _ptr(xp), _stream(x.device)))
    return xp


def moe_grouped_ffn(xp: torch.Tensor, offsets: torch.Tensor, w_gate: torch.Tensor,
                    w_up: torch.Tensor, w_down: torch.Tensor, save_gu: bool = True,
                    ws: Optional[torch.Tensor] = None, out=None):
    """Returns (y [M,d], h [M,I], gu [M,2I] or None)."""
    _need(xp, torch.bfloat16, 2, "xp")
    _need(offsets, torch.int32, 1, "offsets")
    for n, t in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(t, torch.bfloat16, 3, n)
    M, d = xp.shape
    E, _, I = w_gate.shape
    dev = xp.device
    if ws is None:
        ws = new_workspace(workspace_size(MOE_OP_GROUPED_FFN, M, E, 1, 1, d, I), dev)
    if out is None:
        y = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
        h = torch.empty(M, I, dtype=torch.bfloat16, device=dev)
        gu = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=dev) if save_gu else None
    else:
        y, h, gu = out
    _check("moe_grouped_ffn", load().moe_grouped_ffn(
        _ptr(xp), _ptr(offsets), E, M, d, I, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y),
        _ptr(h), _ptr(gu), _ptr(ws), ws.numel(), _stream(dev)))
    return y, h, gu


def moe_grouped_ffn_backward(dy, xp, gu, h, offsets, w_gate, w_up, w_down,
                             ws: Optional[torch.Tensor] = None, out=None):
    """Returns (dxp [M,d] bf16, dw_gate, dw_up [E,d,I] fp32, dw_down [E,I,d] fp32)."""
    for n, t in (("dy", dy), ("xp", xp), ("gu", gu), ("h", h)):
        _need(t, torch.bfloat16, 2, n)
    _need(offsets, torch.int32, 1, "offsets")
    M, d = xp.shape
    E, _, I = w_gate.shape
    dev = xp.device
    if ws is None:
        ws = new_workspace(workspace_size(MOE_OP_GROUPED_FFN_BACKWARD, M, E, 1, 1, d, I), dev)
    if out is None:
        dxp = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
        dwg = torch.empty(E, d, I, dtype=torch.float32, device=dev)
        dwu = torch.empty(E, d, I, dtype=torch.float32, device=dev)
        dwd = torch.empty(E, I, d, dtype=torch.float32, device=dev)
    else:
        dxp, dwg, dwu, dwd = out
    _check("moe_grouped_ffn_backward", load().moe_grouped_ffn_backward(
        _ptr(dy), _ptr(xp), _ptr(gu), _ptr(h), _ptr(offsets), E, M, d, I, _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), _ptr(dxp), _ptr(dwg), _ptr(dwu), _ptr(dwd), _ptr(ws), ws.numel(),
        _stream(dev)))
    return dxp, dwg, dwu, dwd


def moe_grouped_ffn_backward_data(dy, xp, gu, h, offsets, w_gate, w_up, w_down,
                                  ws: torch.Tensor, out: Optional[torch.Tensor] = None):
    """The data part of moe_grouped_ffn_backward: returns dxp [M,d] bf16 and leaves
    [dG | dU] and the padded straddling steps in ws for the weight part."""
    for n, t in (("dy", dy), ("xp", xp), ("gu", gu), ("h", h)):
        _need(t, torch.bfloat16, 2, n)
    _need(offsets, torch.int32, 1, "offsets")
    M, d = xp.shape
    E, _, I = w_gate.shape
    dxp = out if out is not None else torch.empty(M, d, dtype=torch.bfloat16, device=xp.device)
    _check("moe_grouped_ffn_backward_data", load().moe_grouped_ffn_backward_data(
        _ptr(dy), _ptr(xp), _ptr(gu), _ptr(h), _ptr(offsets), E, M, d, I, _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), _ptr(dxp), _ptr(ws), ws.numel(), _stream(xp.device)))
    return dxp


def moe_grouped_ffn_backward_weights(dy, xp, h, offsets, E: int, I: int, ws: torch.Tensor,
                                     out=None):
    """The weight part of moe_grouped_ffn_backward, after the data part on the same
    stream with the same ws: returns (dw_gate, dw_up [E,d,I], dw_down [E,I,d]) fp32."""
    for n, t in (("dy", dy), ("xp", xp), ("h", h)):
        _need(t, torch.bfloat16, 2, n)
    _need(offsets, torch.int32, 1, "offsets")
    M, d = xp.shape
    dev = xp.device
    if out is None:
        out = (torch.empty(E, d, I, dtype=torch.float32, device=dev),
               torch.empty(E, d, I, dtype=torch.float32, device=dev),
               torch.empty(E, I, d, dtype=torch.float32, device=dev))
    dwg, dwu, dwd = out
    _check("moe_grouped_ffn_backward_weights", load().moe_grouped_ffn_backward_weights(
        _ptr(dy), _ptr(xp), _ptr(h), _ptr(offsets), E, M, d, I, _ptr(dwg), _ptr(dwu), _ptr(dwd),
        _ptr(ws), ws.numel(), _stream(dev)))
    return dwg, dwu, dwd


def moe_combine(y: torch.Tensor, topk_w: torch.Tensor, inv_perm: torch.Tensor,
                shared_y: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    _need(y, torch.bfloat16, 2, "y")
    _need(topk_w, torch.float32, 2, "topk_w")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    T, K = topk_w.shape
    d = y.shape[1]
    o = out if out is not None else torch.empty(T, d, dtype=torch.bfloat16, device=y.device)
    _check("moe_combine", load().moe_combine(_ptr(y), _ptr(topk_w), _ptr(inv_perm), T, K, d,
                                             _ptr(shared_y), _ptr(o), _stream(y.device)))
    return o


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, topk_w: torch.Tensor,
                         inv_perm: torch.Tensor, out=None):
    _need(dout, torch.bfloat16, 2, "dout")
    _need(y, torch.bfloat16, 2, "y")
    _need(topk_w, torch.float32, 2, "topk_w")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    T, K = topk_w.shape
    d = dout.shape[1]
    if out is None:
        dy = torch.empty(T * K, d, dtype=torch.bfloat16, device=y.device)
        dw = torch.empty(T, K, dtype=torch.float32, device=y.device)
    else:
        dy, dw = out
    _check("moe_combine_backward", load().moe_combine_backward(
        _ptr(dout), _ptr(y), _ptr(topk_w), _ptr(inv_perm), T, K, d, _ptr(dy), _ptr(dw),
        _stream(y.device)))
    return dy, dw


def moe_dispatch_backward(dxp: torch.Tensor, inv_perm: torch.Tensor, T: int, K: int,
                          dx_shared: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None):
    _need(dxp, torch.bfloat16, 2, "dxp")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    d = dxp.shape[1]
    dx = out if out is not None else torch.empty(T, d, dtype=torch.bfloat16, device=dxp.device)
    _check("moe_dispatch_backward", load().moe_dispatch_backward(
        _ptr(dxp), _ptr(inv_perm), T, K, d, _ptr(dx_shared), _ptr(dx), _stream(dxp.device)))
    return dx


# ---------------------------------------------------------------- expert parallelism over ranks
def moe_ep_recv_layout(counts_local: torch.Tensor, recv_counts: torch.Tensor, R: int,
                       capacity: int, host_splits: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, out=None):
    """Receive-side layout of the all-to-all dispatch from this rank's counts
    [E] and the exchanged counts [R*El]. Returns (splits [2R] = send then
    receive rows per peer, local_offsets [El+1], regroup_index [capacity],
    host_splits); ``host_splits`` (pinned CPU int32 [2R]) receives the one
    device-to-host copy (``False`` skips it)."""
    _need(counts_local, torch.int32, 1, "counts_local")
    _need(recv_counts, torch.int32, 1, "recv_counts")
    E = counts_local.numel()
    dev = counts_local.device
    if E % R or recv_counts.numel() != E:
        raise ValueError("R must divide E and recv_counts must hold R * (E / R) counts")
    El = E // R
    if host_splits is None:
        host_splits = torch.empty(2 * R, dtype=torch.int32, pin_memory=True)
    elif host_splits is False:
        host_splits = None
    if ws is None:
        ws = new_workspace(workspace_size(MOE_OP_EP_RECV_LAYOUT, 1, E, 1, R), dev)
    if out is None:
        out = (torch.empty(2 * R, dtype=torch.int32, device=dev),
               torch.empty(El + 1, dtype=torch.int32, device=dev),
               torch.empty(max(int(capacity), 1), dtype=torch.int32, device=dev))
    splits, loff, reg = out
    _check("moe_ep_recv_layout", load().moe_ep_recv_layout(
        _ptr(counts_local), _ptr(recv_counts), E, R, int(capacity), _ptr(splits), _ptr(loff),
        _ptr(reg), _ptr(host_splits), _ptr(ws), ws.numel(), _stream(dev)))
    return splits, loff, reg, host_splits


def moe_dispatch_slice(x: torch.Tensor, inv_perm: torch.Tensor, offsets: torch.Tensor, K: int,
                       e_lo: int, e_hi: int, out: Tuple[torch.Tensor, torch.Tensor]):
    """Local rows of the dispatch for experts [e_lo, e_hi): out = (xs [rows, d] bf16,
    local_offsets [e_hi - e_lo + 1] int32); returns out."""
    _need(x, torch.bfloat16, 2, "x")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    _need(offsets, torch.int32, 1, "offsets")
    T, d = x.shape
    xs, loff = out
    _need(xs, torch.bfloat16, 2, "xs")
    _need(loff, torch.int32, 1, "local_offsets")
    _check("moe_dispatch_slice", load().moe_dispatch_slice(
        _ptr(x), T, d, K, _ptr(inv_perm), _ptr(offsets), offsets.numel() - 1, int(e_lo), int(e_hi),
        _ptr(xs), _ptr(loff), _stream(x.device)))
    return xs, loff


def moe_combine_slice(y_local: torch.Tensor, topk_w: torch.Tensor, inv_perm: torch.Tensor,
                      offsets: torch.Tensor, e_lo: int, e_hi: int,
                      out: Optional[torch.Tensor] = None):
    """fp32 partial combine [T, d] of the local experts' rows."""
    _need(y_local, torch.bfloat16, 2, "y_local")
    _need(topk_w, torch.float32, 2, "topk_w")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    _need(offsets, torch.int32, 1, "offsets")
    T, K = topk_w.shape
    d = y_local.shape[1]
    o = out if out is not None else torch.empty(T, d, dtype=torch.float32, device=y_local.device)
    _check("moe_combine_slice", load().moe_combine_slice(
        _ptr(y_local), _ptr(topk_w), _ptr(inv_perm), _ptr(offsets), offsets.numel() - 1,
        int(e_lo), int(e_hi), T, K, d, _ptr(o), _stream(y_local.device)))
    return o


def moe_combine_backward_slice(dout: torch.Tensor, y_local: torch.Tensor, topk_w: torch.Tensor,
                               inv_perm: torch.Tensor, offsets: torch.Tensor, e_lo: int,
                               e_hi: int, out: Tuple[torch.Tensor, torch.Tensor]):
    """(dy_local [rows, d] bf16, dtopk_w [T, K] fp32, zero on other ranks' slots)."""
    _need(dout, torch.bfloat16, 2, "dout")
    _need(y_local, torch.bfloat16, 2, "y_local")
    _need(topk_w, torch.float32, 2, "topk_w")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    _need(offsets, torch.int32, 1, "offsets")
    T, K = topk_w.shape
    d = dout.shape[1]
    dy, dw = out
    _check("moe_combine_backward_slice", load().moe_combine_backward_slice(
        _ptr(dout), _ptr(y_local), _ptr(topk_w), _ptr(inv_perm), _ptr(offsets),
        offsets.numel() - 1, int(e_lo), int(e_hi), T, K, d, _ptr(dy), _ptr(dw),
        _stream(dout.device)))
    return dy, dw


def moe_dispatch_backward_slice(dxs: torch.Tensor, inv_perm: torch.Tensor, offsets: torch.Tensor,
                                T: int, K: int, e_lo: int, e_hi: int,
                                out: Optional[torch.Tensor] = None):
    """fp32 partial input gradient [T, d] from the local experts' rows."""
    _need(dxs, torch.bfloat16, 2, "dxs")
    _need(inv_perm, torch.int32, 1, "inv_perm")
    _need(offsets, torch.int32, 1, "offsets")
    d = dxs.shape[1]
    o = out if out is not None else torch.empty(T, d, dtype=torch.float32, device=dxs.device)
    _check("moe_dispatch_backward_slice", load().moe_dispatch_backward_slice(
        _ptr(dxs), _ptr(inv_perm), _ptr(offsets), offsets.numel() - 1, int(e_lo), int(e_hi), T, K,
        d, _ptr(o), _stream(dxs.device)))
    return o


def moe_reduce_finish(partial: torch.Tensor, extra: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None):
    """bf16(partial + extra) for fp32 partial [T, d] and bf16 extra [T, d] (or None)."""
    _need(partial, torch.float32, 2, "partial")
    if extra is not None:
        _need(extra, torch.bfloat16, 2, "extra")
    T, d = partial.shape
    o = out if out is not None else torch.empty(T, d, dtype=torch.bfloat16, device=partial.device)
    _check("moe_reduce_finish", load().moe_reduce_finish(_ptr(partial), _ptr(extra), T, d, _ptr(o),
                                                         _stream(partial.device)))
    return o


# ---------------------------------------------------------------- MXFP8 grouped experts
def mxfp8_row_sf_bytes(M: int, E: int, K: int) -> int:
    """Bytes of the scale atoms of M expert-ordered rows of K elements."""
    return ((M + 127) // 128 + 2 * E) * (K // 128) * 512


def moe_mxfp8_quantize_rows(x: torch.Tensor, offsets: torch.Tensor, out=None):
    """(q [M, K] uint8 E4M3, sf uint8 scale atoms) of the expert-ordered rows x."""
    _need(x, torch.bfloat16, 2, "x")
    _need(offsets, torch.int32, 1, "offsets")
    M, K = x.shape
    E = offsets.numel() - 1
    if out is None:
        out = (torch.empty(M, K, dtype=torch.uint8, device=x.device),
               torch.empty(mxfp8_row_sf_bytes(M, E, K), dtype=torch.uint8, device=x.device))
    q, sf = out
    _check("moe_mxfp8_quantize_rows", load().moe_mxfp8_quantize_rows(
        _ptr(x), _ptr(offsets), E, M, K, _ptr(q), _ptr(sf), _stream(x.device)))
    return q, sf


def moe_mxfp8_quantize_weights(w_a: torch.Tensor, w_b: Optional[torch.Tensor] = None, out=None):
    """(q [E, Nq, K] uint8, sf) of weights [E, K, N] (gate/up interleaved when w_b is given)."""
    _need(w_a, torch.bfloat16, 3, "w_a")
    if w_b is not None:
        _need(w_b, torch.bfloat16, 3, "w_b")
        if w_b.shape != w_a.shape:
            raise ValueError("w_a and w_b must have the same shape")
    E, K, N = w_a.shape
    Nq = 2 * N if w_b is not None else N
    if out is None:
        out = (torch.empty(E, Nq, K, dtype=torch.uint8, device=w_a.device),
               torch.empty(E * (Nq // 128) * (K // 128) * 512, dtype=torch.uint8, device=w_a.device))
    q, sf = out
    _check("moe_mxfp8_quantize_weights", load().moe_mxfp8_quantize_weights(
        _ptr(w_a), _ptr(w_b), E, K, N, _ptr(q), _ptr(sf), _stream(w_a.device)))
    return q, sf


def moe_grouped_ffn_fp8(xp: torch.Tensor, offsets: torch.Tensor, wgu, wd, save_gu: bool = True,
                        ws: Optional[torch.Tensor] = None, out=None):
    """MXFP8 forward of the grouped SwiGLU experts. ``wgu`` = (q, sf) of
    moe_mxfp8_quantize_weights(w_gate, w_up), ``wd`` = (q, sf) of
    moe_mxfp8_quantize_weights(w_down). Returns (y [M,d], h [M,I], gu [M,2I] or None)."""
    _need(xp, torch.bfloat16, 2, "xp")
    _need(offsets, torch.int32, 1, "offsets")
    (gq, gsf), (dq, dsf) = wgu, wd
    for n, t in (("wgu_q", gq), ("wd_q", dq)):
        _need(t, torch.uint8, 3, n)
    M, d = xp.shape
    E, two_i, _ = gq.shape
    I = two_i // 2
    dev = xp.device
    if ws is None:
        ws = new_workspace(workspace_size(MOE_OP_GROUPED_FFN_FP8, M, E, 1, 1, d, I), dev)
    if out is None:
        out = (torch.empty(M, d, dtype=torch.bfloat16, device=dev),
               torch.empty(M, I, dtype=torch.bfloat16, device=dev),
               torch.empty(M, 2 * I, dtype=torch.bfloat16, device=dev) if save_gu else None)
    y, h, gu = out
    _check("moe_grouped_ffn_fp8", load().moe_grouped_ffn_fp8(
        _ptr(xp), _ptr(offsets), E, M, d, I, _ptr(gq), _ptr(gsf), _ptr(dq), _ptr(dsf), _ptr(y),
        _ptr(h), _ptr(gu), _ptr(ws), ws.numel(), _stream(dev)))
    return y, h, gu


# ---------------------------------------------------------------- the block's norms
def _shaped(t: Optional[torch.Tensor], dtype, shape, name: str, dev):
    """_need for a tensor (or None) of a known shape on a known device."""
    if t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                     and t.is_contiguous() and t.device == dev):
        return
    _need(t, dtype, len(shape), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _need_ws(ws: Optional[torch.Tensor], nbytes: int, dev) -> torch.Tensor:
    if ws is None:
        return new_workspace(nbytes, dev)
    if not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    return ws


def moe_norm_in(x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6, out=None):
    """RMS norm before the block: (xn [T,d] bf16, rstd [T] fp32)."""
    _need(x, torch.bfloat16, 2, "x")
    T, d = x.shape
    dev = x.device
    _shaped(gain, torch.float32, (d,), "gain", dev)
    if out is None:
        out = (torch.empty_like(x), torch.empty(T, dtype=torch.float32, device=dev))
    else:
        _shaped(out[0], torch.bfloat16, (T, d), "xn", dev)
        _shaped(out[1], torch.float32, (T,), "rstd", dev)
    xn, rstd = out
    _check("moe_norm_in", load().moe_norm_in(_ptr(x), _ptr(gain), T, d, float(eps), _ptr(xn),
                                             _ptr(rstd), _stream(dev)))
    return xn, rstd


def moe_norm_in_backward(dxn: torch.Tensor, x: torch.Tensor, gain: torch.Tensor,
                         rstd: torch.Tensor, dres: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, out=None):
    """Gradient of moe_norm_in plus the residual's dres: (dx [T,d] bf16, dgain [d] fp32)."""
    _need(dxn, torch.bfloat16, 2, "dxn")
    T, d = dxn.shape
    dev = dxn.device
    _shaped(x, torch.bfloat16, (T, d), "x", dev)
    _shaped(gain, torch.float32, (d,), "gain", dev)
    _shaped(rstd, torch.float32, (T,), "rstd", dev)
    _shaped(dres, torch.bfloat16, (T, d), "dres", dev)
    ws = _need_ws(ws, workspace_size(MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d) if ws is None else 0, dev)
    if out is None:
        out = (torch.empty_like(dxn), torch.empty(d, dtype=torch.float32, device=dev))
    else:
        _shaped(out[0], torch.bfloat16, (T, d), "dx", dev)
        _shaped(out[1], torch.float32, (d,), "dgain", dev)
    dx, dgain = out
    _check("moe_norm_in_backward", load().moe_norm_in_backward(
        _ptr(dxn), _ptr(x), _ptr(gain), _ptr(rstd), _ptr(dres), T, d, _ptr(dx), _ptr(dgain),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return dx, dgain


def _gate_args(gate: Optional[torch.Tensor], span: Optional[int], T: int, d: int, dev):
    """(span, columns) of a gate [ceil(T / span), 1 or d]; span None: T for one row, else 1."""
    if gate is None:
        return 1, 1
    _need(gate, torch.float32, 2, "gate")
    rows, cols = gate.shape
    if span is None:
        span = max(T, 1) if rows == 1 else 1
    span = int(span)
    fits = rows == -(-T // span) or (T == 0 and rows == 1)   # an empty batch keeps its one gate
    if span < 1 or cols not in (1, d) or not fits or gate.device != dev:
        raise ValueError(f"gate must be [ceil({T} / span), 1 or {d}] on {dev}, got "
                         f"{tuple(gate.shape)} with span {span}")
    return min(span, max(T, 1)), cols   # past T it means the same, and 32 bits hold this


def moe_norm_out(y: torch.Tensor, resid: torch.Tensor, gain: Optional[torch.Tensor] = None,
                 topk_w: Optional[torch.Tensor] = None, inv_perm: Optional[torch.Tensor] = None,
                 shared_y: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 span: Optional[int] = None, scale: float = 1.0, eps: float = 1e-6,
                 save: bool = True, out=None):
    """resid + scale * gate * norm(combine(y)) in one launch; without a gain the norm is left
    out. y [T*K,d] in expert order with inv_perm and topk_w, or a plain [T,d]. Returns
    (out [T,d] bf16, zsum [T,d] bf16, rstd [T] fp32): zsum (the combined rows) and rstd are
    what moe_norm_out_backward needs, None with save=False; rstd is None without a gain."""
    _need(y, torch.bfloat16, 2, "y")
    _need(resid, torch.bfloat16, 2, "resid")
    T, d = resid.shape
    rows, dy = y.shape
    dev = resid.device
    if dy != d or (rows % T if T else rows) or y.device != dev:
        raise ValueError(f"y must be [T*K, {d}] with T = {T} on {dev}, got {(rows, dy)} on {y.device}")
    if T:
        K = rows // T
    else:   # an empty batch
        K = topk_w.shape[1] if topk_w is not None and topk_w.dim() == 2 else 1
    _shaped(gain, torch.float32, (d,), "gain", dev)
    _shaped(topk_w, torch.float32, (T, K), "topk_w", dev)
    _shaped(inv_perm, torch.int32, (T * K,), "inv_perm", dev)
    _shaped(shared_y, torch.bfloat16, (T, d), "shared_y", dev)
    span, cols = _gate_args(gate, span, T, d, dev)
    if out is None:
        out = (torch.empty_like(resid), torch.empty_like(resid) if save else None,
               torch.empty(T, dtype=torch.float32, device=dev)
               if save and gain is not None else None)
    else:
        _shaped(out[0], torch.bfloat16, (T, d), "out", dev)
        _shaped(out[1], torch.bfloat16, (T, d), "zsum", dev)
        _shaped(out[2], torch.float32, (T,), "rstd", dev)
    o, zsum, rstd = out
    _check("moe_norm_out", load().moe_norm_out(
        _ptr(y), _ptr(topk_w), _ptr(inv_perm), K, _ptr(shared_y), _ptr(resid), _ptr(gain),
        _ptr(gate), span, cols, float(scale), float(eps), T, d, _ptr(o), _ptr(zsum), _ptr(rstd),
        _stream(dev)))
    return o, zsum, rstd


def moe_norm_out_backward(dout: torch.Tensor, zsum: torch.Tensor, rstd: Optional[torch.Tensor],
                          gain: Optional[torch.Tensor] = None,
                          gate: Optional[torch.Tensor] = None, span: Optional[int] = None,
                          scale: float = 1.0, ws: Optional[torch.Tensor] = None, out=None):
    """(dz [T,d] bf16, dgain [d] fp32 or None, dgate like gate or None); rstd is read with a
    gain only."""
    _need(dout, torch.bfloat16, 2, "dout")
    T, d = dout.shape
    dev = dout.device
    _shaped(zsum, torch.bfloat16, (T, d), "zsum", dev)
    _shaped(rstd, torch.float32, (T,), "rstd", dev)
    _shaped(gain, torch.float32, (d,), "gain", dev)
    if gain is not None and rstd is None:
        raise ValueError("rstd is needed with a gain")
    span, cols = _gate_args(gate, span, T, d, dev)
    ws = _need_ws(ws, workspace_size(MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d) if ws is None else 0, dev)
    if out is None:
        out = (torch.empty_like(dout), None if gain is None else torch.empty_like(gain),
               None if gate is None else torch.empty_like(gate))
    else:
        _shaped(out[0], torch.bfloat16, (T, d), "dz", dev)
        _shaped(out[1], torch.float32, (d,), "dgain", dev)
        _shaped(out[2], torch.float32, tuple(gate.shape) if gate is not None else (), "dgate", dev)
    dz, dgain, dgate = out
    if T == 0 and gate is not None and dgate is not None:
        dgate.zero_()   # the C call sees no gate rows then
    _check("moe_norm_out_backward", load().moe_norm_out_backward(
        _ptr(dout), _ptr(zsum), _ptr(rstd), _ptr(gain), _ptr(gate), span, cols, float(scale), T, d,
        _ptr(dz), _ptr(dgain), _ptr(dgate), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(dev)))
    return dz, dgain, dgate


# ---------------------------------------------------------------- 8-bit checkpoints
def _ckpt8_args(q: torch.Tensor, s: torch.Tensor):
    _need(q, torch.int8, 2, "q")
    _shaped(s, torch.bfloat16, (q.shape[0], -(-q.shape[1] // 32)), "s", q.device)
    return q.shape[0], q.shape[1], q.device


def moe_ckpt8_pack(x: torch.Tensor, out=None):
    """8-bit checkpoint of x [M,N] bf16: (q [M,N] int8, s [M, ceil(N/32)] bf16)."""
    _need(x, torch.bfloat16, 2, "x")
    M, N = x.shape
    dev = x.device
    if out is None:
        out = (torch.empty(M, N, dtype=torch.int8, device=dev),
               torch.empty(M, -(-N // 32), dtype=torch.bfloat16, device=dev))
    else:
        _shaped(out[0], torch.int8, (M, N), "q", dev)
        _ckpt8_args(*out)
    q, s = out
    _check("moe_ckpt8_pack", load().moe_ckpt8_pack(_ptr(x), M, N, _ptr(q), _ptr(s), _stream(dev)))
    return q, s


def moe_ckpt8_dispatch(q: torch.Tensor, s: torch.Tensor, inv_perm: Optional[torch.Tensor] = None,
                       K: int = 1, out: Optional[torch.Tensor] = None):
    """The dispatched rows xp [T*K,d] bf16 of a checkpointed x (K = 1 and no inv_perm: x)."""
    T, d, dev = _ckpt8_args(q, s)
    _shaped(inv_perm, torch.int32, (T * K,), "inv_perm", dev)
    if out is None:
        out = torch.empty(T * K, d, dtype=torch.bfloat16, device=dev)
    else:
        _shaped(out, torch.bfloat16, (T * K, d), "xp", dev)
    _check("moe_ckpt8_dispatch", load().moe_ckpt8_dispatch(
        _ptr(q), _ptr(s), _ptr(inv_perm), T, int(K), d, _ptr(out), _stream(dev)))
    return out


def moe_ckpt8_swiglu(q: torch.Tensor, s: torch.Tensor, out=None):
    """(gu [M,2I] bf16, h [M,I] bf16) of a checkpointed [G | U]."""
    M, N, dev = _ckpt8_args(q, s)
    if N % 2:
        raise ValueError("q must hold [G | U]: an even number of columns")
    I = N // 2
    if out is None:
        out = (torch.empty(M, N, dtype=torch.bfloat16, device=dev),
               torch.empty(M, I, dtype=torch.bfloat16, device=dev))
    else:
        _shaped(out[0], torch.bfloat16, (M, N), "gu", dev)
        _shaped(out[1], torch.bfloat16, (M, I), "h", dev)
    gu, h = out
    _check("moe_ckpt8_swiglu", load().moe_ckpt8_swiglu(_ptr(q), _ptr(s), M, I, _ptr(gu), _ptr(h),
                                                       _stream(dev)))
    return gu, h


def moe_ckpt8_combine_backward(dout: torch.Tensor, q: torch.Tensor, s: torch.Tensor,
                               topk_w: torch.Tensor, inv_perm: torch.Tensor, out=None):
    """moe_combine_backward with y as a checkpoint: (dy [TK,d] bf16, dtopk_w [T,K] fp32)."""
    TK, d, dev = _ckpt8_args(q, s)
    _need(topk_w, torch.float32, 2, "topk_w")
    T, K = topk_w.shape
    if T * K != TK or topk_w.device != dev:
        raise ValueError(f"topk_w must hold {TK} weights on {dev}, got {tuple(topk_w.shape)}")
    _shaped(dout, torch.bfloat16, (T, d), "dout", dev)
    _shaped(inv_perm, torch.int32, (TK,), "inv_perm", dev)
    if out is None:
        out = (torch.empty(TK, d, dtype=torch.bfloat16, device=dev),
               torch.empty(T, K, dtype=torch.float32, device=dev))
    else:
        _shaped(out[0], torch.bfloat16, (TK, d), "dy", dev)
        _shaped(out[1], torch.float32, (T, K), "dtopk_w", dev)
    dy, dw = out
    _check("moe_ckpt8_combine_backward", load().moe_ckpt8_combine_backward(
        _ptr(dout), _ptr(q), _ptr(s), _ptr(topk_w), _ptr(inv_perm), T, K, d, _ptr(dy), _ptr(dw),
        _stream(dev)))
    return dy, dw


# ---------------------------------------------------------------- 4-bit experts
def moe_w4_quantize_weights(w: torch.Tensor, group: int = 128, out=None):
    """Plain 4-bit codes [E,N,K/2] uint8 and scales [E,N,K/group] bf16 of w [E,K,N] bf16."""
    _need(w, torch.bfloat16, 3, "w")
    E, K, N = w.shape
    if group not in (32, 64, 128) or K % group or K % 64:
        raise ValueError(f"K = {K} must be a multiple of 64 and of group (32, 64 or 128), "
                         f"got {group}")
    if out is None:
        out = (torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device),
               torch.empty(E, N, K // group, dtype=torch.bfloat16, device=w.device))
    else:
        _shaped(out[0], torch.uint8, (E, N, K // 2), "codes", w.device)
        _shaped(out[1], torch.bfloat16, (E, N, K // group), "scales", w.device)
    codes, scales = out
    _check("moe_w4_quantize_weights", load().moe_w4_quantize_weights(
        _ptr(w), E, K, N, int(group), _ptr(codes), _ptr(scales), _stream(w.device)))
    return codes, scales


def moe_w4_pack_weights(codes_a: torch.Tensor, scales_a: torch.Tensor,
                        codes_b: Optional[torch.Tensor] = None,
                        scales_b: Optional[torch.Tensor] = None, out=None):
    """Plain 4-bit weights laid out for moe_grouped_ffn_w4: (tiles uint8 [E, tiles, K/64, 1024],
    scales bf16 [E, tiles, K/group, 32]); gate (a) and up (b) share tiles."""
    _need(codes_a, torch.uint8, 3, "codes_a")
    _need(scales_a, torch.bfloat16, 3, "scales_a")
    E, N, K = codes_a.shape[0], codes_a.shape[1], 2 * codes_a.shape[2]
    dev = codes_a.device
    ng = scales_a.shape[2]
    if ng < 1 or K % ng or K % 64 or K // ng not in (32, 64, 128):
        raise ValueError(f"K = {K} in {ng} groups: K must be a multiple of 64, groups of 32, 64 "
                         "or 128")
    group = K // ng
    _shaped(scales_a, torch.bfloat16, (E, N, ng), "scales_a", dev)
    if (codes_b is None) != (scales_b is None):
        raise ValueError("codes_b and scales_b go together")
    _shaped(codes_b, torch.uint8, (E, N, K // 2), "codes_b", dev)
    _shaped(scales_b, torch.bfloat16, (E, N, ng), "scales_b", dev)
    per = 32 if codes_b is None else 16
    if N % per:
        raise ValueError(f"N = {N} must be a multiple of {per}")
    if out is None:
        out = (torch.empty(E, N // per, K // 64, 1024, dtype=torch.uint8, device=dev),
               torch.empty(E, N // per, ng, 32, dtype=torch.bfloat16, device=dev))
    else:
        _shaped(out[0], torch.uint8, (E, N // per, K // 64, 1024), "tiles", dev)
        _shaped(out[1], torch.bfloat16, (E, N // per, ng, 32), "scales", dev)
    tiles, scales = out
    _check("moe_w4_pack_weights", load().moe_w4_pack_weights(
        _ptr(codes_a), _ptr(scales_a), _ptr(codes_b), _ptr(scales_b), E, N, K, group, _ptr(tiles),
        _ptr(scales), _stream(dev)))
    return tiles, scales


def _w4_weight(w, E: int, per: int, name: str, dev):
    """(outputs of one matrix, K, group) of laid-out weights with `per` of its outputs a tile."""
    tiles, scales = w
    _need(tiles, torch.uint8, 4, name + " tiles")
    _need(scales, torch.bfloat16, 4, name + " scales")
    e, nt, kt, tile = tiles.shape
    es, ns, ng, rows = scales.shape
    if (e, tile, es, ns, rows) != (E, 1024, E, nt, 32) or ng < 1 or (64 * kt) % ng:
        raise ValueError(f"{name} must come from moe_w4_pack_weights for {E} experts")
    if tiles.device != dev or scales.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    return nt * per, 64 * kt, 64 * kt // ng


def moe_grouped_ffn_w4(x: torch.Tensor, offsets: torch.Tensor, wgu, wd,
                       perm: Optional[torch.Tensor] = None, K: int = 1,
                       ws: Optional[torch.Tensor] = None, out=None):
    """SwiGLU experts on 4-bit weights: (y [M,d] bf16, h [M,I] bf16). ``wgu`` and ``wd`` come
    from moe_w4_pack_weights (gate and up; down). With perm, x [T,d] are the tokens and row p
    is x[perm[p] / K]; without, x [M,d] holds the rows in expert order."""
    _need(x, torch.bfloat16, 2, "x")
    _need(offsets, torch.int32, 1, "offsets")
    T, d = x.shape
    dev = x.device
    E = offsets.numel() - 1
    M = T * int(K) if perm is not None else T
    _shaped(perm, torch.int32, (M,), "perm", dev)
    I, k_gu, group_gu = _w4_weight(wgu, E, 16, "wgu", dev)
    n_d, k_d, group_d = _w4_weight(wd, E, 32, "wd", dev)
    if k_gu != d or n_d != d or k_d != I or offsets.device != dev:
        raise ValueError(f"weights of [{k_gu} -> {I}] and [{k_d} -> {n_d}] do not fit x of {d}")
    ws = _need_ws(ws, workspace_size(MOE_OP_GROUPED_FFN_W4, T, E, K, 1, d, I) if ws is None else 0,
                  dev)
    if out is None:
        out = (torch.empty(M, d, dtype=torch.bfloat16, device=dev),
               torch.empty(M, I, dtype=torch.bfloat16, device=dev))
    else:
        _shaped(out[0], torch.bfloat16, (M, d), "y", dev)
        _shaped(out[1], torch.bfloat16, (M, I), "h", dev)
    y, h = out
    _check("moe_grouped_ffn_w4", load().moe_grouped_ffn_w4(
        _ptr(x), _ptr(perm), T, int(K), _ptr(offsets), E, M, d, I, group_gu, group_d, _ptr(wgu[0]),
        _ptr(wgu[1]), _ptr(wd[0]), _ptr(wd[1]), _ptr(y), _ptr(h), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return y, h


# ---------------------------------------------------------------- products grouped by expert
def _call(name: str, dev: torch.device, *args):
    """The entry point on dev's current stream, with dev the current device."""
    fn = getattr(_lib or load(), name)
    if dev.index == torch._C._cuda_getDevice():
        return _check(name, fn(*args, _stream(dev)))
    with torch.cuda.device(dev):
        _check(name, fn(*args, _stream(dev)))


def _experts_of(offsets: torch.Tensor, dev) -> int:
    _need(offsets, torch.int32, 1, "offsets")
    if offsets.numel() < 2 or offsets.device != dev:
        raise ValueError(f"offsets must hold E + 1 entries on {dev}")
    return offsets.numel() - 1


def moe_grouped_gemm(x: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor, trans: bool = False,
                     ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """y [M,N] bf16: expert e's rows of x [M,K] times w[e], w [E,K,N], or with trans times the
    transpose of w[e], w [E,N,K] (the input gradient of the product without trans)."""
    _need(x, torch.bfloat16, 2, "x")
    _need(w, torch.bfloat16, 3, "w")
    M, K = x.shape
    dev = x.device
    E = _experts_of(offsets, dev)
    e, a, b = w.shape
    N = a if trans else b
    if (e, b if trans else a) != (E, K) or w.device != dev:
        raise ValueError(f"w must have shape {(E, N, K) if trans else (E, K, N)} on {dev}, got "
                         f"{tuple(w.shape)} on {w.device}")
    ws = _need_ws(ws, WORKSPACE_HEADER, dev)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    else:
        _shaped(out, torch.bfloat16, (M, N), "y", dev)
    _call("moe_grouped_gemm", dev, _ptr(x), _ptr(offsets), E, M, K, N, _ptr(w), int(bool(trans)),
          _ptr(out), _ptr(ws), ws.numel() * ws.element_size())
    return out


def moe_grouped_gemm_wgrad(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor,
                           accumulate: bool = False, ws: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None):
    """dw [E,K,N] fp32: x_e^T dy_e of each expert's rows of x [M,K] and dy [M,N]; with accumulate
    added to out, which has to be given."""
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    dev = x.device
    E = _experts_of(offsets, dev)
    _need(dy, torch.bfloat16, 2, "dy")
    rows, N = dy.shape
    if rows != M or dy.device != dev:
        raise ValueError(f"dy must have shape {(M, N)} on {dev}, got {tuple(dy.shape)} on {dy.device}")
    ws = _need_ws(ws, workspace_size(MOE_OP_GROUPED_GEMM_WGRAD, M, E, 1, 1, K, N) if ws is None else 0,
                  dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to out: give it")
        out = torch.empty(E, K, N, dtype=torch.float32, device=dev)
    else:
        _shaped(out, torch.float32, (E, K, N), "dw", dev)
    _call("moe_grouped_gemm_wgrad", dev, _ptr(x), _ptr(dy), _ptr(offsets), E, M, K, N,
          int(bool(accumulate)), _ptr(out), _ptr(ws), ws.numel() * ws.element_size())
    return out


# ---------------------------------------------------------------- microscaled 4-bit floats
def _fp4_block(block: int, K: int, name: str):
    if block not in (16, 32):
        raise ValueError(f"block must be 16 or 32, got {block}")
    if K < 64 or K % 64:
        raise ValueError(f"{name} must be a multiple of 64, got {K}")


def _fp4_atoms(K: int, block: int) -> int:
    return -(-K // (4 * block))


def _fp4_rows_shapes(M: int, d: int, E: int, block: int):
    return (M, d // 2), (-(-M // 128) + 2 * E, _fp4_atoms(d, block), 512), (M,)


def _given(t, dtype, shape, name: str, dev):
    """_shaped for a tensor that has to be there."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == dev.index):
        _shaped(t, dtype, shape, name, dev)


def _fp4_rows(rows, E: int, block: int, dev):
    """(q, sf, row_scale, M, K) of checked rows from moe_fp4_quantize_rows."""
    q, sf, rs = rows
    _need(q, torch.uint8, 2, "q")
    M, half = q.shape
    d = 2 * half
    _fp4_block(block, d, "K")
    _, s_sf, s_rs = _fp4_rows_shapes(M, d, E, block)
    _given(sf, torch.uint8, s_sf, "sf", dev)
    if block == 16:
        _given(rs, torch.float32, s_rs, "row_scale", dev)
    else:
        rs = None
    return q, sf, rs, M, d


def moe_fp4_quantize_rows(x: torch.Tensor, offsets: torch.Tensor, block: int = 16,
                          inv_perm: Optional[torch.Tensor] = None, K: int = 1, out=None):
    """4-bit rows (q [M,d/2] uint8, sf [tiles,KA,512] uint8, row_scale [M] fp32 or None with
    block 32) in expert order: with inv_perm, token t of x [T,d] goes to rows inv_perm[t*K + j]
    (M = T*K); without, x holds the rows in expert order."""
    _need(x, torch.bfloat16, 2, "x")
    T, d = x.shape
    dev = x.device
    _fp4_block(block, d, "d")
    E = _experts_of(offsets, dev)
    K = int(K)
    if inv_perm is None and K != 1:
        raise ValueError("K is the number of copies that inv_perm places: without it 1")
    M = T * K
    _shaped(inv_perm, torch.int32, (M,), "inv_perm", dev)
    s_q, s_sf, s_rs = _fp4_rows_shapes(M, d, E, block)
    if out is None:
        out = (torch.empty(s_q, dtype=torch.uint8, device=dev),
               torch.empty(s_sf, dtype=torch.uint8, device=dev),
               torch.empty(s_rs, dtype=torch.float32, device=dev) if block == 16 else None)
    else:
        _fp4_rows(out, E, block, dev)
        _shaped(out[0], torch.uint8, s_q, "q", dev)
    q, sf, rs = out
    _call("moe_fp4_quantize_rows", dev, _ptr(x), _ptr(inv_perm), T, K, _ptr(offsets), E, d, block,
          _ptr(q), _ptr(sf), _ptr(rs) if block == 16 else None)
    return out


def moe_fp4_dequantize_rows(rows, offsets: torch.Tensor, block: int = 16,
                            out: Optional[torch.Tensor] = None):
    """The rows of moe_fp4_quantize_rows in bf16 [M,d]."""
    dev = rows[0].device
    E = _experts_of(offsets, dev)
    q, sf, rs, M, d = _fp4_rows(rows, E, block, dev)
    if out is None:
        out = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    else:
        _shaped(out, torch.bfloat16, (M, d), "out", dev)
    _call("moe_fp4_dequantize_rows", dev, _ptr(q), _ptr(sf), _ptr(rs), _ptr(offsets), E, M, d, block,
          _ptr(out))
    return out


def moe_fp4_quantize_weights(w: torch.Tensor, block: int = 16, out=None):
    """A plain 4-bit checkpoint of w [E,K,N] bf16: codes [E,N,K/2] and scales [E,N,K/block] uint8,
    scale [E] fp32 (None with block 32)."""
    _need(w, torch.bfloat16, 3, "w")
    E, K, N = w.shape
    dev = w.device
    _fp4_block(block, K, "K")
    if out is None:
        out = (torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev),
               torch.empty(E, N, K // block, dtype=torch.uint8, device=dev),
               torch.empty(E, dtype=torch.float32, device=dev) if block == 16 else None)
    else:
        _shaped(out[0], torch.uint8, (E, N, K // 2), "codes", dev)
        _shaped(out[1], torch.uint8, (E, N, K // block), "scales", dev)
        _shaped(out[2], torch.float32, (E,), "scale", dev)
    codes, scales, scale = out
    _call("moe_fp4_quantize_weights", dev, _ptr(w), E, K, N, block, _ptr(codes), _ptr(scales),
          _ptr(scale))
    return out


def moe_fp4_pack_scales(scales_a: torch.Tensor, scales_b: Optional[torch.Tensor] = None,
                        block: int = 16, out: Optional[torch.Tensor] = None):
    """Block scales [E,N,K/block] uint8 of a plain checkpoint as the products read them: sf
    [E,tiles,KA,512] of one matrix, or of gate (a) and up (b) together."""
    _need(scales_a, torch.uint8, 3, "scales_a")
    E, N, K = scales_a.shape[0], scales_a.shape[1], scales_a.shape[2] * block
    dev = scales_a.device
    _fp4_block(block, K, "K")
    _shaped(scales_b, torch.uint8, tuple(scales_a.shape), "scales_b", dev)
    if N % (8 if scales_b is None else 64):
        raise ValueError(f"N = {N} must be a multiple of {8 if scales_b is None else 64}")
    shape = (E, -(-N // 128) if scales_b is None else N // 64, _fp4_atoms(K, block), 512)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
    else:
        _shaped(out, torch.uint8, shape, "sf", dev)
    _call("moe_fp4_pack_scales", dev, _ptr(scales_a), _ptr(scales_b), E, N, K, block, _ptr(out))
    return out


def _fp4_factor(t: Optional[torch.Tensor], E: int, block: int, name: str, dev):
    if block == 32:
        return None
    _given(t, torch.float32, (E,), name, dev)
    return t


def moe_grouped_gemm_fp4(rows, offsets: torch.Tensor, w, block: int = 16,
                         ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """y [M,N] bf16 of 4-bit rows (from moe_fp4_quantize_rows) and weights ``w`` = (codes [E,N,K/2],
    scales from moe_fp4_pack_scales, scale [E] or None)."""
    dev = rows[0].device
    E = _experts_of(offsets, dev)
    q, sf, rs, M, K = _fp4_rows(rows, E, block, dev)
    codes, wsf, scale = w
    _need(codes, torch.uint8, 3, "codes")
    N = codes.shape[1]
    _shaped(codes, torch.uint8, (E, N, K // 2), "codes", dev)
    _given(wsf, torch.uint8, (E, -(-N // 128), _fp4_atoms(K, block), 512), "weight scales", dev)
    scale = _fp4_factor(scale, E, block, "scale", dev)
    ws = _need_ws(ws, WORKSPACE_HEADER, dev)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    else:
        _shaped(out, torch.bfloat16, (M, N), "y", dev)
    _call("moe_grouped_gemm_fp4", dev, _ptr(q), _ptr(sf), _ptr(rs), _ptr(offsets), E, M, K, N, block,
          _ptr(codes), _ptr(wsf), _ptr(scale), _ptr(out), _ptr(ws), ws.numel() * ws.element_size())
    return out


def fp4_ffn_op(block: int, h_scale) -> int:
    """The operation id that sizes moe_grouped_ffn_fp4's workspace."""
    return MOE_OP_GROUPED_FFN_FP4 if block == 16 and h_scale is None else MOE_OP_GROUPED_FFN_FP4_FUSED


def moe_grouped_ffn_fp4(rows, offsets: torch.Tensor, wgu, wd, block: int = 16,
                        h_scale: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None):
    """y [M,d] bf16 of the SwiGLU experts on 4-bit rows and weights. ``wgu`` = (gate codes, up codes
    [E,I,d/2], their scales packed together, gate scale, up scale [E]), ``wd`` = (codes [E,d,I/2],
    packed scales, scale [E]); the factors are None with block 32. h_scale [E] fp32 (block 16) fixes
    the hidden rows' factor per expert; without it each hidden row takes its own maximum."""
    dev = rows[0].device
    E = _experts_of(offsets, dev)
    q, sf, rs, M, d = _fp4_rows(rows, E, block, dev)
    gate, up, gsf, gscale, uscale = wgu
    down, dsf, dscale = wd
    _need(gate, torch.uint8, 3, "gate codes")
    I = gate.shape[1]
    if I % 64 or I < 64:
        raise ValueError(f"I must be a multiple of 64, got {I}")
    _shaped(gate, torch.uint8, (E, I, d // 2), "gate codes", dev)
    _given(up, torch.uint8, (E, I, d // 2), "up codes", dev)
    _given(gsf, torch.uint8, (E, I // 64, _fp4_atoms(d, block), 512), "gate and up scales", dev)
    _given(down, torch.uint8, (E, d, I // 2), "down codes", dev)
    _given(dsf, torch.uint8, (E, -(-d // 128), _fp4_atoms(I, block), 512), "down scales", dev)
    gscale = _fp4_factor(gscale, E, block, "gate scale", dev)
    uscale = _fp4_factor(uscale, E, block, "up scale", dev)
    dscale = _fp4_factor(dscale, E, block, "down scale", dev)
    if h_scale is not None:
        if block == 32:
            raise ValueError("h_scale goes with block 16")
        _shaped(h_scale, torch.float32, (E,), "h_scale", dev)
    ws = _need_ws(ws, workspace_size(fp4_ffn_op(block, h_scale), M, E, 1, 1, d, I) if ws is None else 0,
                  dev)
    if out is None:
        out = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    else:
        _shaped(out, torch.bfloat16, (M, d), "y", dev)
    _call("moe_grouped_ffn_fp4", dev, _ptr(q), _ptr(sf), _ptr(rs), _ptr(offsets), E, M, d, I, block,
          _ptr(gate), _ptr(up), _ptr(gsf), _ptr(gscale), _ptr(uscale), _ptr(down), _ptr(dsf),
          _ptr(dscale), _ptr(h_scale), _ptr(out), _ptr(ws), ws.numel() * ws.element_size())
    return out


def moe_profile_start(capacity: int = 4096):
    _check("moe_profile_start", load().moe_profile_start(int(capacity)))


def moe_profile_stop():
    """Stops recording; returns [(kernel name, milliseconds), ...] in launch order."""
    lib = load()
    n = lib.moe_profile_stop()
    out = []
    for i in range(n):
        name = ctypes.c_char_p()
        ms = ctypes.c_float()
        _check("moe_profile_record", lib.moe_profile_record(i, ctypes.byref(name), ctypes.byref(ms)))
        out.append((name.value.decode(), float(ms.value)))
    return out


def moe_debug_wait_timeout(ws: torch.Tensor, timeout_us: int):
    """Runs the GEMM kernels' bounded wait on a barrier nothing completes; the
    status word of ``ws`` then reads MOE_ERR_DEVICE_TIMEOUT."""
    _check("moe_debug_wait_timeout", load().moe_debug_wait_timeout(_ptr(ws), int(timeout_us),
                                                                    _stream(ws.device)))


def moe_debug_check_status() -> int:
    """The debug build's index-check record (synchronises; clears it). Raises
    MoEError(MOE_ERR_UNSUPPORTED) on a release build."""
    st = ctypes.c_int(0)
    _check("moe_debug_check_status", load().moe_debug_check_status(ctypes.byref(st)))
    return st.value


def moe_read_device_status(ws: torch.Tensor) -> int:
    st = ctypes.c_int(0)
    _check("moe_read_device_status", load().moe_read_device_status(
        _ptr(ws), _stream(ws.device), ctypes.byref(st)))
    return st.value
