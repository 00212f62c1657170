"""ctypes binding of librs.so (see include/rs.h): argument marshalling only.

Every function here forwards torch tensors' device pointers and sizes to the C
entry point of the same name and raises ``RsError`` on a non-zero status. All
arithmetic runs in the library's CUDA kernels; there is no other code path, and
a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librs.so")

RS_OK = 0
RS_ERR_NULL = 1
RS_ERR_SHAPE = 2
RS_ERR_KEEP_K = 3
RS_ERR_ALIGN = 4
RS_ERR_CUDA = 5
RS_ERR_DEVICE_TIMEOUT = 6
RS_ERR_NO_MEM = 7

_vp, _i, _fp, _ip = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p
_l, _u = ctypes.c_int64, ctypes.c_uint64
SIGNATURES = {
    "rs_block_forward": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _ip,
                              _fp, _vp]),
    "rs_ln_stats": (_i, [_vp, _i, _i, _fp, _vp]),
    "rs_ln_fc1_gelu": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rs_ln_fc1_gelu_staged": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rs_gelu_apply": (_i, [_fp, _fp, _i, _vp]),
    "rs_debug_fc1_skip_load": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp]),
    "rs_ln_fold": (_i, [_vp, _vp, _vp, _vp, _i, _i, _vp, _fp, _fp, _vp]),
    "rs_fc1_gelu_folded": (_i, [_vp, _fp, _vp, _fp, _fp, _i, _i, _i, _vp, _vp]),
    "rs_ln_fc1_gelu_noalloc": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rs_fc2_residual_shift": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp, _fp, _vp]),
    "rs_fc2_residual_shift_ex": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _fp, _vp]),
    "rs_num_partials_ex": (_i, [_i, _i]),
    "rs_block_forward_ex": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                                 _vp, _ip, _fp, _vp]),
    "rs_select_topk_ex": (_i, [_fp, _i, _i, _i, _i, _i, _i, _fp, _ip, _vp]),
    "rs_select_gather_ex": (_i, [_fp, _i, _vp, _i, _i, _i, _i, _i, _i, _fp, _ip, _vp, _vp]),
    "rs_num_partials": (_i, [_i]),
    "rs_select_topk": (_i, [_fp, _i, _i, _i, _i, _fp, _ip, _vp]),
    "rs_gather_rows": (_i, [_vp, _i, _i, _i, _ip, _i, _vp, _vp]),
    "rs_select_gather": (_i, [_fp, _i, _vp, _i, _i, _i, _i, _fp, _ip, _vp, _vp]),
    "rs_block_forward_block_shift_ex": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                             _vp, _i, _i, _i, _vp, _ip, _fp, _vp]),
    "rs_mlp_forward": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rs_attn_core": (_i, [_vp, _i, _i, _i, _vp, _vp]),
    "rs_debug_attn_skip_load": (_i, [_vp, _i, _i, _i, _vp, _i, _i, _vp]),
    "rs_encoder_forward": (_i, [_vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_vp),
                                ctypes.POINTER(_i), _vp, _vp]),
    "rs_attn_sublayer": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rs_attn_forward_ex": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                                _vp, _ip, _fp, _vp]),
    "rs_mlp_fused_supported": (_i, [_i, _i]),
    "rs_mlp_fused": (_i, [_vp, _fp, _vp, _fp, _fp, _i, _i, _i, _vp, _vp, _vp, _fp, _vp]),
    "rs_ln_forward": (_i, [_vp, _l, _i, _i, _i, _vp, _vp, _i, ctypes.c_float, _vp, _l, _fp, _vp]),
    "rs_ln_quantize": (_i, [_vp, _l, _i, _i, _i, _vp, _vp, _i, ctypes.c_float, _vp, _l, _vp, _fp,
                            _vp]),
    "rs_ln_backward": (_i, [_vp, _l, _vp, _l, _vp, _l, _fp, _vp, _i, _i, _i, _i, _vp, _l, _fp, _fp,
                            _vp, _u, _vp]),
    "rs_ln_backward_ws_bytes": (_u, [_i, _i]),
    "rs_fp8_scale_bytes": (_u, [_i, _i]),
    "rs_fp8_quantize": (_i, [_vp, _l, _i, _i, _i, _vp, _l, _vp, _vp, _l, _vp, _fp, _vp, _u, _vp]),
    "rs_fp8_quantize_ws_bytes": (_u, [_i, _i]),
    "rs_fp8_gemm": (_i, [_vp, _l, _vp, _vp, _l, _vp, _i, _i, _i, _vp, _i, _vp, _l, _vp, _l, _i, _vp,
                         _vp]),
    "rs_debug_fp8_skip_load": (_i, [_vp, _l, _vp, _vp, _l, _vp, _i, _i, _i, _vp, _l, _i, _vp, _i, _i,
                                    _vp]),
    "rs_debug_fp8_linear_skip_load": (_i, [_vp, _l, _i, _i, _i, _vp, _l, _vp, _vp, _l, _i, _vp]),
    "rs_fp8_linear": (_i, [_vp, _l, _i, _i, _i, _vp, _l, _vp, _vp, _i, _vp, _l, _vp, _l, _vp, _u,
                           _vp]),
    "rs_fp8_linear_ws_bytes": (_u, [_i, _i]),
    "rs_fp8_linear_backward": (_i, [_vp, _l, _i, _i, _i, _vp, _l, _vp, _vp, _l, _vp, _vp, _l, _vp,
                                    _l, _i, _fp, _vp, _u, _vp]),
    "rs_fp8_linear_backward_ws_bytes": (_u, [_i, _i]),
    "rs_mlp_forward_fp8": (_i, [_vp, _i, _i, _i, _vp, _l, _vp, _vp, _vp, _l, _vp, _vp, _vp, _vp,
                                _vp, _vp, _u, _vp]),
    "rs_mlp_forward_fp8_ws_bytes": (_u, [_i, _i, _i]),
    "rs_status_string": (ctypes.c_char_p, [_i]),
    "rs_get_last_device_error": (_i, [_vp]),
    "rs_release_workspace": (None, []),
    "rs_workspace_bytes": (ctypes.c_uint64, [_i, _i, _i, _i]),
}

_lib = None


class RsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded librs.so. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m free_vit_token_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().rs_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != RS_OK:
        raise RsError(status, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr() or None


# The current stream's handle without building a torch.cuda.Stream object (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device()) or None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


RS_DIST_L2, RS_DIST_L1, RS_DIST_COSINE = 0, 1, 2
RS_NO_CLS = 1
DISTANCES = {"l2": RS_DIST_L2, "l1": RS_DIST_L1, "cosine": RS_DIST_COSINE}


def _dist(distance) -> int:
    return DISTANCES[distance] if isinstance(distance, str) else int(distance)


def rs_block_forward(x: torch.Tensor, W1, b1, W2, b2, gamma, beta, keep_k: int,
                     y_kept: Optional[torch.Tensor] = None, kept_idx: Optional[torch.Tensor] = None,
                     scores: Optional[torch.Tensor] = None, stream=None, distance="l2",
                     cls: bool = True) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """x [B, L, C] bf16 -> (y_kept [B, n, C] bf16, kept_idx [B, n] int32, scores [B, L] fp32)
    with n = 1 + k (CLS first) or k (cls=False: all L tokens ranked). `distance`: "l2",
    "l1" or "cosine" (or an RS_DIST_* value)."""
    B, L, C = x.shape
    H = W1.shape[0]
    dev = x.device
    n = keep_k + (1 if cls else 0)
    if y_kept is None:
        y_kept = torch.empty(B, n, C, dtype=torch.bfloat16, device=dev)
    if kept_idx is None:
        kept_idx = torch.empty(B, n, dtype=torch.int32, device=dev)
    if scores is None:
        scores = torch.empty(B, L, dtype=torch.float32, device=dev)
    st = lib().rs_block_forward_ex(_ptr(x), B, L, C, H, _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2),
                                   _ptr(gamma), _ptr(beta), int(keep_k), _dist(distance),
                                   0 if cls else RS_NO_CLS, _ptr(y_kept), _ptr(kept_idx),
                                   _ptr(scores), _stream(stream))
    _check(st, "rs_block_forward")
    return y_kept, kept_idx, scores


def rs_ln_stats(x2d: torch.Tensor, stats: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M, C = x2d.shape
    if stats is None:
        stats = torch.empty(M, 2, dtype=torch.float32, device=x2d.device)
    _check(lib().rs_ln_stats(_ptr(x2d), M, C, _ptr(stats), _stream(stream)), "rs_ln_stats")
    return stats


def rs_ln_fc1_gelu(x2d: torch.Tensor, W1, b1, gamma, beta, hidden: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    M, C = x2d.shape
    H = W1.shape[0]
    if hidden is None:
        hidden = torch.empty(M, H, dtype=torch.bfloat16, device=x2d.device)
    st = lib().rs_ln_fc1_gelu(_ptr(x2d), M, C, H, _ptr(W1), _ptr(b1), _ptr(gamma), _ptr(beta),
                              _ptr(hidden), _stream(stream))
    _check(st, "rs_ln_fc1_gelu")
    return hidden


def rs_ln_fold(W1: torch.Tensor, b1, gamma, beta, Wg: Optional[torch.Tensor] = None,
               colG: Optional[torch.Tensor] = None, colC: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    H, C = W1.shape
    dev = W1.device
    if Wg is None:
        Wg = torch.empty(H, C, dtype=torch.bfloat16, device=dev)
    if colG is None:
        colG = torch.empty(H, dtype=torch.float32, device=dev)
    if colC is None:
        colC = torch.empty(H, dtype=torch.float32, device=dev)
    st = lib().rs_ln_fold(_ptr(W1), _ptr(b1), _ptr(gamma), _ptr(beta), C, H, _ptr(Wg), _ptr(colG),
                          _ptr(colC), _stream(stream))
    _check(st, "rs_ln_fold")
    return Wg, colG, colC


def rs_fc1_gelu_folded(x2d: torch.Tensor, stats, Wg, colG, colC,
                       hidden: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M, C = x2d.shape
    H = Wg.shape[0]
    if hidden is None:
        hidden = torch.empty(M, H, dtype=torch.bfloat16, device=x2d.device)
    st = lib().rs_fc1_gelu_folded(_ptr(x2d), _ptr(stats), _ptr(Wg), _ptr(colG), _ptr(colC), M, C, H,
                                  _ptr(hidden), _stream(stream))
    _check(st, "rs_fc1_gelu_folded")
    return hidden


def rs_ln_fc1_gelu_staged(x2d: torch.Tensor, W1, b1, gamma, beta,
                          hidden: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M, C = x2d.shape
    H = W1.shape[0]
    if hidden is None:
        hidden = torch.empty(M, H, dtype=torch.bfloat16, device=x2d.device)
    st = lib().rs_ln_fc1_gelu_staged(_ptr(x2d), M, C, H, _ptr(W1), _ptr(b1), _ptr(gamma),
                                     _ptr(beta), _ptr(hidden), _stream(stream))
    _check(st, "rs_ln_fc1_gelu_staged")
    return hidden


def rs_ln_fc1_gelu_noalloc(x2d: torch.Tensor, W1, b1, gamma, beta, hidden: torch.Tensor,
                           stream=None) -> torch.Tensor:
    """rs_ln_fc1_gelu with its scratch in the library's static device array (the caller
    provides ``hidden``; nothing is allocated)."""
    M, C = x2d.shape
    H = W1.shape[0]
    st = lib().rs_ln_fc1_gelu_noalloc(_ptr(x2d), M, C, H, _ptr(W1), _ptr(b1), _ptr(gamma),
                                      _ptr(beta), _ptr(hidden), _stream(stream))
    _check(st, "rs_ln_fc1_gelu_noalloc")
    return hidden


RS_FUSED_PARTIALS = 4


def rs_mlp_fused_supported(C: int, H: int) -> bool:
    return bool(lib().rs_mlp_fused_supported(int(C), int(H)))


def rs_mlp_fused(x2d: torch.Tensor, stats: torch.Tensor, Wg: torch.Tensor, colG: torch.Tensor,
                 colC: torch.Tensor, W2, b2, y: Optional[torch.Tensor] = None,
                 partials: Optional[torch.Tensor] = None, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The fused MLP on LN statistics and folded weights: (y [M, C] bf16,
    partials [M, RS_FUSED_PARTIALS] fp32)."""
    M, C = x2d.shape
    H = Wg.shape[0]
    if y is None:
        y = torch.empty(M, C, dtype=torch.bfloat16, device=x2d.device)
    if partials is None:
        partials = torch.empty(M, RS_FUSED_PARTIALS, dtype=torch.float32, device=x2d.device)
    st = lib().rs_mlp_fused(_ptr(x2d), _ptr(stats), _ptr(Wg), _ptr(colG), _ptr(colC), M, C, H,
                            _ptr(W2), _ptr(b2), _ptr(y), _ptr(partials), _stream(stream))
    _check(st, "rs_mlp_fused")
    return y, partials


def rs_debug_fc1_skip_load(x2d: torch.Tensor, W1, b1, gamma, beta, hidden: torch.Tensor,
                           skip_kblock: int, timeout_us: int, stream=None) -> None:
    """Test hook: fc1 with one k-block load withheld (see include/rs.h)."""
    M, C = x2d.shape
    H = W1.shape[0]
    st = lib().rs_debug_fc1_skip_load(_ptr(x2d), M, C, H, _ptr(W1), _ptr(b1), _ptr(gamma),
                                      _ptr(beta), _ptr(hidden), int(skip_kblock), int(timeout_us),
                                      _stream(stream))
    _check(st, "rs_debug_fc1_skip_load")


def rs_gelu_apply(z: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty_like(z)
    _check(lib().rs_gelu_apply(_ptr(z), _ptr(out), z.numel(), _stream(stream)), "rs_gelu_apply")
    return out


def rs_num_partials(C: int, distance="l2") -> int:
    return int(lib().rs_num_partials_ex(int(C), _dist(distance)))


def rs_fc2_residual_shift(hidden: torch.Tensor, x2d: torch.Tensor, W2, b2,
                          y: Optional[torch.Tensor] = None, partials: Optional[torch.Tensor] = None,
                          stream=None, distance="l2") -> Tuple[torch.Tensor, torch.Tensor]:
    M, H = hidden.shape
    C = x2d.shape[1]
    if y is None:
        y = torch.empty(M, C, dtype=torch.bfloat16, device=x2d.device)
    if partials is None:
        partials = torch.empty(M, rs_num_partials(C, distance), dtype=torch.float32,
                               device=x2d.device)
    st = lib().rs_fc2_residual_shift_ex(_ptr(hidden), _ptr(x2d), M, C, H, _ptr(W2), _ptr(b2),
                                        _dist(distance), _ptr(y), _ptr(partials), _stream(stream))
    _check(st, "rs_fc2_residual_shift")
    return y, partials


def rs_select_topk(partials: torch.Tensor, B: int, L: int, keep_k: int,
                   scores: Optional[torch.Tensor] = None, kept_idx: Optional[torch.Tensor] = None,
                   stream=None, distance="l2", cls: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    P = partials.shape[-1]
    dev = partials.device
    if scores is None:
        scores = torch.empty(B, L, dtype=torch.float32, device=dev)
    if kept_idx is None:
        kept_idx = torch.empty(B, keep_k + (1 if cls else 0), dtype=torch.int32, device=dev)
    st = lib().rs_select_topk_ex(_ptr(partials), P, B, L, int(keep_k), _dist(distance),
                                 0 if cls else RS_NO_CLS, _ptr(scores), _ptr(kept_idx),
                                 _stream(stream))
    _check(st, "rs_select_topk")
    return scores, kept_idx


def rs_select_gather(partials: torch.Tensor, y: torch.Tensor, keep_k: int,
                     scores: Optional[torch.Tensor] = None, kept_idx: Optional[torch.Tensor] = None,
                     y_kept: Optional[torch.Tensor] = None, stream=None, distance="l2",
                     cls: bool = True) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """partials [B*L, P] fp32, y [B, L, C] bf16 -> (scores, kept_idx, y_kept)."""
    B, L, C = y.shape
    P = partials.shape[-1]
    dev = y.device
    n = keep_k + (1 if cls else 0)
    if scores is None:
        scores = torch.empty(B, L, dtype=torch.float32, device=dev)
    if kept_idx is None:
        kept_idx = torch.empty(B, n, dtype=torch.int32, device=dev)
    if y_kept is None:
        y_kept = torch.empty(B, n, C, dtype=y.dtype, device=dev)
    st = lib().rs_select_gather_ex(_ptr(partials), P, _ptr(y), B, L, C, int(keep_k),
                                   _dist(distance), 0 if cls else RS_NO_CLS, _ptr(scores),
                                   _ptr(kept_idx), _ptr(y_kept), _stream(stream))
    _check(st, "rs_select_gather")
    return scores, kept_idx, y_kept


def rs_gather_rows(y: torch.Tensor, kept_idx: torch.Tensor, keep_k: int,
                   y_kept: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    B, L, C = y.shape
    if y_kept is None:
        y_kept = torch.empty(B, keep_k + 1, C, dtype=y.dtype, device=y.device)
    st = lib().rs_gather_rows(_ptr(y), B, L, C, _ptr(kept_idx), int(keep_k), _ptr(y_kept),
                              _stream(stream))
    _check(st, "rs_gather_rows")
    return y_kept


def rs_get_last_device_error(stream=None) -> int:
    return int(lib().rs_get_last_device_error(_stream(stream)))


def rs_release_workspace() -> None:
    lib().rs_release_workspace()


def rs_workspace_bytes(B: int, L: int, C: int, H: int) -> int:
    return int(lib().rs_workspace_bytes(B, L, C, H))


def rs_attn_core(qkv: torch.Tensor, heads: int, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """qkv [B, L, 3 * 64 heads] bf16 -> out [B, L, 64 heads] bf16: per sample and head,
    Softmax(Q K^T / 8) V."""
    B, L, C3 = qkv.shape
    C = 64 * heads
    if C3 != 3 * C:
        raise ValueError("qkv must be [B, L, 3 * 64 * heads]")
    if out is None:
        out = torch.empty(B, L, C, dtype=torch.bfloat16, device=qkv.device)
    _check(lib().rs_attn_core(_ptr(qkv), B, L, int(heads), _ptr(out), _stream(stream)),
           "rs_attn_core")
    return out


def rs_attn_sublayer(x: torch.Tensor, Wqkv, bqkv, Wo, bo, gamma, beta, heads: int,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [B, L, C] bf16 -> x + SA(LN(x)) [B, L, C] bf16 (C = 64 heads)."""
    B, L, C = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check(lib().rs_attn_sublayer(_ptr(x), B, L, C, int(heads), _ptr(Wqkv), _ptr(bqkv), _ptr(Wo),
                                  _ptr(bo), _ptr(gamma), _ptr(beta), _ptr(out), _stream(stream)),
           "rs_attn_sublayer")
    return out


def rs_attn_forward(x: torch.Tensor, Wqkv, bqkv, Wo, bo, gamma, beta, heads: int, keep_k: int,
                    x_kept: Optional[torch.Tensor] = None,
                    kept_idx: Optional[torch.Tensor] = None,
                    scores: Optional[torch.Tensor] = None, stream=None, distance="l2",
                    cls: bool = True) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The attention sublayer, then pruning by its representation shift:
    (x'_kept [B, n, C], kept_idx [B, n] int32, scores [B, L] fp32), n as in
    rs_block_forward."""
    B, L, C = x.shape
    dev = x.device
    n = keep_k + (1 if cls else 0)
    if x_kept is None:
        x_kept = torch.empty(B, n, C, dtype=torch.bfloat16, device=dev)
    if kept_idx is None:
        kept_idx = torch.empty(B, n, dtype=torch.int32, device=dev)
    if scores is None:
        scores = torch.empty(B, L, dtype=torch.float32, device=dev)
    st = lib().rs_attn_forward_ex(_ptr(x), B, L, C, int(heads), _ptr(Wqkv), _ptr(bqkv), _ptr(Wo),
                                  _ptr(bo), _ptr(gamma), _ptr(beta), int(keep_k), _dist(distance),
                                  0 if cls else RS_NO_CLS, _ptr(x_kept), _ptr(kept_idx),
                                  _ptr(scores), _stream(stream))
    _check(st, "rs_attn_forward")
    return x_kept, kept_idx, scores


def rs_mlp_forward(x: torch.Tensor, W1, b1, W2, b2, gamma, beta,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [..., C] bf16 -> x + MLP(LN(x)) (no scoring, no pruning), same shape."""
    C = x.shape[-1]
    M = x.numel() // C
    H = W1.shape[0]
    if out is None:
        out = torch.empty_like(x)
    _check(lib().rs_mlp_forward(_ptr(x), M, C, H, _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2),
                                _ptr(gamma), _ptr(beta), _ptr(out), _stream(stream)),
           "rs_mlp_forward")
    return out


ENCODER_WEIGHT_ORDER = ("Wqkv", "bqkv", "Wo", "bo", "gamma1", "beta1",
                        "W1", "b1", "W2", "b2", "gamma2", "beta2")


def rs_encoder_forward(x: torch.Tensor, layers, keep, heads: int,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [B, L, C] bf16 through len(layers) encoder layers; `layers[l]` is a sequence
    of the 12 weight tensors in ENCODER_WEIGHT_ORDER, keep[l] the patch tokens kept
    after layer l (negative: no pruning). Returns [B, L_out, C]."""
    B, L, C = x.shape
    depth = len(layers)
    H = layers[0][6].shape[0]
    ptrs = (_vp * (12 * depth))(*[_ptr(t) for lw in layers for t in lw])
    kk = (_i * depth)(*[int(k) for k in keep])
    L_out = L
    for k in keep:
        if k >= 0:
            L_out = 1 + int(k)
    if out is None:
        out = torch.empty(B, L_out, C, dtype=torch.bfloat16, device=x.device)
    _check(lib().rs_encoder_forward(_ptr(x), B, L, C, H, int(heads), depth, ptrs, kk, _ptr(out),
                                    _stream(stream)), "rs_encoder_forward")
    return out


def rs_block_forward_block_shift(x_in: torch.Tensor, x: torch.Tensor, W1, b1, W2, b2, gamma,
                                 beta, keep_k: int, y_kept: Optional[torch.Tensor] = None,
                                 kept_idx: Optional[torch.Tensor] = None,
                                 scores: Optional[torch.Tensor] = None, stream=None,
                                 distance="l2", cls: bool = True):
    """rs_block_forward scored on the whole-block shift D(y, x_in): x_in [B, L, C] is the
    block input before the attention sublayer, x = x' its output."""
    B, L, C = x.shape
    H = W1.shape[0]
    dev = x.device
    n = keep_k + (1 if cls else 0)
    if y_kept is None:
        y_kept = torch.empty(B, n, C, dtype=torch.bfloat16, device=dev)
    if kept_idx is None:
        kept_idx = torch.empty(B, n, dtype=torch.int32, device=dev)
    if scores is None:
        scores = torch.empty(B, L, dtype=torch.float32, device=dev)
    st = lib().rs_block_forward_block_shift_ex(
        _ptr(x_in), _ptr(x), B, L, C, H, _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(gamma),
        _ptr(beta), int(keep_k), _dist(distance), 0 if cls else RS_NO_CLS, _ptr(y_kept),
        _ptr(kept_idx), _ptr(scores), _stream(stream))
    _check(st, "rs_block_forward_block_shift")
    return y_kept, kept_idx, scores


def rs_debug_attn_skip_load(qkv: torch.Tensor, heads: int, out: torch.Tensor, skip_block: int,
                            timeout_us: int, stream=None) -> None:
    """Test hook: the attention core with one CTA's key-block loads withheld from
    `skip_block` on; its waits time out after `timeout_us` (see rs.h)."""
    B, L, _ = qkv.shape
    _check(lib().rs_debug_attn_skip_load(_ptr(qkv), B, L, int(heads), _ptr(out), int(skip_block),
                                         int(timeout_us), _stream(stream)),
           "rs_debug_attn_skip_load")


# ------------------------------------------------------------------ layer norm, 8-bit blocks
RS_BF16, RS_FP16, RS_FP32, RS_E4M3 = 0, 1, 2, 3
RS_MAX_LN_C = 8192
_INT_MAX = 2 ** 31 - 1
_DTYPES = {torch.bfloat16: RS_BF16, torch.float16: RS_FP16, torch.float32: RS_FP32}


class Fp8(NamedTuple):
    """A matrix [rows, K] in 8-bit blocks: ``q`` [rows, ld] float8_e4m3fn (ld >= K, a
    multiple of 16) and ``scales``, a flat uint8 tensor of rs_fp8_scale_bytes(rows, K) bytes
    with one power of two per 128 values of a row (their order: include/rs.h)."""

    q: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int


def _device(t: torch.Tensor, name: str) -> int:
    """The index of the current CUDA device, which `t` must be on."""
    d = t.get_device()
    if d < 0 or d != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return d


def _rows(t: torch.Tensor, name: str, dev: int, dtype: Optional[torch.dtype] = None,
          width: Optional[int] = None, rows: Optional[int] = None) -> Tuple[Optional[int], int, int]:
    """(address, row stride, rows) of a matrix whose rows may be strided; tensors of more
    dimensions count as their rows and must be contiguous."""
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} wanted, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    shape = t.shape
    if t.is_contiguous():
        if len(shape) == 0:
            raise ValueError(f"{name} must be a matrix or a contiguous tensor")
        w = ld = shape[-1]
        n = shape[0] if len(shape) == 2 else t.numel() // max(w, 1)
    else:
        if len(shape) != 2:
            raise ValueError(f"{name} must be a matrix or a contiguous tensor")
        n, w = shape
        ld, step = t.stride()
        if w > 1 and step != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        if n > 1 and ld < w:
            raise ValueError(f"{name}: rows overlap")
        ld = max(ld, w)
    if n > _INT_MAX or w > _INT_MAX:  # ctypes would pass on what 32 bits hold of them
        raise ValueError(f"{name}: sizes below 2^31 wanted, got [{n}, {w}]")
    if width is not None and w != width:
        raise ValueError(f"{name}: rows of {width} wanted, got {w}")
    if rows is not None and n != rows:
        raise ValueError(f"{name}: {rows} rows wanted, got {n}")
    return t.data_ptr() or None, ld, n


def _vec(t: Optional[torch.Tensor], name: str, dev: int, n: int,
         dtype: torch.dtype) -> Optional[int]:
    """Address of a contiguous tensor of n elements (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of {n} elements wanted")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    return t.data_ptr() or None


def _params(x: torch.Tensor, dev: int, C: int, gamma, beta):
    dt = gamma.dtype if gamma is not None else beta.dtype if beta is not None else x.dtype
    if dt is not torch.float32 and dt is not x.dtype:
        raise ValueError("gamma and beta must be float32 or of x's type")
    return _DTYPES[dt], _vec(gamma, "gamma", dev, C, dt), _vec(beta, "beta", dev, C, dt)


def _float_type(x: torch.Tensor) -> int:
    if x.dtype not in _DTYPES:
        raise ValueError("bfloat16, float16 or float32 wanted")
    return _DTYPES[x.dtype]


_ws_sizes = {}


def _ws_size(name: str, *sizes: int, dev: Optional[int] = None) -> int:
    """What the size function `name` says on device `dev`, the current one. Kept, since a call's
    host time counts, by device: the layer norm's answer goes by the SM count."""
    key = (dev, name, sizes)
    n = _ws_sizes.get(key)
    if n is None:
        n = int(getattr(lib(), name)(*sizes))
        # the layer norm's 0 also says that the device could not be asked, which may pass: it is
        # kept only where sizes that need scratch get an answer
        if n or name != "rs_ln_backward_ws_bytes" or lib().rs_ln_backward_ws_bytes(1 << 26, 1):
            if len(_ws_sizes) >= 4096:
                _ws_sizes.clear()
            _ws_sizes[key] = n
    return n


def _ws(ws: Optional[torch.Tensor], device: torch.device, dev: int, name: str, *sizes: int):
    """(address, bytes, tensor) of the caller's scratch, or of scratch from torch's allocator
    (the tensor must live until the call is queued). `name` is the size function."""
    if ws is None:
        n = _ws_size(name, *sizes, dev=dev)
        if n == 0:  # none needed (or sizes that the call will refuse)
            return None, 0, None
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        return ws.data_ptr() or None, n, ws
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if ws.get_device() != dev:
        raise ValueError("ws must be on the current CUDA device")
    return ws.data_ptr() or None, ws.numel() * ws.element_size(), ws


def _like(x: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of x's shape and type."""
    if x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(*x.shape, dtype=x.dtype, device=x.device)


def _matrix(x: torch.Tensor, M: int, N: int, dtype: torch.dtype) -> torch.Tensor:
    """An uninitialised tensor with x's leading dimensions (M rows in all) and N columns."""
    if x.dim() == 2:
        return torch.empty(M, N, dtype=dtype, device=x.device)
    return torch.empty(*x.shape[:-1], N, dtype=dtype, device=x.device)


def _on(stream, fn, *args, **kwargs):
    """fn(*args, **kwargs) with `stream` as the current one: what the call allocates, scratch
    above all, then belongs to the stream that uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def _scale_bytes(rows: int, K: int) -> int:
    return (rows + 127) // 128 * ((K + 511) // 512) * 512


def _fp8_empty(rows: int, K: int, device) -> Fp8:
    return Fp8(torch.empty(rows, (K + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device=device),
               torch.empty(_scale_bytes(rows, K), dtype=torch.uint8, device=device), rows, K)


def _fp8_new(rows: int, K: int, device):
    """A new Fp8 with its (q address, row stride, scales address)."""
    t = _fp8_empty(rows, K, device)
    return t, t.q.data_ptr() or None, (K + 15) // 16 * 16, t.scales.data_ptr() or None


def _fp8(t: Fp8, name: str, dev: int, rows: Optional[int] = None, K: Optional[int] = None):
    """(q address, row stride, scales address) of a quantised operand."""
    q, s, r, k = t
    if (rows is not None and r != rows) or (K is not None and k != K):
        raise ValueError(f"{name}: [{rows}, {K}] wanted, got [{r}, {k}]")
    pq, ld, _ = _rows(q, name, dev, torch.float8_e4m3fn, rows=r)
    if not 0 <= k <= q.shape[-1]:
        raise ValueError(f"{name}: rows shorter than K")
    n = s.numel()
    if n < _scale_bytes(r, k):
        raise ValueError(f"{name}: too few scale bytes")
    return pq, ld, _vec(s, f"{name} scales", dev, n, torch.uint8)


def rs_ln_forward(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                  beta: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  y: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [..., C] (bf16, fp16 or fp32; a matrix may have strided rows) -> (LN(x) of the same
    type, stats [M, 2] fp32 with each row's mean and 1/std for rs_ln_backward). y may be x."""
    if stream is not None:
        return _on(stream, rs_ln_forward, x, gamma, beta, eps, y, stats)
    dev, dt = _device(x, "x"), _float_type(x)
    px, ldx, M = _rows(x, "x", dev)
    C = x.shape[-1]
    pdt, pg, pb = _params(x, dev, C, gamma, beta)
    if y is None:
        y = _like(x)
        py, ldy = y.data_ptr() or None, C
    else:
        py, ldy, _ = _rows(y, "y", dev, x.dtype, C, M)
    if stats is None:
        stats = torch.empty(M, 2, dtype=torch.float32, device=x.device)
        ps = stats.data_ptr() or None
    else:
        ps = _vec(stats, "stats", dev, 2 * M, torch.float32)
    _check(lib().rs_ln_forward(px, ldx, M, C, dt, pg, pb, pdt, eps, py, ldy, ps, _stream(None)),
           "rs_ln_forward")
    return y, stats


def rs_ln_quantize(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                   beta: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   out: Optional[Fp8] = None, stats: Optional[torch.Tensor] = None,
                   stream=None) -> Fp8:
    """LN(x) in 8-bit blocks along C (x bf16 or fp16, C a multiple of 8); `stats` [M, 2] fp32
    also receives each row's mean and 1/std."""
    if stream is not None:
        return _on(stream, rs_ln_quantize, x, gamma, beta, eps, out, stats)
    dev, dt = _device(x, "x"), _float_type(x)
    px, ldx, M = _rows(x, "x", dev)
    C = x.shape[-1]
    pdt, pg, pb = _params(x, dev, C, gamma, beta)
    if out is None:
        out, q, ldq, sc = _fp8_new(M, C, x.device)
    else:
        q, ldq, sc = _fp8(out, "out", dev, M, C)
    _check(lib().rs_ln_quantize(px, ldx, M, C, dt, pg, pb, pdt, eps, q, ldq, sc,
                                _vec(stats, "stats", dev, 2 * M, torch.float32), _stream(None)),
           "rs_ln_quantize")
    return out


def rs_ln_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor,
                   gamma: Optional[torch.Tensor] = None, dres: Optional[torch.Tensor] = None,
                   dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                   dbeta: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of y = LN(x) for dy: (dx, of x's type, with `dres` added; dgamma [C] fp32;
    dbeta [C] fp32). `stats` as rs_ln_forward returned them; dx may be dres."""
    if stream is not None:
        return _on(stream, rs_ln_backward, dy, x, stats, gamma, dres, dx, dgamma, dbeta, ws)
    dev, dt = _device(x, "x"), _float_type(x)
    px, ldx, M = _rows(x, "x", dev)
    C, device, f32 = x.shape[-1], x.device, torch.float32
    pdy, lddy, _ = _rows(dy, "dy", dev, x.dtype, C, M)
    pdr, lddr = (None, C) if dres is None else _rows(dres, "dres", dev, x.dtype, C, M)[:2]
    pdt, pg, _ = _params(x, dev, C, gamma, None)
    if dx is None:
        dx = _like(x)
        pdx, lddx = dx.data_ptr() or None, C
    else:
        pdx, lddx, _ = _rows(dx, "dx", dev, x.dtype, C, M)
    if dgamma is None:
        dgamma = torch.empty(C, dtype=f32, device=device)
        pdg = dgamma.data_ptr() or None
    else:
        pdg = _vec(dgamma, "dgamma", dev, C, f32)
    if dbeta is None:
        dbeta = torch.empty(C, dtype=f32, device=device)
        pdb = dbeta.data_ptr() or None
    else:
        pdb = _vec(dbeta, "dbeta", dev, C, f32)
    pw, nw, ws = _ws(ws, device, dev, "rs_ln_backward_ws_bytes", M, C)
    st = lib().rs_ln_backward(pdy, lddy, px, ldx, pdr, lddr, _vec(stats, "stats", dev, 2 * M, f32),
                              pg, pdt, M, C, dt, pdx, lddx, pdg, pdb, pw, nw, _stream(None))
    _check(st, "rs_ln_backward")
    return dx, dgamma, dbeta


def rs_fp8_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the scales of a [rows, K] matrix; 0 for sizes that the library does not take."""
    if not (0 <= rows <= _INT_MAX and 0 <= K <= _INT_MAX):
        return 0
    return int(lib().rs_fp8_scale_bytes(int(rows), int(K)))


def rs_fp8_quantize(x: torch.Tensor, rows: bool = True, cols: bool = False, colsum: bool = False,
                    out: Optional[Fp8] = None, out_t: Optional[Fp8] = None, stream=None
                    ) -> Tuple[Optional[Fp8], Optional[Fp8], Optional[torch.Tensor]]:
    """x [M, K] (bf16, fp16 or fp32) to 8-bit blocks of 128 along K (`rows`), and/or its
    transpose [K, M] in blocks along M (`cols`), and/or its column sums [K] fp32 (`colsum`,
    needs cols), from one read: a triple, None for what was not asked for."""
    if stream is not None:
        return _on(stream, rs_fp8_quantize, x, rows, cols, colsum, out, out_t)
    dev, dt = _device(x, "x"), _float_type(x)
    px, ldx, M = _rows(x, "x", dev)
    K, device = x.shape[-1], x.device
    if colsum and not cols:
        raise ValueError("colsum needs cols")
    q = qt = sc = sct = sums = ws = pw = ps = None
    ldq = ldqt = nw = 0
    if rows:
        if out is None:
            out, q, ldq, sc = _fp8_new(M, K, device)
        else:
            q, ldq, sc = _fp8(out, "out", dev, M, K)
    if cols:
        if out_t is None:
            out_t, qt, ldqt, sct = _fp8_new(K, M, device)
        else:
            qt, ldqt, sct = _fp8(out_t, "out_t", dev, K, M)
    if colsum:
        sums = torch.empty(K, dtype=torch.float32, device=device)
        ps = sums.data_ptr()
        pw, nw, ws = _ws(None, device, dev, "rs_fp8_quantize_ws_bytes", M, K)
    _check(lib().rs_fp8_quantize(px, ldx, M, K, dt, q, ldq, sc, qt, ldqt, sct, ps, pw, nw,
                                 _stream(None)), "rs_fp8_quantize")
    return out if rows else None, out_t if cols else None, sums


def rs_fp8_gemm(a: Fp8, b: Fp8, bias: Optional[torch.Tensor] = None, gelu: bool = False,
                resid: Optional[torch.Tensor] = None, out=None,
                out_dtype: Optional[torch.dtype] = None, stream=None):
    """act(A B^T + bias) + resid of two quantised operands [M, K] and [N, K]: a bf16 (default)
    or fp32 tensor [M, N], or with out_dtype=torch.float8_e4m3fn an Fp8."""
    if stream is not None:
        return _on(stream, rs_fp8_gemm, a, b, bias, gelu, resid, out, out_dtype)
    M, N, K, device = a.rows, b.rows, a.K, a.q.device
    dev = _device(a.q, "a")
    pa, lda, sa = _fp8(a, "a", dev)
    pb, ldb, sb = _fp8(b, "b", dev, K=K)
    if out_dtype is None:
        out_dtype = (torch.bfloat16 if out is None else
                     torch.float8_e4m3fn if isinstance(out, Fp8) else out.dtype)
    so, pr, ldr = None, None, N
    if out_dtype is torch.float8_e4m3fn:
        if out is None:
            out, po, ldo, so = _fp8_new(M, N, device)
        else:
            po, ldo, so = _fp8(out, "out", dev, M, N)
        dt = RS_E4M3
    else:
        if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
            raise ValueError("out_dtype: bfloat16, float32 or float8_e4m3fn")
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=device)
            po, ldo = out.data_ptr() or None, N
        else:
            po, ldo, _ = _rows(out, "out", dev, out_dtype, N, M)
        dt = _DTYPES[out_dtype]
    if resid is not None:
        pr, ldr, _ = _rows(resid, "resid", dev, out_dtype, N, M)
    _check(lib().rs_fp8_gemm(pa, lda, sa, pb, ldb, sb, M, N, K,
                             _vec(bias, "bias", dev, N, torch.bfloat16), int(gelu), pr, ldr, po,
                             ldo, dt, so, _stream(None)), "rs_fp8_gemm")
    return out


def rs_fp8_linear(x: torch.Tensor, w: Fp8, bias: Optional[torch.Tensor] = None,
                  gelu: bool = False, resid: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """x [..., K] bf16, quantised along K in the call, through a linear layer whose weight
    [N, K] is held in 8 bits: act(x W^T + bias) + resid [..., N] bf16."""
    if stream is not None:
        return _on(stream, rs_fp8_linear, x, w, bias, gelu, resid, out, ws)
    N, K, bf = w.rows, w.K, torch.bfloat16
    dev = _device(x, "x")
    px, ldx, M = _rows(x, "x", dev, bf, K)
    pw, ldw, sw = _fp8(w, "w", dev)
    if out is None:
        out = _matrix(x, M, N, bf)
        po, ldo = out.data_ptr() or None, N
    else:
        po, ldo, _ = _rows(out, "out", dev, bf, N, M)
    pr, ldr = (None, N) if resid is None else _rows(resid, "resid", dev, bf, N, M)[:2]
    pws, nws, ws = _ws(ws, x.device, dev, "rs_fp8_linear_ws_bytes", M, K)
    _check(lib().rs_fp8_linear(px, ldx, M, K, N, pw, ldw, sw, _vec(bias, "bias", dev, N, bf),
                               int(gelu), pr, ldr, po, ldo, pws, nws, _stream(None)),
           "rs_fp8_linear")
    return out


def rs_fp8_linear_backward(dy: torch.Tensor, xt: Optional[Fp8], wt: Optional[Fp8],
                           bias: bool = False, dw_dtype: torch.dtype = torch.bfloat16,
                           ws: Optional[torch.Tensor] = None, stream=None):
    """Gradients of out = x W^T + bias for dy [M, N] bf16, from the transposed quantised
    operands (rs_fp8_quantize(..., cols=True)): xt of x, [K, M], and wt of W, [K, N]. Returns
    (dx [M, K] bf16, dw [N, K], db [N] fp32), None for dx without wt, dw without xt and db
    without `bias`."""
    if stream is not None:
        return _on(stream, rs_fp8_linear_backward, dy, xt, wt, bias, dw_dtype, ws)
    dev = _device(dy, "dy")
    pdy, lddy, M = _rows(dy, "dy", dev, torch.bfloat16)
    N, device = dy.shape[-1], dy.device
    if xt is None and wt is None:
        raise ValueError("xt or wt wanted")
    if dw_dtype is not torch.bfloat16 and dw_dtype is not torch.float32:
        raise ValueError("dw_dtype: bfloat16 or float32")
    K = xt.rows if xt is not None else wt.rows
    px = sx = pw = sw = dx = dw = db = pdx = pdw = pdb = None
    ldx = ldw = 0
    if wt is not None:
        pw, ldw, sw = _fp8(wt, "wt", dev, K, N)
        dx = _matrix(dy, M, K, torch.bfloat16)
        pdx = dx.data_ptr() or None
    if xt is not None:
        px, ldx, sx = _fp8(xt, "xt", dev, K, M)
        dw = torch.empty(N, K, dtype=dw_dtype, device=device)
        pdw = dw.data_ptr()
    if bias:
        db = torch.empty(N, dtype=torch.float32, device=device)
        pdb = db.data_ptr()
    pws, nws, ws = _ws(ws, device, dev, "rs_fp8_linear_backward_ws_bytes", M, N)
    _check(lib().rs_fp8_linear_backward(pdy, lddy, M, N, K, px, ldx, sx, pw, ldw, sw, pdx, K, pdw,
                                        K, _DTYPES[dw_dtype], pdb, pws, nws, _stream(None)),
           "rs_fp8_linear_backward")
    return dx, dw, db


def rs_mlp_forward_fp8(x: torch.Tensor, w1: Fp8, b1, w2: Fp8, b2, gamma, beta,
                       out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """rs_mlp_forward with W1 [H, C] and W2 [C, H] held in 8-bit blocks and both products in 8
    bits: x [..., C] bf16 -> x + MLP(LN(x)), same shape. out may be x."""
    if stream is not None:
        return _on(stream, rs_mlp_forward_fp8, x, w1, b1, w2, b2, gamma, beta, out, ws)
    C, H, bf = w1.K, w1.rows, torch.bfloat16
    dev = _device(x, "x")
    px, ldx, M = _rows(x, "x", dev, bf, C)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    p1, ld1, s1 = _fp8(w1, "w1", dev)
    p2, ld2, s2 = _fp8(w2, "w2", dev, C, H)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr() or None
    elif not out.is_contiguous():
        raise ValueError("out must be contiguous")
    else:
        po = _rows(out, "out", dev, bf, C, M)[0]
    pws, nws, ws = _ws(ws, x.device, dev, "rs_mlp_forward_fp8_ws_bytes", M, C, H)
    st = lib().rs_mlp_forward_fp8(px, M, C, H, p1, ld1, s1, _vec(b1, "b1", dev, H, bf), p2, ld2, s2,
                                  _vec(b2, "b2", dev, C, bf), _vec(gamma, "gamma", dev, C, bf),
                                  _vec(beta, "beta", dev, C, bf), po, pws, nws, _stream(None))
    _check(st, "rs_mlp_forward_fp8")
    return out


def rs_debug_fp8_skip_load(a: Fp8, b: Fp8, out, skip_kblock: int, timeout_us: int,
                           stream=None) -> None:
    """Test hook: rs_fp8_gemm with one K block's load withheld (see include/rs.h)."""
    M, N, K = a.rows, b.rows, a.K
    dev = _device(a.q, "a")
    pa, lda, sa = _fp8(a, "a", dev)
    pb, ldb, sb = _fp8(b, "b", dev, K=K)
    if isinstance(out, Fp8):
        po, ldo, so = _fp8(out, "out", dev, M, N)
        dt = RS_E4M3
    else:
        po, ldo, _ = _rows(out, "out", dev, None, N, M)
        so, dt = None, _float_type(out)
    _check(lib().rs_debug_fp8_skip_load(pa, lda, sa, pb, ldb, sb, M, N, K, po, ldo, dt, so,
                                        int(skip_kblock), int(timeout_us), _stream(stream)),
           "rs_debug_fp8_skip_load")


def rs_debug_fp8_linear_skip_load(x: torch.Tensor, w: Fp8, out: torch.Tensor, timeout_us: int,
                                  stream=None) -> None:
    """Test hook: rs_fp8_linear on a few rows with one weight tile withheld (see include/rs.h)."""
    dev = _device(x, "x")
    px, ldx, M = _rows(x, "x", dev, torch.bfloat16, w.K)
    pw, ldw, sw = _fp8(w, "w", dev)
    po, ldo, _ = _rows(out, "out", dev, torch.bfloat16, w.rows, M)
    _check(lib().rs_debug_fp8_linear_skip_load(px, ldx, M, w.K, w.rows, pw, ldw, sw, po, ldo,
                                               int(timeout_us), _stream(stream)),
           "rs_debug_fp8_linear_skip_load")
