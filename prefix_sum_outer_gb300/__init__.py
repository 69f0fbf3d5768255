"""GB300-native causal dot product (causal linear attention's prefix sum).

Python face of ``libcausal_product.so`` (C ABI in ``include/causal_product.h``).
This module only marshals arguments: every step of the computation runs in
the library's CUDA kernels.  PyTorch supplies device memory and streams.

    out = causal_product(q, k, v)              # autograd-aware
    causal_product_fwd(q, k, v, out)           # raw entry points, same names
    causal_product_bwd(q, k, v, g, dq, dk, dv) #   as the C ABI

q, k: [B, H, N, D]; v: [B, H, N, M]; all contiguous, on one CUDA device,
dtype float32, bfloat16 or float16 (fp16 runs on the fp32 path, widened on
load).  out_i = sum_{j<=i} (q_i . k_j) v_j.

There is no fallback: if the library cannot be built or loaded, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import build as _build

__all__ = [
    "CP_OK", "CausalProductError", "causal_product", "causal_product_fwd", "causal_product_bwd",
    "causal_product_fwd_noalloc", "causal_product_noalloc_status", "causal_product_decode",
    "causal_product_normalizer", "causal_product_normalizer_bwd", "normalizer",
    "causal_product_fwd_norm",
    "causal_product_fwd_feature", "causal_product_bwd_feature", "FEATURES",
    "causal_product_workspace_size", "causal_product_feature_workspace_size",
    "causal_product_launch_count", "causal_product_status",
    "causal_product_checkpoint_size", "causal_product_fwd_ckpt", "causal_product_bwd_ckpt",
    "causal_product_fwd_favor", "causal_product_bwd_favor", "causal_product_favor",
    "causal_product_fwd_delta", "causal_product_bwd_delta", "causal_product_delta",
    "causal_product_decode_delta", "causal_product_delta_workspace_size",
    "causal_product_delta_checkpoint_size",
    "causal_product_qk_rope", "causal_product_qk_rope_bwd", "qk_rope", "QK_NORMS",
    "causal_product_fwd_decay", "causal_product_bwd_decay", "causal_product_decay",
    "causal_product_decode_decay", "causal_product_decay_workspace_size",
    "causal_product_layer_norm", "causal_product_layer_norm_bwd", "layer_norm",
    "causal_product_layer_norm_workspace_size",
    "causal_product_error_string", "library_path", "load_library",
]

CP_DTYPE_F32, CP_DTYPE_BF16, CP_DTYPE_F16 = 0, 1, 2
CP_OK = 0
CP_ERR_TIMEOUT = 7
_DTYPES = {torch.float32: CP_DTYPE_F32, torch.bfloat16: CP_DTYPE_BF16,
           torch.float16: CP_DTYPE_F16}
# feature maps applied to q and k inside the kernels (cp_feature_t)
FEATURES = {None: 0, "none": 0, "elu1": 1}

# norms of queries and keys (cp_qk_norm_t)
QK_NORMS = {"rms": 0, "l2": 1}


def _feature_code(feature) -> int:
    if feature not in FEATURES:
        raise ValueError(f"unknown feature map {feature!r}; expected one of {list(FEATURES)}")
    return FEATURES[feature]

_lib = None
_lock = threading.Lock()


class CausalProductError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {causal_product_error_string(code)}")


def library_path() -> str:
    return _build.LIB


def load_library(rebuild: bool = True) -> ctypes.CDLL:
    """Load the C ABI library (building it first if its sources changed)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if rebuild else _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libcausal_product.so not found at {path}")
            lib = ctypes.CDLL(path)
            p, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            lib.causal_product_workspace_size.argtypes = [i64, i64, i64, i64, i64, c_int, c_int]
            lib.causal_product_workspace_size.restype = sz
            lib.causal_product_launch_count.argtypes = [i64, i64, i64, i64, i64, c_int, c_int]
            lib.causal_product_launch_count.restype = c_int
            lib.causal_product_fwd.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, c_int, p, sz, p]
            lib.causal_product_fwd.restype = c_int
            lib.causal_product_bwd.argtypes = [p, p, p, p, p, p, p, i64, i64, i64, i64, i64, c_int,
                                               p, sz, p]
            lib.causal_product_bwd.restype = c_int
            lib.causal_product_checkpoint_size.argtypes = [i64, i64, i64, i64, i64, c_int]
            lib.causal_product_checkpoint_size.restype = sz
            lib.causal_product_fwd_ckpt.argtypes = [p, p, p, p, p, sz, i64, i64, i64, i64, i64,
                                                    c_int, p, sz, p]
            lib.causal_product_fwd_ckpt.restype = c_int
            lib.causal_product_bwd_ckpt.argtypes = [p, p, p, p, p, sz, p, p, p, i64, i64, i64,
                                                    i64, i64, c_int, p, sz, p]
            lib.causal_product_bwd_ckpt.restype = c_int
            lib.causal_product_fwd_state.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, i64,
                                                     c_int, p, sz, p]
            lib.causal_product_fwd_state.restype = c_int
            lib.causal_product_bwd_state.argtypes = [p, p, p, p, p, p, p, p, p, p, i64, i64, i64,
                                                     i64, i64, c_int, p, sz, p]
            lib.causal_product_bwd_state.restype = c_int
            lib.causal_product_selftest_timeout.argtypes = [p, ctypes.c_uint64, p]
            lib.causal_product_selftest_timeout.restype = c_int
            lib.causal_product_decode.argtypes = [p, p, p, p, p, i64, i64, i64, i64, c_int, p]
            lib.causal_product_decode.restype = c_int
            lib.causal_product_fwd_noalloc.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, c_int,
                                                       p]
            lib.causal_product_fwd_noalloc.restype = c_int
            lib.causal_product_noalloc_status.argtypes = [p]
            lib.causal_product_noalloc_status.restype = c_int
            lib.causal_product_normalizer_workspace_size.argtypes = [i64, i64, i64, i64, c_int]
            lib.causal_product_normalizer_workspace_size.restype = sz
            lib.causal_product_fwd_norm_workspace_size.argtypes = [i64, i64, i64, i64, i64, c_int]
            lib.causal_product_fwd_norm_workspace_size.restype = sz
            lib.causal_product_fwd_norm.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i64, c_int,
                                                    p, sz, p]
            lib.causal_product_fwd_norm.restype = c_int
            lib.causal_product_normalizer.argtypes = [p, p, p, i64, i64, i64, i64, c_int, p, sz, p]
            lib.causal_product_normalizer.restype = c_int
            lib.causal_product_normalizer_bwd.argtypes = [p, p, p, p, p, i64, i64, i64, i64, c_int,
                                                          p, sz, p]
            lib.causal_product_normalizer_bwd.restype = c_int
            lib.causal_product_fwd_feature.argtypes = [p, p, p, p, c_int, i64, i64, i64, i64, i64,
                                                       c_int, p, sz, p]
            lib.causal_product_fwd_feature.restype = c_int
            lib.causal_product_bwd_feature.argtypes = [p, p, p, p, p, p, p, c_int, i64, i64, i64,
                                                       i64, i64, c_int, p, sz, p]
            lib.causal_product_bwd_feature.restype = c_int
            lib.causal_product_feature_workspace_size.argtypes = [i64, i64, i64, i64, i64, c_int,
                                                                  c_int]
            lib.causal_product_feature_workspace_size.restype = sz
            lib.causal_product_normalizer_feature.argtypes = [p, p, p, c_int, i64, i64, i64, i64,
                                                              c_int, p, sz, p]
            lib.causal_product_normalizer_feature.restype = c_int
            lib.causal_product_normalizer_bwd_feature.argtypes = [p, p, p, p, p, c_int, i64, i64,
                                                                  i64, i64, c_int, p, sz, p]
            lib.causal_product_normalizer_bwd_feature.restype = c_int
            lib.causal_product_favor_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64,
                                                                c_int, c_int]
            lib.causal_product_favor_workspace_size.restype = sz
            lib.causal_product_fwd_favor.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i64, i64,
                                                     c_int, p, sz, p]
            lib.causal_product_fwd_favor.restype = c_int
            lib.causal_product_bwd_favor.argtypes = [p, p, p, p, p, p, p, p, i64, i64, i64, i64,
                                                     i64, i64, c_int, p, sz, p]
            lib.causal_product_bwd_favor.restype = c_int
            f32 = ctypes.c_float
            lib.causal_product_delta_workspace_size.argtypes = [i64] * 6 + [c_int, c_int]
            lib.causal_product_delta_workspace_size.restype = sz
            lib.causal_product_delta_checkpoint_size.argtypes = [i64] * 6 + [c_int]
            lib.causal_product_delta_checkpoint_size.restype = sz
            lib.causal_product_fwd_delta.argtypes = ([p] * 9 + [sz, f32] + [i64] * 6
                                                     + [c_int, p, sz, p])
            lib.causal_product_fwd_delta.restype = c_int
            lib.causal_product_bwd_delta.argtypes = ([p] * 7 + [sz] + [p] * 7 + [f32] + [i64] * 6
                                                     + [c_int, p, sz, p])
            lib.causal_product_bwd_delta.restype = c_int
            lib.causal_product_decode_delta.argtypes = [p] * 8 + [i64, f32] + [i64] * 5 + [c_int, p]
            lib.causal_product_decode_delta.restype = c_int
            p64 = ctypes.POINTER(i64)
            lib.causal_product_qk_rope.argtypes = ([p, p64, p, p64, p, p, p, p, i64, p, p, c_int, f32]
                                                   + [i64] * 6 + [c_int, p])
            lib.causal_product_qk_rope.restype = c_int
            lib.causal_product_qk_rope_workspace_size.argtypes = [i64] * 5 + [c_int]
            lib.causal_product_qk_rope_workspace_size.restype = sz
            lib.causal_product_qk_rope_bwd.argtypes = ([p, p64, p, p64, p, p, p, p, i64] + [p] * 6
                                                       + [c_int, f32] + [i64] * 6 + [c_int, p, sz, p])
            lib.causal_product_qk_rope_bwd.restype = c_int
            lib.causal_product_decay_workspace_size.argtypes = [i64] * 6 + [c_int, c_int]
            lib.causal_product_decay_workspace_size.restype = sz
            lib.causal_product_fwd_decay.argtypes = [p] * 8 + [f32] + [i64] * 6 + [c_int, p, sz, p]
            lib.causal_product_fwd_decay.restype = c_int
            lib.causal_product_bwd_decay.argtypes = [p] * 12 + [f32] + [i64] * 6 + [c_int, p, sz, p]
            lib.causal_product_bwd_decay.restype = c_int
            lib.causal_product_decode_decay.argtypes = [p] * 7 + [i64, f32] + [i64] * 5 + [c_int, p]
            lib.causal_product_decode_decay.restype = c_int
            lib.causal_product_layer_norm.argtypes = ([p, p64, p, p, c_int, p, c_int, f32] + [i64] * 4
                                                      + [c_int, p])
            lib.causal_product_layer_norm.restype = c_int
            lib.causal_product_layer_norm_workspace_size.argtypes = [i64] * 4 + [c_int]
            lib.causal_product_layer_norm_workspace_size.restype = sz
            lib.causal_product_layer_norm_bwd.argtypes = ([p, p64, p, c_int, p, c_int] + [p] * 3 + [f32]
                                                          + [i64] * 4 + [c_int, p, sz, p])
            lib.causal_product_layer_norm_bwd.restype = c_int
            lib.causal_product_status.argtypes = [p, p]
            lib.causal_product_status.restype = c_int
            lib.causal_product_error_string.argtypes = [c_int]
            lib.causal_product_error_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def causal_product_error_string(code: int) -> str:
    return load_library().causal_product_error_string(int(code)).decode()


def _dims(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError(f"expected q,k [B,H,N,D] and v [B,H,N,M]; got {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")
    B, H, N, D = q.shape
    return B, H, N, D, v.shape[3]


def _dtype_code(*ts: torch.Tensor) -> int:
    dt = ts[0].dtype
    if dt not in _DTYPES or any(t.dtype != dt for t in ts):
        raise TypeError(f"all tensors must share one dtype in {list(_DTYPES)}; "
                        f"got {[t.dtype for t in ts]}")
    return _DTYPES[dt]


def _check_device(*ts: torch.Tensor):
    dev = ts[0].device
    if dev.type != "cuda":
        raise RuntimeError("causal_product runs on CUDA tensors only (no CPU path)")
    for t in ts:
        if t.device != dev:
            raise RuntimeError("all tensors must be on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _check_like(t: torch.Tensor, shape, dtype: torch.dtype, name: str):
    """A caller-provided output must have exactly the shape and dtype the
    kernels write: the C ABI receives only its pointer, so a smaller buffer
    would be written past its end."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}; "
                         f"got {t.dtype} {tuple(t.shape)}")


def _stream_ptr(stream: Optional[torch.cuda.Stream], device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


def causal_product_workspace_size(B: int, H: int, N: int, D: int, M: int,
                                  dtype: torch.dtype = torch.bfloat16,
                                  backward: bool = False) -> int:
    return int(load_library().causal_product_workspace_size(B, H, N, D, M, _DTYPES[dtype],
                                                            int(bool(backward))))


def causal_product_feature_workspace_size(B: int, H: int, N: int, D: int, M: int,
                                          dtype: torch.dtype = torch.bfloat16,
                                          backward: bool = False) -> int:
    """Workspace bytes of causal_product_fwd_feature / _bwd_feature."""
    return int(load_library().causal_product_feature_workspace_size(
        B, H, N, D, M, _DTYPES[dtype], int(bool(backward))))


def causal_product_launch_count(B: int, H: int, N: int, D: int, M: int,
                                dtype: torch.dtype = torch.bfloat16,
                                backward: bool = False, ckpt: bool = False,
                                norm: bool = False) -> int:
    """Kernels one causal_product_fwd (or, with ``backward``, _bwd; with
    ``ckpt``, the checkpoint calls; with ``norm``, causal_product_fwd_norm)
    launches for this shape; -1 for a shape the entry points reject."""
    mode = 4 if norm else int(bool(backward)) + (2 if ckpt else 0)
    return int(load_library().causal_product_launch_count(B, H, N, D, M, _DTYPES[dtype], mode))


def causal_product_checkpoint_size(B: int, H: int, N: int, D: int, M: int,
                                   dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of the checkpoint buffer of causal_product_fwd_ckpt (0: none)."""
    return int(load_library().causal_product_checkpoint_size(B, H, N, D, M, _DTYPES[dtype]))


def _ckpt_buffer(B, H, N, D, M, dtype, device, ckpt):
    n = causal_product_checkpoint_size(B, H, N, D, M, dtype)
    if ckpt is None:
        ckpt = torch.empty(max(n // 4, 1), dtype=torch.float32, device=device)
    if ckpt.dtype != torch.float32 or ckpt.numel() * 4 < n or not ckpt.is_contiguous():
        raise ValueError(f"ckpt must be a contiguous float32 tensor of at least {n} bytes")
    return ckpt


def causal_product_fwd_ckpt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            out: Optional[torch.Tensor] = None,
                            ckpt: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None):
    """The forward that also writes checkpoints of the state for the
    backward (causal_product_bwd_ckpt); returns (out, ckpt)."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    _check_like(out, (B, H, N, M), q.dtype, "out")
    _check_device(q, k, v, out)
    ckpt = _ckpt_buffer(B, H, N, D, M, q.dtype, q.device, ckpt)
    _check_device(q, ckpt)
    lib = load_library()
    need = lib.causal_product_workspace_size(B, H, N, D, M, code, 0)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_fwd_ckpt(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     ckpt.data_ptr(), ckpt.numel() * 4, B, H, N, D, M, code,
                                     workspace.data_ptr(), workspace.numel(),
                                     _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_ckpt")
    return out, ckpt


def causal_product_bwd_ckpt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            grad_out: torch.Tensor, ckpt: torch.Tensor,
                            grad_q: Optional[torch.Tensor] = None,
                            grad_k: Optional[torch.Tensor] = None,
                            grad_v: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None):
    """(dq, dk, dv) of L = <grad_out, out>, the dq scans seeded from the
    checkpoints causal_product_fwd_ckpt wrote for the same q, k, v."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k"), (grad_v, v, "grad_v")):
        _check_like(t, ref.shape, ref.dtype, name)
    _check_device(q, k, v, grad_out, grad_q, grad_k, grad_v)
    ckpt = _ckpt_buffer(B, H, N, D, M, q.dtype, q.device, ckpt)
    _check_device(q, ckpt)
    lib = load_library()
    need = lib.causal_product_workspace_size(B, H, N, D, M, code, 1)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_bwd_ckpt(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     grad_out.data_ptr(), ckpt.data_ptr(), ckpt.numel() * 4,
                                     grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(),
                                     B, H, N, D, M, code, workspace.data_ptr(),
                                     workspace.numel(), _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd_ckpt")
    return grad_q, grad_k, grad_v


def _workspace(nbytes: int, device) -> torch.Tensor:
    # the status word at its start must begin at zero (it is sticky)
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _state_arg(t: Optional[torch.Tensor], shape, device, name: str) -> int:
    """Device pointer of an optional fp32 [B,H,D,M] state tensor (0 if None)."""
    if t is None:
        return 0
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be float32 of shape {tuple(shape)}; "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    return t.data_ptr()


def causal_product_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None,
                       state_in: Optional[torch.Tensor] = None,
                       return_state: bool = False,
                       state_out: Optional[torch.Tensor] = None):
    """out[b,h,i] = (S_0 + sum_{j<=i} k[b,h,j] v[b,h,j]^T)^T q[b,h,i], enqueued
    on ``stream``.  ``state_in`` is S_0 (float32 [B,H,D,M], None = zero);
    with ``return_state`` the result is (out, S_N), S_N the state after the
    last row (written into ``state_out`` when given)."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    _check_like(out, (B, H, N, M), q.dtype, "out")
    _check_device(q, k, v, out)
    if return_state and state_out is None:
        state_out = torch.empty((B, H, D, M), dtype=torch.float32, device=q.device)
    lib = load_library()
    need = lib.causal_product_workspace_size(B, H, N, D, M, code, 0)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_fwd_state(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        _state_arg(state_in, (B, H, D, M), q.device, "state_in"),
        _state_arg(state_out, (B, H, D, M), q.device, "state_out"),
        B, H, N, D, M, code, workspace.data_ptr(), workspace.numel(),
        _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd")
    return (out, state_out) if return_state else out


def causal_product_fwd_feature(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               feature: str = "elu1", out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out_i = sum_{j<=i} (phi(q_i) . phi(k_j)) v_j with phi applied inside the
    kernels (``feature="elu1"``: phi(x) = elu(x) + 1); q and k are the raw
    inputs."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    _check_like(out, (B, H, N, M), q.dtype, "out")
    _check_device(q, k, v, out)
    lib = load_library()
    need = lib.causal_product_feature_workspace_size(B, H, N, D, M, code, 0)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_fwd_feature(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                        _feature_code(feature), B, H, N, D, M, code,
                                        workspace.data_ptr(), workspace.numel(),
                                        _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_feature")
    return out


def causal_product_bwd_feature(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               grad_out: torch.Tensor, feature: str = "elu1",
                               grad_q: Optional[torch.Tensor] = None,
                               grad_k: Optional[torch.Tensor] = None,
                               grad_v: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None):
    """(dq, dk, dv) of L = <grad_out, out> for causal_product_fwd_feature,
    with respect to the raw q, k and v."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k"), (grad_v, v, "grad_v")):
        _check_like(t, ref.shape, ref.dtype, name)
    _check_device(q, k, v, grad_out, grad_q, grad_k, grad_v)
    lib = load_library()
    need = lib.causal_product_feature_workspace_size(B, H, N, D, M, code, 1)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_bwd_feature(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        grad_out.data_ptr(), grad_q.data_ptr(), grad_k.data_ptr(),
                                        grad_v.data_ptr(), _feature_code(feature), B, H, N, D, M,
                                        code, workspace.data_ptr(), workspace.numel(),
                                        _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd_feature")
    return grad_q, grad_k, grad_v


def causal_product_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               out: torch.Tensor,
                               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Forward pass through the library's allocation-free entry point.

    For callers that must not allocate device memory (their host framework
    owns all device allocations, or they cannot afford an implicit device
    synchronisation): the library uses a fixed static scratch array instead
    of a workspace, so ``out`` must be provided.  Calls that overlap on the
    GPU share that array and race; order them on one stream.
    """
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v, out)
    _check_like(out, (B, H, N, M), q.dtype, "out")
    _check_device(q, k, v, out)
    rc = load_library().causal_product_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                   out.data_ptr(), B, H, N, D, M, code,
                                                   _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_noalloc")
    return out


def _favor_dims(xq: torch.Tensor, xk: torch.Tensor, v: torch.Tensor, W: torch.Tensor):
    if (xq.dim() != 4 or xk.shape != xq.shape or v.dim() != 4 or v.shape[:3] != xq.shape[:3]
            or W.dim() != 2 or W.shape[1] != xq.shape[3]):
        raise ValueError(f"expected xq, xk [B,H,N,R], v [B,H,N,M], W [D,R]; got {tuple(xq.shape)}, "
                         f"{tuple(xk.shape)}, {tuple(v.shape)}, {tuple(W.shape)}")
    B, H, N, R = xq.shape
    return B, H, N, R, W.shape[0], v.shape[3]


def causal_product_fwd_favor(xq: torch.Tensor, xk: torch.Tensor, v: torch.Tensor,
                             W: torch.Tensor, out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out_i = sum_{j<=i} (phi(xq_i) . phi(xk_j)) v_j with the positive random
    features phi(x) = exp(W x - |x|^2 / 2) / sqrt(D), computed in the kernels
    from the raw rows xq, xk [B,H,N,R] and the projection W [D,R] (bf16)."""
    B, H, N, R, D, M = _favor_dims(xq, xk, v, W)
    code = _dtype_code(xq, xk, v, W)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=v.dtype, device=v.device)
    _check_like(out, (B, H, N, M), v.dtype, "out")
    _check_device(xq, xk, v, W, out)
    lib = load_library()
    need = lib.causal_product_favor_workspace_size(B, H, N, R, D, M, code, 0)
    if workspace is None:
        workspace = _workspace(need, v.device)
    rc = lib.causal_product_fwd_favor(xq.data_ptr(), xk.data_ptr(), v.data_ptr(), W.data_ptr(),
                                      out.data_ptr(), B, H, N, R, D, M, code,
                                      workspace.data_ptr(), workspace.numel(),
                                      _stream_ptr(stream, v.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_favor")
    return out


def causal_product_bwd_favor(xq: torch.Tensor, xk: torch.Tensor, v: torch.Tensor,
                             W: torch.Tensor, grad_out: torch.Tensor,
                             grad_xq: Optional[torch.Tensor] = None,
                             grad_xk: Optional[torch.Tensor] = None,
                             grad_v: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None):
    """(dxq, dxk, dv) of L = <grad_out, out> for causal_product_fwd_favor (W
    fixed)."""
    B, H, N, R, D, M = _favor_dims(xq, xk, v, W)
    code = _dtype_code(xq, xk, v, W, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    grad_xq = torch.empty_like(xq) if grad_xq is None else grad_xq
    grad_xk = torch.empty_like(xk) if grad_xk is None else grad_xk
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    for t, ref, name in ((grad_xq, xq, "grad_xq"), (grad_xk, xk, "grad_xk"), (grad_v, v, "grad_v")):
        _check_like(t, ref.shape, ref.dtype, name)
    _check_device(xq, xk, v, W, grad_out, grad_xq, grad_xk, grad_v)
    lib = load_library()
    need = lib.causal_product_favor_workspace_size(B, H, N, R, D, M, code, 1)
    if workspace is None:
        workspace = _workspace(need, v.device)
    rc = lib.causal_product_bwd_favor(xq.data_ptr(), xk.data_ptr(), v.data_ptr(), W.data_ptr(),
                                      grad_out.data_ptr(), grad_xq.data_ptr(), grad_xk.data_ptr(),
                                      grad_v.data_ptr(), B, H, N, R, D, M, code,
                                      workspace.data_ptr(), workspace.numel(),
                                      _stream_ptr(stream, v.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd_favor")
    return grad_xq, grad_xk, grad_v


def causal_product_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, grad_out: torch.Tensor,
                       grad_q: Optional[torch.Tensor] = None,
                       grad_k: Optional[torch.Tensor] = None,
                       grad_v: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None,
                       state_in: Optional[torch.Tensor] = None,
                       grad_state_out: Optional[torch.Tensor] = None,
                       return_state_grad: bool = False,
                       grad_state_in: Optional[torch.Tensor] = None):
    """(dq, dk, dv) of L = <grad_out, out> + <grad_state_out, S_N> for the
    forward from ``state_in`` (S_0; both float32 [B,H,D,M], None = zero).
    With ``return_state_grad`` the result is (dq, dk, dv, dL/dS_0), the last
    written into ``grad_state_in`` when given."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k"), (grad_v, v, "grad_v")):
        _check_like(t, ref.shape, ref.dtype, name)
    _check_device(q, k, v, grad_out, grad_q, grad_k, grad_v)
    if return_state_grad and grad_state_in is None:
        grad_state_in = torch.empty((B, H, D, M), dtype=torch.float32, device=q.device)
    lib = load_library()
    need = lib.causal_product_workspace_size(B, H, N, D, M, code, 1)
    if workspace is None:
        workspace = _workspace(need, q.device)
    shape = (B, H, D, M)
    rc = lib.causal_product_bwd_state(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), grad_out.data_ptr(),
        _state_arg(state_in, shape, q.device, "state_in"),
        _state_arg(grad_state_out, shape, q.device, "grad_state_out"),
        grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(),
        _state_arg(grad_state_in, shape, q.device, "grad_state_in"),
        B, H, N, D, M, code, workspace.data_ptr(), workspace.numel(),
        _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd")
    if return_state_grad:
        return grad_q, grad_k, grad_v, grad_state_in
    return grad_q, grad_k, grad_v


def causal_product_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          state: torch.Tensor, out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decoding step: state <- state + k v^T (in place), out = state^T q.

    q, k: [B,H,D]; v: [B,H,M]; state: float32 [B,H,D,M]."""
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError(f"expected q,k [B,H,D] and v [B,H,M]; got {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")
    B, H, D = q.shape
    M = v.shape[2]
    code = _dtype_code(q, k, v)
    if out is None:
        out = torch.empty((B, H, M), dtype=q.dtype, device=q.device)
    _check_like(out, (B, H, M), q.dtype, "out")
    _check_device(q, k, v, out, state)
    _state_arg(state, (B, H, D, M), q.device, "state")
    rc = load_library().causal_product_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                              out.data_ptr(), state.data_ptr(), B, H, D, M, code,
                                              _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_decode")
    return out


def _qk_dims(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 4 or k.shape != q.shape:
        raise ValueError(f"expected q,k [B,H,N,D]; got {tuple(q.shape)}, {tuple(k.shape)}")
    return tuple(q.shape)


def causal_product_normalizer(q: torch.Tensor, k: torch.Tensor,
                              z: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None,
                              feature: Optional[str] = None) -> torch.Tensor:
    """z[b,h,i] = q[b,h,i] . sum_{j<=i} k[b,h,j] (float32 [B,H,N]): the
    denominator of causal linear attention.  With ``feature="elu1"`` q and k
    are raw inputs mapped by phi(x) = elu(x) + 1 inside the kernel."""
    B, H, N, D = _qk_dims(q, k)
    code = _dtype_code(q, k)
    if z is None:
        z = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if z.dtype != torch.float32 or tuple(z.shape) != (B, H, N):
        raise ValueError(f"z must be float32 of shape {(B, H, N)}")
    _check_device(q, k, z)
    lib = load_library()
    need = lib.causal_product_normalizer_workspace_size(B, H, N, D, code)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_normalizer_feature(q.data_ptr(), k.data_ptr(), z.data_ptr(),
                                               _feature_code(feature), B, H, N, D, code,
                                               workspace.data_ptr(), workspace.numel(),
                                               _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_normalizer")
    return z


def causal_product_fwd_norm(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            out: Optional[torch.Tensor] = None,
                            z: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None):
    """(out, z): the causal product and its normaliser z[b,h,i] = q[b,h,i] .
    sum_{j<=i} k[b,h,j] (float32 [B,H,N]) in one call; one kernel launch for
    bf16 with D, M <= 64 on unsplit problems."""
    B, H, N, D, M = _dims(q, k, v)
    code = _dtype_code(q, k, v)
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    _check_like(out, (B, H, N, M), q.dtype, "out")
    if z is None:
        z = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_like(z, (B, H, N), torch.float32, "z")
    _check_device(q, k, v, out, z)
    lib = load_library()
    need = lib.causal_product_fwd_norm_workspace_size(B, H, N, D, M, code)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_fwd_norm(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     z.data_ptr(), B, H, N, D, M, code, workspace.data_ptr(),
                                     workspace.numel(), _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_norm")
    return out, z


def causal_product_normalizer_bwd(q: torch.Tensor, k: torch.Tensor, grad_z: torch.Tensor,
                                  grad_q: Optional[torch.Tensor] = None,
                                  grad_k: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None,
                                  feature: Optional[str] = None):
    """(dq, dk) of L = <grad_z, z>: dq_i = grad_z_i sum_{j<=i} k_j,
    dk_j = sum_{i>=j} grad_z_i q_i, in q's dtype (with ``feature``, with
    respect to the raw q, k: times phi')."""
    B, H, N, D = _qk_dims(q, k)
    code = _dtype_code(q, k)
    if grad_z.dtype != torch.float32 or tuple(grad_z.shape) != (B, H, N):
        raise ValueError(f"grad_z must be float32 of shape {(B, H, N)}")
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k")):
        _check_like(t, ref.shape, ref.dtype, name)
    _check_device(q, k, grad_z, grad_q, grad_k)
    lib = load_library()
    need = lib.causal_product_normalizer_workspace_size(B, H, N, D, code)
    if workspace is None:
        workspace = _workspace(need, q.device)
    rc = lib.causal_product_normalizer_bwd_feature(q.data_ptr(), k.data_ptr(), grad_z.data_ptr(),
                                                   grad_q.data_ptr(), grad_k.data_ptr(),
                                                   _feature_code(feature), B, H, N, D, code,
                                                   workspace.data_ptr(), workspace.numel(),
                                                   _stream_ptr(stream, q.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_normalizer_bwd")
    return grad_q, grad_k


def causal_product_selftest_timeout(workspace: torch.Tensor, wait_ns: int = 20_000_000,
                                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the failure-path self-test: a bounded wait that runs out and
    records CP_ERR_TIMEOUT in ``workspace``'s status word (read it with
    causal_product_status)."""
    rc = load_library().causal_product_selftest_timeout(workspace.data_ptr(), int(wait_ns),
                                                        _stream_ptr(stream, workspace.device))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_selftest_timeout")


def causal_product_status(workspace: torch.Tensor,
                          stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise ``stream`` and return (and clear) the workspace status word."""
    return int(load_library().causal_product_status(workspace.data_ptr(),
                                                    _stream_ptr(stream, workspace.device)))


def causal_product_noalloc_status(stream: Optional[torch.cuda.Stream] = None,
                                  device=None) -> int:
    """Synchronise ``stream`` and return (and clear) the status word that
    every causal_product_fwd_noalloc call on the current device shares."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return int(load_library().causal_product_noalloc_status(_stream_ptr(stream, dev)))


def _raw_stream(device: int) -> int:
    # (torch.cuda.current_stream builds a Stream object: 2 us of a 10 us step)
    return torch._C._cuda_getCurrentRawStream(device)


def _elsewhere(t: torch.Tensor, stream: Optional[torch.cuda.Stream]):
    """What a call on t's device has to enter first: the named stream, to which
    what it allocates then belongs, or the device where it is not the current
    one (a kernel starts on the current device).  None: nothing."""
    device = t.get_device()
    if stream is not None:
        if device >= 0 and stream.device.index != device:
            raise RuntimeError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
        return torch.cuda.stream(stream)
    if device >= 0 and device != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return None


def _all_plain(device: int, *ts: torch.Tensor) -> bool:
    for t in ts:
        if t.get_device() != device or not t.is_contiguous():
            return False
    return device >= 0


def _check_plain(device: int, *ts: torch.Tensor):
    """_check_device, for the calls whose time is that of their checks."""
    if not _all_plain(device, *ts):
        _check_device(*ts)


def _delta_dims(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                beta: torch.Tensor):
    qs, vs = q.shape, v.shape
    if (len(qs) != 4 or k.shape != qs or len(vs) != 4 or vs[0] != qs[0] or vs[2] != qs[2]
            or qs[1] == 0 or vs[1] % qs[1] != 0):
        raise ValueError(f"expected q,k [B,Hk,N,D] and v [B,H,N,M], H a multiple of Hk; got "
                         f"{tuple(qs)}, {tuple(k.shape)}, {tuple(vs)}")
    B, Hk, N, D = qs
    H, M = vs[1], vs[3]
    for t, name in ((g, "g"), (beta, "beta")):
        if t.shape != (B, H, N) or t.dtype is not torch.float32:
            _check_like(t, (B, H, N), torch.float32, name)
    return B, H, Hk, N, D, M


def causal_product_delta_workspace_size(B: int, H: int, Hk: int, N: int, D: int, M: int,
                                        dtype: torch.dtype = torch.bfloat16,
                                        backward: bool = False) -> int:
    """Workspace bytes of causal_product_fwd_delta / _bwd_delta."""
    return int(load_library().causal_product_delta_workspace_size(B, H, Hk, N, D, M, _DTYPES[dtype],
                                                                  int(bool(backward))))


def causal_product_delta_checkpoint_size(B: int, H: int, Hk: int, N: int, D: int, M: int,
                                         dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of the states causal_product_fwd_delta keeps for the backward."""
    return int(load_library().causal_product_delta_checkpoint_size(B, H, Hk, N, D, M,
                                                                   _DTYPES[dtype]))


def _delta_workspace(workspace: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    # with no workspace of the caller's nobody reads the status word, so it
    # need not begin at zero
    if workspace is None:
        return torch.empty(max(int(need), 256), dtype=torch.uint8, device=device)
    if workspace.device != device:
        raise RuntimeError(f"workspace must be on {device}; got one on {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def causal_product_fwd_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                             beta: torch.Tensor, out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None,
                             state_in: Optional[torch.Tensor] = None, return_state: bool = False,
                             state_out: Optional[torch.Tensor] = None, scale: float = 1.0,
                             save: bool = False, ckpt: Optional[torch.Tensor] = None):
    """The gated delta rule: S_t = a_t S_{t-1} + k_t u_t^T with u_t = beta_t
    (v_t - a_t S_{t-1}^T k_t) and a_t = exp(g_t); out_t = scale S_t^T q_t.

    q, k: [B,Hk,N,D]; v: [B,H,N,M], value head h reading key head h // (H //
    Hk); g (log decay) and beta: float32 [B,H,N]; ``state_in`` is S_0 (float32
    [B,H,D,M], None = zero).  Returns out, followed by S_N with
    ``return_state`` and by the checkpoints causal_product_bwd_delta needs with
    ``save`` (written into ``ckpt`` when given)."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_fwd_delta(q, k, v, g, beta, out, workspace, None, state_in,
                                            return_state, state_out, scale, save, ckpt)
    B, H, Hk, N, D, M = _delta_dims(q, k, v, g, beta)
    code = _dtype_code(q, k, v)
    dev = v.get_device()
    if out is None:
        _check_plain(dev, q, k, v, g, beta)
        out = torch.empty_like(v)
    else:
        _check_like(out, (B, H, N, M), v.dtype, "out")
        _check_plain(dev, q, k, v, g, beta, out)
    if return_state and state_out is None:
        state_out = torch.empty((B, H, D, M), dtype=torch.float32, device=v.device)
    lib = load_library()
    if save or ckpt is not None:
        ckpt = _delta_ckpt(B, H, Hk, N, D, M, v, ckpt)
    need = lib.causal_product_delta_workspace_size(B, H, Hk, N, D, M, code, 0)
    workspace = _delta_workspace(workspace, need, v.device)
    rc = lib.causal_product_fwd_delta(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), out.data_ptr(),
        _state_arg(state_in, (B, H, D, M), v.device, "state_in"),
        _state_arg(state_out, (B, H, D, M), v.device, "state_out"),
        0 if ckpt is None else ckpt.data_ptr(), 0 if ckpt is None else ckpt.numel() * 4,
        float(scale), B, H, Hk, N, D, M, code, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_delta")
    got = (out,) + ((state_out,) if return_state else ()) + ((ckpt,) if save else ())
    return got if len(got) > 1 else out


def _delta_ckpt(B, H, Hk, N, D, M, v, ckpt):
    n = causal_product_delta_checkpoint_size(B, H, Hk, N, D, M, v.dtype)
    if ckpt is None:
        ckpt = torch.empty(max(n // 4, 1), dtype=torch.float32, device=v.device)
    if ckpt.dtype != torch.float32 or ckpt.numel() * 4 < n:
        raise ValueError(f"ckpt must be a contiguous float32 tensor of at least {n} bytes")
    _check_device(v, ckpt)
    return ckpt


def causal_product_bwd_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                             beta: torch.Tensor, grad_out: torch.Tensor, ckpt: torch.Tensor,
                             grad_q: Optional[torch.Tensor] = None,
                             grad_k: Optional[torch.Tensor] = None,
                             grad_v: Optional[torch.Tensor] = None,
                             grad_g: Optional[torch.Tensor] = None,
                             grad_beta: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None, scale: float = 1.0,
                             grad_state_out: Optional[torch.Tensor] = None,
                             return_state_grad: bool = False,
                             grad_state_in: Optional[torch.Tensor] = None):
    """(dq, dk, dv, dg, dbeta) of L = <grad_out, out> + <grad_state_out, S_N>
    for causal_product_fwd_delta(..., save=True) on the same inputs, ``ckpt``
    being the checkpoints it returned; with ``return_state_grad`` dL/dS_0
    follows.  dq and dk are summed over the value heads of a key head."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_bwd_delta(q, k, v, g, beta, grad_out, ckpt, grad_q, grad_k, grad_v,
                                            grad_g, grad_beta, workspace, None, scale,
                                            grad_state_out, return_state_grad, grad_state_in)
    B, H, Hk, N, D, M = _delta_dims(q, k, v, g, beta)
    code = _dtype_code(q, k, v, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    outs = []
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k"), (grad_v, v, "grad_v"),
                         (grad_g, g, "grad_g"), (grad_beta, beta, "grad_beta")):
        t = torch.empty_like(ref) if t is None else t
        _check_like(t, ref.shape, ref.dtype, name)
        outs.append(t)
    dev = v.get_device()
    _check_plain(dev, q, k, v, g, beta, grad_out, *outs)
    if return_state_grad and grad_state_in is None:
        grad_state_in = torch.empty((B, H, D, M), dtype=torch.float32, device=v.device)
    if ckpt is None:
        raise ValueError("ckpt must be the checkpoints causal_product_fwd_delta returned")
    ckpt = _delta_ckpt(B, H, Hk, N, D, M, v, ckpt)
    lib = load_library()
    need = lib.causal_product_delta_workspace_size(B, H, Hk, N, D, M, code, 1)
    workspace = _delta_workspace(workspace, need, v.device)
    shape = (B, H, D, M)
    rc = lib.causal_product_bwd_delta(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        grad_out.data_ptr(), ckpt.data_ptr(), ckpt.numel() * 4,
        _state_arg(grad_state_out, shape, v.device, "grad_state_out"),
        *(t.data_ptr() for t in outs),
        _state_arg(grad_state_in, shape, v.device, "grad_state_in"),
        float(scale), B, H, Hk, N, D, M, code, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd_delta")
    return tuple(outs) + ((grad_state_in,) if return_state_grad else ())


def causal_product_decode_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                                beta: torch.Tensor, state: torch.Tensor,
                                out: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None, scale: float = 1.0,
                                slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the gated delta rule, the state updated in place.

    q, k: [B,Hk,D]; v: [B,H,M]; g, beta: float32 [B,H]; state: float32
    [P,H,D,M].  ``slots`` (int32 [B], on the device) names each sequence's
    state; one outside [0, P) is an idle row (out zero, no state touched).
    Without ``slots`` sequence b has state b.  No two sequences may share a
    slot."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_decode_delta(q, k, v, g, beta, state, out, None, scale, slots)
    qs, vs = q.shape, v.shape
    if (len(qs) != 3 or k.shape != qs or len(vs) != 3 or vs[0] != qs[0] or qs[1] == 0
            or vs[1] % qs[1] != 0):
        raise ValueError(f"expected q,k [B,Hk,D] and v [B,H,M], H a multiple of Hk; got "
                         f"{tuple(qs)}, {tuple(k.shape)}, {tuple(vs)}")
    B, Hk, D = qs
    _, H, M = vs
    code = _dtype_code(q, k, v)
    for t, name in ((g, "g"), (beta, "beta")):
        if t.shape != (B, H) or t.dtype is not torch.float32:
            _check_like(t, (B, H), torch.float32, name)
    dev = q.get_device()
    if out is None:
        _check_plain(dev, q, k, v, g, beta, state)
        out = torch.empty_like(v)
    else:
        _check_like(out, vs, v.dtype, "out")
        _check_plain(dev, q, k, v, g, beta, state, out)
    ss = state.shape
    if len(ss) != 4 or ss[1:] != (H, D, M) or state.dtype is not torch.float32:
        _check_like(state, (ss[0] if len(ss) == 4 else 0, H, D, M), torch.float32, "state")
    P = ss[0]
    if slots is not None:
        _check_like(slots, (B,), torch.int32, "slots")
        _check_plain(dev, q, slots)
    elif P < B:
        raise ValueError(f"state holds {P} sequences, fewer than the {B} of this call")
    rc = load_library().causal_product_decode_delta(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), out.data_ptr(),
        state.data_ptr(), 0 if slots is None else slots.data_ptr(), P, scale, B, H, Hk, D, M,
        code, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_decode_delta")
    return out


class _QkRope:
    """Checked arguments of the q/k norm with rotation, as the C ABI takes them."""

    __slots__ = ("head", "tail", "q_shape", "k_shape", "code", "dev")

    def __init__(self, xq, xk, wq, wk, cos, sin, norm, eps):
        qs, ks = xq.shape, xk.shape
        if len(qs) != 4 or len(ks) != 4 or ks[0] != qs[0] or ks[2:] != qs[2:]:
            raise ValueError(f"expected xq [B,Hq,N,D] and xk [B,Hk,N,D]; got {tuple(qs)}, {tuple(ks)}")
        if norm not in QK_NORMS:
            raise ValueError(f"unknown norm {norm!r}; expected one of {list(QK_NORMS)}")
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin are given together")
        B, Hq, N, D = qs
        plain = []
        weights = []
        for w, name in ((wq, "wq"), (wk, "wk")):
            if w is not None:
                weights.append(w)
                if w.shape != (D,) or w.dtype is not xq.dtype:
                    _dtype_code(xq, w)
                    _check_like(w, (D,), xq.dtype, name)
        self.code = _dtype_code(xq, xk)
        half, per_batch = 0, 0
        if cos is not None:
            cs = cos.shape
            half = cs[-1] if len(cs) > 1 else -1
            if (cos.dtype is not torch.float32 or sin.dtype is not torch.float32 or sin.shape != cs
                    or cs not in ((N, half), (1, N, half), (B, N, half))):
                raise ValueError(f"cos and sin must be float32 of one shape, [N,R/2] or [B,N,R/2]; got "
                                 f"{cos.dtype} {tuple(cs)}, {sin.dtype} {tuple(sin.shape)}")
            plain = [cos, sin]
            if len(cs) == 3 and B > 1 and cs[0] == B:
                per_batch = N * half
        self.dev = xq.get_device()
        if self.dev < 0:
            raise RuntimeError("causal_product runs on CUDA tensors only (no CPU path)")
        if xk.get_device() != self.dev:
            raise RuntimeError("all tensors must be on the same CUDA device")
        plain += weights
        if plain and not _all_plain(self.dev, *plain):
            _check_device(*plain)
            raise RuntimeError("all tensors must be on the same CUDA device")
        sq, sk = xq.stride(), xk.stride()
        if (sq[3] != 1 or sk[3] != 1) and D > 1:
            raise ValueError("the rows of xq and xk must be dense (stride 1 in the last dimension)")
        self.head = (xq.data_ptr(), _Strides(*sq[:3]), xk.data_ptr(), _Strides(*sk[:3]),
                     0 if wq is None else wq.data_ptr(), 0 if wk is None else wk.data_ptr(),
                     0 if cos is None else cos.data_ptr(), 0 if sin is None else sin.data_ptr(),
                     per_batch)
        self.tail = (QK_NORMS[norm], eps, B, Hq, ks[1], N, D, 2 * half, self.code)
        self.q_shape, self.k_shape = qs, ks

    def dense(self, t, shape, dtype, name):
        if t.shape != shape or t.dtype is not dtype:
            _check_like(t, shape, dtype, name)
        if t.get_device() != self.dev or not t.is_contiguous():
            _check_device(t)
            raise RuntimeError("all tensors must be on the same CUDA device")


_Strides = ctypes.c_int64 * 3


def causal_product_qk_rope(xq: torch.Tensor, xk: torch.Tensor, wq: Optional[torch.Tensor] = None,
                           wk: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                           sin: Optional[torch.Tensor] = None, norm: str = "rms",
                           eps: float = 1e-6, q: Optional[torch.Tensor] = None,
                           k: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None):
    """(q, k): the norm of every row of xq [B,Hq,N,D] and xk [B,Hk,N,D] over its
    features (``norm``: "rms", or "l2" for length 1), times the weights wq, wk
    ([D], None = ones), then features (i, i + R/2) of the first R turned by cos,
    sin (float32 [N,R/2] or [B,N,R/2]; None = no rotation).  xq and xk may be
    strided views (rows dense): a projection's ``x.view(B,N,H,D).transpose(1,
    2)`` is read in place.  q and k come dense."""
    place = _elsewhere(xq, stream)
    if place is not None:
        with place:
            return causal_product_qk_rope(xq, xk, wq, wk, cos, sin, norm, eps, q, k)
    a = _QkRope(xq, xk, wq, wk, cos, sin, norm, eps)
    if q is None:
        q = torch.empty_like(xq, memory_format=torch.contiguous_format)
    else:
        a.dense(q, a.q_shape, xq.dtype, "q")
    if k is None:
        k = torch.empty_like(xk, memory_format=torch.contiguous_format)
    else:
        a.dense(k, a.k_shape, xq.dtype, "k")
    rc = load_library().causal_product_qk_rope(*a.head, q.data_ptr(), k.data_ptr(), *a.tail,
                                               _raw_stream(a.dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_qk_rope")
    return q, k


def causal_product_qk_rope_bwd(xq: torch.Tensor, xk: torch.Tensor, wq: Optional[torch.Tensor],
                               wk: Optional[torch.Tensor], grad_q: torch.Tensor,
                               grad_k: torch.Tensor, cos: Optional[torch.Tensor] = None,
                               sin: Optional[torch.Tensor] = None, norm: str = "rms",
                               eps: float = 1e-6, workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None):
    """(dxq, dxk, dwq, dwk) of L = <grad_q, q> + <grad_k, k> for
    causal_product_qk_rope; dxq and dxk dense, dwq and dwk None where the
    weight is."""
    place = _elsewhere(xq, stream)
    if place is not None:
        with place:
            return causal_product_qk_rope_bwd(xq, xk, wq, wk, grad_q, grad_k, cos, sin, norm, eps,
                                              workspace)
    a = _QkRope(xq, xk, wq, wk, cos, sin, norm, eps)
    a.dense(grad_q, a.q_shape, xq.dtype, "grad_q")
    a.dense(grad_k, a.k_shape, xq.dtype, "grad_k")
    dxq, dxk = torch.empty_like(grad_q), torch.empty_like(grad_k)
    dwq = None if wq is None else torch.empty_like(wq)
    dwk = None if wk is None else torch.empty_like(wk)
    lib = load_library()
    need = lib.causal_product_qk_rope_workspace_size(*a.q_shape[:2], a.k_shape[1], *a.q_shape[2:],
                                                     a.code)
    workspace = _delta_workspace(workspace, need, xq.device)
    rc = lib.causal_product_qk_rope_bwd(
        *a.head, grad_q.data_ptr(), grad_k.data_ptr(), dxq.data_ptr(), dxk.data_ptr(),
        0 if dwq is None else dwq.data_ptr(), 0 if dwk is None else dwk.data_ptr(), *a.tail,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(a.dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_qk_rope_bwd")
    return dxq, dxk, dwq, dwk


def _decay_dims(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                lengths: Optional[torch.Tensor]):
    qs, vs = q.shape, v.shape
    if (len(qs) != 4 or k.shape != qs or len(vs) != 4 or vs[0] != qs[0] or vs[2] != qs[2]
            or qs[1] == 0 or vs[1] % qs[1] != 0):
        raise ValueError(f"expected q,k [B,Hk,N,D] and v [B,H,N,M], H a multiple of Hk; got "
                         f"{tuple(qs)}, {tuple(k.shape)}, {tuple(vs)}")
    B, Hk, N, D = qs
    H, M = vs[1], vs[3]
    if log_decay.shape != (H,) or log_decay.dtype is not torch.float32:
        _check_like(log_decay, (H,), torch.float32, "log_decay")
    if lengths is not None:
        _check_like(lengths, (B,), torch.int32, "lengths")
        _check_plain(v.get_device(), v, lengths)
    return B, H, Hk, N, D, M


def causal_product_decay_workspace_size(B: int, H: int, Hk: int, N: int, D: int, M: int,
                                        dtype: torch.dtype = torch.bfloat16,
                                        backward: bool = False) -> int:
    """Workspace bytes of causal_product_fwd_decay / _bwd_decay."""
    return int(load_library().causal_product_decay_workspace_size(B, H, Hk, N, D, M, _DTYPES[dtype],
                                                                  int(bool(backward))))


def causal_product_fwd_decay(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             log_decay: torch.Tensor, out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None,
                             state_in: Optional[torch.Tensor] = None, return_state: bool = False,
                             state_out: Optional[torch.Tensor] = None, scale: float = 1.0,
                             lengths: Optional[torch.Tensor] = None):
    """Linear attention with a decay for each head: S_t = a S_{t-1} + k_t v_t^T
    with a = exp(log_decay[h]); out_t = scale S_t^T q_t.

    q, k: [B,Hk,N,D]; v: [B,H,N,M], value head h reading key head h // (H //
    Hk); log_decay: float32 [H], at most 0 (a positive or NaN one makes its
    head's results NaN; -inf keeps the token alone); ``state_in`` is S_0
    (float32 [B,H,D,M], None = zero).  ``lengths`` (int32 [B], on the device):
    sequence b is its first lengths[b] rows; rows behind them reach nothing and
    give zero.  Returns out, with ``return_state`` followed by the state after
    each sequence's last row, as exact as fp32 arithmetic (asking for it changes
    no bit of out)."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_fwd_decay(q, k, v, log_decay, out, workspace, None, state_in,
                                            return_state, state_out, scale, lengths)
    B, H, Hk, N, D, M = _decay_dims(q, k, v, log_decay, lengths)
    code = _dtype_code(q, k, v)
    dev = v.get_device()
    if out is None:
        _check_plain(dev, q, k, v, log_decay)
        out = torch.empty_like(v)
    else:
        _check_like(out, (B, H, N, M), v.dtype, "out")
        _check_plain(dev, q, k, v, log_decay, out)
    if return_state and state_out is None:
        state_out = torch.empty((B, H, D, M), dtype=torch.float32, device=v.device)
    lib = load_library()
    need = lib.causal_product_decay_workspace_size(B, H, Hk, N, D, M, code, 0)
    workspace = _delta_workspace(workspace, need, v.device)
    rc = lib.causal_product_fwd_decay(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), out.data_ptr(),
        _state_arg(state_in, (B, H, D, M), v.device, "state_in"),
        _state_arg(state_out, (B, H, D, M), v.device, "state_out"),
        0 if lengths is None else lengths.data_ptr(), float(scale), B, H, Hk, N, D, M, code,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_fwd_decay")
    return (out, state_out) if return_state else out


def causal_product_bwd_decay(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             log_decay: torch.Tensor, grad_out: torch.Tensor,
                             grad_q: Optional[torch.Tensor] = None,
                             grad_k: Optional[torch.Tensor] = None,
                             grad_v: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None,
                             state_in: Optional[torch.Tensor] = None,
                             grad_state_out: Optional[torch.Tensor] = None,
                             return_state_grad: bool = False,
                             grad_state_in: Optional[torch.Tensor] = None, scale: float = 1.0,
                             lengths: Optional[torch.Tensor] = None):
    """(dq, dk, dv) of L = <grad_out, out> + <grad_state_out, S_N> for
    causal_product_fwd_decay on the same inputs (nothing is kept from it); with
    ``return_state_grad`` dL/dS_0 follows.  dq and dk are summed over the value
    heads of a key head; rows behind a sequence's length get zero."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_bwd_decay(q, k, v, log_decay, grad_out, grad_q, grad_k, grad_v,
                                            workspace, None, state_in, grad_state_out,
                                            return_state_grad, grad_state_in, scale, lengths)
    B, H, Hk, N, D, M = _decay_dims(q, k, v, log_decay, lengths)
    code = _dtype_code(q, k, v, grad_out)
    if grad_out.shape != v.shape:
        raise ValueError("grad_out must have v's shape")
    outs = []
    for t, ref, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k"), (grad_v, v, "grad_v")):
        t = torch.empty_like(ref) if t is None else t
        _check_like(t, ref.shape, ref.dtype, name)
        outs.append(t)
    dev = v.get_device()
    _check_plain(dev, q, k, v, log_decay, grad_out, *outs)
    if return_state_grad and grad_state_in is None:
        grad_state_in = torch.empty((B, H, D, M), dtype=torch.float32, device=v.device)
    lib = load_library()
    need = lib.causal_product_decay_workspace_size(B, H, Hk, N, D, M, code, 1)
    workspace = _delta_workspace(workspace, need, v.device)
    shape = (B, H, D, M)
    rc = lib.causal_product_bwd_decay(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), grad_out.data_ptr(),
        _state_arg(state_in, shape, v.device, "state_in"),
        _state_arg(grad_state_out, shape, v.device, "grad_state_out"),
        *(t.data_ptr() for t in outs),
        _state_arg(grad_state_in, shape, v.device, "grad_state_in"),
        0 if lengths is None else lengths.data_ptr(), float(scale), B, H, Hk, N, D, M, code,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_bwd_decay")
    return tuple(outs) + ((grad_state_in,) if return_state_grad else ())


def causal_product_decode_decay(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                log_decay: torch.Tensor, state: torch.Tensor,
                                out: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None, scale: float = 1.0,
                                slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of linear attention with a decay for each head, the state
    updated in place.

    q, k: [B,Hk,D]; v: [B,H,M]; log_decay: float32 [H]; state: float32
    [P,H,D,M].  ``slots`` (int32 [B], on the device) names each sequence's
    state; one outside [0, P) is an idle row (out zero, no state touched).
    Without ``slots`` sequence b has state b.  No two sequences may share a
    slot."""
    place = _elsewhere(q, stream)
    if place is not None:
        with place:
            return causal_product_decode_decay(q, k, v, log_decay, state, out, None, scale, slots)
    qs, vs = q.shape, v.shape
    if (len(qs) != 3 or k.shape != qs or len(vs) != 3 or vs[0] != qs[0] or qs[1] == 0
            or vs[1] % qs[1] != 0):
        raise ValueError(f"expected q,k [B,Hk,D] and v [B,H,M], H a multiple of Hk; got "
                         f"{tuple(qs)}, {tuple(k.shape)}, {tuple(vs)}")
    B, Hk, D = qs
    _, H, M = vs
    code = _dtype_code(q, k, v)
    if log_decay.shape != (H,) or log_decay.dtype is not torch.float32:
        _check_like(log_decay, (H,), torch.float32, "log_decay")
    dev = q.get_device()
    if out is None:
        _check_plain(dev, q, k, v, log_decay, state)
        out = torch.empty_like(v)
    else:
        _check_like(out, vs, v.dtype, "out")
        _check_plain(dev, q, k, v, log_decay, state, out)
    ss = state.shape
    if len(ss) != 4 or ss[1:] != (H, D, M) or state.dtype is not torch.float32:
        _check_like(state, (ss[0] if len(ss) == 4 else 0, H, D, M), torch.float32, "state")
    P = ss[0]
    if slots is not None:
        _check_like(slots, (B,), torch.int32, "slots")
        _check_plain(dev, q, slots)
    elif P < B:
        raise ValueError(f"state holds {P} sequences, fewer than the {B} of this call")
    rc = load_library().causal_product_decode_decay(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), out.data_ptr(),
        state.data_ptr(), 0 if slots is None else slots.data_ptr(), P, scale, B, H, Hk, D, M,
        code, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_decode_decay")
    return out


def _layer_norm_args(x, weight, bias, token_major):
    """(rows as the C ABI takes them, their (B,H,N,C), dtype code, device,
    whether the weights are per head, the result's shape) of a layer norm."""
    xs, st = x.shape, x.stride()
    n = len(xs)
    if not 2 <= n <= 4 or (token_major and n != 4):
        raise ValueError(f"expected x [R,C], [B,N,C] or [B,H,N,C] (with token_major: [B,H,N,C]); "
                         f"got {tuple(xs)}")
    C = xs[-1]
    if n == 2:
        dims, strides = (1, 1, xs[0], C), (0, 0, st[0])
    elif n == 3:
        dims, strides = (xs[0], 1, xs[1], C), (st[0], 0, st[1])
    else:
        dims, strides = tuple(xs), st[:3]
    if dims[0] == 0:
        dims = (1, dims[1], 0, C)  # no sequences: no rows (the C side wants B > 0)
    code = _dtype_code(x)
    dev = x.get_device()
    if dev < 0:
        raise RuntimeError("causal_product runs on CUDA tensors only (no CPU path)")
    if st[-1] != 1 and C > 1:
        raise ValueError("the rows of x must be dense (stride 1 in the last dimension)")
    per_head = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if t.dtype is not x.dtype:
            _dtype_code(x, t)
        wide = n == 4 and t.shape == (xs[1], C)
        if not wide and t.shape != (C,):
            raise ValueError(f"{name} must have shape ({C},) or, for x [B,H,N,C], (H, {C}); got "
                             f"{tuple(t.shape)}")
        if per_head is not None and per_head != wide:
            raise ValueError("weight and bias must have one shape")
        per_head = wide
        if not _all_plain(dev, t):
            _check_device(t)
            raise RuntimeError("all tensors must be on the same CUDA device")
    shape = (xs[0], xs[2], xs[1], C) if token_major else tuple(xs)
    return (x.data_ptr(), _Strides(*strides)), dims, code, dev, int(bool(per_head)), shape


def causal_product_layer_norm_workspace_size(B: int, H: int, N: int, C: int,
                                             dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of causal_product_layer_norm_bwd for x [B,H,N,C]; rows [B,N,C]
    count as one head, [R,C] as one sequence of one head (0: a shape that is refused)."""
    return int(load_library().causal_product_layer_norm_workspace_size(B, H, N, C, _DTYPES[dtype]))


def causal_product_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                              bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                              token_major: bool = False, out: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Layer norm of the rows of x ([R,C], [B,N,C] or a causal product's heads
    [B,H,N,C]) over their C features, times ``weight`` plus ``bias`` ([C], or
    [H,C] for weights of each head; None = ones, zeros).  x may be a strided view
    (rows dense), or empty.  The result is dense: x's shape, or with ``token_major``
    [B,N,H,C], the rows an output projection reads."""
    place = _elsewhere(x, stream)
    if place is not None:
        with place:
            return causal_product_layer_norm(x, weight, bias, eps, token_major, out)
    rows, dims, code, dev, per_head, shape = _layer_norm_args(x, weight, bias, token_major)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _check_like(out, shape, x.dtype, "out")
        _check_plain(dev, out)
    rc = load_library().causal_product_layer_norm(
        *rows, 0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
        per_head, out.data_ptr(), int(bool(token_major)), eps, *dims, code, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_layer_norm")
    return out


def causal_product_layer_norm_bwd(x: torch.Tensor, weight: Optional[torch.Tensor],
                                  bias: Optional[torch.Tensor], grad_out: torch.Tensor,
                                  eps: float = 1e-5, token_major: bool = False,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None,
                                  weight_grad: bool = True, bias_grad: bool = True):
    """(dx, dweight, dbias) of L = <grad_out, y> for causal_product_layer_norm;
    dx dense in x's shape, dweight and dbias None where the argument is, and not
    computed (None) where ``weight_grad`` or ``bias_grad`` is false."""
    place = _elsewhere(x, stream)
    if place is not None:
        with place:
            return causal_product_layer_norm_bwd(x, weight, bias, grad_out, eps, token_major,
                                                 workspace, None, weight_grad, bias_grad)
    rows, dims, code, dev, per_head, shape = _layer_norm_args(x, weight, bias, token_major)
    _check_like(grad_out, shape, x.dtype, "grad_out")
    _check_plain(dev, grad_out)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = None if weight is None or not weight_grad else torch.empty_like(weight)
    db = None if bias is None or not bias_grad else torch.empty_like(bias)
    lib = load_library()
    gathers = dw is not None or db is not None
    need = lib.causal_product_layer_norm_workspace_size(*dims, code) if gathers else 0
    workspace = _delta_workspace(workspace, need, x.device)
    rc = lib.causal_product_layer_norm_bwd(
        *rows, 0 if weight is None else weight.data_ptr(), per_head, grad_out.data_ptr(),
        int(bool(token_major)), dx.data_ptr(), 0 if dw is None else dw.data_ptr(),
        0 if db is None else db.data_ptr(), eps, *dims, code, workspace.data_ptr(),
        workspace.nbytes, _raw_stream(dev))
    if rc != CP_OK:
        raise CausalProductError(rc, "causal_product_layer_norm_bwd")
    return dx, dw, db


def _dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """The tensor as the C entry points take it: contiguous, at a whole 16-byte
    address.  A dense view may start anywhere: a slice of a batch of odd widths,
    the gradient that torch.cat hands to one of its parts."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class CausalProduct(torch.autograd.Function):
    """Autograd wrapper: forward and backward both call the C ABI; the
    forward keeps checkpoints of the state for the backward's dq scans."""

    @staticmethod
    def forward(ctx, q, k, v):
        q, k, v = _dense(q), _dense(k), _dense(v)
        out, ckpt = causal_product_fwd_ckpt(q, k, v)
        ctx.save_for_backward(q, k, v, ckpt)
        return out

    @staticmethod
    def backward(ctx, g):
        q, k, v, ckpt = ctx.saved_tensors
        return causal_product_bwd_ckpt(q, k, v, _dense(g.to(q.dtype)), ckpt)


class Normalizer(torch.autograd.Function):
    """Autograd wrapper of the normaliser: (q, k) -> z."""

    @staticmethod
    def forward(ctx, q, k, feature):
        q, k = _dense(q), _dense(k)
        ctx.save_for_backward(q, k)
        ctx.feature = feature
        return causal_product_normalizer(q, k, feature=feature)

    @staticmethod
    def backward(ctx, gz):
        q, k = ctx.saved_tensors
        dq, dk = causal_product_normalizer_bwd(q, k, _dense(gz.float()), feature=ctx.feature)
        return dq, dk, None


def normalizer(q: torch.Tensor, k: torch.Tensor, feature: Optional[str] = None) -> torch.Tensor:
    """z_i = q_i . sum_{j<=i} k_j (float32 [B,H,N]) with autograd support;
    ``feature="elu1"`` maps raw q, k by phi(x) = elu(x) + 1 in the kernel."""
    return Normalizer.apply(q, k, feature)


class CausalProductFeature(torch.autograd.Function):
    """Autograd wrapper with the feature map applied inside the kernels."""

    @staticmethod
    def forward(ctx, q, k, v, feature):
        q, k, v = _dense(q), _dense(k), _dense(v)
        ctx.save_for_backward(q, k, v)
        ctx.feature = feature
        return causal_product_fwd_feature(q, k, v, feature)

    @staticmethod
    def backward(ctx, g):
        q, k, v = ctx.saved_tensors
        dq, dk, dv = causal_product_bwd_feature(q, k, v, _dense(g.to(q.dtype)), ctx.feature)
        return dq, dk, dv, None


class CausalProductState(torch.autograd.Function):
    """Autograd wrapper with a carried state: (q, k, v, S_0) -> (out, S_N)."""

    @staticmethod
    def forward(ctx, q, k, v, state):
        q, k, v = _dense(q), _dense(k), _dense(v)
        state = _dense(state)
        ctx.save_for_backward(q, k, v, state)
        ctx.has_state = state is not None
        return causal_product_fwd(q, k, v, state_in=state, return_state=True)

    @staticmethod
    def backward(ctx, g, g_state):
        q, k, v, state = ctx.saved_tensors
        g = torch.zeros_like(v) if g is None else _dense(g.to(q.dtype))
        g_state = None if g_state is None else _dense(g_state.float())
        dq, dk, dv, ds = causal_product_bwd(q, k, v, g, state_in=state if ctx.has_state else None,
                                            grad_state_out=g_state, return_state_grad=True)
        return dq, dk, dv, (ds if ctx.has_state else None)


class CausalProductFavor(torch.autograd.Function):
    """Autograd wrapper of the positive-random-feature product: (xq, xk, v)
    -> out for a fixed projection W (no gradient for W)."""

    @staticmethod
    def forward(ctx, xq, xk, v, W):
        xq, xk, v, W = _dense(xq), _dense(xk), _dense(v), _dense(W)
        ctx.save_for_backward(xq, xk, v, W)
        return causal_product_fwd_favor(xq, xk, v, W)

    @staticmethod
    def backward(ctx, g):
        xq, xk, v, W = ctx.saved_tensors
        dxq, dxk, dv = causal_product_bwd_favor(xq, xk, v, W, _dense(g.to(v.dtype)))
        return dxq, dxk, dv, None


def causal_product_favor(xq: torch.Tensor, xk: torch.Tensor, v: torch.Tensor,
                         W: torch.Tensor) -> torch.Tensor:
    """Causal product of the positive random features phi(x) = exp(W x -
    |x|^2 / 2) / sqrt(D) of the raw rows xq, xk, with autograd support for
    xq, xk and v (W is treated as a constant)."""
    return CausalProductFavor.apply(xq, xk, v, W)


def _no_tangents(*tensors: Optional[torch.Tensor]) -> None:
    """Refuses forward-mode derivatives: a dual tensor asks for no gradient, so a
    call that goes past autograd where none is wanted would lose its tangent."""
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("this operator has no forward-mode derivative")


class CausalProductDelta(torch.autograd.Function):
    """Autograd wrapper of the gated delta rule: (q, k, v, g, beta, S_0) ->
    (out, S_N)."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, scale):
        q, k, v = _dense(q), _dense(k), _dense(v)
        g, beta = _dense(g), _dense(beta)
        state = _dense(state)
        out, s_n, ckpt = causal_product_fwd_delta(q, k, v, g, beta, state_in=state,
                                                  return_state=True, scale=scale, save=True)
        ctx.save_for_backward(q, k, v, g, beta, ckpt)
        ctx.scale, ctx.has_state = scale, state is not None
        ctx.set_materialize_grads(False)
        return out, s_n

    @staticmethod
    def backward(ctx, go, gs):
        q, k, v, g, beta, ckpt = ctx.saved_tensors
        go = torch.zeros_like(v) if go is None else _dense(go.to(v.dtype))
        gs = None if gs is None else _dense(gs.float())
        d = causal_product_bwd_delta(q, k, v, g, beta, go, ckpt, scale=ctx.scale,
                                     grad_state_out=gs, return_state_grad=ctx.has_state)
        return d[:5] + (d[5] if ctx.has_state else None, None)


def causal_product_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                         beta: torch.Tensor, state: Optional[torch.Tensor] = None,
                         return_state: bool = False, scale: float = 1.0):
    """The gated delta rule with autograd support (causal_product_fwd_delta);
    with ``return_state`` the result is (out, state after the last row).
    Forward-mode derivatives are refused."""
    _no_tangents(q, k, v, g, beta, state)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (q, k, v, g, beta, state)):
        out, s_n = CausalProductDelta.apply(q, k, v, g, beta, state, scale)
        return (out, s_n) if return_state else out
    # no gradient is wanted: no checkpoints
    return causal_product_fwd_delta(_dense(q), _dense(k), _dense(v), _dense(g), _dense(beta),
                                    state_in=_dense(state), return_state=return_state, scale=scale)


class QkRope(torch.autograd.Function):
    """Autograd wrapper of the q/k norm with rotation."""

    @staticmethod
    def forward(ctx, xq, xk, wq, wk, cos, sin, norm, eps):
        ctx.save_for_backward(xq, xk, wq, wk, cos, sin)
        ctx.norm, ctx.eps = norm, eps
        return causal_product_qk_rope(xq, xk, wq, wk, cos, sin, norm, eps)

    @staticmethod
    def backward(ctx, gq, gk):
        xq, xk, wq, wk, cos, sin = ctx.saved_tensors
        gq, gk = _dense(gq.to(xq.dtype)), _dense(gk.to(xq.dtype))
        return causal_product_qk_rope_bwd(xq, xk, wq, wk, gq, gk, cos, sin, ctx.norm,
                                          ctx.eps) + (None, None, None, None)


def qk_rope(xq: torch.Tensor, xk: torch.Tensor, wq: Optional[torch.Tensor] = None,
            wk: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
            sin: Optional[torch.Tensor] = None, norm: str = "rms", eps: float = 1e-6):
    """causal_product_qk_rope with autograd support for xq, xk, wq and wk."""
    return QkRope.apply(xq, xk, wq, wk, cos, sin, norm, eps)


class CausalProductDecay(torch.autograd.Function):
    """Autograd wrapper of linear attention with a decay for each head: (q, k,
    v, S_0) -> (out, S_N or None), the decay a constant."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, scale, lengths, return_state):
        q, k, v = _dense(q), _dense(k), _dense(v)
        log_decay = _dense(log_decay)
        state = _dense(state)
        got = causal_product_fwd_decay(q, k, v, log_decay, state_in=state,
                                       return_state=return_state, scale=scale, lengths=lengths)
        ctx.save_for_backward(q, k, v, log_decay, state, lengths)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return got if return_state else (got, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, go, gs):
        q, k, v, log_decay, state, lengths = ctx.saved_tensors
        go = torch.zeros_like(v) if go is None else _dense(go.to(v.dtype))
        gs = None if gs is None else _dense(gs.float())
        want = ctx.needs_input_grad[4]
        d = causal_product_bwd_decay(q, k, v, log_decay, go, state_in=state, grad_state_out=gs,
                                     return_state_grad=want, scale=ctx.scale, lengths=lengths)
        return d[:3] + (None, d[3] if want else None, None, None, None)


def causal_product_decay(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         log_decay: torch.Tensor, state: Optional[torch.Tensor] = None,
                         return_state: bool = False, scale: float = 1.0,
                         lengths: Optional[torch.Tensor] = None):
    """Linear attention with a decay for each head, with autograd support for q,
    k, v and the state (causal_product_fwd_decay); with ``return_state`` the
    result is (out, state after each sequence's last row).  The decay is a
    constant: one that asks for a gradient is refused, as second and
    forward-mode derivatives are."""
    _no_tangents(q, k, v, log_decay, state)
    if torch.is_grad_enabled():
        if log_decay.requires_grad:
            raise ValueError("log_decay is a constant of the head; it has no gradient")
        if any(t is not None and t.requires_grad for t in (q, k, v, state)):
            out, s_n = CausalProductDecay.apply(q, k, v, log_decay, state, scale, lengths,
                                                bool(return_state))
            return (out, s_n) if return_state else out
    return causal_product_fwd_decay(_dense(q), _dense(k), _dense(v), _dense(log_decay),
                                    state_in=_dense(state), return_state=return_state, scale=scale,
                                    lengths=lengths)


class LayerNorm(torch.autograd.Function):
    """Autograd wrapper of the layer norm."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, token_major):
        ctx.save_for_backward(x, weight, bias)
        ctx.eps, ctx.token_major = eps, token_major
        return causal_product_layer_norm(x, weight, bias, eps, token_major)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x, weight, bias = ctx.saved_tensors
        return causal_product_layer_norm_bwd(x, weight, bias, _dense(gy.to(x.dtype)), ctx.eps,
                                             ctx.token_major, weight_grad=ctx.needs_input_grad[1],
                                             bias_grad=ctx.needs_input_grad[2]) + (None, None)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, token_major: bool = False):
    """causal_product_layer_norm with autograd support for x, weight and bias (first
    derivatives; a second or a forward-mode one is refused)."""
    _no_tangents(x, weight, bias)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)):
        return LayerNorm.apply(x, weight, bias, eps, token_major)
    return causal_product_layer_norm(x, weight, bias, eps, token_major)


def causal_product(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   state: Optional[torch.Tensor] = None, return_state: bool = False,
                   feature: Optional[str] = None):
    """Causal dot product with autograd support (no normaliser, no scale).

    ``state`` (float32 [B,H,D,M]) is the state before the first row; with
    ``return_state`` the result is (out, state after the last row), both
    differentiable.  ``feature="elu1"`` applies phi(x) = elu(x) + 1 to q and
    k inside the kernels (no carried state in that mode)."""
    if _feature_code(feature) != 0:
        if state is not None or return_state:
            raise ValueError("a feature map is not combined with a carried state")
        return CausalProductFeature.apply(q, k, v, feature)
    if state is None and not return_state:
        return CausalProduct.apply(q, k, v)
    out, s_n = CausalProductState.apply(q, k, v, state)
    return (out, s_n) if return_state else out
