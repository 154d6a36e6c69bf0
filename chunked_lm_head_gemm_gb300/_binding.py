"""ctypes binding of liblce.so (include/lce.h): argument marshalling only.

Every step of the loss runs in the library's CUDA kernels; this module only
checks tensors, passes their device pointers and the current CUDA stream,
and raises on a non-OK status. There is no fallback: if the library is not
built or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os
import threading

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import build as _build

_lib = None
_lock = threading.Lock()

LCE_OK = 0
LCE_ERR_INVALID_ARG = 1
LCE_ERR_UNSUPPORTED = 2
LCE_ERR_WORKSPACE = 3
LCE_ERR_LABEL_RANGE = 4
LCE_ERR_TIMEOUT = 5
LCE_ERR_CUDA = 6
LCE_ERR_EXPERT_RANGE = 7

LCE_BF16 = 0
LCE_F32 = 1

SCORING = {"softmax": 0, "sigmoid": 1}

LAYER_NORM = 0
RMS_NORM = 1

IGNORE_INDEX = -100

EXPORTED = ("lce_workspace_size", "lce_default_chunk_rows", "lce_forward",
            "lce_backward", "lce_get_error", "lce_status_string",
            "lce_last_cuda_error", "lce_test_gemm", "lce_test_wait_timeout",
            "lce_profile_start", "lce_profile_stop", "lce_forward_static",
            "lce_forward_backward", "lce_scale_gradients",
            "lce_set_cta_pair", "lce_get_cta_pair", "lce_mlp_workspace_size",
            "lce_mlp_forward", "lce_mlp_backward", "lce_count_valid",
            "lce_forward_slice", "lce_combine_workspace_size",
            "lce_combine_slices", "lce_backward_slice", "lce_set_wave_sync",
            "lce_get_wave_sync", "lce_slice_exp_workspace_size",
            "lce_forward_slice_exp", "lce_backward_slice_exp",
            "lce_forward_ex", "lce_backward_ex", "lce_forward_backward_ex",
            "lce_shard_sums", "lce_combine_shards", "lce_forward_slice_ex",
            "lce_combine_slices_ex", "lce_backward_slice_ex",
            "lce_forward_slice_exp_ex", "lce_backward_slice_exp_ex",
            "lce_route_forward", "lce_route_backward",
            "lce_experts_workspace_size", "lce_experts_forward",
            "lce_experts_backward", "lce_norm_forward", "lce_norm_backward",
            "lce_norm_workspace_size", "lce_balance_forward",
            "lce_balance_backward", "lce_balance_workspace_size",
            "lce_expert_counts", "lce_grad_norm", "lce_clip_grads",
            "lce_grad_norm_workspace_size", "lce_clip_grad_norm")

KERNEL_KINDS = 40


class LossOpts(ctypes.Structure):
    """lce_loss_opts: label smoothing in [0, 1] and the z-loss coefficient."""
    _fields_ = [("label_smoothing", ctypes.c_float),
                ("z_loss", ctypes.c_float)]


class RouteOpts(ctypes.Structure):
    """lce_route_opts: how router logits become experts and weights."""
    _fields_ = [("scoring", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double)]


class LCEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = _lib
        name = lib.lce_status_string(status).decode() if lib else str(status)
        detail = lib.lce_last_cuda_error().decode() if lib else ""
        super().__init__(f"{where}: {name}" + (f" ({detail})" if detail else ""))


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False):
    """Open liblce.so and declare the C signatures. Raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(
                    f"CUDA library not built: {path} is missing "
                    "(run __graft_entry__.build() or python -m "
                    "chunked_lm_head_gemm_gb300.build)")
            _build.build()
        lib = ctypes.CDLL(path)
        p, i64, i32, u64, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                ctypes.c_uint64, ctypes.c_size_t)
        lib.lce_workspace_size.argtypes = [i64, i64, i64, i32, i64]
        lib.lce_workspace_size.restype = sz
        lib.lce_default_chunk_rows.argtypes = [i64, i64, i64]
        lib.lce_default_chunk_rows.restype = i64
        lib.lce_forward.argtypes = [p, p, i32, p, i64, i64, i64, i64, p, p, p,
                                    sz, p]
        lib.lce_forward.restype = i32
        lib.lce_backward.argtypes = [p, p, i32, p, p, i64, i64, i64, i64, p,
                                     i64, p, p, p, sz, p]
        lib.lce_backward.restype = i32
        lib.lce_get_error.argtypes = [p]
        lib.lce_get_error.restype = i32
        lib.lce_status_string.argtypes = [i32]
        lib.lce_status_string.restype = ctypes.c_char_p
        lib.lce_last_cuda_error.argtypes = []
        lib.lce_last_cuda_error.restype = ctypes.c_char_p
        lib.lce_test_gemm.argtypes = [p, p, p, i64, i64, i64, i32, i32, p]
        lib.lce_test_gemm.restype = i32
        lib.lce_test_wait_timeout.argtypes = [u64, p]
        lib.lce_test_wait_timeout.restype = i32
        lib.lce_forward_backward.argtypes = [p, p, i32, p, i64, i64, i64, i64,
                                             i64, p, p, p, p, p, sz, p]
        lib.lce_forward_backward.restype = i32
        opts = ctypes.POINTER(LossOpts)
        lib.lce_forward_ex.argtypes = [p, p, i32, p, i64, i64, i64, i64, opts,
                                       p, p, p, sz, p]
        lib.lce_forward_ex.restype = i32
        lib.lce_backward_ex.argtypes = [p, p, i32, p, p, i64, i64, i64, i64,
                                        opts, p, i64, p, p, p, sz, p]
        lib.lce_backward_ex.restype = i32
        lib.lce_forward_backward_ex.argtypes = [p, p, i32, p, i64, i64, i64,
                                                i64, opts, i64, p, p, p, p, p,
                                                sz, p]
        lib.lce_forward_backward_ex.restype = i32
        lib.lce_shard_sums.argtypes = [p, p, p, p]
        lib.lce_shard_sums.restype = i32
        lib.lce_combine_shards.argtypes = [p, p, p, p, p, p]
        lib.lce_combine_shards.restype = i32
        lib.lce_scale_gradients.argtypes = [p, i32, i64, i64, p, i64, p, p]
        lib.lce_scale_gradients.restype = i32
        lib.lce_count_valid.argtypes = [p, i64, i64, i64, p, p]
        lib.lce_count_valid.restype = i32
        lib.lce_forward_slice.argtypes = [p, p, i32, p, i64, i64, i64, i64,
                                          i64, i64, p, p, p, p, sz, p]
        lib.lce_forward_slice.restype = i32
        lib.lce_combine_workspace_size.argtypes = [i64]
        lib.lce_combine_workspace_size.restype = sz
        lib.lce_combine_slices.argtypes = [p, p, p, i64, p, i64, i64, i64, p,
                                           p, p, sz, p]
        lib.lce_combine_slices.restype = i32
        lib.lce_backward_slice.argtypes = [p, p, i32, p, p, i64, i64, i64,
                                           i64, i64, i64, p, i64, p, p, p, sz,
                                           p]
        lib.lce_backward_slice.restype = i32
        lib.lce_slice_exp_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.lce_slice_exp_workspace_size.restype = sz
        lib.lce_forward_slice_exp.argtypes = [p, p, i32, p, i64, i64, i64,
                                              i64, i64, i64, p, p, p, p, sz,
                                              p]
        lib.lce_forward_slice_exp.restype = i32
        lib.lce_backward_slice_exp.argtypes = [p, p, i32, p, p, i64, i64, i64,
                                               i64, i64, i64, p, p, p, p, sz,
                                               p]
        lib.lce_backward_slice_exp.restype = i32
        lib.lce_forward_slice_ex.argtypes = [p, p, i32, p, i64, i64, i64,
                                             i64, i64, i64, opts, p, p, p, p,
                                             p, sz, p]
        lib.lce_forward_slice_ex.restype = i32
        lib.lce_combine_slices_ex.argtypes = [p, p, p, p, i64, p, i64, i64,
                                              i64, opts, p, p, p, sz, p]
        lib.lce_combine_slices_ex.restype = i32
        lib.lce_backward_slice_ex.argtypes = [p, p, i32, p, p, i64, i64, i64,
                                              i64, i64, i64, opts, p, i64, p,
                                              p, p, sz, p]
        lib.lce_backward_slice_ex.restype = i32
        lib.lce_forward_slice_exp_ex.argtypes = [p, p, i32, p, i64, i64, i64,
                                                 i64, i64, i64, opts, p, p, p,
                                                 p, p, sz, p]
        lib.lce_forward_slice_exp_ex.restype = i32
        lib.lce_backward_slice_exp_ex.argtypes = [p, p, i32, p, p, i64, i64,
                                                  i64, i64, i64, i64, opts, p,
                                                  p, p, p, sz, p]
        lib.lce_backward_slice_exp_ex.restype = i32
        lib.lce_mlp_workspace_size.argtypes = [i64, i64, i64, i64]
        lib.lce_mlp_workspace_size.restype = sz
        lib.lce_mlp_forward.argtypes = [p, p, p, p, i64, i64, i64, i64, p, p,
                                        sz, p]
        lib.lce_mlp_forward.restype = i32
        lib.lce_mlp_backward.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p,
                                         p, p, p, p, sz, p]
        lib.lce_mlp_backward.restype = i32
        ropts = ctypes.POINTER(RouteOpts)
        lib.lce_route_forward.argtypes = [p, i32, p, i64, i64, ropts, p, p, p]
        lib.lce_route_forward.restype = i32
        lib.lce_route_backward.argtypes = [p, i32, p, p, i64, i64, ropts, p,
                                           p]
        lib.lce_route_backward.restype = i32
        lib.lce_experts_workspace_size.argtypes = [i64, i64, i64, i64, i64,
                                                   i32]
        lib.lce_experts_workspace_size.restype = sz
        lib.lce_experts_forward.argtypes = [p, p, p, p, p, i32, p, i64, i64,
                                            i64, i64, i64, p, p, sz, p]
        lib.lce_experts_forward.restype = i32
        lib.lce_experts_backward.argtypes = [p, p, p, p, p, i32, p, p, i64,
                                             i64, i64, i64, i64, i32, p, p, p,
                                             p, p, p, sz, p]
        lib.lce_experts_backward.restype = i32
        f32 = ctypes.c_float
        lib.lce_norm_workspace_size.argtypes = [i64, i64]
        lib.lce_norm_workspace_size.restype = sz
        lib.lce_norm_forward.argtypes = [i32, p, i32, p, p, i32, i64, i64, f32,
                                         p, p, p, p]
        lib.lce_norm_forward.restype = i32
        lib.lce_norm_backward.argtypes = [i32, p, i32, p, i32, p, p, p, i64,
                                          i64, i32, p, p, p, p, sz, p]
        lib.lce_norm_backward.restype = i32
        lib.lce_balance_workspace_size.argtypes = [i64, i64]
        lib.lce_balance_workspace_size.restype = sz
        lib.lce_balance_forward.argtypes = [p, i32, p, p, i64, i64, i64, i32,
                                            f32, p, p, p, p, sz, p]
        lib.lce_balance_forward.restype = i32
        lib.lce_balance_backward.argtypes = [p, i32, p, i64, i64, i32, p, p, p,
                                             p]
        lib.lce_balance_backward.restype = i32
        lib.lce_expert_counts.argtypes = [p, p, i64, i64, i64, p, p]
        lib.lce_expert_counts.restype = i32
        lib.lce_grad_norm_workspace_size.argtypes = [i64]
        lib.lce_grad_norm_workspace_size.restype = sz
        lib.lce_grad_norm.argtypes = [p, p, p, i64, p, p, sz, p]
        lib.lce_grad_norm.restype = i32
        lib.lce_clip_grads.argtypes = [p, p, p, p, i64, p, f32, p]
        lib.lce_clip_grads.restype = i32
        lib.lce_clip_grad_norm.argtypes = [p, p, p, p, i64, f32, p, p, sz, p]
        lib.lce_clip_grad_norm.restype = i32
        lib.lce_set_cta_pair.argtypes = [i32]
        lib.lce_set_cta_pair.restype = i32
        lib.lce_get_cta_pair.argtypes = []
        lib.lce_get_cta_pair.restype = i32
        lib.lce_set_wave_sync.argtypes = [i32]
        lib.lce_set_wave_sync.restype = i32
        lib.lce_get_wave_sync.argtypes = []
        lib.lce_get_wave_sync.restype = i32
        lib.lce_forward_static.argtypes = [p, p, p, i64, i64, i64, i64, p, p,
                                           p]
        lib.lce_forward_static.restype = i32
        lib.lce_profile_start.argtypes = []
        lib.lce_profile_start.restype = i32
        lib.lce_profile_stop.argtypes = [ctypes.POINTER(KernelStat)]
        lib.lce_profile_stop.restype = i32
        _lib = lib
        return lib


def _check(status: int, where: str):
    if status != LCE_OK:
        raise LCEError(status, where)


def _stream_ptr(device) -> int:
    """The device's current stream (device None: the current device's)."""
    if isinstance(device, str):
        device = torch.device(device)
    if isinstance(device, torch.device):
        if device.type != "cuda":  # its pointers must not reach a kernel
            raise ValueError(f"expected a CUDA device, got {device}")
        if device.index is not None:
            return torch._C._cuda_getCurrentRawStream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LCE_BF16
    if t.dtype == torch.float32:
        return LCE_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _written(*tensors):
    """Tells autograd that a call has written tensors (None: not this one)
    that may be the caller's, whose memory the library knows by address alone:
    one that an operation has saved for its gradient is then an error there."""
    increment_version([t for t in tensors if t is not None])


def _check_inputs(h, W, labels):
    if not (h.is_cuda and W.is_cuda and labels.is_cuda):
        raise ValueError("h, W and labels must be CUDA tensors")
    if h.dim() != 2 or W.dim() != 2 or labels.dim() != 1:
        raise ValueError("expected h [L,H], W [V,H], labels [L]")
    if h.shape[1] != W.shape[1] or labels.shape[0] != h.shape[0]:
        raise ValueError(f"shape mismatch: h {tuple(h.shape)}, W "
                         f"{tuple(W.shape)}, labels {tuple(labels.shape)}")
    if h.dtype != W.dtype:
        raise TypeError("h and W must have the same dtype")
    if labels.dtype != torch.int64:
        raise TypeError("labels must be int64")
    if not (h.is_contiguous() and W.is_contiguous() and labels.is_contiguous()):
        raise ValueError("h, W and labels must be contiguous")


def workspace_size(L: int, H: int, V: int, dtype=torch.bfloat16,
                   chunk_rows: int = 0) -> int:
    code = LCE_BF16 if dtype == torch.bfloat16 else LCE_F32
    n = load().lce_workspace_size(L, H, V, code, chunk_rows)
    if n == 0:
        raise ValueError(f"invalid sizes L={L} H={H} V={V} chunk={chunk_rows}")
    return n


def default_chunk_rows(L: int, H: int, V: int) -> int:
    return load().lce_default_chunk_rows(L, H, V)


def alloc_workspace(L, H, V, dtype, chunk_rows, device) -> torch.Tensor:
    return torch.empty(workspace_size(L, H, V, dtype, chunk_rows),
                       dtype=torch.uint8, device=device)


def _opts(label_smoothing: float, z_loss: float):
    """The lce_loss_opts pointer for a loss variant, or None (plain loss)."""
    if label_smoothing == 0.0 and z_loss == 0.0:
        return None
    return ctypes.pointer(LossOpts(float(label_smoothing), float(z_loss)))


def forward(h: torch.Tensor, W: torch.Tensor, labels: torch.Tensor,
            ignore_index: int = IGNORE_INDEX, workspace=None,
            loss_out=None, lse_out=None, label_smoothing: float = 0.0,
            z_loss: float = 0.0):
    """Returns (loss [scalar fp32], lse [L] fp32), both on h's device.
    label_smoothing / z_loss select a loss variant (lce_forward_ex)."""
    lib = load()
    _check_inputs(h, W, labels)
    L, H = h.shape
    V = W.shape[0]
    dev = h.device
    if workspace is None:
        workspace = alloc_workspace(L, H, V, h.dtype, 0, dev)
    loss = loss_out if loss_out is not None else torch.empty((), dtype=torch.float32, device=dev)
    lse = lse_out if lse_out is not None else torch.empty(L, dtype=torch.float32, device=dev)
    opts = _opts(label_smoothing, z_loss)
    if opts is None:
        st = lib.lce_forward(h.data_ptr(), W.data_ptr(), _dtype_code(h),
                             labels.data_ptr(), L, H, V, ignore_index,
                             loss.data_ptr(), lse.data_ptr(),
                             workspace.data_ptr(), workspace.numel(),
                             _stream_ptr(dev))
        _check(st, "lce_forward")
    else:
        st = lib.lce_forward_ex(h.data_ptr(), W.data_ptr(), _dtype_code(h),
                                labels.data_ptr(), L, H, V, ignore_index,
                                opts, loss.data_ptr(), lse.data_ptr(),
                                workspace.data_ptr(), workspace.numel(),
                                _stream_ptr(dev))
        _check(st, "lce_forward_ex")
    _written(loss, lse)
    return loss, lse


def backward(h: torch.Tensor, W: torch.Tensor, labels: torch.Tensor,
             lse: torch.Tensor, dloss: torch.Tensor,
             ignore_index: int = IGNORE_INDEX, chunk_rows: int = 0,
             workspace=None, dH_out=None, dW_out=None,
             label_smoothing: float = 0.0, z_loss: float = 0.0,
             compute_dH: bool = True, compute_dW: bool = True):
    """Returns (dH [L,H] of h's dtype, dW [V,H] fp32). The loss variant
    must be the forward's. compute_dH / compute_dW = False skips that
    gradient's contraction (returned as None; at least one is needed)."""
    lib = load()
    _check_inputs(h, W, labels)
    L, H = h.shape
    V = W.shape[0]
    dev = h.device
    if lse.dtype != torch.float32 or lse.shape != (L,) or not lse.is_cuda:
        raise ValueError("lse must be a CUDA float32 [L] tensor")
    dloss = dloss.reshape(1).to(device=dev, dtype=torch.float32).contiguous()
    if workspace is None:
        workspace = alloc_workspace(L, H, V, h.dtype, chunk_rows, dev)
    dH, dW = _grad_outputs(h, V, dH_out, dW_out, compute_dH, compute_dW)
    opts = _opts(label_smoothing, z_loss)
    if opts is None:
        st = lib.lce_backward(h.data_ptr(), W.data_ptr(), _dtype_code(h),
                              labels.data_ptr(), lse.data_ptr(), L, H, V,
                              ignore_index, dloss.data_ptr(), chunk_rows,
                              _ptr(dH), _ptr(dW), workspace.data_ptr(),
                              workspace.numel(), _stream_ptr(dev))
        _check(st, "lce_backward")
    else:
        st = lib.lce_backward_ex(h.data_ptr(), W.data_ptr(), _dtype_code(h),
                                 labels.data_ptr(), lse.data_ptr(), L, H, V,
                                 ignore_index, opts, dloss.data_ptr(),
                                 chunk_rows, _ptr(dH), _ptr(dW),
                                 workspace.data_ptr(), workspace.numel(),
                                 _stream_ptr(dev))
        _check(st, "lce_backward_ex")
    _written(dH, dW)
    return dH, dW


def _ptr(t):
    """A tensor's device pointer, or None (NULL) for an absent one."""
    return None if t is None else t.data_ptr()


def _grad_outputs(h, V, dH_out, dW_out, compute_dH, compute_dW):
    """The dH [L,H] (h's dtype) and dW [V,H] fp32 outputs, None where the
    gradient is not wanted."""
    L, H = h.shape
    dH = dW = None
    if compute_dH:
        dH = dH_out if dH_out is not None else torch.empty_like(h)
    if compute_dW:
        dW = dW_out if dW_out is not None else torch.empty(
            V, H, dtype=torch.float32, device=h.device)
    return dH, dW


def forward_backward(h: torch.Tensor, W: torch.Tensor, labels: torch.Tensor,
                     ignore_index: int = IGNORE_INDEX, chunk_rows: int = 0,
                     workspace=None, loss_out=None, lse_out=None, dH_out=None,
                     dW_out=None, label_smoothing: float = 0.0,
                     z_loss: float = 0.0, compute_dH: bool = True,
                     compute_dW: bool = True):
    """Loss, lse and the gradients of the loss itself (dloss = 1) in one
    call, without recomputing the logits. Returns (loss, lse, dH, dW);
    compute_dH / compute_dW = False skips that gradient (None)."""
    lib = load()
    _check_inputs(h, W, labels)
    L, H = h.shape
    V = W.shape[0]
    dev = h.device
    if workspace is None:
        workspace = alloc_workspace(L, H, V, h.dtype, chunk_rows, dev)
    loss = loss_out if loss_out is not None else torch.empty((), dtype=torch.float32, device=dev)
    lse = lse_out if lse_out is not None else torch.empty(L, dtype=torch.float32, device=dev)
    dH, dW = _grad_outputs(h, V, dH_out, dW_out, compute_dH, compute_dW)
    opts = _opts(label_smoothing, z_loss)
    if opts is None:
        st = lib.lce_forward_backward(h.data_ptr(), W.data_ptr(),
                                      _dtype_code(h), labels.data_ptr(), L, H,
                                      V, ignore_index, chunk_rows,
                                      loss.data_ptr(), lse.data_ptr(),
                                      _ptr(dH), _ptr(dW),
                                      workspace.data_ptr(), workspace.numel(),
                                      _stream_ptr(dev))
        _check(st, "lce_forward_backward")
    else:
        st = lib.lce_forward_backward_ex(h.data_ptr(), W.data_ptr(),
                                         _dtype_code(h), labels.data_ptr(), L,
                                         H, V, ignore_index, opts, chunk_rows,
                                         loss.data_ptr(), lse.data_ptr(),
                                         _ptr(dH), _ptr(dW),
                                         workspace.data_ptr(),
                                         workspace.numel(), _stream_ptr(dev))
        _check(st, "lce_forward_backward_ex")
    _written(loss, lse, dH, dW)
    return loss, lse, dH, dW


def scale_gradients(dH, dW, dloss: torch.Tensor):
    """dH *= dloss and dW *= dloss in place (dloss a device scalar); either
    gradient may be None."""
    ref = dH if dH is not None else dW
    if ref is None:
        return dH, dW
    L, H = dH.shape if dH is not None else (1, dW.shape[1])
    V = dW.shape[0] if dW is not None else 1
    code = _dtype_code(dH) if dH is not None else LCE_BF16
    dloss = dloss.reshape(1).to(device=ref.device,
                                dtype=torch.float32).contiguous()
    st = load().lce_scale_gradients(_ptr(dH), code, L, H, _ptr(dW), V,
                                    dloss.data_ptr(), _stream_ptr(ref.device))
    _check(st, "lce_scale_gradients")
    _written(dH, dW)
    return dH, dW


def count_valid(labels: torch.Tensor, V: int,
                ignore_index: int = IGNORE_INDEX, out=None) -> torch.Tensor:
    """Device int64 [1]: rows whose label is not ignore_index and lies in
    [0, V) (the N of the mean loss); no host synchronisation."""
    if labels.dtype != torch.int64 or labels.dim() != 1 or not labels.is_cuda:
        raise ValueError("labels must be a 1-D int64 CUDA tensor")
    labels = labels.contiguous()
    if out is None:
        out = torch.empty(1, dtype=torch.int64, device=labels.device)
    st = load().lce_count_valid(labels.data_ptr(), labels.numel(), V,
                                ignore_index, out.data_ptr(),
                                _stream_ptr(labels.device))
    _check(st, "lce_count_valid")
    _written(out)
    return out


def shard_sums(loss_local: torch.Tensor, n_local: torch.Tensor,
               out=None) -> torch.Tensor:
    """Device float64 [2] = (N_r loss_r, N_r) of one row shard, to be summed
    over the shards (lce_shard_sums)."""
    loss_local = loss_local.reshape(1).to(torch.float32).contiguous()
    n_local = n_local.reshape(1).to(torch.int64).contiguous()
    dev = loss_local.device
    if out is None:
        out = torch.empty(2, dtype=torch.float64, device=dev)
    st = load().lce_shard_sums(loss_local.data_ptr(), n_local.data_ptr(),
                               out.data_ptr(), _stream_ptr(dev))
    _check(st, "lce_shard_sums")
    _written(out)
    return out


def combine_shards(sums: torch.Tensor, n_local: torch.Tensor,
                   dloss: torch.Tensor | None = None):
    """From the shards' summed (S, N): (loss = S / N, this shard's gradient
    weight dloss N_r / N), device float32 scalars, 0 when N = 0
    (lce_combine_shards)."""
    if sums.dtype != torch.float64 or sums.numel() != 2 or not sums.is_cuda:
        raise ValueError("sums must be a CUDA float64 tensor of 2 elements")
    sums = sums.contiguous()
    dev = sums.device
    n_local = n_local.reshape(1).to(torch.int64).contiguous()
    d = None
    if dloss is not None:
        d = dloss.reshape(1).to(device=dev, dtype=torch.float32).contiguous()
    loss = torch.empty((), dtype=torch.float32, device=dev)
    weight = torch.empty((), dtype=torch.float32, device=dev)
    st = load().lce_combine_shards(sums.data_ptr(), n_local.data_ptr(),
                                   d.data_ptr() if d is not None else None,
                                   loss.data_ptr(), weight.data_ptr(),
                                   _stream_ptr(dev))
    _check(st, "lce_combine_shards")
    return loss, weight


def _slice_out(out, L, label_smoothing, dev):
    """Rows m, s, zy (and zsum under label smoothing) of a [3 or 4, L]
    float32 tensor."""
    rows = 4 if label_smoothing != 0.0 else 3
    if out is None:
        out = torch.empty(rows, L, dtype=torch.float32, device=dev)
    if out.dtype != torch.float32 or out.shape != (rows, L):
        raise ValueError(f"out must be float32 [{rows}, {L}]")
    return out, tuple(out[r] for r in range(rows))


def forward_slice(h: torch.Tensor, W_slice: torch.Tensor,
                  labels: torch.Tensor, v0: int, V_total: int,
                  ignore_index: int = IGNORE_INDEX, workspace=None,
                  out=None, label_smoothing: float = 0.0,
                  z_loss: float = 0.0):
    """One vocabulary slice (W_slice = rows v0 .. v0 + Vs - 1 of the head):
    returns (m, s, zy), each float32 [L]: the slice's per-row max logit, sum
    of exp(z - m), and label logit (0 where the label is elsewhere); under
    label smoothing also zsum, the slice's per-row sum of logits, as a
    fourth (lce_forward_slice_ex)."""
    lib = load()
    _check_inputs(h, W_slice, labels)
    L, H = h.shape
    Vs = W_slice.shape[0]
    dev = h.device
    if workspace is None:
        workspace = alloc_workspace(L, H, Vs, h.dtype, 0, dev)
    out, rows = _slice_out(out, L, label_smoothing, dev)
    opts = _opts(label_smoothing, z_loss)
    if opts is None:
        st = lib.lce_forward_slice(h.data_ptr(), W_slice.data_ptr(),
                                   _dtype_code(h), labels.data_ptr(), L, H,
                                   Vs, v0, V_total, ignore_index,
                                   rows[0].data_ptr(), rows[1].data_ptr(),
                                   rows[2].data_ptr(), workspace.data_ptr(),
                                   workspace.numel(), _stream_ptr(dev))
    else:
        st = lib.lce_forward_slice_ex(
            h.data_ptr(), W_slice.data_ptr(), _dtype_code(h),
            labels.data_ptr(), L, H, Vs, v0, V_total, ignore_index, opts,
            rows[0].data_ptr(), rows[1].data_ptr(), rows[2].data_ptr(),
            rows[3].data_ptr() if len(rows) == 4 else None,
            workspace.data_ptr(), workspace.numel(), _stream_ptr(dev))
    _check(st, "lce_forward_slice")
    _written(out)
    return rows


def combine_slices(m: torch.Tensor, s: torch.Tensor, zy: torch.Tensor,
                   labels: torch.Tensor, V_total: int,
                   ignore_index: int = IGNORE_INDEX, workspace=None,
                   zsum=None, label_smoothing: float = 0.0,
                   z_loss: float = 0.0):
    """m, s, zy (and zsum under label smoothing): float32 [P, L] (every
    slice's forward_slice output, in the same slice order on every
    process). Returns (loss, lse [L])."""
    lib = load()
    P, L = m.shape
    ts = (m, s, zy) if zsum is None else (m, s, zy, zsum)
    for t in ts:
        if t.dtype != torch.float32 or t.shape != (P, L) or not t.is_cuda:
            raise ValueError("m, s, zy, zsum must be CUDA float32 [P, L] "
                             "tensors")
    m, s, zy = m.contiguous(), s.contiguous(), zy.contiguous()
    zsum = zsum.contiguous() if zsum is not None else None
    labels = labels.contiguous()
    dev = m.device
    if workspace is None:
        workspace = torch.empty(lib.lce_combine_workspace_size(L),
                                dtype=torch.uint8, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(L, dtype=torch.float32, device=dev)
    opts = _opts(label_smoothing, z_loss)
    if opts is None:
        st = lib.lce_combine_slices(m.data_ptr(), s.data_ptr(), zy.data_ptr(),
                                    P, labels.data_ptr(), L, V_total,
                                    ignore_index, loss.data_ptr(),
                                    lse.data_ptr(), workspace.data_ptr(),
                                    workspace.numel(), _stream_ptr(dev))
    else:
        st = lib.lce_combine_slices_ex(
            m.data_ptr(), s.data_ptr(), zy.data_ptr(),
            zsum.data_ptr() if zsum is not None else None, P,
            labels.data_ptr(), L, V_total, ignore_index, opts,
            loss.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
            workspace.numel(), _stream_ptr(dev))
    _check(st, "lce_combine_slices")
    return loss, lse


def backward_slice(h: torch.Tensor, W_slice: torch.Tensor,
                   labels: torch.Tensor, lse: torch.Tensor,
                   dloss: torch.Tensor, v0: int, V_total: int,
                   ignore_index: int = IGNORE_INDEX, chunk_rows: int = 0,
                   workspace=None, label_smoothing: float = 0.0,
                   z_loss: float = 0.0, compute_dH: bool = True,
                   compute_dW: bool = True):
    """One vocabulary slice's backward from the merged lse: returns
    (dH_part [L,H] float32, whose sum over slices is dH; dW_slice [Vs,H]);
    compute_dH / compute_dW = False skips that one (None)."""
    lib = load()
    _check_inputs(h, W_slice, labels)
    L, H = h.shape
    Vs = W_slice.shape[0]
    dev = h.device
    if lse.dtype != torch.float32 or lse.shape != (L,) or not lse.is_cuda:
        raise ValueError("lse must be a CUDA float32 [L] tensor")
    dloss = dloss.reshape(1).to(device=dev, dtype=torch.float32).contiguous()
    if workspace is None:
        workspace = alloc_workspace(L, H, Vs, h.dtype, chunk_rows, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dH = torch.empty(L, H, **f32) if compute_dH else None
    dW = torch.empty(Vs, H, **f32) if compute_dW else None
    st = lib.lce_backward_slice_ex(h.data_ptr(), W_slice.data_ptr(),
                                   _dtype_code(h), labels.data_ptr(),
                                   lse.data_ptr(), L, H, Vs, v0, V_total,
                                   ignore_index,
                                   _opts(label_smoothing, z_loss),
                                   dloss.data_ptr(), chunk_rows,
                                   _ptr(dH), _ptr(dW),
                                   workspace.data_ptr(), workspace.numel(),
                                   _stream_ptr(dev))
    _check(st, "lce_backward_slice")
    return dH, dW


def slice_exp_workspace(L: int, H: int, Vs: int, dtype, device):
    """The workspace forward_slice_exp fills and backward_slice_exp reads."""
    n = load().lce_slice_exp_workspace_size(
        L, H, Vs, LCE_F32 if dtype == torch.float32 else LCE_BF16)
    if n == 0:
        raise ValueError("invalid sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward_slice_exp(h, W_slice, labels, v0: int, V_total: int, workspace,
                      ignore_index: int = IGNORE_INDEX, out=None,
                      label_smoothing: float = 0.0, z_loss: float = 0.0):
    """forward_slice that also keeps the slice's tile exponentials in
    `workspace` (from slice_exp_workspace) for backward_slice_exp."""
    lib = load()
    _check_inputs(h, W_slice, labels)
    L, H = h.shape
    Vs = W_slice.shape[0]
    out, rows = _slice_out(out, L, label_smoothing, h.device)
    st = lib.lce_forward_slice_exp_ex(
        h.data_ptr(), W_slice.data_ptr(), _dtype_code(h), labels.data_ptr(),
        L, H, Vs, v0, V_total, ignore_index, _opts(label_smoothing, z_loss),
        rows[0].data_ptr(), rows[1].data_ptr(), rows[2].data_ptr(),
        rows[3].data_ptr() if len(rows) == 4 else None,
        workspace.data_ptr(), workspace.numel(), _stream_ptr(h.device))
    _check(st, "lce_forward_slice_exp")
    _written(out)
    return rows


def backward_slice_exp(h, W_slice, labels, lse, dloss, v0: int, V_total: int,
                       workspace, ignore_index: int = IGNORE_INDEX,
                       label_smoothing: float = 0.0, z_loss: float = 0.0,
                       compute_dH: bool = True, compute_dW: bool = True):
    """The slice's backward from the exponentials forward_slice_exp kept:
    returns (dH_part [L,H] float32, dW_slice [Vs,H] float32), None for a
    gradient not asked for."""
    lib = load()
    _check_inputs(h, W_slice, labels)
    L, H = h.shape
    Vs = W_slice.shape[0]
    dev = h.device
    if lse.dtype != torch.float32 or lse.shape != (L,) or not lse.is_cuda:
        raise ValueError("lse must be a CUDA float32 [L] tensor")
    dloss = dloss.reshape(1).to(device=dev, dtype=torch.float32).contiguous()
    f32 = dict(dtype=torch.float32, device=dev)
    dH = torch.empty(L, H, **f32) if compute_dH else None
    dW = torch.empty(Vs, H, **f32) if compute_dW else None
    st = lib.lce_backward_slice_exp_ex(h.data_ptr(), W_slice.data_ptr(),
                                       _dtype_code(h), labels.data_ptr(),
                                       lse.data_ptr(), L, H, Vs, v0, V_total,
                                       ignore_index,
                                       _opts(label_smoothing, z_loss),
                                       dloss.data_ptr(), _ptr(dH), _ptr(dW),
                                       workspace.data_ptr(),
                                       workspace.numel(),
                                       _stream_ptr(dev))
    _check(st, "lce_backward_slice_exp")
    return dH, dW


def get_error(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device
    error status: LCE_OK, LCE_ERR_TIMEOUT, LCE_ERR_LABEL_RANGE or
    LCE_ERR_EXPERT_RANGE."""
    return load().lce_get_error(_stream_ptr(device))


def tc_gemm(A: torch.Tensor, B: torch.Tensor, M: int, N: int, K: int,
              a_mn: bool, b_mn: bool) -> torch.Tensor:
    """D = A B (fp32) through the tensor-core building block.
    A: [M,K] if not a_mn else [K,M]; B: [N,K] if not b_mn else [K,N]."""
    lib = load()
    D = torch.empty(M, N, dtype=torch.float32, device=A.device)
    st = lib.lce_test_gemm(A.data_ptr(), B.data_ptr(), D.data_ptr(), M, N, K,
                           int(a_mn), int(b_mn), _stream_ptr(A.device))
    _check(st, "lce_test_gemm")
    return D


def wait_timeout_probe(timeout_ns: int, device=None):
    st = load().lce_test_wait_timeout(timeout_ns, _stream_ptr(device))
    _check(st, "lce_test_wait_timeout")


def _check_mlp(x, Wg, Wu, Wd):
    ts = (x, Wg, Wu, Wd)
    if not all(t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
               for t in ts):
        raise ValueError("x, Wg, Wu, Wd must be contiguous bf16 CUDA tensors")
    L, H = x.shape
    I = Wg.shape[0]
    if Wg.shape != (I, H) or Wu.shape != (I, H) or Wd.shape != (H, I):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, Wg "
                         f"{tuple(Wg.shape)}, Wu {tuple(Wu.shape)}, Wd "
                         f"{tuple(Wd.shape)}")
    return L, H, I


def mlp_workspace_size(L: int, H: int, I: int, chunk_rows: int = 0) -> int:
    n = load().lce_mlp_workspace_size(L, H, I, chunk_rows)
    if n == 0:
        raise ValueError(f"invalid MLP sizes L={L} H={H} I={I}")
    return n


def mlp_forward(x, Wg, Wu, Wd, chunk_rows: int = 0, workspace=None,
                y_out=None):
    """y = (silu(x Wg^T) * (x Wu^T)) Wd^T over row chunks (bf16)."""
    lib = load()
    L, H, I = _check_mlp(x, Wg, Wu, Wd)
    if workspace is None:
        workspace = torch.empty(mlp_workspace_size(L, H, I, chunk_rows),
                                dtype=torch.uint8, device=x.device)
    y = y_out if y_out is not None else torch.empty_like(x)
    st = lib.lce_mlp_forward(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                             Wd.data_ptr(), L, H, I, chunk_rows, y.data_ptr(),
                             workspace.data_ptr(), workspace.numel(),
                             _stream_ptr(x.device))
    _check(st, "lce_mlp_forward")
    _written(y_out)
    return y


def mlp_backward(x, Wg, Wu, Wd, dy, chunk_rows: int = 0, workspace=None,
                 dx_out=None, dWg_out=None, dWu_out=None, dWd_out=None,
                 compute_dx: bool = True, compute_dWgu: bool = True,
                 compute_dWd: bool = True):
    """Returns (dx bf16 [L,H], dWg fp32 [I,H], dWu fp32 [I,H], dWd fp32
    [H,I]) for upstream gradient dy, recomputing the chunk intermediates.
    compute_dx / compute_dWgu (dWg and dWu) / compute_dWd = False skips
    that gradient's contraction (returned as None)."""
    lib = load()
    L, H, I = _check_mlp(x, Wg, Wu, Wd)
    if not (dy.is_cuda and dy.dtype == torch.bfloat16 and dy.is_contiguous()
            and dy.shape == (L, H)):
        raise ValueError("dy must be a contiguous bf16 CUDA [L,H] tensor")
    dev = x.device
    if workspace is None:
        workspace = torch.empty(mlp_workspace_size(L, H, I, chunk_rows),
                                dtype=torch.uint8, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dx = dWg = dWu = dWd = None
    if compute_dx:
        dx = dx_out if dx_out is not None else torch.empty_like(x)
    if compute_dWgu:
        dWg = dWg_out if dWg_out is not None else torch.empty(I, H, **f32)
        dWu = dWu_out if dWu_out is not None else torch.empty(I, H, **f32)
    if compute_dWd:
        dWd = dWd_out if dWd_out is not None else torch.empty(H, I, **f32)
    st = lib.lce_mlp_backward(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                              Wd.data_ptr(), dy.data_ptr(), L, H, I,
                              chunk_rows, _ptr(dx), _ptr(dWg), _ptr(dWu),
                              _ptr(dWd), workspace.data_ptr(),
                              workspace.numel(), _stream_ptr(dev))
    _check(st, "lce_mlp_backward")
    _written(dx, dWg, dWu, dWd)
    return dx, dWg, dWu, dWd


@functools.lru_cache(maxsize=256)
def _route_opts_of(*values):
    """The lce_route_opts pointer of plain values, its fields in order."""
    if not all(-2 ** 31 <= v < 2 ** 31 for v in values[1:5]):
        raise ValueError("top_k, n_group, topk_group and group_top must fit "
                         "in 32 bits")
    return ctypes.pointer(RouteOpts(*values))


def _route_opts(scoring, top_k, n_group, topk_group, group_top, renormalize,
                scale):
    if scoring not in SCORING:
        raise ValueError(f"scoring must be one of {sorted(SCORING)}, got "
                         f"{scoring!r}")
    # kept by value: a number that lives in a tensor is read at each call
    return _route_opts_of(SCORING[scoring], operator.index(top_k),
                          operator.index(n_group), operator.index(topk_group),
                          operator.index(group_top), int(bool(renormalize)),
                          float(scale))


def _check_logits(logits):
    if not logits.is_cuda or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA [L,E] tensor")
    return _dtype_code(logits)


def _check_out(name, t, shape, dtype, device):
    """An output the caller gives is written as it stands."""
    if (t.shape != shape or t.dtype is not dtype or t.device != device or
            not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of "
                         f"shape {tuple(shape)} on {device}")
    return t


def _check_workspace(workspace, device):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def route_forward(logits: torch.Tensor, top_k: int, scoring: str = "softmax",
                  bias=None, n_group: int = 1, topk_group: int = 1,
                  group_top: int = 1, renormalize: bool = True,
                  scale: float = 1.0, weights_out=None, experts_out=None):
    """Routes each row of router logits [L,E] (bf16 or fp32) to top_k
    experts: returns (weights [L,top_k] of logits' dtype, experts [L,top_k]
    int32). bias: float32 [E] added to the scores for the selection alone;
    n_group / topk_group / group_top: group-limited selection
    (lce_route_forward)."""
    lib = load()
    code = _check_logits(logits)
    L, E = logits.shape
    dev = logits.device
    opts = _route_opts(scoring, top_k, n_group, topk_group, group_top,
                       renormalize, scale)
    if bias is not None and not (bias.is_cuda and bias.shape == (E,) and
                                 bias.dtype == torch.float32 and
                                 bias.is_contiguous()):
        raise ValueError("bias must be a contiguous CUDA float32 [E] tensor")
    shape = (L, max(top_k, 0))
    if weights_out is not None:
        weights = _check_out("weights_out", weights_out, shape, logits.dtype,
                             dev)
    else:
        weights = torch.empty(shape, dtype=logits.dtype, device=dev)
    if experts_out is not None:
        experts = _check_out("experts_out", experts_out, shape, torch.int32,
                             dev)
    else:
        experts = torch.empty(shape, dtype=torch.int32, device=dev)
    st = lib.lce_route_forward(logits.data_ptr(), code, _ptr(bias), L, E,
                               opts, weights.data_ptr(),
                               experts.data_ptr(), _stream_ptr(dev))
    _check(st, "lce_route_forward")
    if weights_out is not None or experts_out is not None:
        _written(weights_out, experts_out)
    return weights, experts


def route_backward(logits: torch.Tensor, experts: torch.Tensor,
                   dweights: torch.Tensor, scoring: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0,
                   dlogits_out=None) -> torch.Tensor:
    """dlogits [L,E] (logits' dtype) of route_forward from dweights
    [L,top_k], the selection being constant (lce_route_backward)."""
    lib = load()
    code = _check_logits(logits)
    L, E = logits.shape
    dev = logits.device
    _check_experts(experts, L)
    k = experts.shape[1]
    if not (dweights.is_cuda and dweights.shape == (L, k) and
            dweights.dtype == logits.dtype and dweights.is_contiguous()):
        raise ValueError("dweights must be a contiguous CUDA [L,top_k] tensor "
                         "of logits' dtype")
    opts = _route_opts(scoring, k, 1, 1, 1, renormalize, scale)
    if dlogits_out is not None:
        out = _check_out("dlogits_out", dlogits_out, logits.shape,
                         logits.dtype, dev)
    else:
        out = torch.empty_like(logits)
    st = lib.lce_route_backward(logits.data_ptr(), code, experts.data_ptr(),
                                dweights.data_ptr(), L, E, opts,
                                out.data_ptr(), _stream_ptr(dev))
    _check(st, "lce_route_backward")
    if dlogits_out is not None:
        _written(dlogits_out)
    return out


def _check_experts(experts, L):
    if (experts.dtype is not torch.int32 or not experts.is_cuda or
            experts.dim() != 2 or experts.size(0) != L or
            not experts.is_contiguous()):
        raise ValueError("experts must be a contiguous CUDA int32 [L,top_k] "
                         "tensor")


def _check_experts_mlp(x, Wg, Wu, Wd, weights, experts):
    for t in (x, Wg, Wu, Wd):
        if (t.dtype is not torch.bfloat16 or not t.is_cuda or
                not t.is_contiguous()):
            raise ValueError("x, Wg, Wu, Wd must be contiguous bf16 CUDA "
                             "tensors")
    if x.dim() != 2 or Wg.dim() != 3:
        raise ValueError("expected x [L,H], Wg and Wu [E,I,H], Wd [E,H,I]")
    L, H = x.shape
    shape = Wg.shape
    E, I, Hw = shape
    if Hw != H or Wu.shape != shape or Wd.shape != (E, H, I):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, Wg "
                         f"{tuple(Wg.shape)}, Wu {tuple(Wu.shape)}, Wd "
                         f"{tuple(Wd.shape)}")
    _check_experts(experts, L)
    shape = experts.shape
    if (weights.shape != shape or not weights.is_cuda or
            not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous CUDA tensor of "
                         "experts' shape")
    return L, H, I, E, shape[1], _dtype_code(weights)


@functools.lru_cache(maxsize=1024)
def experts_workspace_size(L: int, H: int, I: int, E: int, top_k: int,
                           backward: bool = False) -> int:
    n = load().lce_experts_workspace_size(L, H, I, E, top_k, int(backward))
    if n == 0:
        raise ValueError(f"invalid experts sizes L={L} H={H} I={I} E={E} "
                         f"top_k={top_k}")
    return n


def experts_forward(x, Wg, Wu, Wd, weights, experts, workspace=None,
                    y_out=None):
    """y_t = sum_k weights[t,k] Wd_e (silu(Wg_e x_t) * (Wu_e x_t)), e =
    experts[t,k] (-1: dropped): x bf16 [L,H], Wg and Wu bf16 [E,I,H], Wd bf16
    [E,H,I], weights [L,top_k] (bf16 or fp32), experts int32 [L,top_k]."""
    L, H, I, E, K, code = _check_experts_mlp(x, Wg, Wu, Wd, weights, experts)
    dev = x.device
    if workspace is None:
        workspace = torch.empty(experts_workspace_size(L, H, I, E, K),
                                dtype=torch.uint8, device=dev)
    else:
        _check_workspace(workspace, dev)
    if y_out is not None:
        y = _check_out("y_out", y_out, x.shape, x.dtype, dev)
    else:
        y = torch.empty_like(x)
    st = load().lce_experts_forward(
        x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
        weights.data_ptr(), code, experts.data_ptr(), L, H, I, E, K,
        y.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream_ptr(dev))
    if st:
        _check(st, "lce_experts_forward")
    if y_out is not None:
        _written(y_out)
    return y


def experts_backward(x, Wg, Wu, Wd, weights, experts, dy, workspace=None,
                     grad_dtype=torch.float32, compute_dx: bool = True,
                     compute_dWgu: bool = True, compute_dWd: bool = True,
                     compute_dweights: bool = True):
    """Returns (dx bf16 [L,H], dWg, dWu, dWd of grad_dtype (fp32 or bf16) in
    the weights' shapes, dweights of weights' dtype) for upstream gradient dy,
    recomputing the intermediates. compute_* = False skips that gradient
    (returned as None)."""
    lib = load()
    L, H, I, E, K, code = _check_experts_mlp(x, Wg, Wu, Wd, weights, experts)
    if not (dy.is_cuda and dy.dtype == torch.bfloat16 and dy.is_contiguous()
            and dy.shape == (L, H)):
        raise ValueError("dy must be a contiguous bf16 CUDA [L,H] tensor")
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("grad_dtype must be float32 or bfloat16")
    if workspace is None:
        workspace = torch.empty(experts_workspace_size(L, H, I, E, K, True),
                                dtype=torch.uint8, device=x.device)
    else:
        _check_workspace(workspace, x.device)
    dx = dWg = dWu = dWd = dw = None
    if compute_dx:
        dx = torch.empty_like(x)
    if compute_dWgu:
        dWg = torch.empty_like(Wg, dtype=grad_dtype)
        dWu = torch.empty_like(Wu, dtype=grad_dtype)
    if compute_dWd:
        dWd = torch.empty_like(Wd, dtype=grad_dtype)
    if compute_dweights:
        dw = torch.empty_like(weights)
    st = lib.lce_experts_backward(
        x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
        weights.data_ptr(), code, experts.data_ptr(), dy.data_ptr(), L, H, I,
        E, K, LCE_F32 if grad_dtype == torch.float32 else LCE_BF16, _ptr(dx),
        _ptr(dWg), _ptr(dWu), _ptr(dWd), _ptr(dw), workspace.data_ptr(),
        workspace.numel(), _stream_ptr(x.device))
    _check(st, "lce_experts_backward")
    return dx, dWg, dWu, dWd, dw


def _call(name, device, *args):
    """One call of the library with the tensors' device current, on that
    device's current stream (the last argument)."""
    index = device.index
    fn = getattr(_lib or load(), name)
    if index is None:
        st = fn(*args, _stream_ptr(device))
    elif index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _check(st, name)


def _check_rows(name, t, shape, dtype, device):
    """An input of known shape and type, as the C ABI reads it."""
    if (t.dtype is not dtype or t.shape != shape or t.device != device or
            not t.is_cuda or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of "
                         f"shape {tuple(shape)} on {device}")
    return t


_TYPE_CODES = {torch.bfloat16: LCE_BF16, torch.float32: LCE_F32}


def _check_norm(x, weight, bias):
    """Device, sizes and type codes (of x, of the parameters) of a norm's
    inputs."""
    if not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA [L,H] tensor")
    code = param = _TYPE_CODES.get(x.dtype)
    if code is None:
        _dtype_code(x)  # raises
    L, H = x.shape
    device = x.device
    if weight is not None:
        param = _TYPE_CODES.get(weight.dtype)
        if param is None:
            _dtype_code(weight)
        _check_rows("weight", weight, (H,), weight.dtype, device)
    if bias is not None:
        dtype = bias.dtype if weight is None else weight.dtype
        param = _TYPE_CODES.get(dtype)
        if param is None:
            _dtype_code(bias)
        _check_rows("bias", bias, (H,), dtype, device)
    return device, L, H, code, param


@functools.lru_cache(maxsize=1024)
def norm_workspace_size(L: int, H: int) -> int:
    """Bytes of workspace that a norm's backward needs for the parameters'
    gradients."""
    n = load().lce_norm_workspace_size(L, H)
    if n == 0:
        raise ValueError(f"invalid norm sizes L={L} H={H}")
    return n


def _norm_forward(kind, x, weight, bias, eps, y_out, save_stats):
    dev, L, H, code, param = _check_norm(x, weight, bias)
    if y_out is not None:
        y = _check_out("y_out", y_out, x.shape, x.dtype, dev)
    else:
        y = torch.empty_like(x)
    mean = rstd = None
    if save_stats:
        rstd = torch.empty(L, dtype=torch.float32, device=dev)
        if kind == LAYER_NORM:
            mean = torch.empty_like(rstd)
    _call("lce_norm_forward", dev, kind, x.data_ptr(), code,
          None if weight is None else weight.data_ptr(),
          None if bias is None else bias.data_ptr(), param, L, H, float(eps),
          y.data_ptr(), None if mean is None else mean.data_ptr(),
          None if rstd is None else rstd.data_ptr())
    if y_out is not None:
        _written(y_out)
    return y, mean, rstd


def _norm_backward(kind, x, weight, mean, rstd, dy, grad_dtype, workspace,
                   dx_out, compute_dx, compute_dweight, compute_dbias):
    dev, L, H, code, param = _check_norm(x, weight, None)
    _check_rows("dy", dy, x.shape, x.dtype, dev)
    _check_rows("rstd", rstd, (L,), torch.float32, dev)
    if kind == LAYER_NORM:
        _check_rows("mean", mean, (L,), torch.float32, dev)
    grad_code = _TYPE_CODES.get(grad_dtype)
    if grad_code is None:
        raise TypeError("grad_dtype must be float32 or bfloat16")
    dx = dw = db = None
    if compute_dx:
        if dx_out is not None:
            dx = _check_out("dx_out", dx_out, x.shape, x.dtype, dev)
        else:
            dx = torch.empty_like(x)
    if compute_dweight:
        dw = torch.empty(H, dtype=grad_dtype, device=dev)
    if compute_dbias:
        db = torch.empty(H, dtype=grad_dtype, device=dev)
    size = 0
    if workspace is not None:
        _check_workspace(workspace, dev)
        size = workspace.numel() * workspace.element_size()
    elif compute_dweight or compute_dbias:
        size = norm_workspace_size(L, H)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _call("lce_norm_backward", dev, kind, x.data_ptr(), code,
          None if weight is None else weight.data_ptr(), param,
          None if mean is None else mean.data_ptr(), rstd.data_ptr(),
          dy.data_ptr(), L, H, grad_code,
          None if dx is None else dx.data_ptr(),
          None if dw is None else dw.data_ptr(),
          None if db is None else db.data_ptr(),
          None if workspace is None else workspace.data_ptr(), size)
    if compute_dx and dx_out is not None:
        _written(dx_out)
    return dx, dw, db


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5,
                       y_out=None, save_stats: bool = True):
    """Layer norm of the rows of x [L,H] (bf16 or fp32): returns (y of x's
    type, mean [L], rstd [L] fp32, what the backward needs; None with
    save_stats=False). weight and bias: [H], both bf16 or both fp32, or None.
    y_out may be x (lce_norm_forward)."""
    return _norm_forward(LAYER_NORM, x, weight, bias, eps, y_out, save_stats)


def layer_norm_backward(x, weight, mean, rstd, dy, grad_dtype=torch.float32,
                        workspace=None, dx_out=None, compute_dx: bool = True,
                        compute_dweight: bool = True,
                        compute_dbias: bool = True):
    """Returns (dx [L,H] of x's type, dweight, dbias [H] of grad_dtype) for
    upstream gradient dy. compute_* = False skips that gradient (None);
    dx_out may be dy or x (lce_norm_backward)."""
    return _norm_backward(LAYER_NORM, x, weight, mean, rstd, dy, grad_dtype,
                          workspace, dx_out, compute_dx, compute_dweight,
                          compute_dbias)


def rms_norm_forward(x, weight=None, eps: float = 1e-6, y_out=None,
                     save_stats: bool = True):
    """RMS norm of the rows of x [L,H]: returns (y, rstd [L]), as
    layer_norm_forward without the mean and the bias."""
    y, _, rstd = _norm_forward(RMS_NORM, x, weight, None, eps, y_out,
                               save_stats)
    return y, rstd


def rms_norm_backward(x, weight, rstd, dy, grad_dtype=torch.float32,
                      workspace=None, dx_out=None, compute_dx: bool = True,
                      compute_dweight: bool = True):
    """Returns (dx, dweight) of rms_norm_forward, as layer_norm_backward."""
    dx, dw, _ = _norm_backward(RMS_NORM, x, weight, None, rstd, dy, grad_dtype,
                               workspace, dx_out, compute_dx, compute_dweight,
                               False)
    return dx, dw


def _check_mask(mask, L, device):
    if mask is not None:
        _check_rows("mask", mask, (L,), torch.bool, device)
    return mask


def _check_slots(experts, L, device):
    _check_experts(experts, L)
    if experts.device != device:
        raise ValueError(f"experts must be on {device}")
    return experts.shape[1]


@functools.lru_cache(maxsize=1024)
def balance_workspace_size(L: int, E: int) -> int:
    n = load().lce_balance_workspace_size(L, E)
    if n == 0:
        raise ValueError(f"invalid balance sizes L={L} E={E}")
    return n


def _scoring_code(scoring):
    if scoring not in SCORING:
        raise ValueError(f"scoring must be one of {sorted(SCORING)}, got "
                         f"{scoring!r}")
    return SCORING[scoring]


def balance_forward(logits, experts, scoring: str = "softmax",
                    coef: float = 1.0, mask=None, workspace=None):
    """The routing's balance loss coef * sum_e f_e mean_t p_te of router logits
    [L,E] (bf16 or fp32) and their experts int32 [L,top_k] (-1: dropped), over
    the tokens whose mask (bool [L]) is set: returns (loss [] fp32, counts [E]
    int32, slopes [E] fp32, what the backward needs) (lce_balance_forward)."""
    code = _check_logits(logits)
    L, E = logits.shape
    dev = logits.device
    K = _check_slots(experts, L, dev)
    _check_mask(mask, L, dev)
    score = _scoring_code(scoring)
    if workspace is None:
        workspace = torch.empty(balance_workspace_size(L, E),
                                dtype=torch.uint8, device=dev)
    else:
        _check_workspace(workspace, dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    slopes = torch.empty(E, dtype=torch.float32, device=dev)
    _call("lce_balance_forward", dev, logits.data_ptr(), code,
          experts.data_ptr(), None if mask is None else mask.data_ptr(), L, E,
          K, score, float(coef),
          loss.data_ptr(), counts.data_ptr(), slopes.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return loss, counts, slopes


def balance_backward(logits, slopes, dloss, scoring: str = "softmax",
                     mask=None, dlogits_out=None):
    """dlogits [L,E] (logits' type) of balance_forward for the gradient dloss
    of the loss (one fp32 value on the device), the counts being constant."""
    code = _check_logits(logits)
    L, E = logits.shape
    dev = logits.device
    _check_rows("slopes", slopes, (E,), torch.float32, dev)
    _check_mask(mask, L, dev)
    score = _scoring_code(scoring)
    if dloss.numel() != 1:
        raise ValueError("dloss must be one value")
    if dloss.dtype is not torch.float32 or dloss.device != dev:
        dloss = dloss.to(device=dev, dtype=torch.float32)
    if dlogits_out is not None:
        out = _check_out("dlogits_out", dlogits_out, logits.shape,
                         logits.dtype, dev)
    else:
        out = torch.empty_like(logits)
    _call("lce_balance_backward", dev, logits.data_ptr(), code,
          None if mask is None else mask.data_ptr(), L, E, score,
          slopes.data_ptr(), dloss.data_ptr(), out.data_ptr())
    if dlogits_out is not None:
        _written(dlogits_out)
    return out


def expert_counts(experts, num_experts: int, mask=None, counts_out=None):
    """Slots of each expert, int32 [num_experts], of experts int32 [L,top_k]
    (-1: dropped) over the tokens whose mask (bool [L]) is set."""
    L = experts.shape[0] if experts.dim() else 0
    dev = experts.device
    K = _check_slots(experts, L, dev)
    _check_mask(mask, L, dev)
    E = operator.index(num_experts)
    if counts_out is not None:
        counts = _check_out("counts_out", counts_out, (E,), torch.int32, dev)
    else:
        counts = torch.empty(max(E, 0), dtype=torch.int32, device=dev)
    _call("lce_expert_counts", dev, experts.data_ptr(),
          None if mask is None else mask.data_ptr(), L, E, K,
          counts.data_ptr())
    if counts_out is not None:
        _written(counts_out)
    return counts


def _dense(t):
    """Whether t's elements fill one run of memory without overlap, in any
    order of dimensions."""
    if t.numel() == 0:
        return True
    step = 1
    for stride, n in sorted((s, n) for s, n in zip(t.stride(), t.shape)
                            if n != 1):
        if stride != step:
            return False
        step *= n
    return True


_dtype_of = operator.attrgetter("dtype")


def _host_array(kind, code, values):
    """A C array of a list of numbers (array's conversion is the fast one)."""
    return (kind * len(values)).from_buffer(array.array(code, values))


class _GradTable:
    """Host arrays of a list of gradients, as the C ABI takes them. A list has
    hundreds of tensors: each property is asked of all of them at once."""

    def __init__(self, grads):
        given = self.given = list(grads)
        grads = self.grads = [g for g in given if g is not None]
        n = self.n = len(grads)
        if not n:
            self.device = torch.device("cuda", torch.cuda.current_device())
        else:
            self.device = grads[0].device
            if (not grads[0].is_cuda or
                    len(set(map(torch.Tensor.get_device, grads))) > 1):
                raise ValueError("gradients must be CUDA tensors on one "
                                 "device")
        try:
            codes = self.code_list = [_TYPE_CODES[t]
                                      for t in map(_dtype_of, grads)]
        except KeyError as e:
            raise TypeError(f"unsupported dtype {e.args[0]}; use bfloat16 or "
                            "float32") from None
        self.flat = all(map(torch.Tensor.is_contiguous, grads))
        if not self.flat and not all(map(_dense, grads)):
            raise ValueError("gradients must fill their memory without gaps "
                             "or overlap")
        self.ptrs = _host_array(ctypes.c_void_p, "Q",
                                list(map(torch.Tensor.data_ptr, grads)))
        self.codes = _host_array(ctypes.c_int, "i", codes)
        self.size_list = list(map(torch.Tensor.numel, grads))
        self.sizes = _host_array(ctypes.c_int64, "q", self.size_list)

    def outputs(self, grads_out):
        """The outputs' pointers: the gradients' own without grads_out."""
        if grads_out is None:
            self.outs = self.grads
            return self.ptrs
        grads, outs = self.grads, list(grads_out)
        if len(outs) != len(self.given):
            raise ValueError(f"{len(outs)} outputs for {len(self.given)} "
                             "gradients")
        kept = self.outs = [o for o in outs if o is not None]
        if (len(kept) != self.n or self.n != len(outs) and any(
                (o is None) != (g is None) for o, g in zip(outs, self.given))):
            raise ValueError("an output must be None where its gradient is, "
                             "and there alone")
        outs = kept
        codes = list(map(_TYPE_CODES.get, map(_dtype_of, outs)))
        same = (codes == self.code_list and
                list(map(torch.Tensor.numel, outs)) == self.size_list and
                set(map(torch.Tensor.get_device, outs)) ==
                set(map(torch.Tensor.get_device, grads[:1])))
        if same and not (self.flat and
                         all(map(torch.Tensor.is_contiguous, outs))):
            same = all(o.shape == g.shape and o.stride() == g.stride() or
                       o.is_contiguous() and g.is_contiguous()
                       for o, g in zip(outs, grads))
        if not same:
            raise ValueError("an output must have its gradient's type, device "
                             "and number of elements, and be contiguous or "
                             "laid out as the gradient")
        return _host_array(ctypes.c_void_p, "Q",
                           list(map(torch.Tensor.data_ptr, outs)))

    def workspace(self, workspace):
        if workspace is not None:
            return _check_workspace(workspace, self.device)
        return torch.empty(grad_norm_workspace_size(self.n),
                           dtype=torch.uint8, device=self.device)


def _max_norm(value):
    value = float(value)
    if not value >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {value}")
    return value


@functools.lru_cache(maxsize=1024)
def grad_norm_workspace_size(n: int) -> int:
    """Bytes of workspace that grad_norm needs for n gradients."""
    size = load().lce_grad_norm_workspace_size(n)
    if size == 0:
        raise ValueError(f"invalid number of gradients {n}")
    return size


def grad_norm(grads, workspace=None):
    """sqrt of the sum of all squares of a list of gradients (bf16 or fp32
    CUDA tensors of any shapes; None, a parameter without one, is passed by):
    a fp32 scalar on their device."""
    table = _GradTable(grads)
    dev = table.device
    ws = table.workspace(workspace)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    _call("lce_grad_norm", dev, table.ptrs, table.codes, table.sizes, table.n,
          norm.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return norm


def clip_grads(grads, norm, max_norm: float, grads_out=None):
    """Multiplies every gradient by min(1, max_norm / (norm + 1e-6)), in place
    or into grads_out (tensors laid out as the gradients; contiguous ones may
    differ in shape, such as slices of a flat buffer; None where the gradient
    is). norm: one fp32 value on the device, of grad_norm or of a sum over
    processes. Gradients or outputs that overlap are refused."""
    max_norm = _max_norm(max_norm)
    table = _GradTable(grads)
    _check_rows("norm", norm.reshape(-1), (1,), torch.float32, table.device)
    _call("lce_clip_grads", table.device, table.ptrs, table.outputs(grads_out),
          table.codes, table.sizes, table.n, norm.data_ptr(), max_norm)
    increment_version(table.outs)


def clip_grad_norm(grads, max_norm: float, grads_out=None, workspace=None):
    """clip_grads by the gradients' own norm, which is returned (as it was
    before the clipping)."""
    max_norm = _max_norm(max_norm)
    table = _GradTable(grads)
    dev = table.device
    outs = table.outputs(grads_out)
    ws = table.workspace(workspace)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    _call("lce_clip_grad_norm", dev, table.ptrs, outs, table.codes,
          table.sizes, table.n, max_norm, norm.data_ptr(), ws.data_ptr(),
          ws.numel() * ws.element_size())
    increment_version(table.outs)
    return norm


def set_cta_pair(enable: bool):
    """Run the contractions on CTA pairs (cta_group::2) or single CTAs."""
    _check(load().lce_set_cta_pair(1 if enable else 0), "lce_set_cta_pair")


def get_cta_pair() -> bool:
    return bool(load().lce_get_cta_pair())


def set_wave_sync(enable: bool):
    """Wave pacing of the contractions on (default) or off; same results."""
    _check(load().lce_set_wave_sync(1 if enable else 0), "lce_set_wave_sync")


def get_wave_sync() -> bool:
    return bool(load().lce_get_wave_sync())


def profile_start():
    """Time every kernel this thread launches through the library."""
    _check(load().lce_profile_start(), "lce_profile_start")


def profile_stop() -> dict:
    """Waits for the recorded launches; returns {kind: (launches, total_ms,
    flops)} for the kinds that ran."""
    arr = (KernelStat * KERNEL_KINDS)()
    _check(load().lce_profile_stop(arr), "lce_profile_stop")
    return {a.name.decode(): (a.launches, a.total_ms, a.flops) for a in arr
            if a.launches}


class LinearCrossEntropy(torch.autograd.Function):
    """loss = mean cross entropy of h W^T against labels, without the logits.

    fused=False: forward saves only lse [L] (4 bytes per row); backward
    recomputes the logits chunk by chunk in the library.
    fused=True: forward computes the loss and the gradients in one call
    (no recompute) and keeps dH, dW (for dloss = 1) until backward, which
    returns copies scaled by dloss. The kept tensors are never modified, so
    a retained graph gives the same gradients again; the cost is memory:
    dH and dW (L H + 4 V H bytes for bf16 h) stay allocated from the forward
    until the graph is freed, and backward briefly holds the scaled copies
    as well."""

    @staticmethod
    def forward(ctx, h, W, labels, ignore_index=IGNORE_INDEX, chunk_rows=0,
                fused=False, label_smoothing=0.0, z_loss=0.0):
        ctx.ignore_index = ignore_index
        ctx.chunk_rows = chunk_rows
        ctx.fused = fused
        ctx.w_dtype = W.dtype
        ctx.variant = dict(label_smoothing=label_smoothing, z_loss=z_loss)
        # only the gradients autograd asks for are computed (a frozen head:
        # no dW contraction)
        ctx.want = dict(compute_dH=ctx.needs_input_grad[0],
                        compute_dW=ctx.needs_input_grad[1])
        if fused and any(ctx.want.values()):
            loss, _, dH, dW = forward_backward(h, W, labels, ignore_index,
                                               chunk_rows, **ctx.variant,
                                               **ctx.want)
            ctx.save_for_backward(dH, dW)
        else:
            ctx.fused = False
            loss, lse = forward(h, W, labels, ignore_index, **ctx.variant)
            ctx.save_for_backward(h, W, labels, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        if not any(ctx.want.values()):
            return None, None, None, None, None, None, None, None
        if ctx.fused:
            kept_dH, kept_dW = ctx.saved_tensors
            dH, dW = scale_gradients(
                kept_dH.clone() if kept_dH is not None else None,
                kept_dW.clone() if kept_dW is not None else None, dloss)
        else:
            h, W, labels, lse = ctx.saved_tensors
            dH, dW = backward(h, W, labels, lse, dloss, ctx.ignore_index,
                              ctx.chunk_rows, **ctx.variant, **ctx.want)
        return (dH, dW.to(ctx.w_dtype) if dW is not None else None, None,
                None, None, None, None, None)


class SequenceTiledMLP(torch.autograd.Function):
    """y = down(silu(gate(x)) * up(x)) over row chunks, as an autograd
    Function: forward keeps only its inputs (no L x I intermediate outlives
    a chunk); backward recomputes each chunk's gate/up activations in the
    library and returns dx (bf16) and the three weight gradients in the
    weights' dtype, computing only those autograd asks for. dy is made a
    contiguous bf16 tensor first."""

    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, chunk_rows=0):
        ctx.chunk_rows = chunk_rows
        ctx.save_for_backward(x, Wg, Wu, Wd)
        return mlp_forward(x, Wg, Wu, Wd, chunk_rows)

    @staticmethod
    def backward(ctx, dy):
        x, Wg, Wu, Wd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:4]):
            return None, None, None, None, None
        dy = dy.to(torch.bfloat16).contiguous()
        # only the gradients autograd asks for (frozen weights: dx alone)
        dx, dWg, dWu, dWd = mlp_backward(x, Wg, Wu, Wd, dy, ctx.chunk_rows,
                                         compute_dx=need[0],
                                         compute_dWgu=need[1] or need[2],
                                         compute_dWd=need[3])
        cast = [t.to(w.dtype) if (t is not None and n) else None
                for t, w, n in ((dWg, Wg, need[1]), (dWu, Wu, need[2]),
                                (dWd, Wd, need[3]))]
        return (dx, cast[0], cast[1], cast[2], None)


class RouteExperts(torch.autograd.Function):
    """route_forward under autograd: the weights carry gradient to the
    logits, the selection (experts) does not. bias steers the selection
    alone and gets none."""

    @staticmethod
    def forward(ctx, logits, top_k, scoring="softmax", bias=None, n_group=1,
                topk_group=1, group_top=1, renormalize=True, scale=1.0):
        weights, experts = route_forward(logits, top_k, scoring, bias, n_group,
                                         topk_group, group_top, renormalize,
                                         scale)
        ctx.opts = (scoring, renormalize, scale)
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        logits, experts = ctx.saved_tensors
        dlogits = None
        if ctx.needs_input_grad[0]:
            dlogits = route_backward(logits, experts,
                                     dweights.to(logits.dtype).contiguous(),
                                     *ctx.opts)
        return (dlogits,) + (None,) * 8


def route_experts(logits, top_k: int, scoring: str = "softmax", bias=None,
                  n_group: int = 1, topk_group: int = 1, group_top: int = 1,
                  renormalize: bool = True, scale: float = 1.0):
    """(weights, experts) of router logits, with autograd (route_forward)."""
    return RouteExperts.apply(logits, top_k, scoring, bias, n_group,
                              topk_group, group_top, renormalize, scale)


class ExpertsMLP(torch.autograd.Function):
    """experts_forward under autograd: forward keeps only its inputs,
    backward recomputes the activations and returns dx, the weight gradients
    in bf16 (the weights' type) and dweights, computing only those autograd
    asks for. dy is made a contiguous bf16 tensor first."""

    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, weights, experts):
        ctx.save_for_backward(x, Wg, Wu, Wd, weights, experts)
        return experts_forward(x, Wg, Wu, Wd, weights, experts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need = ctx.needs_input_grad
        if not any(need[:5]):
            return (None,) * 6
        dy = dy.to(torch.bfloat16).contiguous()
        dx, dWg, dWu, dWd, dw = experts_backward(
            *ctx.saved_tensors, dy, grad_dtype=torch.bfloat16,
            compute_dx=need[0], compute_dWgu=need[1] or need[2],
            compute_dWd=need[3], compute_dweights=need[4])
        return (dx, dWg if need[1] else None, dWu if need[2] else None, dWd,
                dw, None)


def experts_mlp(x, Wg, Wu, Wd, weights, experts):
    """The experts' gated MLP (experts_forward) with autograd."""
    return ExpertsMLP.apply(x, Wg, Wu, Wd, weights, experts)


class LayerNorm(torch.autograd.Function):
    """layer_norm_forward under autograd; the parameters' gradients in their
    own type. dy is made a contiguous tensor of x's type first."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = (x if weight is None and bias is None else
                           bias if weight is None else weight).dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:3]):
            return (None,) * 4
        return layer_norm_backward(
            x, weight, mean, rstd, dy.to(x.dtype).contiguous(),
            grad_dtype=ctx.param_dtype, compute_dx=need[0],
            compute_dweight=need[1], compute_dbias=need[2]) + (None,)


class RMSNorm(torch.autograd.Function):
    """rms_norm_forward under autograd, as LayerNorm."""

    @staticmethod
    def forward(ctx, x, weight, eps):
        y, rstd = rms_norm_forward(x, weight, eps)
        ctx.save_for_backward(x, weight, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:2]):
            return (None,) * 3
        dtype = x.dtype if weight is None else weight.dtype
        return rms_norm_backward(
            x, weight, rstd, dy.to(x.dtype).contiguous(), grad_dtype=dtype,
            compute_dx=need[0], compute_dweight=need[1]) + (None,)


def _wants_grad(*tensors):
    """Whether a call has to go through its autograd Function: for a gradient,
    or for a tangent, which the Function refuses (it has no forward mode)."""
    backward = torch.is_grad_enabled()
    for t in tensors:
        if t is not None and (backward and t.requires_grad or
                              forward_ad.unpack_dual(t).tangent is not None):
            return True
    return False


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm of the rows of x [L,H] with autograd (layer_norm_forward)."""
    if not _wants_grad(x, weight, bias):  # serving: no statistics are kept
        return layer_norm_forward(x, weight, bias, eps, save_stats=False)[0]
    return LayerNorm.apply(x, weight, bias, eps)


def rms_norm(x, weight=None, eps: float = 1e-6):
    """RMS norm of the rows of x [L,H] with autograd (rms_norm_forward)."""
    if not _wants_grad(x, weight):
        return rms_norm_forward(x, weight, eps, save_stats=False)[0]
    return RMSNorm.apply(x, weight, eps)


class BalanceLoss(torch.autograd.Function):
    """balance_forward under autograd: the loss carries gradient to the
    logits through the scores; the counts are constant."""

    @staticmethod
    def forward(ctx, logits, experts, scoring, coef, mask):
        loss, counts, slopes = balance_forward(logits, experts, scoring, coef,
                                               mask)
        ctx.scoring = scoring
        ctx.save_for_backward(logits, slopes, mask)
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        logits, slopes, mask = ctx.saved_tensors
        dlogits = None
        if ctx.needs_input_grad[0]:
            dlogits = balance_backward(logits, slopes, dloss, ctx.scoring,
                                       mask)
        return (dlogits,) + (None,) * 4


def balance_loss(logits, experts, scoring: str = "softmax", coef: float = 1.0,
                 mask=None):
    """(loss, counts) of the routing's balance, with autograd
    (balance_forward)."""
    return BalanceLoss.apply(logits, experts, scoring, coef, mask)


def sequence_tiled_mlp(x, Wg, Wu, Wd, chunk_rows: int = 0):
    """The gated MLP down(silu(gate(x)) * up(x)) (nn.Linear weight layouts:
    Wg, Wu [I, H], Wd [H, I]; bf16) with autograd, over row chunks."""
    return SequenceTiledMLP.apply(x, Wg, Wu, Wd, chunk_rows)


def linear_cross_entropy(h, W, labels, ignore_index: int = IGNORE_INDEX,
                         chunk_rows: int = 0, fused: bool = False,
                         label_smoothing: float = 0.0, z_loss: float = 0.0):
    """Mean cross entropy of h W^T against labels (autograd). label_smoothing
    and z_loss select the loss variants of lce_forward_ex."""
    return LinearCrossEntropy.apply(h, W, labels, ignore_index, chunk_rows,
                                    fused, label_smoothing, z_loss)
