"""convolution_backward_b200 -- B200 (sm_100a) convolution backward-data (dgrad).

A thin ctypes binding over ``libdgrad.so`` (the C ABI in ``include/dgrad.h``).
This module only marshals arguments: it checks tensor shapes, dtypes and
devices, passes raw device pointers and the current CUDA stream, and raises on
a non-OK status.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback.  If the library is missing the
calls raise ``DgradUnavailable``.

    dX = pointwise(dY, W)                          # dY (N,H,W,K), W (K,C) -> (N,H,W,C)
    dX = depthwise(dY, W, H=H, W=W_, stride=1, pad_h=1, pad_w=1)   # W (KH,KW,C)

    Y, mean, rstd = layernorm_forward(X, gamma, beta, stats=True)  # X (..., C)
    H, Z = gated_forward(X, W, act="silu", preact=True)            # W (2F, C) -> (..., F), (..., 2F)
    Y = dropout_forward(X, p, seed, offset, residual=R)
    Y, mean, rstd = groupnorm_forward(X, groups, gamma, beta, act="silu", stats=True)   # X (N, ..., C)

and their ``_backward`` counterparts; and over all parameters at once

    state = adamw_state(params, bits=8)             # or 32; master=True keeps fp32 copies
    norm, scale = grad_norm(grads, max_norm=1.0)
    adamw_step(state, grads, step, lr, grad_scale=scale)
  Tensors are NHWC (rows of channels) and contiguous;
float32, bfloat16 or float16 (16-bit in, 16-bit out, fp32 accumulate).
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import threading

__all__ = ["pointwise", "pointwise_splitk", "pointwise_splitk_noalloc", "depthwise_tc", "depthwise_tc_workspace_bytes", "dense", "grouped", "splitk_workspace_bytes", "depthwise", "out_dims", "check_status", "DgradError", "DgradUnavailable",
           "layernorm_forward", "layernorm_backward", "layernorm_backward_workspace_bytes", "dropout_forward", "dropout_backward",
           "gated_forward", "gated_backward", "gated_backward_workspace_bytes", "ACTIVATIONS",
           "groupnorm_forward", "groupnorm_backward", "groupnorm_forward_workspace_bytes", "groupnorm_backward_workspace_bytes",
           "AdamWState", "adamw_state", "adamw_step", "adamw_moments", "grad_norm", "grad_norm_workspace_bytes",
           "Problem", "lib", "library_path", "selftest_timeout", "fma_probe", "STATUS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
# DGRAD_LIBRARY=debug loads libdgrad_debug.so: the same kernels built with index
# checks on every hand-indexed store (a failed check skips the store and makes
# check_status raise with DGRAD_ERR_BOUNDS).
_LIB_PATH = os.path.join(_PKG, "libdgrad_debug.so" if os.environ.get("DGRAD_LIBRARY") == "debug" else "libdgrad.so")
_lock = threading.Lock()
_lib = None

STATUS = {0: "DGRAD_OK", 1: "DGRAD_ERR_INVALID", 2: "DGRAD_ERR_UNSUPPORTED", 3: "DGRAD_ERR_ALIGNMENT",
          4: "DGRAD_ERR_CUDA", 5: "DGRAD_ERR_TIMEOUT", 6: "DGRAD_ERR_BOUNDS"}
DW_MODES = {"auto": 0, "rotated": 1, "rowstream": 2}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}   # dgrad_act_t
_ACT_NONE = 5                    # DGRAD_ACT_NONE: group norm's act=None
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}
SPLITK_SCRATCH_BYTES = 8 << 20   # DGRAD_SPLITK_SCRATCH_BYTES: the fixed per-device split-K buffer


class DgradUnavailable(RuntimeError):
    """libdgrad.so could not be loaded (not built, or built for another platform)."""


class DgradError(RuntimeError):
    def __init__(self, status: int, what: str, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = f"{what}: {STATUS.get(status, status)}"
        if status == 4:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


class _AdamW(ctypes.Structure):
    """dgrad_adamw_t."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("lr_device", ctypes.c_void_p),
                ("step_device", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p), ("state_bits", ctypes.c_int32),
                ("stochastic", ctypes.c_int32), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class Problem(ctypes.Structure):
    """dgrad_problem_t: N, H, W, C, K (int64), KH, KW, stride, pad_h, pad_w (int32)."""
    _fields_ = [("N", ctypes.c_int64), ("H", ctypes.c_int64), ("W", ctypes.c_int64),
                ("C", ctypes.c_int64), ("K", ctypes.c_int64), ("KH", ctypes.c_int32),
                ("KW", ctypes.c_int32), ("stride", ctypes.c_int32), ("pad_h", ctypes.c_int32),
                ("pad_w", ctypes.c_int32)]


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libdgrad (ctypes.CDLL) with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise DgradUnavailable(
                    f"{_LIB_PATH} is missing; build it with `python -m convolution_backward_b200._build` "
                    "(nvcc, sm_100a)")
            try:
                L = ctypes.CDLL(_LIB_PATH)
            except OSError as e:
                raise DgradUnavailable(f"cannot load {_LIB_PATH}: {e}") from e
            P = ctypes.POINTER
            vp = ctypes.c_void_p
            L.dgrad_pointwise.argtypes = [P(Problem), ctypes.c_int, vp, vp, vp, vp]
            L.dgrad_pointwise.restype = ctypes.c_int
            L.dgrad_depthwise.argtypes = [P(Problem), ctypes.c_int, ctypes.c_int, vp, vp, vp, vp]
            L.dgrad_depthwise.restype = ctypes.c_int
            L.dgrad_out_dims.argtypes = [P(Problem), P(ctypes.c_int64), P(ctypes.c_int64)]
            L.dgrad_out_dims.restype = ctypes.c_int
            L.dgrad_check_status.argtypes = [vp]
            L.dgrad_check_status.restype = ctypes.c_int
            L.dgrad_status_string.argtypes = [ctypes.c_int]
            L.dgrad_status_string.restype = ctypes.c_char_p
            L.dgrad_last_cuda_error.argtypes = []
            L.dgrad_last_cuda_error.restype = ctypes.c_int
            L.dgrad_selftest_timeout.argtypes = [ctypes.c_longlong, vp]
            L.dgrad_selftest_timeout.restype = ctypes.c_int
            L.dgrad_fma_probe.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp]
            L.dgrad_fma_probe.restype = ctypes.c_int
            L.dgrad_pointwise_splitk.argtypes = [P(Problem), ctypes.c_int, ctypes.c_int, vp, vp, vp, vp,
                                                 ctypes.c_size_t, vp]
            L.dgrad_pointwise_splitk.restype = ctypes.c_int
            L.dgrad_pointwise_splitk_workspace.argtypes = [P(Problem), ctypes.c_int, P(ctypes.c_size_t),
                                                           P(ctypes.c_int)]
            L.dgrad_pointwise_splitk_workspace.restype = ctypes.c_int
            L.dgrad_pointwise_splitk_noalloc.argtypes = [P(Problem), ctypes.c_int, ctypes.c_int, vp, vp, vp, vp]
            L.dgrad_pointwise_splitk_noalloc.restype = ctypes.c_int
            L.dgrad_dense.argtypes = [P(Problem), ctypes.c_int, vp, vp, vp, vp]
            L.dgrad_dense.restype = ctypes.c_int
            L.dgrad_grouped.argtypes = [P(Problem), ctypes.c_int64, ctypes.c_int, vp, vp, vp, vp]
            L.dgrad_grouped.restype = ctypes.c_int
            L.dgrad_depthwise_tc.argtypes = [P(Problem), ctypes.c_int, vp, vp, vp, vp, ctypes.c_size_t, vp]
            L.dgrad_depthwise_tc.restype = ctypes.c_int
            L.dgrad_depthwise_tc_workspace.argtypes = [P(Problem), P(ctypes.c_size_t)]
            L.dgrad_depthwise_tc_workspace.restype = ctypes.c_int
            i64, u64, dbl, sz, ci = ctypes.c_int64, ctypes.c_uint64, ctypes.c_double, ctypes.c_size_t, ctypes.c_int
            for name, args in {
                    "layernorm_forward": [i64, i64, ci, dbl, vp, vp, vp, vp, vp, vp, vp],
                    "layernorm_backward": [i64, i64, ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                    "layernorm_backward_workspace": [i64, i64, ci, P(sz)],
                    "gated_forward": [i64, i64, i64, ci, ci, vp, vp, vp, vp, vp],
                    "gated_backward": [i64, i64, i64, ci, ci, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                    "gated_backward_workspace": [i64, i64, i64, P(sz)],
                    "groupnorm_forward": [i64, i64, i64, i64, ci, dbl, ci, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                    "groupnorm_backward": [i64, i64, i64, i64, ci, ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                    "groupnorm_forward_workspace": [i64, i64, i64, i64, ci, P(sz)],
                    "groupnorm_backward_workspace": [i64, i64, i64, i64, ci, P(sz)],
                    "adamw_step": [i64, vp, ci, ci, P(_AdamW), vp],
                    "adamw_check": [i64, vp, ci, ci, ctypes.c_int32],
                    "adamw_moments": [i64, vp, vp, vp, vp],
                    "grad_norm": [i64, vp, vp, ci, dbl, vp, vp, sz, vp],
                    "grad_norm_workspace": [i64, P(sz)],
                    "dropout_forward": [i64, ci, dbl, u64, u64, vp, vp, vp, vp],
                    "dropout_backward": [i64, ci, dbl, u64, u64, vp, vp, vp]}.items():
                f = getattr(L, "dgrad_" + name)
                f.argtypes = args
                f.restype = ctypes.c_int
            _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != 0:
        raise DgradError(status, what, lib().dgrad_last_cuda_error())


def _stream_ptr(stream, device=None):
    """The raw cudaStream_t of `stream` (default: the current stream of `device`).
    A given stream must belong to `device`."""
    import torch
    if stream is None:
        index = None if device is None else device.index
        # the raw handle, without the Stream object around it (2 us a call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and index is not None:
            return raw(index) or None
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device} but the tensors are on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _device_of(*ts):
    """The one CUDA device every tensor in `ts` lives on.  The C ABI works on the
    current device, so the wrappers make this device current around each call;
    tensors on different devices are refused."""
    dev = ts[0].device
    for t in ts:
        if t.device != dev:
            raise ValueError("all tensors of one call must be on the same CUDA device, got "
                             + ", ".join(sorted({f"{d.type}:{d.index}" for d in (u.device for u in ts)})))
    return dev


def _call(dev, what, fn, *args, stream=None):
    """Run C entry point `fn` with `dev` current and its stream appended."""
    import torch
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, _stream_ptr(stream, dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream_ptr(stream, dev))
    if status != 0:
        _check(status, what)


def _code_of(dtype) -> int:
    import torch
    if dtype == torch.float32:
        return 0
    if dtype == torch.bfloat16:
        return 1
    if dtype == torch.float16:
        return 2
    raise TypeError(f"unsupported dtype {dtype}; use float32, bfloat16 or float16")


def _dtype_code(t) -> int:
    return _code_of(t.dtype)


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors (no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous (NHWC)")


def _at(t):
    """A tensor's address.  One whose storage was released is refused: its address is that of its offset, 0 for most,
    which stands for an optional tensor that is not there."""
    p = t.data_ptr()
    if p < 1 << 40 and t.numel() and t.untyped_storage().data_ptr() == 0:
        raise ValueError("a tensor's storage does not hold its elements")
    return p


def out_dims(H, W, KH, KW, stride=1, pad_h=0, pad_w=-1):
    """(Ho, Wo) of the forward convolution (host-only C call)."""
    prob = Problem(1, H, W, 1, 1, KH, KW, stride, pad_h, pad_w)
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().dgrad_out_dims(ctypes.byref(prob), ctypes.byref(ho), ctypes.byref(wo)), "dgrad_out_dims")
    return ho.value, wo.value


def pointwise(dY, W, out=None, stream=None):
    """Pointwise dgrad: dX[n,h,w,:] = dY[n,h,w,:] @ W, dY (N,H,W,K), W (K,C).  Calls dgrad_pointwise."""
    import torch
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 2 or W.shape[0] != dY.shape[3]:
        raise ValueError("expected dY (N,H,W,K) and W (K,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, H, Wd, K = dY.shape
    C = W.shape[1]
    if out is None:
        out = torch.empty((N, H, Wd, C), dtype=dY.dtype, device=dY.device)
    else:
        _need_cuda(out)
        if tuple(out.shape) != (N, H, Wd, C) or out.dtype != dY.dtype:
            raise ValueError("out has the wrong shape or dtype")
    prob = Problem(N, H, Wd, C, K, 1, 1, 1, 0, 0)
    _call(_device_of(dY, W, out), "dgrad_pointwise", lib().dgrad_pointwise, ctypes.byref(prob), _dtype_code(dY),
          _at(dY), _at(W), _at(out), stream=stream)
    return out


def splitk_workspace_bytes(N, H, W, K, C, splits=0):
    """(bytes, splits) of workspace pointwise_splitk needs (dgrad_pointwise_splitk_workspace)."""
    prob = Problem(N, H, W, C, K, 1, 1, 1, 0, 0)
    nb, used = ctypes.c_size_t(), ctypes.c_int()
    _check(lib().dgrad_pointwise_splitk_workspace(ctypes.byref(prob), int(splits), ctypes.byref(nb),
                                                  ctypes.byref(used)), "dgrad_pointwise_splitk_workspace")
    return nb.value, used.value


def pointwise_splitk(dY, W, splits=0, workspace=None, out=None, stream=None):
    """Split-K pointwise dgrad for small M (bf16; dgrad_pointwise_splitk).

    workspace: a caller-owned CUDA tensor of at least splitk_workspace_bytes(...)
    bytes; allocated here with torch when None."""
    import torch
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 2 or W.shape[0] != dY.shape[3]:
        raise ValueError("expected dY (N,H,W,K) and W (K,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, H, Wd, K = dY.shape
    C = W.shape[1]
    nbytes, used = splitk_workspace_bytes(N, H, Wd, K, C, splits)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dY.device)
    if out is None:
        out = torch.empty((N, H, Wd, C), dtype=dY.dtype, device=dY.device)
    prob = Problem(N, H, Wd, C, K, 1, 1, 1, 0, 0)
    _call(_device_of(dY, W, out, workspace), "dgrad_pointwise_splitk", lib().dgrad_pointwise_splitk,
          ctypes.byref(prob), _dtype_code(dY), int(used), _at(dY), _at(W), _at(out),
          _at(workspace), workspace.numel() * workspace.element_size(), stream=stream)
    return out


def pointwise_splitk_noalloc(dY, W, out, splits=0, stream=None):
    """Split-K pointwise dgrad that allocates nothing (dgrad_pointwise_splitk_noalloc).

    For callers that must not allocate device memory at call time: the partial
    tiles go to the library's fixed per-device scratch buffer of
    SPLITK_SCRATCH_BYTES, so ``out`` (N,H,W,C, dY's dtype) is required.  Calls
    that overlap in time on one device share that buffer and race; calls ordered
    on one stream do not.  The first call on a device sets the buffer up: make
    it before any stream capture begins.  A problem whose partial tiles do not
    fit the buffer raises DgradError (status 2, unsupported)."""
    _need_cuda(dY, W, out)
    if dY.dim() != 4 or W.dim() != 2 or W.shape[0] != dY.shape[3]:
        raise ValueError("expected dY (N,H,W,K) and W (K,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, H, Wd, K = dY.shape
    C = W.shape[1]
    if tuple(out.shape) != (N, H, Wd, C) or out.dtype != dY.dtype:
        raise ValueError("out must be (N,H,W,C) with dY's dtype")
    prob = Problem(N, H, Wd, C, K, 1, 1, 1, 0, 0)
    _call(_device_of(dY, W, out), "dgrad_pointwise_splitk_noalloc", lib().dgrad_pointwise_splitk_noalloc,
          ctypes.byref(prob), _dtype_code(dY), int(splits), _at(dY), _at(W), _at(out),
          stream=stream)
    return out


def depthwise(dY, W, *, H, W_out=None, stride=1, pad_h=0, pad_w=-1, mode="auto", out=None,
              stream=None, **kw):
    """Depthwise dgrad (groups = C): dY (N,Ho,Wo,C), W (KH,KW,C) -> dX (N,H,W,C).  Calls dgrad_depthwise.

    H and W_out (alias ``Wd``) are dX's spatial extents; pad_w = -1 means pad_h.
    mode: "auto" (rotated-filter at stride 1, row-streaming otherwise),
    "rotated" or "rowstream".
    """
    import torch
    if W_out is None:
        W_out = kw.pop("Wd")
    if kw:
        raise TypeError(f"unexpected arguments {sorted(kw)}")
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 3 or W.shape[2] != dY.shape[3]:
        raise ValueError("expected dY (N,Ho,Wo,C) and W (KH,KW,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, Ho, Wo, C = dY.shape
    KH, KW = W.shape[0], W.shape[1]
    prob = Problem(N, H, W_out, C, C, KH, KW, stride, pad_h, pad_w)
    eho, ewo = out_dims(H, W_out, KH, KW, stride, pad_h, pad_w)
    if (eho, ewo) != (Ho, Wo):
        raise ValueError(f"dY spatial extent {(Ho, Wo)} does not match the geometry ({eho}, {ewo})")
    if out is None:
        out = torch.empty((N, H, W_out, C), dtype=dY.dtype, device=dY.device)
    else:
        _need_cuda(out)
        if tuple(out.shape) != (N, H, W_out, C) or out.dtype != dY.dtype:
            raise ValueError("out has the wrong shape or dtype")
    _call(_device_of(dY, W, out), "dgrad_depthwise", lib().dgrad_depthwise, ctypes.byref(prob), _dtype_code(dY),
          DW_MODES[mode], _at(dY), _at(W), _at(out), stream=stream)
    return out


def dense(dY, W, *, H, W_out=None, stride=1, pad_h=0, pad_w=-1, out=None, stream=None, **kw):
    """Dense (ungrouped) dgrad on the tensor cores (bf16 or f16; dgrad_dense): dY (N,Ho,Wo,K),
    W (KH,KW,K,C) -> dX (N,H,W,C).  H and W_out (alias ``Wd``) are dX's spatial extents."""
    import torch
    if W_out is None:
        W_out = kw.pop("Wd")
    if kw:
        raise TypeError(f"unexpected arguments {sorted(kw)}")
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 4 or W.shape[2] != dY.shape[3]:
        raise ValueError("expected dY (N,Ho,Wo,K) and W (KH,KW,K,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, Ho, Wo, K = dY.shape
    KH, KW, _, C = W.shape
    eho, ewo = out_dims(H, W_out, KH, KW, stride, pad_h, pad_w)
    if (eho, ewo) != (Ho, Wo):
        raise ValueError(f"dY spatial extent {(Ho, Wo)} does not match the geometry ({eho}, {ewo})")
    if out is None:
        out = torch.empty((N, H, W_out, C), dtype=dY.dtype, device=dY.device)
    else:
        _need_cuda(out)
        if tuple(out.shape) != (N, H, W_out, C) or out.dtype != dY.dtype:
            raise ValueError("out has the wrong shape or dtype")
    prob = Problem(N, H, W_out, C, K, KH, KW, stride, pad_h, pad_w)
    _call(_device_of(dY, W, out), "dgrad_dense", lib().dgrad_dense, ctypes.byref(prob), _dtype_code(dY),
          _at(dY), _at(W), _at(out), stream=stream)
    return out


def grouped(dY, W, groups, *, H, W_out=None, stride=1, pad_h=0, pad_w=-1, out=None, stream=None, **kw):
    """Grouped dgrad on the tensor cores (bf16 or f16; dgrad_grouped): dY (N,Ho,Wo,K),
    W (KH,KW,K,C/groups) -> dX (N,H,W,C).  A 1x1 filter is grouped pointwise dgrad."""
    import torch
    if W_out is None:
        W_out = kw.pop("Wd")
    if kw:
        raise TypeError(f"unexpected arguments {sorted(kw)}")
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 4 or W.shape[2] != dY.shape[3]:
        raise ValueError("expected dY (N,Ho,Wo,K) and W (KH,KW,K,C/groups)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, Ho, Wo, K = dY.shape
    KH, KW, _, Cg = W.shape
    C = Cg * int(groups)
    eho, ewo = out_dims(H, W_out, KH, KW, stride, pad_h, pad_w)
    if (eho, ewo) != (Ho, Wo):
        raise ValueError(f"dY spatial extent {(Ho, Wo)} does not match the geometry ({eho}, {ewo})")
    if out is None:
        out = torch.empty((N, H, W_out, C), dtype=dY.dtype, device=dY.device)
    else:
        _need_cuda(out)
        if tuple(out.shape) != (N, H, W_out, C) or out.dtype != dY.dtype:
            raise ValueError("out has the wrong shape or dtype")
    prob = Problem(N, H, W_out, C, K, KH, KW, stride, pad_h, pad_w)
    _call(_device_of(dY, W, out), "dgrad_grouped", lib().dgrad_grouped, ctypes.byref(prob), int(groups),
          _dtype_code(dY), _at(dY), _at(W), _at(out), stream=stream)
    return out


def depthwise_tc_workspace_bytes(N, H, W, C, KH, KW, pad_h=0, pad_w=-1) -> int:
    """Workspace bytes dgrad_depthwise_tc needs (host only); raises DgradError when unsupported."""
    prob = Problem(N, H, W, C, C, KH, KW, 1, pad_h, pad_w)
    nb = ctypes.c_size_t()
    _check(lib().dgrad_depthwise_tc_workspace(ctypes.byref(prob), ctypes.byref(nb)), "dgrad_depthwise_tc_workspace")
    return nb.value


def depthwise_tc(dY, W, *, H, W_out=None, pad_h=0, pad_w=-1, workspace=None, out=None, stream=None, **kw):
    """Stride-1 depthwise dgrad on the tensor cores (bf16; dgrad_depthwise_tc).

    Same arguments and result as depthwise() at stride 1.  workspace: a CUDA
    tensor of at least depthwise_tc_workspace_bytes(...) bytes, allocated here
    with torch when None."""
    import torch
    if W_out is None:
        W_out = kw.pop("Wd")
    if kw:
        raise TypeError(f"unexpected arguments {sorted(kw)}")
    _need_cuda(dY, W)
    if dY.dim() != 4 or W.dim() != 3 or W.shape[2] != dY.shape[3]:
        raise ValueError("expected dY (N,Ho,Wo,C) and W (KH,KW,C)")
    if W.dtype != dY.dtype:
        raise TypeError("dY and W must have the same dtype")
    N, Ho, Wo, C = dY.shape
    KH, KW = W.shape[0], W.shape[1]
    eho, ewo = out_dims(H, W_out, KH, KW, 1, pad_h, pad_w)
    if (eho, ewo) != (Ho, Wo):
        raise ValueError(f"dY spatial extent {(Ho, Wo)} does not match the geometry ({eho}, {ewo})")
    prob = Problem(N, H, W_out, C, C, KH, KW, 1, pad_h, pad_w)
    nbytes = depthwise_tc_workspace_bytes(N, H, W_out, C, KH, KW, pad_h, pad_w)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dY.device)
    if out is None:
        out = torch.empty((N, H, W_out, C), dtype=dY.dtype, device=dY.device)
    else:
        _need_cuda(out)
        if tuple(out.shape) != (N, H, W_out, C) or out.dtype != dY.dtype:
            raise ValueError("out has the wrong shape or dtype")
    _call(_device_of(dY, W, out, workspace), "dgrad_depthwise_tc", lib().dgrad_depthwise_tc, ctypes.byref(prob),
          _dtype_code(dY), _at(dY), _at(W), _at(out), _at(workspace),
          workspace.numel() * workspace.element_size(), stream=stream)
    return out


# ------------------------------------------------ the residual branch's operators

def _rows_of(X):
    """(M, C): the rows of X (..., C) and their length."""
    if X.dim() < 1:
        raise ValueError("expected a tensor of rows (..., C)")
    C = X.shape[-1]
    if C < 1:
        raise ValueError("expected at least one channel")
    M = 1
    for d in X.shape[:-1]:
        M *= d
    return M, C


def _like(t, shape, dtype, what):
    """Check a tensor argument's shape and dtype."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")


class _Allocator:
    """Outputs and workspaces of one call on a stream other than the device's current one: they
    come from that stream's pool, so that memory still in use on another stream is never
    handed out to it, and the tensors of the call are recorded on the stream they are used
    on besides their own: freeing one early does not pull it away."""

    def __init__(self, stream, current):
        self.stream, self.current = stream, current

    def empty(self, like, shape, dtype):
        import torch
        with torch.cuda.stream(self.stream):
            t = like.new_empty(shape, dtype=dtype)
        t.record_stream(self.current)
        return t

    def uses(self, *ts):
        for t in ts:
            if t is not None:
                t.record_stream(self.stream)


def _allocator(device, stream):
    """None where the call runs on the device's current stream."""
    if stream is None:
        return None
    import torch
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device} but the tensors are on {device}")
    current = torch.cuda.current_stream(device)
    return None if stream == current else _Allocator(stream, current)


def _torch():
    import torch
    return torch


def _empty(al, like, shape, dtype):
    if al is not None:
        return al.empty(like, shape, dtype)
    if dtype == like.dtype and shape == like.shape:
        return _torch().empty_like(like)   # half the host time of the general form
    return like.new_empty(shape, dtype=dtype)


def _out(al, out, like, shape):
    """The result tensor: `out` once checked, or a new one of `like`'s dtype."""
    if out is not None:
        _like(out, shape, like.dtype, "out")
        return out
    return _empty(al, like, shape, like.dtype)


def _ptr(t):
    return None if t is None else _at(t)


def layernorm_forward(X, gamma=None, beta=None, eps=1e-5, stats=False, out=None, stream=None):
    """Layer norm over the last axis of X (..., C) (dgrad_layernorm_forward).

    gamma, beta: (C,) of X's dtype, or None for ones and zeros.  With ``stats`` the
    result is (Y, mean, rstd), the fp32 statistics of shape X.shape[:-1] that
    layernorm_backward takes.  ``out`` may be X."""
    import torch
    _need_cuda(X)
    code = _dtype_code(X)
    M, C = _rows_of(X)
    given = [t for t in (gamma, beta, out) if t is not None]
    _need_cuda(*given)
    dev = _device_of(X, *given)
    for t, what in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _like(t, (C,), X.dtype, what)
    al = _allocator(dev, stream)
    out = _out(al, out, X, X.shape)
    mean = rstd = None
    if stats:
        mean = _empty(al, X, X.shape[:-1], torch.float32)
        rstd = _empty(al, mean, mean.shape, torch.float32)
    if al is not None:
        al.uses(X, *given)
    _call(dev, "dgrad_layernorm_forward", lib().dgrad_layernorm_forward, M, C, code, float(eps), _at(X),
          _ptr(gamma), _ptr(beta), _at(out), _ptr(mean), _ptr(rstd), stream=stream)
    return (out, mean, rstd) if stats else out


@functools.lru_cache(maxsize=256)
def _ln_workspace(M, C, code) -> int:
    nb = ctypes.c_size_t()
    _check(lib().dgrad_layernorm_backward_workspace(M, C, code, ctypes.byref(nb)), "dgrad_layernorm_backward_workspace")
    return nb.value


def layernorm_backward_workspace_bytes(M, C, dtype) -> int:
    """Workspace bytes layernorm_backward needs for M rows of C elements of a torch dtype (host only)."""
    return _ln_workspace(int(M), int(C), _code_of(dtype))


def layernorm_backward(dY, X, mean, rstd, gamma=None, param_grads=True, workspace=None, out=None, stream=None):
    """Gradients of layernorm_forward: (dX, dgamma, dbeta) (dgrad_layernorm_backward).

    mean, rstd: the forward's statistics.  dgamma and dbeta (C,) have X's dtype; without
    ``param_grads`` they are None and not computed.  ``out`` (dX) may be dY or X.
    workspace: a CUDA tensor of at least layernorm_backward_workspace_bytes(...) bytes,
    taken from torch when None."""
    import torch
    _need_cuda(dY, X, mean, rstd)
    code = _dtype_code(X)
    M, C = _rows_of(X)
    _like(dY, X.shape, X.dtype, "dY")
    _like(mean, X.shape[:-1], torch.float32, "mean")
    _like(rstd, X.shape[:-1], torch.float32, "rstd")
    given = [t for t in (gamma, workspace, out) if t is not None]
    _need_cuda(*given)
    dev = _device_of(dY, X, mean, rstd, *given)
    if gamma is not None:
        _like(gamma, (C,), X.dtype, "gamma")
    al = _allocator(dev, stream)
    out = _out(al, out, X, X.shape)
    dgamma = dbeta = None
    ws_bytes = 0
    if param_grads:
        dgamma = _empty(al, X if gamma is None else gamma, (C,), X.dtype)
        dbeta = _empty(al, dgamma, (C,), X.dtype)
        if workspace is None:
            ws_bytes = max(_ln_workspace(M, C, code), 16)
            workspace = _empty(al, X, (ws_bytes,), torch.uint8)
        else:
            ws_bytes = workspace.numel() * workspace.element_size()
    if al is not None:
        al.uses(dY, X, mean, rstd, *given)
    _call(dev, "dgrad_layernorm_backward", lib().dgrad_layernorm_backward, M, C, code, _at(dY), _at(X),
          _ptr(gamma), _at(mean), _at(rstd), _at(out), _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
          ws_bytes, stream=stream)
    return out, dgamma, dbeta


def _samples_of(X, groups):
    """(N, S, C, G): samples, positions, channels and groups of X (N, ..., C)."""
    if X.dim() < 2:
        raise ValueError("expected samples of positions (N, ..., C)")
    groups = int(groups)
    C = X.shape[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the {C} channels, got {groups}")
    S = 1
    for d in X.shape[1:-1]:
        S *= d
    return X.shape[0], S, C, groups


def _norm_act(act):
    return _ACT_NONE if act is None else _act_code(act)


@functools.lru_cache(maxsize=256)
def _gn_workspace(backward, N, S, C, G, code) -> int:
    name = "dgrad_groupnorm_" + ("backward" if backward else "forward") + "_workspace"
    nb = ctypes.c_size_t()
    _check(getattr(lib(), name)(N, S, C, G, code, ctypes.byref(nb)), name)
    return nb.value


def groupnorm_forward_workspace_bytes(N, S, C, groups, dtype) -> int:
    """Workspace bytes groupnorm_forward needs for N samples of S positions of C channels (host only)."""
    return _gn_workspace(False, int(N), int(S), int(C), int(groups), _code_of(dtype))


def groupnorm_backward_workspace_bytes(N, S, C, groups, dtype) -> int:
    """Workspace bytes groupnorm_backward needs (host only)."""
    return _gn_workspace(True, int(N), int(S), int(C), int(groups), _code_of(dtype))


def _workspace(al, workspace, like, nbytes):
    """(pointer's tensor, bytes): the given workspace, or one from torch where any is needed."""
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, 0
    return _empty(al, like, (nbytes,), _torch().uint8), nbytes


def groupnorm_forward(X, groups, gamma=None, beta=None, eps=1e-5, act=None, stats=False, workspace=None, out=None,
                      stream=None):
    """Group norm of X (N, ..., C), channels last, with an activation (dgrad_groupnorm_forward).

    Each of ``groups`` runs of C/groups adjacent channels is normalised over all positions of its
    sample.  gamma, beta: (C,) of X's dtype, or None for ones and zeros; act: None or one of
    ACTIVATIONS.  With ``stats`` the result is (Y, mean, rstd), the fp32 statistics (N, groups) that
    groupnorm_backward takes.  ``out`` may be X.  workspace: a CUDA tensor of at least
    groupnorm_forward_workspace_bytes(...) bytes, taken from torch when None."""
    import torch
    _need_cuda(X)
    code = _dtype_code(X)
    N, S, C, G = _samples_of(X, groups)
    acode = _norm_act(act)
    given = [t for t in (gamma, beta, workspace, out) if t is not None]
    _need_cuda(*given)
    dev = _device_of(X, *given)
    for t, what in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _like(t, (C,), X.dtype, what)
    al = _allocator(dev, stream)
    out = _out(al, out, X, X.shape)
    mean = rstd = None
    if stats:
        mean = _empty(al, X, (N, G), torch.float32)
        rstd = _empty(al, mean, mean.shape, torch.float32)
    workspace, ws_bytes = _workspace(al, workspace, X, _gn_workspace(False, N, S, C, G, code))
    if al is not None:
        al.uses(X, *given)
    _call(dev, "dgrad_groupnorm_forward", lib().dgrad_groupnorm_forward, N, S, C, G, code, float(eps), acode,
          _at(X), _ptr(gamma), _ptr(beta), _at(out), _ptr(mean), _ptr(rstd), _ptr(workspace), ws_bytes,
          stream=stream)
    return (out, mean, rstd) if stats else out


def groupnorm_backward(dY, X, mean, rstd, gamma=None, beta=None, act=None, param_grads=True, workspace=None, out=None,
                       stream=None):
    """Gradients of groupnorm_forward: (dX, dgamma, dbeta) (dgrad_groupnorm_backward).

    mean, rstd: the forward's statistics (N, groups); gamma, beta and act as in the forward pass.
    dgamma and dbeta (C,) have X's dtype; without ``param_grads`` they are None and not computed.
    ``out`` (dX) may be dY or X.  workspace: a CUDA tensor of at least
    groupnorm_backward_workspace_bytes(...) bytes, taken from torch when None."""
    import torch
    _need_cuda(dY, X, mean, rstd)
    code = _dtype_code(X)
    if mean.dim() != 2:
        raise ValueError(f"mean must have shape (N, groups), got {tuple(mean.shape)}")
    N, S, C, G = _samples_of(X, mean.shape[1])
    acode = _norm_act(act)
    _like(dY, X.shape, X.dtype, "dY")
    _like(mean, (N, G), torch.float32, "mean")
    _like(rstd, (N, G), torch.float32, "rstd")
    given = [t for t in (gamma, beta, workspace, out) if t is not None]
    _need_cuda(*given)
    dev = _device_of(dY, X, mean, rstd, *given)
    for t, what in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _like(t, (C,), X.dtype, what)
    al = _allocator(dev, stream)
    out = _out(al, out, X, X.shape)
    dgamma = dbeta = None
    if param_grads:
        dgamma = _empty(al, X if gamma is None else gamma, (C,), X.dtype)
        dbeta = _empty(al, dgamma, (C,), X.dtype)
    workspace, ws_bytes = _workspace(al, workspace, X, _gn_workspace(True, N, S, C, G, code))
    if al is not None:
        al.uses(dY, X, mean, rstd, *given)
    _call(dev, "dgrad_groupnorm_backward", lib().dgrad_groupnorm_backward, N, S, C, G, code, acode, _at(dY),
          _at(X), _ptr(gamma), _ptr(beta), _at(mean), _at(rstd), _at(out), _ptr(dgamma),
          _ptr(dbeta), _ptr(workspace), ws_bytes, stream=stream)
    return out, dgamma, dbeta


def _act_code(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}; use one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _gated_width(W, C):
    """F of W (2F, C)."""
    if W.dim() != 2 or W.shape[1] != C or W.shape[0] % 2 or W.shape[0] == 0:
        raise ValueError(f"expected W (2F, {C}), got {tuple(W.shape)}")
    return W.shape[0] // 2


def gated_forward(X, W, act="silu", preact=False, out=None, stream=None):
    """Gated pointwise block (bf16 or f16; dgrad_gated_forward): H = act(X Wg^T) * (X Wu^T).

    X (..., C); W (2F, C), the gate's F rows first -> H (..., F).  With ``preact`` the result
    is (H, Z), the pre-activations (..., 2F) that gated_backward takes."""
    _need_cuda(X, W)
    code = _dtype_code(X)
    acode = _act_code(act)
    M, C = _rows_of(X)
    F = _gated_width(W, C)
    _like(W, W.shape, X.dtype, "W")
    given = [out] if out is not None else []
    _need_cuda(*given)
    dev = _device_of(X, W, *given)
    al = _allocator(dev, stream)
    shape = (*X.shape[:-1], F)
    out = _out(al, out, X, shape)
    Z = _empty(al, X, (*X.shape[:-1], 2 * F), X.dtype) if preact else None
    if al is not None:
        al.uses(X, W, *given)
    _call(dev, "dgrad_gated_forward", lib().dgrad_gated_forward, M, C, F, code, acode, _at(X), _at(W),
          _at(out), _ptr(Z), stream=stream)
    return (out, Z) if preact else out


@functools.lru_cache(maxsize=256)
def _gated_workspace(M, C, F) -> int:
    nb = ctypes.c_size_t()
    _check(lib().dgrad_gated_backward_workspace(M, C, F, ctypes.byref(nb)), "dgrad_gated_backward_workspace")
    return nb.value


def gated_backward_workspace_bytes(M, C, F) -> int:
    """Workspace bytes gated_backward needs (host only)."""
    return _gated_workspace(int(M), int(C), int(F))


def gated_backward(dH, X, Z, W, act="silu", input_grad=True, weight_grad=True, workspace=None, stream=None):
    """Gradients of gated_forward: (dX, dW) (bf16 or f16; dgrad_gated_backward).

    Z: the pre-activations gated_forward kept.  The gradient at Z is rounded to the element
    type before the two products (fp32 up to 4096 values of dH); in f16 it is scaled where its
    range needs that.  Without ``input_grad`` dX, without
    ``weight_grad`` dW is None and not computed.  workspace: a CUDA tensor of at least
    gated_backward_workspace_bytes(...) bytes, taken from torch when None."""
    import torch
    _need_cuda(dH, X, Z, W)
    code = _dtype_code(X)
    acode = _act_code(act)
    M, C = _rows_of(X)
    F = _gated_width(W, C)
    _like(W, W.shape, X.dtype, "W")
    _like(dH, (*X.shape[:-1], F), X.dtype, "dH")
    _like(Z, (*X.shape[:-1], 2 * F), X.dtype, "Z")
    if not input_grad and not weight_grad:
        raise ValueError("nothing to compute: neither input_grad nor weight_grad")
    given = [workspace] if workspace is not None else []
    _need_cuda(*given)
    dev = _device_of(dH, X, Z, W, *given)
    al = _allocator(dev, stream)
    dX = _out(al, None, X, X.shape) if input_grad else None
    dW = _out(al, None, W, W.shape) if weight_grad else None
    if workspace is None:
        workspace = _empty(al, X, (max(_gated_workspace(M, C, F), 16),), torch.uint8)
    if al is not None:
        al.uses(dH, X, Z, W, *given)
    _call(dev, "dgrad_gated_backward", lib().dgrad_gated_backward, M, C, F, code, acode, _at(dH), _at(X),
          _at(Z), _at(W), _ptr(dX), _ptr(dW), _at(workspace),
          workspace.numel() * workspace.element_size(), stream=stream)
    return dX, dW


def _counter(v, what):
    v = int(v)
    if not 0 <= v < 1 << 64:
        raise ValueError(f"{what} must lie in [0, 2^64)")
    return v


def dropout_forward(X, p, seed, offset=0, residual=None, out=None, stream=None):
    """Dropout with probability p, plus ``residual`` when given (dgrad_dropout_forward).

    The mask is a function of (seed, offset) and the element's index, and is not stored:
    give every call its own pair, and the backward pass its forward's.  The pair is taken when
    the call is made: a call captured into a CUDA graph repeats its mask in every replay.
    p is rounded to a multiple of 2^-16.  ``out`` may be X or residual."""
    _need_cuda(X)
    code = _dtype_code(X)
    given = [t for t in (residual, out) if t is not None]
    _need_cuda(*given)
    dev = _device_of(X, *given)
    if residual is not None:
        _like(residual, X.shape, X.dtype, "residual")
    al = _allocator(dev, stream)
    out = _out(al, out, X, X.shape)
    if al is not None:
        al.uses(X, *given)
    _call(dev, "dgrad_dropout_forward", lib().dgrad_dropout_forward, X.numel(), code, float(p),
          _counter(seed, "seed"), _counter(offset, "offset"), _at(X), _ptr(residual), _at(out),
          stream=stream)
    return out


def dropout_backward(dY, p, seed, offset=0, out=None, stream=None):
    """Gradient of dropout_forward in X (dgrad_dropout_backward); the residual's is dY itself.
    ``out`` may be dY."""
    _need_cuda(dY)
    code = _dtype_code(dY)
    given = [out] if out is not None else []
    _need_cuda(*given)
    dev = _device_of(dY, *given)
    al = _allocator(dev, stream)
    out = _out(al, out, dY, dY.shape)
    if al is not None:
        al.uses(dY, *given)
    _call(dev, "dgrad_dropout_backward", lib().dgrad_dropout_backward, dY.numel(), code, float(p),
          _counter(seed, "seed"), _counter(offset, "offset"), _at(dY), _at(out), stream=stream)
    return out


# ------------------------------------------------ the optimizer's step over many tensors

QUANT_BLOCK = 256   # elements of a tensor that share a maximum in 8-bit states

_TABLE = [("param", "u8"), ("grad", "u8"), ("m", "u8"), ("v", "u8"), ("master", "u8"), ("m_max", "u8"), ("v_max", "u8"),
          ("n", "i8")]   # dgrad_adamw_tensor_t


def _lists():
    """The native reader of tensor lists (csrc/tensor_lists.cpp)."""
    global _reader
    if _reader is None:
        import importlib

        import torch       # its libraries come first
        try:
            reader = importlib.import_module("._tensor_lists", __name__)
        except ImportError as e:
            raise DgradUnavailable(f"cannot load _tensor_lists: {e}; build it with "
                                   "`python -m convolution_backward_b200._build`") from e
        if reader.torch_version != torch.__version__.split("+")[0]:
            raise DgradUnavailable(f"_tensor_lists was built against torch {reader.torch_version}, this is {torch.__version__}; "
                                   "build it again with `python -m convolution_backward_b200._build`")
        _reader = reader
    return _reader


_reader = None


class _Array:
    """A numpy array and its address."""

    def __init__(self, a):
        self.a, self.at = a, a.ctypes.data


def _same(ts, what):
    """The one dtype and CUDA device of a list of contiguous tensors."""
    if not ts:
        raise ValueError(f"{what}: expected at least one tensor")
    _need_cuda(*ts)
    for t in ts:
        if t.dtype != ts[0].dtype:
            raise TypeError(f"{what} must have one dtype, got {ts[0].dtype} and {t.dtype}")
    return ts[0].dtype, _device_of(*ts)


class AdamWState:
    """Parameters and optimizer states that adamw_step works on: lists of contiguous CUDA tensors of
    one device, one tensor of each list per parameter.

    params: one dtype.  32-bit states: m, v fp32 of the parameters' shapes.  8-bit states: m int8 and v
    uint8 codes of the parameters' shapes, and m_max, v_max fp32 with an element for every 256 of a tensor.
    master: fp32 copies of 16-bit parameters, which are then what is stepped.  No two tensors may
    share memory.  copy.copy shares the tensors, copy.deepcopy and pickle copy them.  The tensors stay the
    caller's: save them as they are, load them with copy_; where the storage of one has been replaced, or its size
    or type changed, adamw_step refuses the state.  A step counts as an in-place change of the parameters and
    master copies that it writes: a graph that has saved one of them raises when it is run backward.  (The states
    are not counted, and the replay of a captured step counts nothing.)"""

    def __init__(self, params, m, v, master=None, m_max=None, v_max=None):
        import numpy as np
        import torch
        self.params, self.m, self.v = tuple(params), tuple(m), tuple(v)
        self.master = None if master is None else tuple(master)
        dtype, self.device = _same(self.params, "params")
        self._code = _code_of(dtype)
        self.dtype = dtype
        n = len(self.params)
        self.bits = 8 if (self.m and self.m[0].dtype == torch.int8) else 32
        if (self.bits == 8) != (m_max is not None) or (self.bits == 8) != (v_max is not None):
            raise ValueError("m_max and v_max go with int8 m and uint8 v")
        self.m_max = None if m_max is None else tuple(m_max)
        self.v_max = None if v_max is None else tuple(v_max)
        lists = [("m", self.m, torch.int8 if self.bits == 8 else torch.float32),
                 ("v", self.v, torch.uint8 if self.bits == 8 else torch.float32), ("master", self.master, torch.float32)]
        self.shapes = [tuple(p.shape) for p in self.params]
        for what, ts, want in lists:
            if ts is None:
                continue
            if len(ts) != n:
                raise ValueError(f"{what}: expected {n} tensors, got {len(ts)}")
            for t, shape in zip(ts, self.shapes):
                _like(t, shape, want, what)
        for what, ts in (("m_max", self.m_max), ("v_max", self.v_max)):
            if ts is None:
                continue
            if len(ts) != n:
                raise ValueError(f"{what}: expected {n} tensors, got {len(ts)}")
            for t, p in zip(ts, self.params):
                _like(t, (-(-p.numel() // QUANT_BLOCK),), torch.float32, what)
        everything = [t for ts in (self.params, self.m, self.v, self.master, self.m_max, self.v_max) if ts for t in ts]
        _need_cuda(*everything)
        _device_of(*everything)
        self._list, self._all = list(self.params), everything
        self._weights = self._list + list(self.master or ())
        self._was = [_Array(np.empty(len(everything), dtype=t)) for t in (np.uint64, np.int64, np.int64)]
        self._was_at = tuple(w.at for w in self._was)
        _lists().describe(everything, *self._was_at)
        self._table = np.zeros(n, dtype=_TABLE)
        for name, ts in (("param", self.params), ("m", self.m), ("v", self.v), ("master", self.master),
                         ("m_max", self.m_max), ("v_max", self.v_max)):
            if ts is not None:
                self._table[name] = [t.data_ptr() for t in ts]
        self._table["n"] = [p.numel() for p in self.params]
        self._address = self._table.ctypes.data
        status = lib().dgrad_adamw_check(n, self._address, self._code, self._code, self.bits)
        if status == 1:
            raise ValueError("parameters and states must not share memory")
        _check(status, "dgrad_adamw_check")
        self._n = _Array(np.ascontiguousarray(self._table["n"]))
        # the written ranges in order, for gradients and results to be held against
        lo = np.array([t.data_ptr() for t in everything if t.numel()], dtype=np.uint64)
        size = np.array([t.numel() * t.element_size() for t in everything if t.numel()], dtype=np.uint64)
        order = np.argsort(lo)
        self._lo, self._hi = _Array(lo[order]), _Array((lo + size)[order])
        self._ranges = (self._lo.at, self._hi.at, len(order))
        # one step's gradients; a call of adamw_step fills them and has read them when it returns
        self._grads = _Array(np.zeros(n, dtype=np.uint64))

    def _apart(self, at, nbytes):
        return _lists().apart(at, self._n.at, len(self.params), nbytes, *self._ranges)

    def __reduce__(self):
        """Copies and pickles are made anew from (copies of) the tensors: the addresses held here are this state's own."""
        lists = (self.params, self.m, self.v, self.master, self.m_max, self.v_max)
        return type(self), tuple(None if ts is None else list(ts) for ts in lists)

    def _unchanged(self, lists):
        if not lists.same(self._all, *self._was_at):
            raise ValueError("the storage, size or type of a parameter or state has changed since its AdamWState was made")

    def __len__(self):
        return len(self.params)


def adamw_state(params, bits=32, master=False):
    """A fresh AdamWState for `params`: zero moments in 32 or in 8 bits, and with ``master`` fp32 copies of
    16-bit parameters."""
    import torch
    params = list(params)
    if bits not in (32, 8):
        raise ValueError(f"bits must be 32 or 8, got {bits}")

    def zeros(dtype):
        return [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params]

    def maxima():
        return [torch.zeros(-(-p.numel() // QUANT_BLOCK), device=p.device) for p in params]

    _same(params, "params")
    more = {"master": [p.detach().float().clone() for p in params]} if master else {}
    if bits == 32:
        return AdamWState(params, zeros(torch.float32), zeros(torch.float32), **more)
    return AdamWState(params, zeros(torch.int8), zeros(torch.uint8), m_max=maxima(), v_max=maxima(), **more)


def _scalar(t, dtype, dev, what):
    """The device pointer of a one-element tensor."""
    _need_cuda(t)
    if t.numel() != 1:
        raise ValueError(f"{what} must have one element, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    _device_of(t, _On(dev))
    return _at(t)


class _On:
    """A device, for _device_of."""

    def __init__(self, device):
        self.device = device


def adamw_step(state, grads, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=None, seed=None,
               offset=0, stream=None) -> None:
    """One AdamW step over all tensors of `state`, in place (dgrad_adamw_step).

    grads: one tensor per parameter, of its shape and of the parameters' dtype or float32 (one dtype
    for the list), or None for a parameter that is left as it is.  step counts from 1.  step and lr
    may be one-element CUDA tensors (int64, float32), which a captured step reads in every replay (a step
    below 1 or a rate that is no finite number changes nothing).
    grad_scale: a one-element fp32 CUDA tensor that multiplies the gradients (grad_norm's factor); where
    it is no finite number the step changes nothing.  seed (8-bit states): codes are
    rounded stochastically by the bits of (seed, offset): give every step its own pair, and dropout others;
    None: to the nearer value.  Moments and weights are fp32 within the step, and the weights
    (master copies) are rounded once to the parameters' dtype."""
    import torch
    n = len(state.params)
    grads = list(grads)
    dev = state.device
    to = state._grads
    lists = _lists()
    gcode, gdev = lists.read(grads, state._list, "gradients", to.at, 0)
    if gcode < 0:
        gcode, gdev = state._code, dev.index     # nothing to step
    if gcode != state._code and gcode != 0:
        raise TypeError(f"gradients must be {state.dtype} or float32")
    if gdev != dev.index:
        raise ValueError("all tensors of one call must be on the same CUDA device")
    state._unchanged(lists)
    if not lists.apart(to.at, state._n.at, n, 4 if gcode == 0 else 2, *state._ranges):
        raise ValueError("gradients must not share memory with parameters or states")
    state._table["grad"] = to.a
    h = _AdamW()
    given = []
    if isinstance(lr, torch.Tensor):
        h.lr_device = _scalar(lr, torch.float32, dev, "lr")
        given.append(lr)
    else:
        h.lr = float(lr)
    if isinstance(step, torch.Tensor):
        h.step_device = _scalar(step, torch.int64, dev, "step")
        given.append(step)
    else:
        h.step = int(step)
    if grad_scale is not None:
        h.grad_scale = _scalar(grad_scale, torch.float32, dev, "grad_scale")
        given.append(grad_scale)
    if given:
        scalars = array.array("q", [a for a in (h.lr_device, h.step_device, h.grad_scale) if a] + [1] * len(given))
        where = scalars.buffer_info()[0]
        if not lists.apart(where, where + 8 * len(given), len(given), 8, *state._ranges):
            raise ValueError("lr, step and grad_scale must not share memory with parameters or states")
    h.beta1, h.beta2 = betas
    h.eps, h.weight_decay, h.state_bits = eps, weight_decay, state.bits
    if seed is not None:
        if state.bits != 8:
            raise ValueError("seed goes with 8-bit states")
        h.stochastic, h.seed, h.offset = 1, _counter(seed, "seed"), _counter(offset, "offset")
    al = _allocator(dev, stream)
    if al is not None:
        al.uses(*grads, *given, *state._all)
    _call(dev, "dgrad_adamw_step", lib().dgrad_adamw_step, n, state._address, state._code, gcode, ctypes.byref(h),
          stream=stream)
    lists.written(state._weights, to.at, n)


def adamw_moments(state, out=None, stream=None):
    """(m, v): what a state's moments stand for, as fp32 tensors (dgrad_adamw_moments): for
    checkpoints, or to go on with 32-bit states.  32-bit states are returned as they are.  out: two lists of
    fp32 tensors of the parameters' shapes to write to."""
    import numpy as np
    import torch
    if state.bits == 32 and out is None:
        return state.m, state.v
    if state.bits == 32:
        raise ValueError("32-bit moments are state.m and state.v")
    dev = state.device
    al = _allocator(dev, stream)
    given = []
    if out is None:
        out = tuple([_empty(al, state.m_max[i], s, torch.float32) for i, s in enumerate(state.shapes)] for _ in range(2))
    else:
        out = tuple(list(ts) for ts in out)
        if len(out) != 2:
            raise ValueError("out: expected two lists of tensors")
        given = out[0] + out[1]
        if any(t is None for t in given):
            raise TypeError("out must be tensors")
    state._unchanged(_lists())
    to = [_Array(np.empty(len(state), dtype=np.uint64)) for _ in range(2)]
    for ts, at, what in zip(out, to, ("out: m", "out: v")):
        code, index = _lists().read(ts, state._list, what, at.at, 0)
        if code != 0:
            raise TypeError(f"{what} must be float32")
        if index != dev.index:
            raise ValueError("all tensors of one call must be on the same CUDA device")
    if given and not (state._apart(to[0].at, 4) and state._apart(to[1].at, 4) and
                      _lists().disjoint(to[0].at, to[1].at, state._n.at, len(state), 4)):
        raise ValueError("out must not share memory with itself or the state")
    if al is not None:
        al.uses(*given, *state._all)
    _call(dev, "dgrad_adamw_moments", lib().dgrad_adamw_moments, len(state), state._address, to[0].at, to[1].at, stream=stream)
    if given:
        _lists().written(given, to[0].at, len(state))
    return out


@functools.lru_cache(maxsize=256)
def _norm_workspace(count) -> int:
    nb = ctypes.c_size_t()
    _check(lib().dgrad_grad_norm_workspace(count, ctypes.byref(nb)), "dgrad_grad_norm_workspace")
    return nb.value


def grad_norm_workspace_bytes(count) -> int:
    """Workspace bytes grad_norm needs for a list of `count` tensors (host only)."""
    return _norm_workspace(int(count))


def grad_norm(grads, max_norm=None, workspace=None, stream=None):
    """The norm over all elements of `grads` (contiguous, one dtype and device), a fp32 CUDA scalar
    (dgrad_grad_norm).  With max_norm: (norm, scale) with scale = min(1, max_norm/(norm + 1e-6)), the
    grad_scale that clips an adamw_step; NaN where the norm is no finite number, which leaves that step
    out.  Nothing waits for the GPU."""
    import torch
    grads = list(grads)
    if not grads:
        raise ValueError("grads: expected at least one tensor")
    lists = array.array("q", bytes(16 * len(grads)))     # addresses, elements
    at = lists.buffer_info()[0]
    elements = at + 8 * len(grads)
    code, _ = _lists().read(grads, None, "gradients", at, elements)
    first = grads[0]
    dev = first.device
    limit = float("inf") if max_norm is None else float(max_norm)
    given = [] if workspace is None else [workspace]
    _need_cuda(*given)
    _device_of(first, *given)
    al = _allocator(dev, stream)
    ws_bytes = _norm_workspace(len(grads))
    if workspace is None:       # behind the two results
        out = _empty(al, first, (4 + ws_bytes // 4,), torch.float32)
        ws_at = _at(out) + 16
    else:
        out = _empty(al, first, (2,), torch.float32)
        ws_at, ws_bytes = _at(workspace), workspace.numel() * workspace.element_size()
    if al is not None:
        al.uses(*grads, *given)
    _call(dev, "dgrad_grad_norm", lib().dgrad_grad_norm, len(grads), at, elements, code, limit,
          _at(out), ws_at, ws_bytes, stream=stream)
    return out[0] if max_norm is None else (out[0], out[1])


def check_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel reported a timeout (dgrad_check_status)."""
    import torch
    dev = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().dgrad_check_status(_stream_ptr(stream, dev)), "dgrad_check_status")


def selftest_timeout(limit_cycles: int = 20_000_000, stream=None) -> None:
    """Launch the diagnostic kernel whose bounded wait runs out (dgrad_selftest_timeout)."""
    import torch
    dev = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().dgrad_selftest_timeout(int(limit_cycles), _stream_ptr(stream, dev)), "dgrad_selftest_timeout")


def fma_probe(blocks: int, iters: int, packed: bool, sink, stream=None) -> int:
    """Launch the fp32 FMA-rate probe; returns the FLOP count it performs."""
    _call(_device_of(sink), "dgrad_fma_probe", lib().dgrad_fma_probe, int(blocks), int(iters), 1 if packed else 0,
          _at(sink), stream=stream)
    return int(blocks) * 256 * int(iters) * 16 * 2
