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

and their ``_backward`` counterparts.  Tensors are NHWC (rows of channels) and contiguous;
float32, bfloat16 or float16 (16-bit in, 16-bit out, fp32 accumulate).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

__all__ = ["pointwise", "pointwise_splitk", "pointwise_splitk_noalloc", "depthwise_tc", "depthwise_tc_workspace_bytes", "dense", "grouped", "splitk_workspace_bytes", "depthwise", "out_dims", "check_status", "DgradError", "DgradUnavailable",
           "layernorm_forward", "layernorm_backward", "layernorm_backward_workspace_bytes", "dropout_forward", "dropout_backward",
           "gated_forward", "gated_backward", "gated_backward_workspace_bytes", "ACTIVATIONS",
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
          dY.data_ptr(), W.data_ptr(), out.data_ptr(), stream=stream)
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
          ctypes.byref(prob), _dtype_code(dY), int(used), dY.data_ptr(), W.data_ptr(), out.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream=stream)
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
          ctypes.byref(prob), _dtype_code(dY), int(splits), dY.data_ptr(), W.data_ptr(), out.data_ptr(),
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
          DW_MODES[mode], dY.data_ptr(), W.data_ptr(), out.data_ptr(), stream=stream)
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
          dY.data_ptr(), W.data_ptr(), out.data_ptr(), stream=stream)
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
          _dtype_code(dY), dY.data_ptr(), W.data_ptr(), out.data_ptr(), stream=stream)
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
          _dtype_code(dY), dY.data_ptr(), W.data_ptr(), out.data_ptr(), workspace.data_ptr(),
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
    return None if t is None else t.data_ptr()


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
    _call(dev, "dgrad_layernorm_forward", lib().dgrad_layernorm_forward, M, C, code, float(eps), X.data_ptr(),
          _ptr(gamma), _ptr(beta), out.data_ptr(), _ptr(mean), _ptr(rstd), stream=stream)
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
    _call(dev, "dgrad_layernorm_backward", lib().dgrad_layernorm_backward, M, C, code, dY.data_ptr(), X.data_ptr(),
          _ptr(gamma), mean.data_ptr(), rstd.data_ptr(), out.data_ptr(), _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
          ws_bytes, stream=stream)
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
    _call(dev, "dgrad_gated_forward", lib().dgrad_gated_forward, M, C, F, code, acode, X.data_ptr(), W.data_ptr(),
          out.data_ptr(), _ptr(Z), stream=stream)
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
    _call(dev, "dgrad_gated_backward", lib().dgrad_gated_backward, M, C, F, code, acode, dH.data_ptr(), X.data_ptr(),
          Z.data_ptr(), W.data_ptr(), _ptr(dX), _ptr(dW), workspace.data_ptr(),
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
          _counter(seed, "seed"), _counter(offset, "offset"), X.data_ptr(), _ptr(residual), out.data_ptr(),
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
          _counter(seed, "seed"), _counter(offset, "offset"), dY.data_ptr(), out.data_ptr(), stream=stream)
    return out


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
          sink.data_ptr(), stream=stream)
    return int(blocks) * 256 * int(iters) * 16 * 2
