"""ctypes binding of libfp8_scaled_mm.so: argument marshalling only.

Every step of the multiply runs in the HIP library; this module turns torch
tensors into device pointers, sizes and the current stream, and turns
status codes into exceptions.  A missing library is an error (there is no
fallback path).  The ordinary calls of the layer norm and the linear layer go
through _calls (csrc/torch_calls.cpp), which does the same with less host time;
without it they take the same path as the others.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import math
import os
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
try:
    from . import _calls
except ImportError as e:
    _calls = None
    if os.path.exists(os.path.join(HERE, "_calls.so")):
        warnings.warn(f"the extension _calls does not load ({e}): short calls take some microseconds more; build it "
                      "again with `python -m precision_linear_amd.build`")

library_path = os.path.join(HERE, "libfp8_scaled_mm.so")

PER_TENSOR = 0
ROWWISE = 1
_MODES = {"per_tensor": PER_TENSOR, "tensorwise": PER_TENSOR, "rowwise": ROWWISE,
          PER_TENSOR: PER_TENSOR, ROWWISE: ROWWISE}

# operand formats (enum fp8mm_format)
E4M3FN = 0
E5M2 = 1
_FORMATS = {"e4m3fn": E4M3FN, "e5m2": E5M2, E4M3FN: E4M3FN, E5M2: E5M2}

# splits value of a stream-K plan (FP8MM_SPLITS_STREAM_K in include/fp8_scaled_mm.h)
SPLITS_STREAM_K = -1

# status codes from include/fp8_scaled_mm.h
(OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_MODE, ERR_DEVICE, ERR_LAUNCH, ERR_CONFIG, ERR_WORKSPACE,
 ERR_FORMAT, ERR_SCRATCH, ERR_ACTIVATION) = range(12)
_ARG_ERRORS = {ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_MODE, ERR_CONFIG, ERR_WORKSPACE, ERR_FORMAT,
               ERR_SCRATCH, ERR_ACTIVATION}

EXPORTS = ("fp8_scaled_mm", "fp8_scaled_mm_with_config", "fp8_scaled_mm_with_plan",
           "fp8_scaled_mm_typed", "fp8_scaled_mm_noalloc",
           "fp8_scaled_mm_workspace_size", "fp8_scaled_mm_select_splits",
           "fp8_scaled_mm_num_configs", "fp8_scaled_mm_config_name", "fp8_scaled_mm_select_config",
           "fp8_scaled_mm_grid_size", "fp8_scaled_mm_status_string", "fp8mm_status_string",
           "fp8_quantize_e4m3", "fp8_quantize_e5m2", "fp8_quantize_e4m3_ws", "fp8_quantize_e5m2_ws",
           "fp8_quantize_workspace_size", "fp8_quantize_set_wait_limit_us",
           "fp8_quantize_status_string")

# status codes from include/fp8_quantize.h
(Q_OK, Q_ERR_NULL, Q_ERR_SHAPE, Q_ERR_ALIGN, Q_ERR_MODE, Q_ERR_DEVICE, Q_ERR_LAUNCH,
 Q_ERR_WORKSPACE) = range(8)
_Q_ARG_ERRORS = {Q_ERR_NULL, Q_ERR_SHAPE, Q_ERR_ALIGN, Q_ERR_MODE, Q_ERR_WORKSPACE}

# functions from include/fp8_linear.h (status codes: those of fp8_scaled_mm.h)
# and its activations (enum fp8mm_activation)
LINEAR_EXPORTS = ("fp8_linear", "fp8_linear_backward", "fp8_linear_backward_workspace_size")
_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# functions and status codes from include/fp8_layer_norm.h
LAYER_NORM_EXPORTS = ("fp8_layer_norm", "fp8_layer_norm_backward",
                      "fp8_layer_norm_backward_workspace_size", "fp8_layer_norm_status_string")
(LN_OK, LN_ERR_NULL, LN_ERR_SHAPE, LN_ERR_ALIGN, LN_ERR_DTYPE, LN_ERR_DEVICE, LN_ERR_LAUNCH,
 LN_ERR_WORKSPACE, LN_ERR_VALUE) = range(9)
_LN_ARG_ERRORS = {LN_ERR_NULL, LN_ERR_SHAPE, LN_ERR_ALIGN, LN_ERR_DTYPE, LN_ERR_WORKSPACE,
                  LN_ERR_VALUE}


# The entry points that _calls uses, in its order.
_CALLS_ENTRIES = ("fp8_layer_norm", "fp8_layer_norm_backward", "fp8_layer_norm_backward_workspace_size",
                  "fp8_linear", "fp8_scaled_mm_workspace_size", "fp8_linear_backward",
                  "fp8_linear_backward_workspace_size")


class Fp8MMError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"fp8_scaled_mm failed: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is missing: build it with "
                "`python -m precision_linear_amd.build` (there is no non-HIP fallback)")
        L = ctypes.CDLL(library_path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.fp8_scaled_mm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
        L.fp8_scaled_mm.restype = i32
        L.fp8_scaled_mm_with_config.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32]
        L.fp8_scaled_mm_with_config.restype = i32
        L.fp8_scaled_mm_with_plan.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32,
                                              i32, vp, i64]
        L.fp8_scaled_mm_with_plan.restype = i32
        L.fp8_scaled_mm_typed.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i64, i64, i64, i32, vp,
                                          i32, i32, vp, i64]
        L.fp8_scaled_mm_typed.restype = i32
        L.fp8_scaled_mm_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, i32]
        L.fp8_scaled_mm_noalloc.restype = i32
        L.fp8_scaled_mm_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32, i32]
        L.fp8_scaled_mm_workspace_size.restype = i64
        L.fp8_scaled_mm_select_splits.argtypes = [i64, i64, i64, i32, i32, i32]
        L.fp8_scaled_mm_select_splits.restype = i32
        L.fp8_scaled_mm_num_configs.argtypes = []
        L.fp8_scaled_mm_num_configs.restype = i32
        L.fp8_scaled_mm_config_name.argtypes = [i32]
        L.fp8_scaled_mm_config_name.restype = ctypes.c_char_p
        L.fp8_scaled_mm_select_config.argtypes = [i64, i64, i64, i32, i32, i32]
        L.fp8_scaled_mm_select_config.restype = i32
        L.fp8_scaled_mm_grid_size.argtypes = [i32, i64, i64, i32]
        L.fp8_scaled_mm_grid_size.restype = i64
        L.fp8_scaled_mm_status_string.argtypes = [i32]
        L.fp8_scaled_mm_status_string.restype = ctypes.c_char_p
        L.fp8mm_status_string.argtypes = [i32]
        L.fp8mm_status_string.restype = ctypes.c_char_p
        L.fp8_quantize_e4m3.argtypes = [vp, vp, vp, i64, i64, i32, vp]
        L.fp8_quantize_e4m3.restype = i32
        L.fp8_quantize_e5m2.argtypes = [vp, vp, vp, i64, i64, i32, vp]
        L.fp8_quantize_e5m2.restype = i32
        for name in ("fp8_quantize_e4m3_ws", "fp8_quantize_e5m2_ws"):
            getattr(L, name).argtypes = [vp, vp, vp, i64, i64, i32, vp, i64, vp]
            getattr(L, name).restype = i32
        L.fp8_quantize_workspace_size.argtypes = [i64, i64, i32]
        L.fp8_quantize_workspace_size.restype = i64
        L.fp8_quantize_set_wait_limit_us.argtypes = [i64]
        L.fp8_quantize_set_wait_limit_us.restype = i64
        L.fp8_quantize_status_string.argtypes = [i32]
        L.fp8_quantize_status_string.restype = ctypes.c_char_p
        L.fp8_linear.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp, i64, i64, i64, i32, vp,
                                 i32, i32, vp, i64]
        L.fp8_linear.restype = i32
        L.fp8_linear_backward.argtypes = [vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, i64, i64, i64, vp, vp,
                                          i64]
        L.fp8_linear_backward.restype = i32
        L.fp8_linear_backward_workspace_size.argtypes = [i64, i64, i64, i32, i32]
        L.fp8_linear_backward_workspace_size.restype = i64
        f32 = ctypes.c_float
        L.fp8_layer_norm.argtypes = [vp, i32, vp, vp, i32, f32, vp, vp, i32, vp, vp, vp, i64, i64, vp]
        L.fp8_layer_norm.restype = i32
        L.fp8_layer_norm_backward.argtypes = [vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, i64, i64,
                                              vp, i64, vp]
        L.fp8_layer_norm_backward.restype = i32
        L.fp8_layer_norm_backward_workspace_size.argtypes = [i64, i64]
        L.fp8_layer_norm_backward_workspace_size.restype = i64
        L.fp8_layer_norm_status_string.argtypes = [i32]
        L.fp8_layer_norm_status_string.restype = ctypes.c_char_p
        if _calls is not None:
            _calls.use_library(tuple(ctypes.cast(getattr(L, name), ctypes.c_void_p).value
                                     for name in _CALLS_ENTRIES), _workspace)
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fp8_scaled_mm_status_string(int(status)).decode()


def config_names() -> list:
    L = lib()
    return [L.fp8_scaled_mm_config_name(i).decode() for i in range(L.fp8_scaled_mm_num_configs())]


def select_config(M, N, K, mode, has_bias=False, with_workspace=True) -> int:
    """The automatic configuration; with_workspace=True is the plan this
    module's fp8_scaled_mm runs (it supplies a workspace whenever the plan
    splits K), False the one of the C entry point fp8_scaled_mm."""
    return int(lib().fp8_scaled_mm_select_config(M, N, K, _MODES[mode], int(bool(has_bias)),
                                                 int(bool(with_workspace))))


def select_splits(M, N, K, mode, has_bias=False, config=-1) -> int:
    return int(lib().fp8_scaled_mm_select_splits(M, N, K, _MODES[mode], int(bool(has_bias)),
                                                 int(config)))


def workspace_size(M, N, K, mode, has_bias=False, config=-1, splits=0) -> int:
    return int(lib().fp8_scaled_mm_workspace_size(M, N, K, _MODES[mode], int(bool(has_bias)),
                                                  int(config), int(splits)))


# Workspaces handed to the library, per (device, stream, kind): torch allocations
# (the library allocates nothing itself), zeros where the kind counts on them.
# Calls on one stream are ordered, so they can share one; a larger one replaces it
# for later calls, but none is freed, because another thread may be enqueuing a
# call with it.
_workspaces: dict = {}
# While a graph is captured, the calls on a stream share one of the capture's
# own, (capture, workspace): its fill is recorded, to run with each replay, so no
# other call may count on it, and the graph may be replayed beside any other work.
# (torch.cuda.graph keeps the memory of a capture to its graph.)
_captured: dict = {}


def _workspace(device: torch.device, stream: int, nbytes: int, kind: str = "mm") -> torch.Tensor:
    key = (device.index, stream, kind)
    capture = _capture_id(device, stream)
    if capture is not None:
        have = _captured.get(key)
        if have is None or have[0] != capture or have[1].numel() < nbytes:
            # (What is replaced goes back to its graph's memory, as any temporary
            # tensor of a capture does.)
            have = _captured[key] = (capture, _new_workspace(device, nbytes, kind))
        return have[1]
    have = _workspaces.get(key)
    if have and have[-1].numel() >= nbytes:
        return have[-1]
    ws = _new_workspace(device, max(nbytes, 2 * have[-1].numel() if have else 0), kind)
    _workspaces.setdefault(key, []).append(ws)
    return ws


# Bytes at a workspace's start that have to be zero before its first use: the
# arrival counters of a split K, all of the per-tensor quantisation's.
_ZEROED = {"mm": 256 << 10, "quantize": 1 << 20, "layer_norm": 0}


def _new_workspace(device: torch.device, nbytes: int, kind: str) -> torch.Tensor:
    ws = torch.empty((nbytes + (1 << 20) - 1) >> 20 << 20, dtype=torch.uint8, device=device)
    if _ZEROED[kind]:
        ws[:_ZEROED[kind]].zero_()      # a fill kernel on the current stream
    return ws


# Whether the current stream is captured (torch's direct accessor where it has one).
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _capture_id(device: torch.device, stream: int):
    """Which graph capture `stream`, the device's current one, is part of (None: no capture)."""
    if not (_capturing() if _current_device() == device.index else _call(device.index, _capturing)):
        return None
    status, ident = ctypes.c_int(), ctypes.c_ulonglong()
    err = lib().hipStreamGetCaptureInfo(ctypes.c_void_p(stream), ctypes.byref(status), ctypes.byref(ident))
    if err != 0:
        raise RuntimeError(f"hipStreamGetCaptureInfo failed: {err}")
    return ident.value


_TORCH_FORMATS = {torch.float8_e4m3fn: E4M3FN, torch.float8_e5m2: E5M2}


def _as_codes(t: torch.Tensor, name: str, fmt) -> tuple:
    """(tensor, format id).  A float8 tensor carries its format; uint8 codes
    take `fmt` (default e4m3fn)."""
    dt = t.dtype
    if fmt is None and dt == torch.uint8:
        return t, E4M3FN
    if fmt is not None and fmt not in _FORMATS:
        raise ValueError(f"{name}_format must be 'e4m3fn' or 'e5m2', got {fmt!r}")
    if dt in _TORCH_FORMATS:
        f = _TORCH_FORMATS[dt]
        if fmt is not None and _FORMATS[fmt] != f:
            raise ValueError(f"{name} is {dt} but {name}_format={fmt!r}")
        return t, f
    if dt == torch.uint8:
        return t, _FORMATS[fmt]
    raise ValueError(f"{name} must be float8_e4m3fn, float8_e5m2 or uint8 codes, got {dt}")


def _check_devices(dev: int, tensors) -> None:
    """Every (name, tensor) given (None skipped) must live on GPU `dev`: the
    library passes their pointers to kernels on that device.  Compares
    device indices (a CPU tensor's is -1)."""
    for name, t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


# The current stream's raw handle for a device index: torch's direct accessor
# where it has one (no Stream object built per call), else the public API.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


# The current HIP device's index (torch's direct accessor where it has one).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev: int, fn, *args) -> int:
    """fn(*args) with `dev` as the current HIP device (the library launches on
    the current one): calls from that device, the usual case, skip the switch."""
    if _current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


# Workspace bytes of automatic plans, per (device, M, N, K, mode, bias, config,
# splits): the plan depends on nothing else, so the size is asked once.
_ws_sizes: dict = {}


def _keep_size(key, need: int) -> None:
    if len(_ws_sizes) >= 4096:      # many distinct shapes: start over
        _ws_sizes.clear()
    _ws_sizes[key] = need


def _mm_args(a, b, scale_a, scale_b, bias, out, mode, workspace, a_format, b_format, extra=()):
    """Checks the multiply's arguments (`extra`: more (name, tensor) pairs that
    must be on the same GPU).  Returns (a, fa, b, fb, out, M, N, K, mode,
    device index), with `out` allocated if it is None."""
    m = _MODES.get(mode) if isinstance(mode, (str, int)) else None
    if m is None:
        raise ValueError(f"mode must be 'per_tensor' or 'rowwise', got {mode!r}")
    a, fa = _as_codes(a, "a", a_format)
    b, fb = _as_codes(b, "b", b_format)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    if b.shape[1] == K and b.is_contiguous():
        N = b.shape[0]
    elif b.shape[0] == K and b.stride() == (1, K):
        b = b.t()
        N = b.shape[0]
    else:
        raise ValueError(f"b must be N x K contiguous or K x N column-major, got {tuple(b.shape)} "
                         f"strides {b.stride()} for K={K}")
    if not a.is_contiguous():
        raise ValueError("a must be contiguous (row-major M x K)")
    if not (a.is_cuda and b.is_cuda and scale_a.is_cuda and scale_b.is_cuda):
        raise ValueError("all tensors must be on the GPU")
    dev = a.get_device()
    _check_devices(dev, (("b", b), ("scale_a", scale_a), ("scale_b", scale_b), ("bias", bias),
                         ("out", out), ("workspace", workspace), *extra))
    for name, s in (("scale_a", scale_a), ("scale_b", scale_b)):
        if s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32")
    want_a, want_b = (1, 1) if m == PER_TENSOR else (M, N)
    if scale_a.numel() != want_a or scale_b.numel() != want_b:
        raise ValueError(f"{'per-tensor' if m == PER_TENSOR else 'row-wise'} scales need "
                         f"{want_a} and {want_b} elements, got {scale_a.numel()} and {scale_b.numel()}")
    if bias is not None:
        if bias.dtype != torch.bfloat16 or bias.numel() != N or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous bf16 GPU vector of length N")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    elif out.dtype != torch.bfloat16 or out.shape != (M, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 M x N tensor")
    return a, fa, b, fb, out, M, N, K, m, dev


def _mm_workspace(L, device, dev, stream, M, N, K, m, has_bias, config, splits, workspace):
    """(address, bytes) of the workspace of a call's plan: the caller's, or this
    module's for the stream where the plan splits K."""
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous GPU tensor")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if splits == 1:
        return None, 0
    key = (dev, M, N, K, m, has_bias, config, splits)
    need = _ws_sizes.get(key)
    if need is None:
        need = int(L.fp8_scaled_mm_workspace_size(M, N, K, m, int(has_bias), int(config), int(splits)))
        _keep_size(key, need)
    if need <= 0:
        return None, 0
    ws = _workspace(device, stream, need)
    return ws.data_ptr(), ws.numel()


def fp8_scaled_mm(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                  bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  mode="per_tensor", config: int = -1, splits: int = 0,
                  workspace: torch.Tensor | None = None, a_format=None,
                  b_format=None) -> torch.Tensor:
    """out = bf16(scale_a * scale_b * (a @ b^T) + bias) with a: M x K and b: N x K
    (float8 codes, K contiguous).  b may also be given as a K x N column-major
    view (stride (1, K)), which is the same memory.  Each operand is e4m3fn or
    e5m2: taken from its torch dtype, or from a_format / b_format for uint8
    codes (default e4m3fn).  `config` (-1: automatic) and `splits` (0:
    automatic; SPLITS_STREAM_K: stream-K) select the plan.  When the plan
    splits K, its workspace is
    `workspace` (a GPU byte tensor, zero-filled before first use) or, if that
    is None, one this module keeps per stream (allocated by torch)."""
    a, fa, b, fb, out, M, N, K, m, dev = _mm_args(a, b, scale_a, scale_b, bias, out, mode, workspace,
                                                  a_format, b_format)
    L = lib()
    stream = _stream_of(dev)
    ws_ptr, ws_bytes = _mm_workspace(L, a.device, dev, stream, M, N, K, m, bias is not None, config,
                                     splits, workspace)
    st = _call(dev, L.fp8_scaled_mm_typed, a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(),
               scale_b.data_ptr(), bias.data_ptr() if bias is not None else None, out.data_ptr(),
               M, N, K, m, stream, int(config), int(splits), ws_ptr, ws_bytes)
    if st != OK:
        _mm_error("fp8_scaled_mm", st)
    return out


def fp8_linear(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
               bias: torch.Tensor | None = None, residual: torch.Tensor | None = None, *,
               activation="none", preact: torch.Tensor | None = None,
               out: torch.Tensor | None = None, mode="rowwise", config: int = -1, splits: int = 0,
               workspace: torch.Tensor | None = None, a_format=None, b_format=None) -> torch.Tensor:
    """out = bf16(act(z) + residual) with z = scale_a * scale_b * (a @ b^T) + bias:
    fp8_scaled_mm with the rest of a linear layer in its epilogue, rounded once.

    `activation` is 'none', 'relu', 'gelu' (z Phi(z)), 'gelu_tanh' or 'silu'.
    `residual` (M x N bf16) may also be `out`.  `preact` (M x N bf16) receives
    bf16(z), which fp8_linear_backward takes.  Operands, formats, plans and
    workspaces are fp8_scaled_mm's (stream-K plans take no epilogue)."""
    act = _activation(activation)
    if (_calls is not None and out is None and config == -1 and splits == 0 and workspace is None
            and a_format is None and b_format is None and isinstance(mode, (str, int))):
        got = _calls.linear(a, b, scale_a, scale_b, bias, residual, act, preact, _MODES.get(mode, -1))
        if got.__class__ is tuple:
            return got[0]
        if got is not None:
            _mm_error("fp8_linear", got)
    a, fa, b, fb, out, M, N, K, m, dev = _mm_args(a, b, scale_a, scale_b, bias, out, mode, workspace,
                                                  a_format, b_format,
                                                  (("residual", residual), ("preact", preact)))
    for name, t in (("residual", residual), ("preact", preact)):
        if t is not None and (t.dtype != torch.bfloat16 or t.shape != (M, N) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bf16 M x N tensor")
    L = lib()
    stream = _stream_of(dev)
    ws_ptr, ws_bytes = _mm_workspace(L, a.device, dev, stream, M, N, K, m, bias is not None, config,
                                     splits, workspace)
    st = _call(dev, L.fp8_linear, a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(),
               scale_b.data_ptr(), _ptr(bias), _ptr(residual), act, _ptr(preact), out.data_ptr(), M, N,
               K, m, stream, int(config), int(splits), ws_ptr, ws_bytes)
    if st != OK:
        _mm_error("fp8_linear", st)
    return out


def fp8_linear_backward(dy: torch.Tensor, x: torch.Tensor | None, wt: torch.Tensor | None,
                        wt_scale: torch.Tensor | None, z: torch.Tensor | None = None, *,
                        activation="none", dx=True, dw=True, dbias: bool = True, wt_format=None,
                        workspace: torch.Tensor | None = None):
    """(dx, dw, dbias) of out = act(x W^T + bias) from dy, the gradient of act(z):

        dz = dy act'(z),  dx = dz W,  dw = dz^T x,  dbias = sum of dz over the rows

    with dz in e5m2 (a scale for each row in dx, for each column in dw), x in
    e4m3fn (a scale for each column) and W as float8 codes.

    dy and z (fp8_linear's preact; not needed for 'none') are M x N bf16, x is
    M x K bf16, wt the K x N codes of W transposed with K scales wt_scale.  dx
    (M x K) and dw (N x K) are bf16, dbias is fp32; True allocates one, False
    leaves it (and what only it needs) out, and dx and dw may be buffers.  What is
    left out is None in the result.  N and K are multiples of 16.  Codes, scales and partial sums
    live in `workspace` (a GPU byte tensor with any contents) or in memory that torch
    has back after the call (a graph captured without torch.cuda.graph needs one
    that stays)."""
    act = _activation(activation)
    if _calls is not None and dx is dw is dbias is True and workspace is None and wt_format is None:
        got = _calls.linear_backward(dy, x, wt, wt_scale, z, act)
        if got.__class__ is tuple:
            return got
        if got is not None:
            _mm_error("fp8_linear_backward", got)
    want_dx, want_dw = dx is not False, dw is not False
    out_dx, out_dw = want_dx and dx is not True, want_dw and dw is not True      # buffers given
    if (out_dx and not isinstance(dx, torch.Tensor)) or (out_dw and not isinstance(dw, torch.Tensor)):
        raise ValueError("dx and dw must be True, False or a tensor to write")
    if dbias is not True and dbias is not False:
        raise ValueError("dbias must be True or False")
    if not (want_dx or want_dw or dbias):
        raise ValueError("nothing to compute: dx, dw and dbias are all False")
    if not dy.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    if dy.dtype != torch.bfloat16 or dy.dim() != 2 or not dy.is_contiguous():
        raise ValueError("dy must be a contiguous bf16 M x N tensor")
    M, N = dy.shape
    if z is not None:
        _bf16_matrix("z", z, (M, N))
    elif act != 0:
        raise ValueError(f"activation {activation!r} needs z")
    K, fw = 16, E4M3FN      # (a problem without dx and dw has no K)
    if want_dw:
        if x is None:
            raise ValueError("dw needs x")
        if x.dim() != 2:
            raise ValueError("x must be a contiguous bf16 M x K tensor")
        K = x.shape[1]
        _bf16_matrix("x", x, (M, K))
    if want_dx:
        if wt is None or wt_scale is None:
            raise ValueError("dx needs wt and wt_scale")
        wt, fw = _as_codes(wt, "wt", wt_format)
        if wt.dim() != 2 or not wt.is_contiguous() or wt.shape[1] != N or (want_dw and wt.shape[0] != K):
            raise ValueError(f"wt must be contiguous K x N codes with N = {N}" +
                             (f" and K = {K}" if want_dw else "") + f", got {tuple(wt.shape)}")
        K = wt.shape[0]
        _ln_vector(wt_scale, "wt_scale", K)
    if N < 16 or N % 16 != 0 or K < 16 or K % 16 != 0:
        raise ValueError(f"N and K must be multiples of 16, got {N} and {K}")
    if out_dx:
        _bf16_matrix("dx", dx, (M, K))
    if out_dw:
        _bf16_matrix("dw", dw, (N, K))
    dev = dy.get_device()
    device = dy.device
    x = x if want_dw else None
    wt, wt_scale = (wt, wt_scale) if want_dx else (None, None)
    _check_devices(dev, (("z", z), ("x", x), ("wt", wt), ("wt_scale", wt_scale), ("workspace", workspace),
                         ("dx", dx if out_dx else None), ("dw", dw if out_dw else None)))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    if not out_dx:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=device) if want_dx else None
    if not out_dw:
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=device) if want_dw else None
    db = torch.empty(N, dtype=torch.float32, device=device) if dbias else None
    L = lib()
    stream = _stream_of(dev)
    if workspace is not None:
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    else:
        key = ("linear_grad", M, N, K, want_dx, want_dw)
        need = _ws_sizes.get(key)
        if need is None:
            need = int(L.fp8_linear_backward_workspace_size(M, N, K, want_dx, want_dw))
            if need < 0:
                raise ValueError(f"fp8_linear_backward: {status_string(ERR_SHAPE)}")
            _keep_size(key, need)
        ws, ws_bytes = torch.empty(need, dtype=torch.uint8, device=device), need
    st = _call(dev, L.fp8_linear_backward, dy.data_ptr(), _ptr(x), _ptr(wt), fw, _ptr(wt_scale), _ptr(z), act,
               _ptr(dx), _ptr(dw), _ptr(db), M, N, K, stream, ws.data_ptr(), ws_bytes)
    if st != OK:
        _mm_error("fp8_linear_backward", st)
    return dx, dw, db


def _bf16_matrix(name: str, t: torch.Tensor, shape: tuple) -> None:
    if t.dtype != torch.bfloat16 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 {shape[0]} x {shape[1]} tensor")


def _activation(activation) -> int:
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of 'none', 'relu', 'gelu', 'gelu_tanh' and 'silu', "
                         f"got {activation!r}")
    return _ACTIVATIONS[activation]


def _mm_error(fn: str, st: int) -> None:
    if st in _ARG_ERRORS:
        raise ValueError(f"{fn}: {status_string(st)} (status {st})")
    raise Fp8MMError(st)


def fp8_quantize(x: torch.Tensor, mode="rowwise", q: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, fmt="e4m3fn", workspace=True):
    """(q, scale) = dynamic float8 quantisation of a rows x cols bf16 GPU matrix:
    scale = amax/qmax (one value, or one per row), q = RNE(clamp(x/scale, +-qmax))
    as uint8 codes, with qmax = 448 (fmt 'e4m3fn') or 57344 ('e5m2').  `q` and
    `scale` may be passed to reuse buffers.  workspace=True gives the per-tensor
    mode a per-stream workspace (its one-pass path); False runs the two-pass
    path, which needs none."""
    if mode not in _MODES:
        raise ValueError(f"mode must be 'per_tensor' or 'rowwise', got {mode!r}")
    if fmt not in _FORMATS:
        raise ValueError(f"fmt must be 'e4m3fn' or 'e5m2', got {fmt!r}")
    f = _FORMATS[fmt]
    fn_name = "fp8_quantize_e4m3_ws" if f == E4M3FN else "fp8_quantize_e5m2_ws"
    m = _MODES[mode]
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous 2-D bf16 GPU tensor")
    rows, cols = x.shape
    n_scale = 1 if m == PER_TENSOR else rows
    dev = x.get_device()
    _check_devices(dev, (("q", q), ("scale", scale)))
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    elif q.dtype not in (torch.uint8, torch.float8_e4m3fn if f == E4M3FN else torch.float8_e5m2) \
            or tuple(q.shape) != (rows, cols) or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous uint8 (or float8_{fmt}) rows x cols tensor")
    if scale is None:
        scale = torch.empty(n_scale, dtype=torch.float32, device=x.device)
    elif scale.dtype != torch.float32 or scale.numel() != n_scale or not scale.is_contiguous():
        raise ValueError(f"scale must be a contiguous float32 tensor of {n_scale} elements")
    stream = _stream_of(dev)
    with torch.cuda.device(dev) if torch.cuda.current_device() != dev else contextlib.nullcontext():
        need = int(lib().fp8_quantize_workspace_size(rows, cols, m)) if workspace else 0
        ws = _workspace(x.device, stream, need, "quantize") if need > 0 else None
        st = getattr(lib(), fn_name)(x.data_ptr() if x.numel() else None,
                                     q.data_ptr() if q.numel() else None, scale.data_ptr(),
                                     rows, cols, m, ws.data_ptr() if ws is not None else None,
                                     need, stream)
    if st != Q_OK:
        msg = f"{fn_name}: {lib().fp8_quantize_status_string(st).decode()} (status {st})"
        if st in _Q_ARG_ERRORS:
            raise ValueError(msg)
        raise RuntimeError(msg)
    return q, scale


# element types of the layer norm (enum fp8ln_dtype)
_LN_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

LayerNormResult = collections.namedtuple("LayerNormResult", "y q scale mean rstd")
_result = tuple.__new__


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ln_matrix(t, name: str, like: torch.Tensor | None = None) -> None:
    if like is None:
        if t.dtype not in _LN_DTYPES or t.dim() != 2 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous 2-D bf16 or fp32 GPU tensor")
    elif t.dtype != like.dtype or t.shape != like.shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} tensor of shape {tuple(like.shape)}")


def _ln_param(t, name: str, cols: int, dev: int) -> int:
    """The library's code for the type of w or b (None: -1)."""
    if t is None:
        return -1
    code = _LN_DTYPES.get(t.dtype)
    if code is None or t.numel() != cols or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 or bf16 vector of {cols} elements")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return code


def _ln_vector(t, name: str, n: int) -> None:
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")


def _ln_error(fn: str, st: int) -> None:
    msg = f"{fn}: {lib().fp8_layer_norm_status_string(st).decode()} (status {st})"
    raise ValueError(msg) if st in _LN_ARG_ERRORS else RuntimeError(msg)


def fp8_layer_norm(x: torch.Tensor, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
                   eps: float = 1e-5, *, y=True, fmt=None, stats: bool = False,
                   q: torch.Tensor | None = None,
                   scale: torch.Tensor | None = None) -> LayerNormResult:
    """Layer norm over the last axis of a rows x cols bf16 or fp32 matrix, with
    the row-wise float8 quantisation of its result:

        y = (x - mean) * rstd * w + b,   rstd = 1 / sqrt(var + eps)
        scale = max|y| / qmax for each row,   q = RNE(y / scale)

    w and b (fp32 or bf16; None: ones, zeros) have cols elements.  `y` is True
    (allocate), False (not wanted) or a tensor to write; fmt 'e4m3fn' or 'e5m2'
    asks for the codes (uint8) and their scales, in `q` and `scale` if given
    (then cols must be a multiple of 16); stats=True returns mean and rstd,
    which fp8_layer_norm_backward takes.  The codes come from the fp32 y.  A row
    that holds a NaN or an infinity gives NaN in all of its outputs."""
    if _calls is not None and q is None and scale is None:
        got = _calls.layer_norm(x, w, b, eps, y, -1 if fmt is None else _FORMATS.get(fmt, -2), stats)
        if got.__class__ is tuple:
            return _result(LayerNormResult, got)
        if got is not None:
            _ln_error("fp8_layer_norm", got)
    _ln_matrix(x, "x")
    rows, cols = x.shape
    given = isinstance(y, torch.Tensor)
    if cols == 0:
        raise ValueError("x needs at least one column")
    if fmt is None:
        if q is not None or scale is not None:
            raise ValueError("q and scale need fmt")
        if y is False:
            raise ValueError("nothing to compute: y=False and fmt=None")
    elif fmt not in _FORMATS:
        raise ValueError(f"fmt must be 'e4m3fn', 'e5m2' or None, got {fmt!r}")
    elif cols % 16 != 0:
        raise ValueError(f"codes need a number of columns that is a multiple of 16, got {cols}")
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    dev = x.get_device()
    pw, pb = _ln_param(w, "w", cols, dev), _ln_param(b, "b", cols, dev)
    if pw != pb and pw >= 0 and pb >= 0:
        raise ValueError("w and b must have one type")
    pdt = pw if pw >= 0 else pb if pb >= 0 else 1
    if given:
        _ln_matrix(y, "y", x)
    elif y is not True and y is not False:
        raise ValueError("y must be True, False or a tensor to write")
    if given or q is not None or scale is not None:
        _check_devices(dev, (("q", q), ("scale", scale), ("y", y if given else None)))
    device = x.device
    out = y if given else torch.empty_like(x) if y else None
    f = 0
    if fmt is not None:
        f = _FORMATS[fmt]
        if q is None:
            q = torch.empty((rows, cols), dtype=torch.uint8, device=device)
        elif q.dtype not in (torch.uint8, torch.float8_e4m3fn if f == E4M3FN else torch.float8_e5m2) \
                or tuple(q.shape) != (rows, cols) or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous uint8 (or float8_{fmt}) rows x cols tensor")
        if scale is None:
            scale = torch.empty(rows, dtype=torch.float32, device=device)
        else:
            _ln_vector(scale, "scale", rows)
    mean = rstd = None
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=device)
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
    st = _call(dev, lib().fp8_layer_norm, x.data_ptr(), _LN_DTYPES[x.dtype], _ptr(w), _ptr(b), pdt, eps,
               _ptr(out), _ptr(q), f, _ptr(scale), _ptr(mean), _ptr(rstd), rows, cols, _stream_of(dev))
    if st != LN_OK:
        _ln_error("fp8_layer_norm", st)
    return LayerNormResult(out, q, scale, mean, rstd)


def fp8_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                            rstd: torch.Tensor, w: torch.Tensor | None = None, *,
                            residual_grad: torch.Tensor | None = None,
                            dx: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None):
    """(dx, dw, db) of the layer norm above, from the gradient dy of y, its
    input x and the forward call's mean and rstd.  residual_grad is added to dx
    (in fp32) where x also went along a residual path.  dx has x's type (`dx`
    may be passed to reuse a buffer), dw and db are fp32.  The partial column
    sums go to `workspace` (a GPU byte tensor) or to one that this module keeps
    per stream.  The sums' order is fixed: equal calls give equal bits."""
    if _calls is not None and dx is None and workspace is None:
        got = _calls.layer_norm_backward(dy, x, mean, rstd, w, residual_grad)
        if got.__class__ is tuple:
            return got
        if got is not None:
            _ln_error("fp8_layer_norm_backward", got)
    _ln_matrix(x, "x")
    _ln_matrix(dy, "dy", x)
    rows, cols = x.shape
    if cols == 0:
        raise ValueError("x needs at least one column")
    _ln_vector(mean, "mean", rows)
    _ln_vector(rstd, "rstd", rows)
    dev = x.get_device()
    pdt = _ln_param(w, "w", cols, dev)
    if pdt < 0:
        pdt = 1
    for name, t in (("residual_grad", residual_grad), ("dx", dx)):
        if t is not None:
            _ln_matrix(t, name, x)
    _check_devices(dev, (("dy", dy), ("mean", mean), ("rstd", rstd), ("dx", dx),
                         ("residual_grad", residual_grad), ("workspace", workspace)))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    if dx is None:
        dx = torch.empty_like(x)
    dw = torch.empty(cols, dtype=torch.float32, device=x.device)
    db = torch.empty(cols, dtype=torch.float32, device=x.device)
    L = lib()
    stream = _stream_of(dev)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        key = ("layer_norm", rows, cols)
        need = _ws_sizes.get(key)
        if need is None:
            need = int(L.fp8_layer_norm_backward_workspace_size(rows, cols))
            _keep_size(key, need)
        ws, ws_bytes = None, 0
        if need > 0:
            ws, ws_bytes = _workspace(x.device, stream, need, "layer_norm").data_ptr(), need
    st = _call(dev, L.fp8_layer_norm_backward, dy.data_ptr(), x.data_ptr(), _LN_DTYPES[x.dtype],
               mean.data_ptr(), rstd.data_ptr(), _ptr(w), pdt, _ptr(residual_grad), dx.data_ptr(),
               dw.data_ptr(), db.data_ptr(), rows, cols, ws, ws_bytes, stream)
    if st != LN_OK:
        _ln_error("fp8_layer_norm_backward", st)
    return dx, dw, db
