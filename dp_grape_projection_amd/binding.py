"""ctypes binding of libdpg.so (include/dpg.h): argument marshalling only.

Every step of the DP-GRAPE update runs in the library's HIP kernels; this
module turns torch tensors into device pointers and the current HIP stream,
and allocates outputs and workspaces with torch when the caller does not pass
them. It never computes any part of the method itself, and it raises when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
import os
from typing import List, Optional, Sequence

import torch  # loaded first: libdpg.so then shares torch's HIP runtime

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdpg.so")

DPG_OK = 0
DPG_ERR_INVALID_ARG = 1
DPG_ERR_WORKSPACE = 2
DPG_ERR_UNSUPPORTED = 3
DPG_ERR_HIP = 4
DPG_FP32 = 0
DPG_BF16 = 1

EXPORTED = (
    "dpg_project_workspace_size", "dpg_project_clip_noise",
    "dpg_adam_workspace_size", "dpg_adam_backproject", "dpg_philox_normals",
    "dpg_project_layer_workspace_size", "dpg_project_layer",
    "dpg_clip_workspace_size", "dpg_clip_sum_noise",
    "dpg_step_workspace_size", "dpg_private_step", "dpg_private_step_static",
    "dpg_static_scratch_bytes", "dpg_rc_norms_workspace_size", "dpg_rc_norms",
    "dpg_embed", "dpg_embed_workspace_size", "dpg_embed_norms", "dpg_embed_grad",
    "dpg_vocab_loss_workspace_size", "dpg_vocab_loss", "dpg_vocab_loss_grad",
    "dpg_distill_loss_workspace_size", "dpg_distill_loss", "dpg_distill_loss_grad",
    "dpg_status_string", "dpg_last_error", "dpg_version",
    "dpg_timing_enable", "dpg_timing_read", "dpg_kernel_name",
)
N_KERNEL_KINDS = 10


class DpgError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class LayerGrad(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("layer_id", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("A", ctypes.c_void_p), ("dY", ctypes.c_void_p),
                ("G_priv", ctypes.c_void_p)]


class LayerHat(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int64), ("layer_id", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("G_hat", ctypes.c_void_p),
                ("G_priv", ctypes.c_void_p)]


class LayerParam(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("layer_id", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("G_priv", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libdpg.so (once). Raises FileNotFoundError when it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(
            f"{p} is missing: build it with `python -m dp_grape_projection_amd.build`")
    lib = ctypes.CDLL(p)
    i32, i64, u32, u64 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                          ctypes.c_uint64)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.dpg_project_workspace_size.argtypes = [
        ctypes.POINTER(LayerGrad), i32, i64, i64, i32, i32, ctypes.POINTER(sz)]
    f64 = ctypes.c_double
    lib.dpg_project_clip_noise.argtypes = [
        ctypes.POINTER(LayerGrad), i32, i64, i64, i32, i32, f64, f64, u64,
        u64, u64, vp, vp, sz, vp]
    lib.dpg_rc_norms_workspace_size.argtypes = [
        ctypes.POINTER(LayerGrad), i32, i64, i64, i32, i32, ctypes.POINTER(sz)]
    lib.dpg_rc_norms.argtypes = [
        ctypes.POINTER(LayerGrad), i32, i64, i64, i32, i32, f64, u64, u64, vp, vp,
        vp, sz, vp]
    lib.dpg_adam_workspace_size.argtypes = [
        ctypes.POINTER(LayerParam), i32, i32, i32, ctypes.POINTER(sz)]
    lib.dpg_adam_backproject.argtypes = [
        ctypes.POINTER(LayerParam), i32, i32, i32, f64, f64, f64, f64, u64,
        u64, u64, vp, sz, vp]
    lib.dpg_philox_normals.argtypes = [u64, u32, u32, u32, u64, u64, vp, vp, vp]
    lib.dpg_project_layer_workspace_size.argtypes = [
        ctypes.POINTER(LayerGrad), i64, i64, i32, i32, ctypes.POINTER(sz)]
    lib.dpg_project_layer.argtypes = [
        ctypes.POINTER(LayerGrad), i64, i64, i32, i32, u64, u64, vp, vp, vp, sz, vp]
    lib.dpg_clip_workspace_size.argtypes = [i64, ctypes.POINTER(sz)]
    lib.dpg_step_workspace_size.argtypes = [
        ctypes.POINTER(LayerGrad), i32, i64, i64, i32, i32, ctypes.POINTER(sz)]
    lib.dpg_private_step.argtypes = [
        ctypes.POINTER(LayerGrad), ctypes.POINTER(LayerParam), i32, i64, i64, i32,
        i32, f64, f64, f64, f64, f64, f64, u64, u64, u64, vp, vp, sz, vp]
    lib.dpg_private_step_static.argtypes = [
        ctypes.POINTER(LayerGrad), ctypes.POINTER(LayerParam), i32, i64, i64, i32,
        i32, f64, f64, f64, f64, f64, f64, u64, u64, u64, vp, vp]
    lib.dpg_static_scratch_bytes.argtypes = []
    lib.dpg_clip_sum_noise.argtypes = [
        ctypes.POINTER(LayerHat), i32, i64, i32, f64, f64, u64, u64, vp, vp, vp,
        sz, vp]
    psz = ctypes.POINTER(sz)
    lib.dpg_embed.argtypes = [vp, i64, vp, i64, i64, i32, f64, i32, vp, vp]
    lib.dpg_embed_workspace_size.argtypes = [i64, i64, i64, i64, psz]
    lib.dpg_embed_norms.argtypes = [vp, vp, i64, i64, i64, i64, i32, f64, vp, vp, sz, vp]
    lib.dpg_embed_grad.argtypes = [vp, vp, i64, i64, i64, i64, i32, f64, vp, i32, i32, vp,
                                   vp, sz, vp]
    lib.dpg_vocab_loss_workspace_size.argtypes = [i64, i64, i64, i32, i32, psz]
    lib.dpg_vocab_loss.argtypes = [vp, vp, vp, i64, i64, i64, i32, f64, vp, vp, vp, sz, vp]
    lib.dpg_vocab_loss_grad.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, f64, vp, vp,
                                        vp, sz, vp]
    lib.dpg_distill_loss_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32, psz]
    lib.dpg_distill_loss.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, f64, f64, vp,
                                     vp, vp, sz, vp]
    lib.dpg_distill_loss_grad.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32,
                                          f64, f64, vp, vp, vp, sz, vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.dpg_static_scratch_bytes.restype = ctypes.c_size_t
    lib.dpg_status_string.restype = ctypes.c_char_p
    lib.dpg_status_string.argtypes = [ctypes.c_int]
    lib.dpg_last_error.restype = ctypes.c_char_p
    lib.dpg_last_error.argtypes = []
    lib.dpg_timing_enable.argtypes = [ctypes.c_int]
    lib.dpg_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_int64), i32,
                                    ctypes.c_int]
    lib.dpg_kernel_name.restype = ctypes.c_char_p
    lib.dpg_kernel_name.argtypes = [ctypes.c_int]
    if path is None:
        _lib = lib
    return lib


def _check(lib, status: int):
    if status != DPG_OK:
        msg = lib.dpg_last_error().decode() or lib.dpg_status_string(status).decode()
        raise DpgError(status, msg)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return DPG_BF16
    if t == torch.float32:
        return DPG_FP32
    raise TypeError(f"A/dY must be bfloat16 or float32, got {t}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _require(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# The current stream's handle without building a torch.cuda.Stream (3 us of
# host time a call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _on_stream(fn):
    """Runs `fn` with its `stream` argument (when given) as torch's current
    stream, so that the outputs and temporary workspaces it allocates belong
    to the stream the library's kernels are enqueued on: the caching
    allocator then does not hand their memory to other work while those
    kernels may still use it."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def wrapper(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return wrapper


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]):
    if workspace is not None:
        _require(workspace, "workspace", torch.uint8)
        return workspace, workspace.numel()
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device), nbytes


def project_workspace_size(shapes: Sequence, B: int, T: int, r: int,
                           dtype: torch.dtype,
                           layer_ids: Optional[Sequence[int]] = None) -> int:
    """Workspace bytes dpg_project_clip_noise needs; shapes = [(d_in, d_out)]."""
    lib = load_library()
    n = len(shapes)
    ids = list(range(n)) if layer_ids is None else list(layer_ids)
    arr = (LayerGrad * n)()
    for i, ((di, do), lid) in enumerate(zip(shapes, ids)):
        arr[i].d_in, arr[i].d_out, arr[i].layer_id = int(di), int(do), int(lid)
    out = ctypes.c_size_t(0)
    _check(lib, lib.dpg_project_workspace_size(arr, n, int(B), int(T), int(r),
                                               _dtype_code(dtype),
                                               ctypes.byref(out)))
    return out.value


def adam_workspace_size(shapes: Sequence, r: int, dtype: torch.dtype,
                        layer_ids: Optional[Sequence[int]] = None) -> int:
    lib = load_library()
    n = len(shapes)
    ids = list(range(n)) if layer_ids is None else list(layer_ids)
    arr = (LayerParam * n)()
    for i, ((di, do), lid) in enumerate(zip(shapes, ids)):
        arr[i].d_in, arr[i].d_out, arr[i].layer_id = int(di), int(do), int(lid)
    out = ctypes.c_size_t(0)
    _check(lib, lib.dpg_adam_workspace_size(arr, n, int(r), _dtype_code(dtype),
                                            ctypes.byref(out)))
    return out.value


@_on_stream
def dpg_project_clip_noise(A: Sequence[torch.Tensor], dY: Sequence[torch.Tensor],
                           r: int, clip_C: float, sigma: float, seed: int,
                           step: int, proj_step: Optional[int] = None,
                           layer_ids: Optional[Sequence[int]] = None,
                           G_priv: Optional[List[torch.Tensor]] = None,
                           sample_norms: Optional[torch.Tensor] = None,
                           return_norms: bool = True,
                           workspace: Optional[torch.Tensor] = None,
                           stream=None):
    """Projection, global per-sample clip, batch sum and noise (libdpg).

    A[l]: [B, T, d_in_l], dY[l]: [B, T, d_out_l] (bf16 or fp32, on the GPU).
    Returns (G_priv list of [r, d_out_l] fp32, sample norms [B] or None)."""
    lib = load_library()
    n = len(A)
    if n < 1 or len(dY) != n:
        raise ValueError("A and dY must be non-empty lists of equal length")
    dt = A[0].dtype
    B, T = int(A[0].shape[0]), int(A[0].shape[1])
    ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
    proj_step = step if proj_step is None else proj_step
    dev = A[0].device
    if G_priv is None:
        G_priv = [torch.empty((r, int(d.shape[2])), dtype=torch.float32,
                              device=dev) for d in dY]
    if sample_norms is None and return_norms:
        sample_norms = torch.empty(B, dtype=torch.float32, device=dev)
    arr = (LayerGrad * n)()
    for i in range(n):
        _require(A[i], f"A[{i}]", dt)
        _require(dY[i], f"dY[{i}]", dt)
        if A[i].dim() != 3 or dY[i].dim() != 3 or \
                tuple(A[i].shape[:2]) != (B, T) or tuple(dY[i].shape[:2]) != (B, T):
            raise ValueError(f"layer {i}: A and dY must be [B, T, d] with common B, T")
        d_in, d_out = int(A[i].shape[2]), int(dY[i].shape[2])
        _require(G_priv[i], f"G_priv[{i}]", torch.float32, (r, d_out))
        arr[i].d_in, arr[i].d_out, arr[i].layer_id = d_in, d_out, ids[i]
        arr[i].A, arr[i].dY, arr[i].G_priv = _ptr(A[i]), _ptr(dY[i]), _ptr(G_priv[i])
    if sample_norms is not None:
        _require(sample_norms, "sample_norms", torch.float32, (B,))
    need = ctypes.c_size_t(0)
    _check(lib, lib.dpg_project_workspace_size(arr, n, B, T, int(r),
                                               _dtype_code(dt), ctypes.byref(need)))
    ws, ws_bytes = _workspace(need.value, dev, workspace)
    _check(lib, lib.dpg_project_clip_noise(
        arr, n, B, T, int(r), _dtype_code(dt), float(clip_C), float(sigma),
        int(seed), int(step), int(proj_step), _ptr(sample_norms),
        ws.data_ptr(), ws_bytes, _stream_handle(stream)))
    return G_priv, sample_norms


@_on_stream
def dpg_adam_backproject(G_priv: Sequence[torch.Tensor], W: Sequence[torch.Tensor],
                         m: Sequence[torch.Tensor], v: Sequence[torch.Tensor],
                         r: int, lr: float, beta1: float, beta2: float,
                         eps: float, seed: int, step: int,
                         proj_step: Optional[int] = None,
                         layer_ids: Optional[Sequence[int]] = None,
                         dtype: torch.dtype = torch.bfloat16,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Projected Adam and back-projection W -= lr P^T U, in place (libdpg).

    dtype is the operand precision of P^T U (bf16 or fp32)."""
    lib = load_library()
    n = len(W)
    ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
    proj_step = step if proj_step is None else proj_step
    arr = (LayerParam * n)()
    for i in range(n):
        _require(W[i], f"W[{i}]", torch.float32)
        if W[i].dim() != 2:
            raise ValueError(f"W[{i}] must be [d_in, d_out]")
        d_in, d_out = int(W[i].shape[0]), int(W[i].shape[1])
        for name, t in (("G_priv", G_priv[i]), ("m", m[i]), ("v", v[i])):
            _require(t, f"{name}[{i}]", torch.float32, (r, d_out))
        arr[i].d_in, arr[i].d_out, arr[i].layer_id = d_in, d_out, ids[i]
        arr[i].G_priv, arr[i].W = _ptr(G_priv[i]), _ptr(W[i])
        arr[i].m, arr[i].v = _ptr(m[i]), _ptr(v[i])
    code = _dtype_code(dtype)
    need = ctypes.c_size_t(0)
    _check(lib, lib.dpg_adam_workspace_size(arr, n, int(r), code, ctypes.byref(need)))
    ws, ws_bytes = _workspace(need.value, W[0].device, workspace)
    _check(lib, lib.dpg_adam_backproject(
        arr, n, int(r), code, float(lr), float(beta1), float(beta2), float(eps),
        int(seed), int(step), int(proj_step), ws.data_ptr(), ws_bytes,
        _stream_handle(stream)))
    return W, m, v


@_on_stream
def dpg_private_step(A: Sequence[torch.Tensor], dY: Sequence[torch.Tensor],
                     W: Sequence[torch.Tensor], m: Sequence[torch.Tensor],
                     v: Sequence[torch.Tensor], r: int, clip_C: float, sigma: float,
                     lr: float, beta1: float, beta2: float, eps: float, seed: int,
                     step: int, proj_step: Optional[int] = None,
                     layer_ids: Optional[Sequence[int]] = None, stream=None):
    """The whole step in one call (libdpg): W, m, v updated in place.
    Returns (G_priv list of [r, d_out] fp32, sample norms [B])."""
    ps = PreparedStep(A, dY, W, m, v, r, clip_C, sigma, seed, lr, beta1, beta2,
                      eps, layer_ids=layer_ids)
    proj_step = step if proj_step is None else proj_step
    _check(ps.lib, ps.lib.dpg_private_step(
        ps.grads, ps.params, ps.n, ps.B, ps.T, ps.r, ps.dtype_code, float(clip_C),
        float(sigma), float(lr), float(beta1), float(beta2), float(eps), int(seed),
        int(step), int(proj_step), ps.sample_norms.data_ptr(), ps.ws3.data_ptr(),
        ps.ws3_bytes, _stream_handle(stream)))
    return ps.G_priv, ps.sample_norms


@_on_stream
def dpg_rc_norms(A: Sequence[torch.Tensor], dY: Sequence[torch.Tensor], k: int,
                 clip_C: float, seed: int, step: int,
                 layer_ids: Optional[Sequence[int]] = None,
                 norms: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Randomized clipping's per-sample norm estimate (libdpg): Hutchinson's
    estimator with k Gaussian probes per layer on the d_out side.
    A[l]: [B, T, d_in_l], dY[l]: [B, T, d_out_l] (bf16 or fp32, on the GPU).
    Returns (estimated norms [B], clip factors min(1, C / nhat) [B])."""
    lib = load_library()
    n = len(A)
    if n < 1 or len(dY) != n:
        raise ValueError("A and dY must be non-empty lists of equal length")
    dt = A[0].dtype
    B, T = int(A[0].shape[0]), int(A[0].shape[1])
    ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
    dev = A[0].device
    norms = torch.empty(B, dtype=torch.float32, device=dev) if norms is None else norms
    scales = torch.empty(B, dtype=torch.float32, device=dev) if scales is None else scales
    _require(norms, "norms", torch.float32, (B,))
    _require(scales, "scales", torch.float32, (B,))
    arr = (LayerGrad * n)()
    for i in range(n):
        _require(A[i], f"A[{i}]", dt)
        _require(dY[i], f"dY[{i}]", dt)
        if A[i].dim() != 3 or dY[i].dim() != 3 or \
                tuple(A[i].shape[:2]) != (B, T) or tuple(dY[i].shape[:2]) != (B, T):
            raise ValueError(f"layer {i}: A and dY must be [B, T, d] with common B, T")
        arr[i].d_in, arr[i].d_out, arr[i].layer_id = int(A[i].shape[2]), int(dY[i].shape[2]), ids[i]
        arr[i].A, arr[i].dY, arr[i].G_priv = _ptr(A[i]), _ptr(dY[i]), None
    need = ctypes.c_size_t(0)
    _check(lib, lib.dpg_rc_norms_workspace_size(arr, n, B, T, int(k), _dtype_code(dt),
                                                ctypes.byref(need)))
    ws, ws_bytes = _workspace(need.value, dev, workspace)
    _check(lib, lib.dpg_rc_norms(arr, n, B, T, int(k), _dtype_code(dt), float(clip_C),
                                 int(seed), int(step), norms.data_ptr(), scales.data_ptr(),
                                 ws.data_ptr(), ws_bytes, _stream_handle(stream)))
    return norms, scales


def static_scratch_bytes() -> int:
    """Bytes of the library's static scratch (per GPU)."""
    return int(load_library().dpg_static_scratch_bytes())


@_on_stream
def dpg_private_step_static(A: Sequence[torch.Tensor], dY: Sequence[torch.Tensor],
                            W: Sequence[torch.Tensor], m: Sequence[torch.Tensor],
                            v: Sequence[torch.Tensor], G_priv: Sequence[torch.Tensor],
                            sample_norms: torch.Tensor, r: int, clip_C: float,
                            sigma: float, lr: float, beta1: float, beta2: float,
                            eps: float, seed: int, step: int,
                            proj_step: Optional[int] = None,
                            layer_ids: Optional[Sequence[int]] = None, stream=None):
    """The one-call step in the library's static scratch (libdpg
    dpg_private_step_static): nothing is allocated, here or in the library;
    the caller passes every output (G_priv [r, d_out] fp32 per layer,
    sample_norms [B] fp32). W, m, v are updated in place."""
    lib = load_library()
    grads, params, n, B, T, code = _step_tables(A, dY, W, m, v, G_priv, r, layer_ids)
    _require(sample_norms, "sample_norms", torch.float32, (B,))
    proj_step = step if proj_step is None else proj_step
    _check(lib, lib.dpg_private_step_static(
        grads, params, n, B, T, int(r), code, float(clip_C), float(sigma), float(lr),
        float(beta1), float(beta2), float(eps), int(seed), int(step), int(proj_step),
        sample_norms.data_ptr(), _stream_handle(stream)))
    return G_priv, sample_norms


def _step_tables(A, dY, W, m, v, G_priv, r, layer_ids):
    """Checked layer tables (dpg_layer_grad, dpg_layer_param) of one step."""
    n = len(A)
    if n < 1 or not (len(dY) == len(W) == len(m) == len(v) == len(G_priv) == n):
        raise ValueError("A, dY, W, m, v and G_priv must be lists of equal length >= 1")
    dt = A[0].dtype
    B, T = int(A[0].shape[0]), int(A[0].shape[1])
    ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
    grads, params = (LayerGrad * n)(), (LayerParam * n)()
    for i in range(n):
        _require(A[i], f"A[{i}]", dt)
        _require(dY[i], f"dY[{i}]", dt)
        if A[i].dim() != 3 or dY[i].dim() != 3 or \
                tuple(A[i].shape[:2]) != (B, T) or tuple(dY[i].shape[:2]) != (B, T):
            raise ValueError(f"layer {i}: A and dY must be [B, T, d] with common B, T")
        d_in, d_out = int(A[i].shape[2]), int(dY[i].shape[2])
        _require(W[i], f"W[{i}]", torch.float32, (d_in, d_out))
        for name, t in (("G_priv", G_priv[i]), ("m", m[i]), ("v", v[i])):
            _require(t, f"{name}[{i}]", torch.float32, (r, d_out))
        g, p = grads[i], params[i]
        g.d_in = p.d_in = d_in
        g.d_out = p.d_out = d_out
        g.layer_id = p.layer_id = ids[i]
        g.A, g.dY, g.G_priv = A[i].data_ptr(), dY[i].data_ptr(), G_priv[i].data_ptr()
        p.G_priv, p.W = G_priv[i].data_ptr(), W[i].data_ptr()
        p.m, p.v = m[i].data_ptr(), v[i].data_ptr()
    return grads, params, n, B, T, _dtype_code(dt)


@_on_stream
def dpg_project_layer(A: torch.Tensor, dY: torch.Tensor, r: int, seed: int,
                      proj_step: int, layer_id: int, norm_sq: torch.Tensor,
                      G_hat: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Streaming form, one layer (libdpg): G_hat[i] = P A_i^T dY_i
    ([B, r, d_out] fp32) and norm_sq[i] += ||G_hat[i]||^2. Returns G_hat."""
    lib = load_library()
    dt = A.dtype
    _require(A, "A", dt)
    _require(dY, "dY", dt)
    if A.dim() != 3 or dY.dim() != 3 or tuple(A.shape[:2]) != tuple(dY.shape[:2]):
        raise ValueError("A and dY must be [B, T, d] with common B, T")
    B, T = int(A.shape[0]), int(A.shape[1])
    d_in, d_out = int(A.shape[2]), int(dY.shape[2])
    if G_hat is None:
        G_hat = torch.empty((B, r, d_out), dtype=torch.float32, device=A.device)
    _require(G_hat, "G_hat", torch.float32, (B, r, d_out))
    _require(norm_sq, "norm_sq", torch.float32, (B,))
    arr = (LayerGrad * 1)()
    arr[0].d_in, arr[0].d_out, arr[0].layer_id = d_in, d_out, int(layer_id)
    arr[0].A, arr[0].dY = _ptr(A), _ptr(dY)
    need = ctypes.c_size_t(0)
    _check(lib, lib.dpg_project_layer_workspace_size(arr, B, T, int(r), _dtype_code(dt),
                                                     ctypes.byref(need)))
    ws, ws_bytes = _workspace(need.value, A.device, workspace)
    _check(lib, lib.dpg_project_layer(arr, B, T, int(r), _dtype_code(dt), int(seed),
                                      int(proj_step), _ptr(G_hat), _ptr(norm_sq),
                                      ws.data_ptr(), ws_bytes, _stream_handle(stream)))
    return G_hat


@_on_stream
def dpg_clip_sum_noise(G_hat: Sequence[torch.Tensor], r: int, clip_C: float,
                       sigma: float, seed: int, step: int, norm_sq: torch.Tensor,
                       layer_ids: Optional[Sequence[int]] = None,
                       G_priv: Optional[List[torch.Tensor]] = None,
                       sample_norms: Optional[torch.Tensor] = None,
                       return_norms: bool = True,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Streaming form, after the last layer (libdpg): G_priv_l =
    (sum_i s_i G_hat_l[i] + sigma C Z_l) / B with s_i from norm_sq.
    Returns (G_priv list of [r, d_out] fp32, sample norms [B] or None)."""
    lib = load_library()
    n = len(G_hat)
    if n < 1:
        raise ValueError("G_hat must be a non-empty list")
    B = int(G_hat[0].shape[0])
    dev = G_hat[0].device
    ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
    if G_priv is None:
        G_priv = [torch.empty((r, int(g.shape[2])), dtype=torch.float32, device=dev)
                  for g in G_hat]
    if sample_norms is None and return_norms:
        sample_norms = torch.empty(B, dtype=torch.float32, device=dev)
    _require(norm_sq, "norm_sq", torch.float32, (B,))
    arr = (LayerHat * n)()
    for i in range(n):
        d_out = int(G_hat[i].shape[2])
        _require(G_hat[i], f"G_hat[{i}]", torch.float32, (B, r, d_out))
        _require(G_priv[i], f"G_priv[{i}]", torch.float32, (r, d_out))
        arr[i].d_out, arr[i].layer_id = d_out, ids[i]
        arr[i].G_hat, arr[i].G_priv = _ptr(G_hat[i]), _ptr(G_priv[i])
    if sample_norms is not None:
        _require(sample_norms, "sample_norms", torch.float32, (B,))
    need = ctypes.c_size_t(0)
    _check(lib, lib.dpg_clip_workspace_size(B, ctypes.byref(need)))
    ws, ws_bytes = _workspace(need.value, dev, workspace)
    _check(lib, lib.dpg_clip_sum_noise(arr, n, B, int(r), float(clip_C), float(sigma),
                                       int(seed), int(step), _ptr(norm_sq),
                                       _ptr(sample_norms), ws.data_ptr(), ws_bytes,
                                       _stream_handle(stream)))
    return G_priv, sample_norms


@_on_stream
def dpg_philox_normals(seed: int, layer_id: int, step_word: int, tag: int,
                       start: int, n: int, device="cuda", words: bool = False,
                       stream=None):
    """The library's random stream z(e), e in [start, start+n) (and raw words)."""
    lib = load_library()
    z = torch.empty(n, dtype=torch.float32, device=device)
    w = None
    if words and n > 0:
        n_ctr = ((start + n - 1) >> 2) - (start >> 2) + 1
        w = torch.empty(4 * n_ctr, dtype=torch.int32, device=device)
    _check(lib, lib.dpg_philox_normals(int(seed), int(layer_id), int(step_word),
                                       int(tag), int(start), int(n), _ptr(z),
                                       _ptr(w), _stream_handle(stream)))
    return (z, w) if words else z


def _ids(t, name: str, shape=None):
    _require(t, name, torch.int64, shape)
    return t


def _same_device(ref: torch.Tensor, **tensors):
    at = ref.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} must be on {ref.device}, got {t.device}")


@_on_stream
def dpg_embed(ids: torch.Tensor, E: torch.Tensor, scale: float = 1.0,
              dtype: Optional[torch.dtype] = None, Y: Optional[torch.Tensor] = None,
              stream=None):
    """Token lookup with scaling (libdpg): Y = scale * E[ids], zero where an
    id lies outside [0, V).

    ids: int64 of any shape; E: [V, d] fp32 or bf16; dtype (default E's) is
    Y's: an fp32 table is looked up in fp32 or bf16, a bf16 table in bf16.
    Returns Y of shape ids.shape + (d,)."""
    lib = load_library()
    _require(E, "E")
    if E.dim() != 2:
        raise ValueError("E must be [V, d]")
    V, d = int(E.shape[0]), int(E.shape[1])
    _ids(ids, "ids")
    dtype = E.dtype if dtype is None else dtype
    table = _dtype_code(E.dtype)
    code = _dtype_code(dtype)
    if Y is None:
        Y = torch.empty((*ids.shape, d), dtype=dtype, device=E.device)
    _require(Y, "Y", dtype, (*ids.shape, d))
    _same_device(E, ids=ids, Y=Y)
    if ids.numel() == 0:
        return Y
    _check(lib, lib.dpg_embed(_ptr(ids), ids.numel(), _ptr(E), V, d, table, float(scale),
                              code, _ptr(Y), _stream_handle(stream)))
    return Y


def _embed_args(ids, dY, V):
    """Checked (B, T, d) of a [B, T] batch of ids and its [B, T, d] gradient."""
    _ids(ids, "ids")
    _require(dY, "dY")
    if ids.dim() != 2 or dY.dim() != 3 or tuple(dY.shape[:2]) != tuple(ids.shape):
        raise ValueError("ids must be [B, T] and dY [B, T, d]")
    _same_device(dY, ids=ids)
    return int(ids.shape[0]), int(ids.shape[1]), int(dY.shape[2])


# (a size depends on its arguments alone, and asking costs as much as a launch)
@functools.lru_cache(maxsize=1024)
def _embed_workspace_size(B, T, V, d):
    lib, need = load_library(), ctypes.c_size_t(0)
    _check(lib, lib.dpg_embed_workspace_size(B, T, V, d, ctypes.byref(need)))
    return need.value


def _embed_workspace(B, T, V, d, device, workspace):
    return _workspace(_embed_workspace_size(B, T, int(V), d), device, workspace)


@_on_stream
def dpg_embed_norms(ids: torch.Tensor, dY: torch.Tensor, V: int, norm_sq: torch.Tensor,
                    scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                    stream=None):
    """Each sample's squared gradient norm of the table, added to norm_sq
    (libdpg): norm_sq[i] += sum_v ||scale sum_{t: ids[i, t] = v} dY[i, t]||^2.
    ids: [B, T] int64, dY: [B, T, d] (bf16 or fp32), norm_sq: [B] fp32, the
    buffer dpg_project_layer adds to. Returns norm_sq."""
    lib = load_library()
    B, T, d = _embed_args(ids, dY, V)
    _require(norm_sq, "norm_sq", torch.float32, (B,))
    _same_device(dY, norm_sq=norm_sq)
    code = _dtype_code(dY.dtype)
    if ids.numel() == 0:
        return norm_sq
    ws, ws_bytes = _embed_workspace(B, T, V, d, dY.device, workspace)
    _check(lib, lib.dpg_embed_norms(_ptr(ids), _ptr(dY), B, T, int(V), d, code, float(scale),
                                    _ptr(norm_sq), ws.data_ptr(), ws_bytes,
                                    _stream_handle(stream)))
    return norm_sq


@_on_stream
def dpg_embed_grad(ids: torch.Tensor, dY: torch.Tensor, V: int, scale: float = 1.0,
                   sample_scales: Optional[torch.Tensor] = None,
                   table_dtype: Optional[torch.dtype] = None,
                   dE: Optional[torch.Tensor] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """The table's gradient (libdpg): dE[v] = scale sum_i s_i
    sum_{t: ids[i, t] = v} dY[i, t], s_i = sample_scales[i] ([B] fp32 clip
    factors; 1 when None). table_dtype (default dE's, else fp32) is dE's type:
    fp32, or bf16 for a bf16 dY. With accumulate the rows of tokens that occur
    are added to (dE must be given), otherwise every row is written."""
    lib = load_library()
    B, T, d = _embed_args(ids, dY, V)
    if dE is None:
        if accumulate:
            raise ValueError("accumulate needs dE")
        dE = torch.empty((int(V), d), dtype=table_dtype or torch.float32, device=dY.device)
    _require(dE, "dE", table_dtype, (int(V), d))
    if sample_scales is not None:
        _require(sample_scales, "sample_scales", torch.float32, (B,))
    _same_device(dY, dE=dE, sample_scales=sample_scales)
    code, table = _dtype_code(dY.dtype), _dtype_code(dE.dtype)
    if ids.numel() == 0:
        return dE if accumulate else dE.zero_()
    ws, ws_bytes = _embed_workspace(B, T, V, d, dY.device, workspace)
    _check(lib, lib.dpg_embed_grad(_ptr(ids), _ptr(dY), B, T, int(V), d, code, float(scale),
                                   _ptr(sample_scales), table, 1 if accumulate else 0,
                                   _ptr(dE), ws.data_ptr(), ws_bytes,
                                   _stream_handle(stream)))
    return dE


def _loss_args(X, E, ids, name, k_shape=()):
    """Checked (N, d, V, dtype code) of X [..., d], E [V, d] and ids [..., *k_shape]."""
    _require(X, "X")
    _require(E, "E", X.dtype)
    if X.dim() < 1 or E.dim() != 2 or int(X.shape[-1]) != int(E.shape[1]):
        raise ValueError("X must be [..., d] and E [V, d]")
    _ids(ids, name, (*X.shape[:-1], *k_shape))
    _same_device(X, E=E, **{name: ids})
    d = int(X.shape[-1])
    # (a width of zero has rows all the same, which the library refuses)
    N = X.numel() // d if d else math.prod(X.shape[:-1])
    return N, d, int(E.shape[0]), _dtype_code(X.dtype)


def _loss_outputs(X, loss, lse):
    rows = tuple(X.shape[:-1])
    loss = torch.empty(rows, dtype=torch.float32, device=X.device) if loss is None else loss
    lse = torch.empty(rows, dtype=torch.float32, device=X.device) if lse is None else lse
    _require(loss, "loss", torch.float32, rows)
    _require(lse, "lse", torch.float32, rows)
    _same_device(X, loss=loss, lse=lse)
    return loss, lse


def _loss_grads(X, E, lse, dloss, need_dX, need_dE, dX, dE):
    rows = tuple(X.shape[:-1])
    _require(lse, "lse", torch.float32, rows)
    _require(dloss, "dloss", torch.float32, rows)
    if need_dX and dX is None:
        dX = torch.empty_like(X)
    if need_dE and dE is None:
        dE = torch.empty_like(E)
    if not (need_dX or need_dE):
        raise ValueError("need_dX or need_dE must be set")
    dX, dE = (dX if need_dX else None), (dE if need_dE else None)
    if dX is not None:
        _require(dX, "dX", X.dtype, X.shape)
    if dE is not None:
        _require(dE, "dE", E.dtype, E.shape)
    _same_device(X, lse=lse, dloss=dloss, dX=dX, dE=dE)
    return dX, dE


@functools.lru_cache(maxsize=1024)
def _vocab_workspace_size(N, d, V, k, code, grad):
    lib, need = load_library(), ctypes.c_size_t(0)
    if k is None:
        st = lib.dpg_vocab_loss_workspace_size(N, d, V, code, grad, ctypes.byref(need))
    else:
        st = lib.dpg_distill_loss_workspace_size(N, d, V, k, code, grad, ctypes.byref(need))
    _check(lib, st)
    return need.value


def _vocab_workspace(N, d, V, k, code, grad, device, workspace):
    return _workspace(_vocab_workspace_size(N, d, V, k, code, grad), device, workspace)


@_on_stream
def dpg_vocab_loss(X: torch.Tensor, E: torch.Tensor, targets: torch.Tensor,
                   scale: float = 1.0, loss: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Softmax cross entropy against a [V, d] table without an array of
    logits (libdpg): z = scale X E^T, lse = ln sum_v exp z_v,
    loss = lse - z_target; both 0 where the target lies outside [0, V).
    X: [..., d] and E in the same type (bf16 or fp32), targets: [...] int64.
    Returns (loss, lse), fp32 of X's leading shape."""
    lib = load_library()
    N, d, V, code = _loss_args(X, E, targets, "targets")
    loss, lse = _loss_outputs(X, loss, lse)
    if N == 0:
        return loss, lse
    ws, ws_bytes = _vocab_workspace(N, d, V, None, code, 0, X.device, workspace)
    _check(lib, lib.dpg_vocab_loss(_ptr(X), _ptr(E), _ptr(targets), N, d, V, code,
                                   float(scale), _ptr(loss), _ptr(lse), ws.data_ptr(),
                                   ws_bytes, _stream_handle(stream)))
    return loss, lse


@_on_stream
def dpg_vocab_loss_grad(X: torch.Tensor, E: torch.Tensor, targets: torch.Tensor,
                        lse: torch.Tensor, dloss: torch.Tensor, scale: float = 1.0,
                        need_dX: bool = True, need_dE: bool = True,
                        dX: Optional[torch.Tensor] = None,
                        dE: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of sum_n dloss_n loss_n of dpg_vocab_loss (libdpg), with the
    lse it returned. dloss: fp32 of X's leading shape. Returns (dX, dE) in X's
    type; None for the one not needed."""
    lib = load_library()
    N, d, V, code = _loss_args(X, E, targets, "targets")
    dX, dE = _loss_grads(X, E, lse, dloss, need_dX, need_dE, dX, dE)
    if N == 0:
        return dX, None if dE is None else dE.zero_()
    ws, ws_bytes = _vocab_workspace(N, d, V, None, code, 1, X.device, workspace)
    _check(lib, lib.dpg_vocab_loss_grad(_ptr(X), _ptr(E), _ptr(targets), _ptr(lse),
                                        _ptr(dloss), N, d, V, code, float(scale), _ptr(dX),
                                        _ptr(dE), ws.data_ptr(), ws_bytes,
                                        _stream_handle(stream)))
    return dX, dE


def _top_args(X, E, top_ids, top_logits):
    if not isinstance(top_ids, torch.Tensor) or top_ids.dim() < 1:
        raise TypeError("top_ids must be a [..., k] torch.Tensor")
    k = int(top_ids.shape[-1])
    N, d, V, code = _loss_args(X, E, top_ids, "top_ids", (k,))
    _require(top_logits, "top_logits", torch.float32, top_ids.shape)
    _same_device(X, top_logits=top_logits)
    return N, d, V, k, code


@_on_stream
def dpg_distill_loss(X: torch.Tensor, E: torch.Tensor, top_ids: torch.Tensor,
                     top_logits: torch.Tensor, temperature: float = 1.0,
                     scale: float = 1.0, loss: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Distillation from a teacher's top k logits per row (libdpg):
    loss = tau^2 sum_j q_j (ln q_j - ln p_id(j)), q = softmax of
    top_logits / tau over the entries whose id lies in [0, V), p = softmax of
    scale X E^T / tau over the vocabulary. Rows without any weight get 0.
    top_ids: [..., k] int64, top_logits: [..., k] fp32.
    Returns (loss, lse), lse = ln sum_v exp(z_v / tau)."""
    lib = load_library()
    N, d, V, k, code = _top_args(X, E, top_ids, top_logits)
    loss, lse = _loss_outputs(X, loss, lse)
    if N == 0:
        return loss, lse
    ws, ws_bytes = _vocab_workspace(N, d, V, k, code, 0, X.device, workspace)
    _check(lib, lib.dpg_distill_loss(_ptr(X), _ptr(E), _ptr(top_ids), _ptr(top_logits), N, d,
                                     V, k, code, float(scale), float(temperature),
                                     _ptr(loss), _ptr(lse), ws.data_ptr(), ws_bytes,
                                     _stream_handle(stream)))
    return loss, lse


@_on_stream
def dpg_distill_loss_grad(X: torch.Tensor, E: torch.Tensor, top_ids: torch.Tensor,
                          top_logits: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor,
                          temperature: float = 1.0, scale: float = 1.0,
                          need_dX: bool = True, need_dE: bool = True,
                          dX: Optional[torch.Tensor] = None,
                          dE: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of sum_n dloss_n loss_n of dpg_distill_loss (libdpg), with
    the lse it returned. Returns (dX, dE); None for the one not needed."""
    lib = load_library()
    N, d, V, k, code = _top_args(X, E, top_ids, top_logits)
    dX, dE = _loss_grads(X, E, lse, dloss, need_dX, need_dE, dX, dE)
    if N == 0:
        return dX, None if dE is None else dE.zero_()
    ws, ws_bytes = _vocab_workspace(N, d, V, k, code, 1, X.device, workspace)
    _check(lib, lib.dpg_distill_loss_grad(
        _ptr(X), _ptr(E), _ptr(top_ids), _ptr(top_logits), _ptr(lse), _ptr(dloss), N, d, V, k,
        code, float(scale), float(temperature), _ptr(dX), _ptr(dE), ws.data_ptr(), ws_bytes,
        _stream_handle(stream)))
    return dX, dE


class PreparedStep:
    """One DP-GRAPE step with its layer tables and workspaces marshalled
    once, for callers that repeat the step on the same buffers (a training
    loop, the bench): dpg_private_step, or with one_call=False the two calls
    dpg_project_clip_noise and dpg_adam_backproject.

    run(step) enqueues the step on the current stream with
    step = proj_step = `step`."""

    def __init__(self, A, dY, W, m, v, r, clip_C, sigma, seed, lr, beta1,
                 beta2, eps, layer_ids=None, G_priv=None, sample_norms=None,
                 one_call=True):
        self.lib = load_library()
        self.one_call = one_call
        n = len(A)
        dt = A[0].dtype
        self.dtype_code = _dtype_code(dt)
        self.B, self.T = int(A[0].shape[0]), int(A[0].shape[1])
        ids = list(range(n)) if layer_ids is None else [int(x) for x in layer_ids]
        dev = A[0].device
        self.G_priv = G_priv or [torch.empty((r, int(d.shape[2])),
                                             dtype=torch.float32, device=dev)
                                 for d in dY]
        self.sample_norms = (torch.empty(self.B, dtype=torch.float32, device=dev)
                             if sample_norms is None else sample_norms)
        self.grads, self.params, _, _, _, _ = _step_tables(A, dY, W, m, v, self.G_priv,
                                                           r, ids)
        self.n = n
        self.r = int(r)
        self.hyper = (float(clip_C), float(sigma), int(seed), float(lr),
                      float(beta1), float(beta2), float(eps))
        need1, need2 = ctypes.c_size_t(0), ctypes.c_size_t(0)
        _check(self.lib, self.lib.dpg_project_workspace_size(
            self.grads, n, self.B, self.T, self.r, self.dtype_code,
            ctypes.byref(need1)))
        _check(self.lib, self.lib.dpg_adam_workspace_size(
            self.params, n, self.r, self.dtype_code, ctypes.byref(need2)))
        self.ws1, self.ws1_bytes = _workspace(need1.value, dev, None)
        self.ws2, self.ws2_bytes = _workspace(need2.value, dev, None)
        need3 = ctypes.c_size_t(0)
        _check(self.lib, self.lib.dpg_step_workspace_size(
            self.grads, n, self.B, self.T, self.r, self.dtype_code,
            ctypes.byref(need3)))
        self.ws3, self.ws3_bytes = _workspace(need3.value if one_call else 0, dev, None)
        self._keep = (A, dY, W, m, v)

    def _buffers(self):
        return [self.sample_norms, self.ws1, self.ws2, self.ws3, *self.G_priv]

    def _mark_stream(self, stream) -> None:
        """Buffers allocated on the construction stream and used on another
        one are marked as in use there, so that freeing this object does not
        release them to other work before that stream reaches this point."""
        if stream is not None and stream != torch.cuda.current_stream():
            for t in self._buffers():
                t.record_stream(stream)

    def run(self, step: int, stream=None) -> None:
        C, sigma, seed, lr, b1, b2, eps = self.hyper
        h = _stream_handle(stream)
        lib = self.lib
        self._mark_stream(stream)
        if self.one_call:
            _check(lib, lib.dpg_private_step(
                self.grads, self.params, self.n, self.B, self.T, self.r,
                self.dtype_code, C, sigma, lr, b1, b2, eps, seed, step, step,
                self.sample_norms.data_ptr(), self.ws3.data_ptr(), self.ws3_bytes, h))
            return
        _check(lib, lib.dpg_project_clip_noise(
            self.grads, self.n, self.B, self.T, self.r, self.dtype_code, C,
            sigma, seed, step, step, self.sample_norms.data_ptr(),
            self.ws1.data_ptr(), self.ws1_bytes, h))
        _check(lib, lib.dpg_adam_backproject(
            self.params, self.n, self.r, self.dtype_code, lr, b1, b2, eps,
            seed, step, step, self.ws2.data_ptr(), self.ws2_bytes, h))


class PreparedStreamingStep(PreparedStep):
    """The same step in the streaming form: dpg_project_layer for each layer
    in order (stored projections [B, r, d_out] fp32, squared norms summed
    over the layers), then dpg_clip_sum_noise and dpg_adam_backproject, with
    every table, buffer and workspace marshalled once."""

    def __init__(self, A, dY, W, m, v, r, clip_C, sigma, seed, lr, beta1,
                 beta2, eps, layer_ids=None):
        super().__init__(A, dY, W, m, v, r, clip_C, sigma, seed, lr, beta1,
                         beta2, eps, layer_ids=layer_ids)
        dev = A[0].device
        self.norm_sq = torch.zeros(self.B, dtype=torch.float32, device=dev)
        self.G_hat = [torch.empty((self.B, self.r, int(d.shape[2])),
                                  dtype=torch.float32, device=dev) for d in dY]
        self.one = []
        need = 0
        for i in range(self.n):
            g = (LayerGrad * 1)()
            ctypes.memmove(ctypes.addressof(g), ctypes.addressof(self.grads[i]),
                           ctypes.sizeof(LayerGrad))
            self.one.append(g)
            b = ctypes.c_size_t(0)
            _check(self.lib, self.lib.dpg_project_layer_workspace_size(
                g, self.B, self.T, self.r, self.dtype_code, ctypes.byref(b)))
            need = max(need, b.value)
        self.wsl, self.wsl_bytes = _workspace(need, dev, None)
        b = ctypes.c_size_t(0)
        _check(self.lib, self.lib.dpg_clip_workspace_size(self.B, ctypes.byref(b)))
        self.wsc, self.wsc_bytes = _workspace(b.value, dev, None)
        self.hats = (LayerHat * self.n)()
        for i in range(self.n):
            h = self.hats[i]
            h.d_out, h.layer_id = self.grads[i].d_out, self.grads[i].layer_id
            h.G_hat, h.G_priv = self.G_hat[i].data_ptr(), self.G_priv[i].data_ptr()

    def _buffers(self):
        return super()._buffers() + [self.norm_sq, self.wsl, self.wsc, *self.G_hat]

    def run(self, step: int, stream=None) -> None:
        C, sigma, seed, lr, b1, b2, eps = self.hyper
        h = _stream_handle(stream)
        lib = self.lib
        self._mark_stream(stream)
        with torch.cuda.stream(stream) if stream is not None else _nullctx():
            self.norm_sq.zero_()
        for i in range(self.n):
            _check(lib, lib.dpg_project_layer(
                self.one[i], self.B, self.T, self.r, self.dtype_code, seed, step,
                self.G_hat[i].data_ptr(), self.norm_sq.data_ptr(),
                self.wsl.data_ptr(), self.wsl_bytes, h))
        _check(lib, lib.dpg_clip_sum_noise(
            self.hats, self.n, self.B, self.r, C, sigma, seed, step,
            self.norm_sq.data_ptr(), self.sample_norms.data_ptr(),
            self.wsc.data_ptr(), self.wsc_bytes, h))
        _check(lib, lib.dpg_adam_backproject(
            self.params, self.n, self.r, self.dtype_code, lr, b1, b2, eps,
            seed, step, step, self.ws2.data_ptr(), self.ws2_bytes, h))


class _nullctx:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


def timing_enable(on: bool = True) -> None:
    """Bracket every kernel launch of the two step calls with HIP events."""
    lib = load_library()
    _check(lib, lib.dpg_timing_enable(1 if on else 0))


def timing_read(reset: bool = True) -> dict:
    """{kernel name: (total ms, launches)} since the last reset."""
    lib = load_library()
    ms = (ctypes.c_double * N_KERNEL_KINDS)()
    cnt = (ctypes.c_int64 * N_KERNEL_KINDS)()
    _check(lib, lib.dpg_timing_read(ms, cnt, N_KERNEL_KINDS, 1 if reset else 0))
    return {lib.dpg_kernel_name(k).decode(): (ms[k], cnt[k])
            for k in range(N_KERNEL_KINDS)}


def version() -> int:
    return load_library().dpg_version()
