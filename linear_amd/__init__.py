"""MI355X (gfx950) FP16 linear layer: y = FP16(FP16(x @ weight.T) + b).

Also its bfloat16 form, the unrounded FP32 sums, multi-step epilogue programs,
the grouped and indexed (per-row expert) contractions, the gated feed-forward
block with its gradients, the layer's gradients, the global gradient norm
with clipping, a linear head's softmax cross entropy with its gradients, and an
AdamW step over many tensors.  A thin ctypes binding over the C ABI of ``liblinear_amd.so`` (declared in
``include/linear_amd.h``).  The functions carry the C entry points' names and
only marshal arguments: every step of the computation runs in the library's
HIP kernels.  PyTorch supplies device memory and the stream.  If the library
is missing the calls raise; there is no fallback.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import importlib.util
import itertools
import operator
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblinear_amd.so")
MARSHAL_PATH = os.path.join(_HERE, "_marshal.so")

LINEAR_OK = 0
LINEAR_E_NULL = 1
LINEAR_E_SHAPE = 2
LINEAR_E_STRIDE = 3
LINEAR_E_ALIAS = 4
LINEAR_E_PATH = 5
LINEAR_E_DEVICE = 6
LINEAR_E_LAUNCH = 7
LINEAR_E_EPILOGUE = 8
LINEAR_E_CAPTURE = 9
LINEAR_E_WORKSPACE = 10
LINEAR_E_SCRATCH = 11
LINEAR_E_VALUE = 12
LINEAR_E_MEMORY = 13

# scratch the no-allocation indexed call holds per GPU (include/linear_amd.h)
NOALLOC_SCRATCH_BYTES = 1 << 20

# Epilogue steps (include/linear_amd.h, LINEAR_EPI_*)
EPI_MAX_STEPS = 8
EPI_BIAS = 1
EPI_RESIDUAL = 2
EPI_MUL = 3
EPI_SILU = 4
EPI_GELU_TANH = 5
EPI_GELU_ERF = 6

PATH_AUTO = 0
PATH_GEMM = 1
PATH_SKINNY = 2

ENTRY_POINTS = ("linear_f16", "linear_f16_nobias", "linear_f16_ex", "linear_f16_f32out",
                "linear_bf16", "linear_bf16_nobias", "linear_bf16_ex", "linear_bf16_f32out",
                "linear_f16_epilogue", "linear_bf16_epilogue",
                "linear_f16_grouped", "linear_bf16_grouped", "linear_f16_grouped_f32out", "linear_bf16_grouped_f32out",
                "linear_indexed_workspace_bytes",
                "linear_f16_indexed", "linear_bf16_indexed", "linear_f16_indexed_f32out", "linear_bf16_indexed_f32out",
                "linear_f16_indexed_noalloc",
                "linear_f16_gated", "linear_bf16_gated", "linear_gated_forward_workspace_bytes", "linear_gated_workspace_bytes",
                "linear_f16_gated_backward", "linear_bf16_gated_backward", "linear_backward_workspace_bytes",
                "linear_f16_backward_input", "linear_bf16_backward_input",
                "linear_f16_backward_weight", "linear_bf16_backward_weight",
                "linear_f16_backward_weight_f32out", "linear_bf16_backward_weight_f32out",
                "linear_cross_entropy_workspace_bytes", "linear_cross_entropy_backward_workspace_bytes",
                "linear_cross_entropy_workspace_bytes_aligned", "linear_cross_entropy_backward_workspace_bytes_aligned",
                "linear_f16_cross_entropy", "linear_bf16_cross_entropy",
                "linear_f16_cross_entropy_backward", "linear_bf16_cross_entropy_backward",
                "linear_f16_cross_entropy_backward_f32out", "linear_bf16_cross_entropy_backward_f32out",
                "linear_grad_workspace_bytes", "linear_grad_norm", "linear_grad_clip",
                "linear_adamw_state_bytes", "linear_adamw", "linear_adamw_values",
                "linear_f16_plan", "linear_gated_backward_plan", "linear_status_string", "linear_last_hip_error")


class LinearError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (status %d%s)" % (
            what, linear_status_string(code), code,
            ", hip error %d" % _lib().linear_last_hip_error()
            if code in (LINEAR_E_DEVICE, LINEAR_E_LAUNCH) else ""))


class LinearArgumentError(LinearError, ValueError):
    pass


class _Plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("threads", ctypes.c_int32), ("vector_io", ctypes.c_int32),
                ("grid", ctypes.c_int64), ("split_n", ctypes.c_int64), ("tile_m2", ctypes.c_int32),
                ("tile_n2", ctypes.c_int32), ("grid2", ctypes.c_int64), ("stages", ctypes.c_int32)]


class _ProductPlan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("tile_m", "tile_n", "stages", "sets", "splits", "tile_m2", "tile_n2")] + [
        ("split_c", ctypes.c_int64)]


class _GatedPlan(ctypes.Structure):
    _fields_ = [("dx", _ProductPlan), ("dw", _ProductPlan), ("joint", ctypes.c_int32), ("two_words", ctypes.c_int32)]


class _AdamwOptions(ctypes.Structure):
    _fields_ = [(f, ctypes.c_double) for f in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("state_bits", ctypes.c_int32), ("max_norm", ctypes.c_float),
        ("norm", ctypes.c_void_p), ("device_lr", ctypes.c_void_p), ("device_step", ctypes.c_void_p)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("nsteps", ctypes.c_int32), ("op", ctypes.c_int32 * EPI_MAX_STEPS),
                ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("mul", ctypes.c_void_p), ("ldm", ctypes.c_int64)]


_LIB = None


def _lib():
    """Load liblinear_amd.so (after torch, so both share one HIP runtime)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("liblinear_amd.so is not built (run `python -m linear_amd.build` or "
                           "__graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.linear_f16.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp]
    lib.linear_f16.restype = i32
    lib.linear_f16_nobias.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp]
    lib.linear_f16_nobias.restype = i32
    lib.linear_f16_ex.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i32, vp]
    lib.linear_f16_ex.restype = i32
    for name in ("linear_bf16",):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp]
        getattr(lib, name).restype = i32
    lib.linear_bf16_nobias.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp]
    lib.linear_bf16_nobias.restype = i32
    lib.linear_bf16_ex.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i32, vp]
    lib.linear_bf16_ex.restype = i32
    for name in ("linear_f16_f32out", "linear_bf16_f32out"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_epilogue", "linear_bf16_epilogue"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, ctypes.POINTER(_Epilogue), vp, i64, i64, i64, i64, i32, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_grouped", "linear_bf16_grouped"):
        getattr(lib, name).argtypes = [vp, i64, i64, vp, i64, vp, vp, i64, i64, i64, i64, i64, i64, i32, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_grouped_f32out", "linear_bf16_grouped_f32out"):
        getattr(lib, name).argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, i64, i64, i64, i64, i32, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_indexed", "linear_bf16_indexed", "linear_f16_indexed_f32out",
                 "linear_bf16_indexed_f32out"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, i64, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
    lib.linear_f16_indexed_noalloc.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, i64, i64, i64, i64, vp]
    lib.linear_f16_indexed_noalloc.restype = i32
    lib.linear_indexed_workspace_bytes.argtypes = [i64, i64]
    lib.linear_indexed_workspace_bytes.restype = i64
    for name in ("linear_f16_gated", "linear_bf16_gated"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp,
                                       i64, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_gated_backward", "linear_bf16_gated_backward"):
        getattr(lib, name).argtypes = ([vp, i64] * 6 + [i32] + [vp, i64] * 3 + [i64, i64, i64, vp, i64, vp])
        getattr(lib, name).restype = i32
    for name in ("linear_f16_backward_input", "linear_bf16_backward_input"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_backward_weight", "linear_bf16_backward_weight"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_backward_weight_f32out", "linear_bf16_backward_weight_f32out"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_cross_entropy", "linear_bf16_cross_entropy"):
        getattr(lib, name).argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
    for name in ("linear_f16_cross_entropy_backward", "linear_bf16_cross_entropy_backward"):
        getattr(lib, name).argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, i64, i64, i64, vp, i64, vp]
        getattr(lib, name).restype = i32
        getattr(lib, name + "_f32out").argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, i32, i64, i64,
                                                   i64, vp, i64, vp]
        getattr(lib, name + "_f32out").restype = i32
    for name in ("linear_gated_forward_workspace_bytes", "linear_gated_workspace_bytes", "linear_backward_workspace_bytes",
                 "linear_cross_entropy_workspace_bytes", "linear_cross_entropy_backward_workspace_bytes",
                 "linear_cross_entropy_workspace_bytes_aligned", "linear_cross_entropy_backward_workspace_bytes_aligned"):
        getattr(lib, name).argtypes = [i64, i64, i64]
        getattr(lib, name).restype = i64
    lib.linear_grad_workspace_bytes.argtypes = [i64]
    lib.linear_grad_workspace_bytes.restype = i64
    lib.linear_grad_norm.argtypes = [vp, i64, vp, vp, i64, vp]
    lib.linear_grad_norm.restype = i32
    lib.linear_grad_clip.argtypes = [vp, vp, i64, vp, ctypes.c_float, vp]
    lib.linear_grad_clip.restype = i32
    lib.linear_adamw_state_bytes.argtypes = [i64, i32]
    lib.linear_adamw_state_bytes.restype = i64
    lib.linear_adamw.argtypes = [vp, vp, vp, vp, vp, i64, ctypes.POINTER(_AdamwOptions), vp]
    lib.linear_adamw.restype = i32
    lib.linear_adamw_values.argtypes = [vp, vp, i32, i64, vp]
    lib.linear_adamw_values.restype = i32
    lib.linear_f16_plan.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i32,
                                    ctypes.POINTER(_Plan)]
    lib.linear_f16_plan.restype = i32
    lib.linear_gated_backward_plan.argtypes = [i64, i64, i64, ctypes.POINTER(_GatedPlan)]
    lib.linear_gated_backward_plan.restype = i32
    lib.linear_status_string.argtypes = [i32]
    lib.linear_status_string.restype = ctypes.c_char_p
    lib.linear_last_hip_error.argtypes = []
    lib.linear_last_hip_error.restype = i32
    _LIB = lib
    return lib


class _NoMarshal:
    """In place of csrc/marshal.cpp where it could not be built: every call takes the way through the
    binding's own checks, at more host time."""

    def _none(*args):
        return None

    adamw = states = cross_entropy = cross_entropy_backward = scratch = staticmethod(_none)


@functools.lru_cache(maxsize=None)
def _marshal():
    """The module that reads lists of tensors (csrc/marshal.cpp)."""
    if not os.path.exists(MARSHAL_PATH):
        warnings.warn("_marshal.so is not built: calls take more host time (python -m linear_amd.build says what it needs)")
        return _NoMarshal
    spec = importlib.util.spec_from_file_location("_marshal", MARSHAL_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def library_path() -> str:
    return LIB_PATH


def linear_status_string(code: int) -> str:
    return _lib().linear_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code == LINEAR_OK:
        return
    if code in (LINEAR_E_DEVICE, LINEAR_E_LAUNCH):
        raise LinearError(code, what)
    raise LinearArgumentError(code, what)


def _mat(t: torch.Tensor, name: str, dtype=torch.float16):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    rows, cols = t.shape
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError("%s must have unit inner stride" % name)
    return t.data_ptr(), ld if rows > 1 else max(cols, ld, 1)


def _stream_handle(stream, *tensors):
    """The stream a launch goes to, after checking its tensor arguments: every one
    must be a GPU ('cuda') tensor on the current device, where the library
    launches (a host address handed to a kernel would fault the GPU, so it is
    refused here instead).  stream: a torch stream, a raw handle or None (the
    current stream of that device)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError("every tensor argument must be on the GPU (a 'cuda' device); got one on %s" % t.device)
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensor arguments on two devices: %s and %s" % (dev, t.device))
    if dev is not None and dev.index is not None and dev.index != torch.cuda.current_device():
        raise ValueError("the tensors are on %s but the current device is cuda:%d (the library launches on the "
                         "current device; call under torch.cuda.device(%s))" % (dev, torch.cuda.current_device(), dev))
    if stream is not None:
        sdev = getattr(stream, "device", None)
        if sdev is not None and dev is not None and torch.device(sdev) != dev:
            raise ValueError("the stream belongs to %s but the tensors are on %s" % (sdev, dev))
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    if dev is not None:
        return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
    return ctypes.c_void_p(0)


def _prepare(x, weight, b, out, dtype=torch.float16, out_dtype=None):
    out_dtype = out_dtype or dtype
    xp, ldx = _mat(x, "x", dtype)
    wp, ldw = _mat(weight, "weight", dtype)
    M, K = x.shape
    N, K2 = weight.shape
    if K != K2:
        raise ValueError("x is [%d, %d] but weight is [%d, %d]" % (M, K, N, K2))
    bp = None
    if b is not None:
        if b.dtype != dtype or b.dim() != 1 or b.shape[0] != N or (N > 1 and b.stride(0) != 1):
            raise ValueError("b must be a contiguous %s [N] tensor" % dtype)
        bp = b.data_ptr()
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    yp, ldy = _mat(out, "out", out_dtype)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [%d, %d]" % (M, N))
    return xp, ldx, wp, ldw, bp, out, yp, ldy, M, N, K


def linear_f16(x: torch.Tensor, weight: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y = FP16(FP16(x @ weight.T) + b) on the GPU (x [M,K], weight [N,K], b [N], float16)."""
    if b is None:
        raise ValueError("linear_f16 needs a bias; use linear_f16_nobias")
    xp, ldx, wp, ldw, bp, out, yp, ldy, M, N, K = _prepare(x, weight, b, out)
    rc = _lib().linear_f16(xp, ldx, wp, ldw, bp, yp, ldy, M, N, K, _stream_handle(stream, x, weight, b, out))
    _check(rc, "linear_f16")
    return out


def linear_f16_nobias(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """proj = FP16(x @ weight.T) on the GPU."""
    xp, ldx, wp, ldw, _, out, yp, ldy, M, N, K = _prepare(x, weight, None, out)
    rc = _lib().linear_f16_nobias(xp, ldx, wp, ldw, yp, ldy, M, N, K, _stream_handle(stream, x, weight, out))
    _check(rc, "linear_f16_nobias")
    return out


def linear_f16_ex(x: torch.Tensor, weight: torch.Tensor, b: torch.Tensor | None,
                  out: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """linear_f16 with a forced path (PATH_AUTO / PATH_GEMM / PATH_SKINNY) and optional bias."""
    xp, ldx, wp, ldw, bp, out, yp, ldy, M, N, K = _prepare(x, weight, b, out)
    rc = _lib().linear_f16_ex(xp, ldx, wp, ldw, bp, yp, ldy, M, N, K, int(path),
                              _stream_handle(stream, x, weight, b, out))
    _check(rc, "linear_f16_ex")
    return out


def linear_f16_f32out(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor | None = None,
                      path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """The unrounded FP32 sums x @ weight.T (float16 operands, float32 output)."""
    xp, ldx, wp, ldw, _, out, yp, ldy, M, N, K = _prepare(x, weight, None, out, torch.float16, torch.float32)
    rc = _lib().linear_f16_f32out(xp, ldx, wp, ldw, yp, ldy, M, N, K, int(path),
                                  _stream_handle(stream, x, weight, out))
    _check(rc, "linear_f16_f32out")
    return out


def linear_bf16(x: torch.Tensor, weight: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """y = BF16(BF16(x @ weight.T) + b) (bfloat16 x [M,K], weight [N,K], b [N])."""
    if b is None:
        raise ValueError("linear_bf16 needs a bias; use linear_bf16_nobias")
    xp, ldx, wp, ldw, bp, out, yp, ldy, M, N, K = _prepare(x, weight, b, out, torch.bfloat16)
    rc = _lib().linear_bf16(xp, ldx, wp, ldw, bp, yp, ldy, M, N, K, _stream_handle(stream, x, weight, b, out))
    _check(rc, "linear_bf16")
    return out


def linear_bf16_nobias(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """proj = BF16(x @ weight.T)."""
    xp, ldx, wp, ldw, _, out, yp, ldy, M, N, K = _prepare(x, weight, None, out, torch.bfloat16)
    rc = _lib().linear_bf16_nobias(xp, ldx, wp, ldw, yp, ldy, M, N, K, _stream_handle(stream, x, weight, out))
    _check(rc, "linear_bf16_nobias")
    return out


def linear_bf16_ex(x: torch.Tensor, weight: torch.Tensor, b: torch.Tensor | None,
                   out: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """linear_bf16 with a forced path and optional bias."""
    xp, ldx, wp, ldw, bp, out, yp, ldy, M, N, K = _prepare(x, weight, b, out, torch.bfloat16)
    rc = _lib().linear_bf16_ex(xp, ldx, wp, ldw, bp, yp, ldy, M, N, K, int(path),
                               _stream_handle(stream, x, weight, b, out))
    _check(rc, "linear_bf16_ex")
    return out


def linear_bf16_f32out(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor | None = None,
                       path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """The unrounded FP32 sums x @ weight.T (bfloat16 operands, float32 output)."""
    xp, ldx, wp, ldw, _, out, yp, ldy, M, N, K = _prepare(x, weight, None, out, torch.bfloat16, torch.float32)
    rc = _lib().linear_bf16_f32out(xp, ldx, wp, ldw, yp, ldy, M, N, K, int(path),
                                   _stream_handle(stream, x, weight, out))
    _check(rc, "linear_bf16_f32out")
    return out


def _epilogue_call(fn_name, dtype, x, weight, ops, bias, residual, mul, out, path, stream):
    ops = [int(o) for o in ops]
    if len(ops) > EPI_MAX_STEPS:
        raise ValueError("at most %d epilogue steps" % EPI_MAX_STEPS)
    xp, ldx, wp, ldw, _, out, yp, ldy, M, N, K = _prepare(x, weight, None, out, dtype)
    ep = _Epilogue()
    ep.nsteps = len(ops)
    for i, o in enumerate(ops):
        ep.op[i] = o
    if bias is not None:
        if bias.dtype != dtype or bias.dim() != 1 or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1):
            raise ValueError("bias must be a contiguous %s [N] tensor" % dtype)
        ep.bias = bias.data_ptr()
    for name, t in (("residual", residual), ("mul", mul)):
        if t is None:
            continue
        tp, ld = _mat(t, name, dtype)
        if tuple(t.shape) != (M, N):
            raise ValueError("%s must be [%d, %d]" % (name, M, N))
        setattr(ep, name, tp)
        setattr(ep, "ldr" if name == "residual" else "ldm", ld)
    rc = getattr(_lib(), fn_name)(xp, ldx, wp, ldw, ctypes.byref(ep), yp, ldy, M, N, K, int(path),
                                  _stream_handle(stream, x, weight, bias, residual, mul, out))
    _check(rc, fn_name)
    return out


def linear_f16_epilogue(x: torch.Tensor, weight: torch.Tensor, ops, bias=None, residual=None, mul=None,
                        out: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """The projection followed by the epilogue steps `ops` (EPI_*), each rounded to binary16.
    bias [N], residual and mul [M, N] as the steps need them; out may be the residual itself."""
    return _epilogue_call("linear_f16_epilogue", torch.float16, x, weight, ops, bias, residual, mul, out, path,
                          stream)


def linear_bf16_epilogue(x: torch.Tensor, weight: torch.Tensor, ops, bias=None, residual=None, mul=None,
                         out: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """linear_f16_epilogue on bfloat16 operands, inputs and output."""
    return _epilogue_call("linear_bf16_epilogue", torch.bfloat16, x, weight, ops, bias, residual, mul, out, path,
                          stream)


def _grouped_call(dtype, x, weight, b, out, f32, path, stream):
    """x [G, M, K] (inner two dims row-major), weight [G*N, K], b [G*N] or None."""
    if x.dtype != dtype or weight.dtype != dtype:
        raise TypeError("x and weight must be %s" % dtype)
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [G, M, K] and weight [G*N, K]")
    G, M, K = x.shape
    if G == 0 or weight.shape[0] % max(G, 1) != 0 or weight.shape[1] != K:
        raise ValueError("weight must be [G*N, %d] for G = %d" % (K, G))
    N = weight.shape[0] // G
    if (K > 1 and x.stride(2) != 1) or (K > 1 and weight.stride(1) != 1):
        raise ValueError("x and weight need unit inner stride")
    ldx = x.stride(1) if M > 1 else max(K, x.stride(1), 1)
    sx = x.stride(0)
    ldw = weight.stride(0) if weight.shape[0] > 1 else max(K, 1)
    out_dtype = torch.float32 if f32 else dtype
    if out is None:
        out = torch.empty((G, M, N), dtype=out_dtype, device=x.device)
    if out.dtype != out_dtype or tuple(out.shape) != (G, M, N) or (N > 1 and out.stride(2) != 1):
        raise ValueError("out must be a %s [%d, %d, %d] tensor with unit inner stride" % (out_dtype, G, M, N))
    ldy = out.stride(1) if M > 1 else max(N, out.stride(1), 1)
    sy = out.stride(0)
    bp = None
    if b is not None:
        if f32:
            raise ValueError("the FP32-output grouped call takes no bias")
        if b.dtype != dtype or b.dim() != 1 or b.shape[0] != G * N or (G * N > 1 and b.stride(0) != 1):
            raise ValueError("b must be a contiguous %s [G*N] tensor" % dtype)
        bp = b.data_ptr()
    tag = "bf16" if dtype == torch.bfloat16 else "f16"
    if f32:
        name = "linear_%s_grouped_f32out" % tag
        rc = getattr(_lib(), name)(x.data_ptr(), ldx, sx, weight.data_ptr(), ldw, out.data_ptr(), ldy, sy, G, M, N,
                                   K, int(path), _stream_handle(stream, x, weight, out))
    else:
        name = "linear_%s_grouped" % tag
        rc = getattr(_lib(), name)(x.data_ptr(), ldx, sx, weight.data_ptr(), ldw, bp, out.data_ptr(), ldy, sy, G, M,
                                   N, K, int(path), _stream_handle(stream, x, weight, b, out))
    _check(rc, name)
    return out


def linear_f16_grouped(x, weight, b=None, out=None, path: int = PATH_AUTO, stream=None):
    """Grouped contraction: x [G, M, K] against weight [G*N, K] read as G blocks of N rows."""
    return _grouped_call(torch.float16, x, weight, b, out, False, path, stream)


def linear_bf16_grouped(x, weight, b=None, out=None, path: int = PATH_AUTO, stream=None):
    return _grouped_call(torch.bfloat16, x, weight, b, out, False, path, stream)


def linear_f16_grouped_f32out(x, weight, out=None, path: int = PATH_AUTO, stream=None):
    return _grouped_call(torch.float16, x, weight, None, out, True, path, stream)


def linear_bf16_grouped_f32out(x, weight, out=None, path: int = PATH_AUTO, stream=None):
    return _grouped_call(torch.bfloat16, x, weight, None, out, True, path, stream)


def indexed_workspace_bytes(E: int, M: int) -> int:
    """Bytes of device workspace an indexed call with E experts and M rows needs."""
    n = _lib().linear_indexed_workspace_bytes(E, M)
    if n < 0:
        raise ValueError("E=%d, M=%d out of range" % (E, M))
    return n


def _indexed_args(dtype, x, w, idx, out, f32):
    """Checks and marshalling shared by the indexed calls: x [M, K], w [E, K, N]
    (inner two dims row-major), idx [M] int32.  Returns (out, pointer/stride/shape
    arguments of the C call up to K)."""
    if x.dtype != dtype or w.dtype != dtype:
        raise TypeError("x and w must be %s" % dtype)
    if idx.dtype != torch.int32 or idx.dim() != 1 or (idx.shape[0] > 1 and idx.stride(0) != 1):
        raise TypeError("idx must be a contiguous int32 [M] tensor")
    xp, ldx = _mat(x, "x", dtype)
    if w.dim() != 3:
        raise ValueError("w must be [E, K, N]")
    E, K, N = w.shape
    M = x.shape[0]
    if x.shape[1] != K or idx.shape[0] != M:
        raise ValueError("x is %s, w is %s, idx is %s" % (tuple(x.shape), tuple(w.shape), tuple(idx.shape)))
    if N > 1 and w.stride(2) != 1:
        raise ValueError("w needs unit inner stride")
    ldw = w.stride(1) if K > 1 else max(N, w.stride(1), 1)
    sw = w.stride(0) if E > 1 else max(K * ldw, w.stride(0), 1)
    out_dtype = torch.float32 if f32 else dtype
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    yp, ldy = _mat(out, "out", out_dtype)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [%d, %d]" % (M, N))
    return out, (xp, ldx, w.data_ptr(), ldw, sw, idx.data_ptr(), yp, ldy, E, M, N, K)


def _indexed_call(dtype, x, w, idx, out, f32, stream, workspace):
    out, args = _indexed_args(dtype, x, w, idx, out, f32)
    E, M = args[8], args[9]
    need = indexed_workspace_bytes(E, M)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    elif workspace.dtype != torch.uint8 or workspace.dim() != 1 or workspace.numel() < need:
        raise ValueError("workspace must be a uint8 tensor of at least %d bytes" % need)
    tag = "bf16" if dtype == torch.bfloat16 else "f16"
    name = "linear_%s_indexed%s" % (tag, "_f32out" if f32 else "")
    rc = getattr(_lib(), name)(*args, workspace.data_ptr(), workspace.numel(),
                               _stream_handle(stream, x, w, idx, out, workspace))
    _check(rc, name)
    return out


def linear_f16_indexed_noalloc(x, w, idx, out, stream=None):
    """linear_f16_indexed without a workspace, for callers that cannot allocate: the
    library's per-GPU scratch array (NOALLOC_SCRATCH_BYTES) holds the routing.
    out must be given (a [M, N] binary16 tensor; this call allocates nothing).
    Calls in flight at once on one GPU share that array and race."""
    if out is None:
        raise ValueError("out is required: the no-allocation call creates no tensor")
    out, args = _indexed_args(torch.float16, x, w, idx, out, False)
    rc = _lib().linear_f16_indexed_noalloc(*args, _stream_handle(stream, x, w, idx, out))
    _check(rc, "linear_f16_indexed_noalloc")
    return out


def linear_f16_indexed(x, w, idx, out=None, stream=None, workspace=None):
    """Indexed contraction: row m of x against expert table w[idx[m]] ([K, N]); rows whose
    idx has no expert keep out's contents.  workspace: a uint8 device tensor of at least
    indexed_workspace_bytes(E, M) bytes (allocated per call when None)."""
    return _indexed_call(torch.float16, x, w, idx, out, False, stream, workspace)


def linear_bf16_indexed(x, w, idx, out=None, stream=None, workspace=None):
    return _indexed_call(torch.bfloat16, x, w, idx, out, False, stream, workspace)


def linear_f16_indexed_f32out(x, w, idx, out=None, stream=None, workspace=None):
    return _indexed_call(torch.float16, x, w, idx, out, True, stream, workspace)


def linear_bf16_indexed_f32out(x, w, idx, out=None, stream=None, workspace=None):
    return _indexed_call(torch.bfloat16, x, w, idx, out, True, stream, workspace)


def _launch_stream(stream, *tensors):
    """_stream_handle's checks for tensors on one device and the current stream, the usual
    call, at less host time; anything else goes through it."""
    if stream is None:
        devices = {t.get_device() for t in tensors if t is not None}    # -1 on the host
        if len(devices) == 1:
            index = devices.pop()
            if index >= 0 and index == torch._C._cuda_getDevice():
                return torch._C._cuda_getCurrentRawStream(index)
    return _stream_handle(stream, *tensors)


def _many_launch_stream(stream, *lists):
    """_launch_stream for lists of many tensors."""
    if stream is None:
        stream_of = _current_stream(set(map(torch.Tensor.get_device, itertools.chain(*lists))))
        if stream_of is not None:
            return stream_of
    return _stream_handle(stream, *itertools.chain(*lists))


def _current_stream(devices):
    """The raw current stream where the devices (-1: the host) are the current one alone, else None."""
    if len(devices) == 1:
        index = devices.pop()
        if index >= 0 and index == torch._C._cuda_getDevice():
            return torch._C._cuda_getCurrentRawStream(index)
    return None


_NO_CONTEXT = contextlib.nullcontext()


def _on(stream, device):
    """A context in which new tensors belong to the stream of the launch, so that their
    memory is not reused by other work before the launch has run."""
    if stream is None or device.type != "cuda":
        return _NO_CONTEXT
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        if handle == 0:
            stream = torch.cuda.default_stream(device)
        else:
            stream = torch.cuda.ExternalStream(handle, device=device)
    return torch.cuda.stream(stream)


def _operand(t, name, dtype, shape):
    """Pointer and row stride of a tensor that must have this type and shape."""
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    return _mat(t, name, dtype)


def _output(t, name, dtype, shape, like):
    """The output tensor (a new one on the device of `like` when not given), its pointer and row stride."""
    if t is None:
        t = like.new_empty(shape) if like.dtype == dtype else like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr(), max(shape[1], 1)
    return (t, *_operand(t, name, dtype, shape))


@functools.lru_cache(maxsize=None)
def _entry(name):
    return getattr(_lib(), name)


def _scratch(workspace, need, device):
    """The call's workspace, its address and its size: the caller's uint8 tensor, or a new one
    where the call needs any."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or workspace.numel() < need or (
            workspace.numel() > 1 and workspace.stride(0) != 1):
        raise ValueError("workspace must be a contiguous uint8 tensor of at least %d bytes" % need)
    return workspace, workspace.data_ptr(), workspace.numel()


_GATED = {t: "linear_%s_gated" % t for t in ("f16", "bf16")}
_GATED_BACKWARD = {t: "linear_%s_gated_backward" % t for t in ("f16", "bf16")}
_BACKWARD_INPUT = {t: "linear_%s_backward_input" % t for t in ("f16", "bf16")}
_BACKWARD_WEIGHT = {(t, f): "linear_%s_backward_weight%s" % (t, "_f32out" if f else "")
                    for t in ("f16", "bf16") for f in (False, True)}


@functools.lru_cache(maxsize=256)
def gated_forward_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of device workspace a gated forward call needs: 0 where K is a multiple of 8."""
    n = _lib().linear_gated_forward_workspace_bytes(M, N, K)
    if n < 0:
        raise ValueError("M=%d, N=%d, K=%d out of range" % (M, N, K))
    return n


def _gated_call(tag, dtype, x, wg, wu, act, keep, out, gate, up, workspace, stream):
    if x.dim() != 2 or wg.dim() != 2:
        raise ValueError("x must be [M, K] and wg, wu [N, K]")
    M, K = x.shape
    N = wg.shape[0]
    xp, ldx = _mat(x, "x", dtype)
    gp, ldg = _operand(wg, "wg", dtype, (N, K))
    up_, ldu = _operand(wu, "wu", dtype, (N, K))
    handle = _launch_stream(stream, x, wg, wu, out, gate, up, workspace)
    with _on(stream, x.device):
        out, hp, ldh = _output(out, "out", dtype, (M, N), x)
        kept = []
        for name, t in (("gate", gate), ("up", up)):
            kept += _output(t, name, dtype, (M, N), x) if keep or t is not None else (None, None, 0)
        workspace, wsp, wsn = _scratch(workspace, gated_forward_workspace_bytes(M, N, K), x.device)
    name = _GATED[tag]
    rc = _entry(name)(xp, ldx, gp, ldg, up_, ldu, int(act), hp, ldh, kept[1], kept[2], kept[4], kept[5], M, N, K, wsp, wsn,
                      handle)
    _check(rc, name)
    return (out, kept[0], kept[3]) if keep else out


def linear_f16_gated(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, act: int = EPI_SILU, keep: bool = False,
                     out=None, gate=None, up=None, workspace=None, stream=None):
    """h = act(x @ wg.T) * (x @ wu.T) in one kernel, rounded once to binary16 (x [M, K], wg and wu
    [N, K]; act EPI_SILU, EPI_GELU_TANH or EPI_GELU_ERF).  keep: also return the two rounded
    projections, which the backward call takes: (h, gate, up).  out, gate, up: tensors to write.  workspace: a uint8 device
    tensor of at least gated_forward_workspace_bytes(M, N, K) bytes (allocated per call when None)."""
    return _gated_call("f16", torch.float16, x, wg, wu, act, keep, out, gate, up, workspace, stream)


def linear_bf16_gated(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, act: int = EPI_SILU, keep: bool = False,
                      out=None, gate=None, up=None, workspace=None, stream=None):
    """linear_f16_gated on bfloat16 operands and outputs."""
    return _gated_call("bf16", torch.bfloat16, x, wg, wu, act, keep, out, gate, up, workspace, stream)


@functools.lru_cache(maxsize=256)
def gated_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of device workspace a gated backward call needs."""
    n = _lib().linear_gated_workspace_bytes(M, N, K)
    if n < 0:
        raise ValueError("M=%d, N=%d, K=%d out of range" % (M, N, K))
    return n


def _gated_backward_call(tag, dtype, dh, x, wg, wu, gate, up, act, need_dx, need_dw, dx, dwg, dwu, workspace, stream):
    if x.dim() != 2 or wg.dim() != 2:
        raise ValueError("x must be [M, K] and wg, wu [N, K]")
    need_dx, need_dw = need_dx or dx is not None, need_dw or dwg is not None or dwu is not None
    if not (need_dx or need_dw):
        raise ValueError("nothing to compute: neither dx nor the weights' gradients are wanted")
    M, K = x.shape
    N = wg.shape[0]
    args = []
    for name, t, shape in (("dh", dh, (M, N)), ("x", x, (M, K)), ("wg", wg, (N, K)), ("wu", wu, (N, K)),
                           ("gate", gate, (M, N)), ("up", up, (M, N))):
        args += _operand(t, name, dtype, shape)
    handle = _launch_stream(stream, dh, x, wg, wu, gate, up, dx, dwg, dwu, workspace)
    none = (None, None, 0)
    with _on(stream, x.device):
        dx, *dxa = _output(dx, "dx", dtype, (M, K), x) if need_dx else none
        dwg, *dga = _output(dwg, "dwg", dtype, (N, K), x) if need_dw else none
        dwu, *dua = _output(dwu, "dwu", dtype, (N, K), x) if need_dw else none
        workspace, wsp, wsn = _scratch(workspace, gated_workspace_bytes(M, N, K), x.device)
    name = _GATED_BACKWARD[tag]
    rc = _entry(name)(*args, int(act), *dxa, *dga, *dua, M, N, K, wsp, wsn, handle)
    _check(rc, name)
    return dx, dwg, dwu


def linear_f16_gated_backward(dh, x, wg, wu, gate, up, act: int = EPI_SILU, need_dx: bool = True, need_dw: bool = True,
                              dx=None, dwg=None, dwu=None, workspace=None, stream=None):
    """The gated block's gradients (dx [M, K], dwg [N, K], dwu [N, K]) from dh [M, N] and the
    projections that the forward call kept; those not wanted are None.  workspace: a uint8 device
    tensor of at least gated_workspace_bytes(M, N, K) bytes (allocated per call when None)."""
    return _gated_backward_call("f16", torch.float16, dh, x, wg, wu, gate, up, act, need_dx, need_dw, dx, dwg, dwu,
                                workspace, stream)


def linear_bf16_gated_backward(dh, x, wg, wu, gate, up, act: int = EPI_SILU, need_dx: bool = True, need_dw: bool = True,
                               dx=None, dwg=None, dwu=None, workspace=None, stream=None):
    """linear_f16_gated_backward on bfloat16 operands and outputs."""
    return _gated_backward_call("bf16", torch.bfloat16, dh, x, wg, wu, gate, up, act, need_dx, need_dw, dx, dwg, dwu,
                                workspace, stream)


@functools.lru_cache(maxsize=256)
def backward_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of device workspace the layer's backward calls need."""
    n = _lib().linear_backward_workspace_bytes(M, N, K)
    if n < 0:
        raise ValueError("M=%d, N=%d, K=%d out of range" % (M, N, K))
    return n


def _backward_input_call(tag, dtype, dy, weight, out, workspace, stream):
    if dy.dim() != 2 or weight.dim() != 2:
        raise ValueError("dy must be [M, N] and weight [N, K]")
    M, N = dy.shape
    K = weight.shape[1]
    yp, ldy = _mat(dy, "dy", dtype)
    wp, ldw = _operand(weight, "weight", dtype, (N, K))
    handle = _launch_stream(stream, dy, weight, out, workspace)
    with _on(stream, dy.device):
        out, xp, ldx = _output(out, "out", dtype, (M, K), dy)
        workspace, wsp, wsn = _scratch(workspace, backward_workspace_bytes(M, N, K), dy.device)
    name = _BACKWARD_INPUT[tag]
    rc = _entry(name)(yp, ldy, wp, ldw, xp, ldx, M, N, K, wsp, wsn, handle)
    _check(rc, name)
    return out


def linear_f16_backward_input(dy: torch.Tensor, weight: torch.Tensor, out=None, workspace=None, stream=None):
    """dx = dy @ weight (dy [M, N], weight [N, K], float16), FP32 sums rounded once.  workspace: a uint8
    device tensor of at least backward_workspace_bytes(M, N, K) bytes (allocated per call when None)."""
    return _backward_input_call("f16", torch.float16, dy, weight, out, workspace, stream)


def linear_bf16_backward_input(dy: torch.Tensor, weight: torch.Tensor, out=None, workspace=None, stream=None):
    """linear_f16_backward_input on bfloat16 operands."""
    return _backward_input_call("bf16", torch.bfloat16, dy, weight, out, workspace, stream)


def _backward_weight_call(tag, dtype, f32, dy, x, bias, accumulate, out, db, workspace, stream):
    if dy.dim() != 2 or x.dim() != 2:
        raise ValueError("dy must be [M, N] and x [M, K]")
    M, N = dy.shape
    K = x.shape[1]
    bias = bias or db is not None
    if accumulate and (out is None or (bias and db is None)):
        raise ValueError("accumulate adds to tensors that are there: give out (and db)")
    yp, ldy = _mat(dy, "dy", dtype)
    xp, ldx = _operand(x, "x", dtype, (M, K))
    handle = _launch_stream(stream, dy, x, out, db, workspace)
    odt = torch.float32 if f32 else dtype
    with _on(stream, dy.device):
        out, wp, ldw = _output(out, "out", odt, (N, K), dy)
        if bias and db is None:
            db = torch.empty((N,), dtype=odt, device=dy.device)
        workspace, wsp, wsn = _scratch(workspace, backward_workspace_bytes(M, N, K), dy.device)
    if bias and (db.dtype != odt or tuple(db.shape) != (N,) or (N > 1 and db.stride(0) != 1)):
        raise ValueError("db must be a contiguous %s [N] tensor" % odt)
    bp = db.data_ptr() if bias else None
    name = _BACKWARD_WEIGHT[tag, f32]
    flag = (int(bool(accumulate)),) if f32 else ()
    rc = _entry(name)(yp, ldy, xp, ldx, wp, ldw, bp, *flag, M, N, K, wsp, wsn, handle)
    _check(rc, name)
    return out, (db if bias else None)


def linear_f16_backward_weight(dy: torch.Tensor, x: torch.Tensor, bias: bool = False, out=None, db=None, workspace=None,
                               stream=None):
    """(dw, db): dw = dy.T @ x [N, K] and, with bias, db = dy.sum(0) [N] (else None); dy [M, N], x [M, K],
    float16, FP32 sums rounded once.  workspace as for linear_f16_backward_input."""
    return _backward_weight_call("f16", torch.float16, False, dy, x, bias, False, out, db, workspace, stream)


def linear_bf16_backward_weight(dy: torch.Tensor, x: torch.Tensor, bias: bool = False, out=None, db=None, workspace=None,
                                stream=None):
    """linear_f16_backward_weight on bfloat16 operands."""
    return _backward_weight_call("bf16", torch.bfloat16, False, dy, x, bias, False, out, db, workspace, stream)


def linear_f16_backward_weight_f32out(dy: torch.Tensor, x: torch.Tensor, bias: bool = False, accumulate: bool = False,
                                      out=None, db=None, workspace=None, stream=None):
    """linear_f16_backward_weight with the unrounded FP32 sums; accumulate: added to what out (and db) hold."""
    return _backward_weight_call("f16", torch.float16, True, dy, x, bias, accumulate, out, db, workspace, stream)


def linear_bf16_backward_weight_f32out(dy: torch.Tensor, x: torch.Tensor, bias: bool = False, accumulate: bool = False,
                                       out=None, db=None, workspace=None, stream=None):
    """linear_f16_backward_weight_f32out on bfloat16 operands."""
    return _backward_weight_call("bf16", torch.bfloat16, True, dy, x, bias, accumulate, out, db, workspace, stream)


_CROSS_ENTROPY = {t: "linear_%s_cross_entropy" % t for t in ("f16", "bf16")}
_CROSS_ENTROPY_BACKWARD = {(t, f): "linear_%s_cross_entropy_backward%s" % (t, "_f32out" if f else "")
                           for t in ("f16", "bf16") for f in (False, True)}


@functools.lru_cache(maxsize=256)
def cross_entropy_workspace_bytes(M: int, N: int, K: int, aligned: bool = False) -> int:
    """Bytes of device workspace a cross entropy call needs; aligned: where x and weight are 16-byte aligned and
    their row strides multiples of 8, so that neither is copied."""
    lib = _lib()
    n = (lib.linear_cross_entropy_workspace_bytes_aligned if aligned else lib.linear_cross_entropy_workspace_bytes)(M, N, K)
    if n < 0:
        raise ValueError("M=%d, N=%d, K=%d out of range" % (M, N, K))
    return n


@functools.lru_cache(maxsize=256)
def cross_entropy_backward_workspace_bytes(M: int, N: int, K: int, aligned: bool = False) -> int:
    """Bytes of device workspace a cross entropy backward call needs; aligned: where weight is 16-byte aligned and
    its row stride a multiple of 8, so that it is not copied."""
    lib = _lib()
    n = (lib.linear_cross_entropy_backward_workspace_bytes_aligned if aligned
         else lib.linear_cross_entropy_backward_workspace_bytes)(M, N, K)
    if n < 0:
        raise ValueError("M=%d, N=%d, K=%d out of range" % (M, N, K))
    return n


CROSS_ENTROPY_MAX_K = (1 << 22) - 8


def _in_place(p, rows, ld):
    """Whether rows of a multiple of 8 values are read where they are (see the workspaces)."""
    return not p or (p % 16 == 0 and (rows <= 1 or (ld % 8 == 0 and ld <= CROSS_ENTROPY_MAX_K)))


def _vector(t, name, dtype, n):
    """Pointer of a contiguous vector of n values (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous %s tensor of %d values" % (name, dtype, n))
    return t.data_ptr()


def _new_scratch(need, device):
    """A new workspace on a GPU and its address, at less host time than _scratch."""
    made = _marshal().scratch(need, device)
    return made if made is not None else _scratch(None, need, torch.device("cuda", device))[:2]


def _cross_entropy_call(tag, dtype, x, weight, target, b, loss, lse, workspace, stream):
    name = _CROSS_ENTROPY[tag]
    if stream is None and workspace is None and loss is None and lse is None:
        packed = _marshal().cross_entropy(x, weight, target, b, tag == "bf16")    # None: not the plain case
        if packed is not None:
            device, M, N, K, loss, lse, args = packed
            need = cross_entropy_workspace_bytes(M, N, K, (args[0] | args[2]) % 16 == 0)
            workspace, wsp = _new_scratch(need, device)
            _check(_entry(name)(*args, M, N, K, wsp, need, torch._C._cuda_getCurrentRawStream(device)), name)
            return loss, lse
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [M, K] and weight [N, K]")
    M, K = x.shape
    N = weight.shape[0]
    xp, ldx = _mat(x, "x", dtype)
    wp, ldw = _operand(weight, "weight", dtype, (N, K))
    tp = _vector(target, "target", torch.int64, M)
    bp = _vector(b, "b", dtype, N)
    handle = _launch_stream(stream, x, weight, target, b, loss, lse, workspace)
    with _on(stream, x.device):
        if loss is None:
            loss = torch.empty(M, dtype=torch.float32, device=x.device)
        if lse is None:
            lse = torch.empty(M, dtype=torch.float32, device=x.device)
        need = cross_entropy_workspace_bytes(M, N, K, _in_place(xp, M, ldx) and _in_place(wp, N, ldw))
        workspace, wsp, wsn = _scratch(workspace, need, x.device)
    rc = _entry(name)(xp, ldx, wp, ldw, bp, tp, _vector(loss, "loss", torch.float32, M), _vector(lse, "lse", torch.float32, M),
                      M, N, K, wsp, wsn, handle)
    _check(rc, name)
    return loss, lse


def linear_f16_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, b=None, loss=None, lse=None,
                             workspace=None, stream=None):
    """(loss, lse) of the head x @ weight.T (+ b) (x [M, K], weight [N, K], b [N], float16; target int64 [M]):
    lse = log sum exp of a row's logits, loss = lse - the target's logit, float32 [M]; a target outside [0, N)
    (-100, say) gives loss 0.  The logits are never stored.  loss, lse: tensors to write.  workspace: a uint8
    device tensor of at least cross_entropy_workspace_bytes(M, N, K, aligned) bytes (allocated per call when None)."""
    return _cross_entropy_call("f16", torch.float16, x, weight, target, b, loss, lse, workspace, stream)


def linear_bf16_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, b=None, loss=None, lse=None,
                              workspace=None, stream=None):
    """linear_f16_cross_entropy on bfloat16 operands."""
    return _cross_entropy_call("bf16", torch.bfloat16, x, weight, target, b, loss, lse, workspace, stream)


def _cross_entropy_backward_call(tag, dtype, f32, dloss, x, weight, target, lse, b, dlse, need_dx, need_dw, bias, accumulate,
                                 dx, dw, db, workspace, stream):
    name = _CROSS_ENTROPY_BACKWARD[tag, f32]
    need_dx, need_dw = bool(need_dx or dx is not None), bool(need_dw or dw is not None)
    bias = db is not None or (need_dw and b is not None if bias is None else bool(bias))
    if stream is None and workspace is None and dx is None and dw is None and db is None and not accumulate and (
            need_dx or need_dw or bias):
        packed = _marshal().cross_entropy_backward(dloss, x, weight, target, lse, b, dlse, need_dx, need_dw, bias,
                                                   tag == "bf16", f32)
        if packed is not None:
            device, M, N, K, dx, dw, db, args = packed
            need = cross_entropy_backward_workspace_bytes(M, N, K, args[4] % 16 == 0)
            workspace, wsp = _new_scratch(need, device)
            flag = (0,) if f32 else ()
            _check(_entry(name)(*args, *flag, M, N, K, wsp, need, torch._C._cuda_getCurrentRawStream(device)), name)
            return dx, dw, db
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [M, K] and weight [N, K]")
    if not (need_dx or need_dw or bias):
        raise ValueError("nothing to compute: no gradient is wanted")
    if accumulate and ((need_dw and dw is None) or (bias and db is None)):
        raise ValueError("accumulate adds to tensors that are there: give dw (and db)")
    M, K = x.shape
    N = weight.shape[0]
    xp, ldx = _mat(x, "x", dtype)
    wp, ldw = _operand(weight, "weight", dtype, (N, K))
    vectors = [_vector(t, n, torch.float32, M) for t, n in ((dloss, "dloss"), (dlse, "dlse"), (lse, "lse"))]
    tp = _vector(target, "target", torch.int64, M)
    bp = _vector(b, "b", dtype, N)
    handle = _launch_stream(stream, dloss, dlse, x, weight, target, lse, b, dx, dw, db, workspace)
    none = (None, None, 0)
    odt = torch.float32 if f32 else dtype
    with _on(stream, x.device):
        dx, *dxa = _output(dx, "dx", dtype, (M, K), x) if need_dx else none
        dw, *dwa = _output(dw, "dw", odt, (N, K), x) if need_dw else none
        if bias and db is None:
            db = torch.empty(N, dtype=odt, device=x.device)
        need = cross_entropy_backward_workspace_bytes(M, N, K, _in_place(wp, N, ldw))
        workspace, wsp, wsn = _scratch(workspace, need, x.device)
    flag = (int(bool(accumulate)),) if f32 else ()
    rc = _entry(name)(vectors[0], vectors[1], xp, ldx, wp, ldw, bp, tp, vectors[2], *dxa, *dwa,
                      _vector(db, "db", odt, N) if bias else None, *flag, M, N, K, wsp, wsn, handle)
    _check(rc, name)
    return dx, dw, (db if bias else None)


def linear_f16_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                                      lse: torch.Tensor, b=None, dlse=None, need_dx: bool = True, need_dw: bool = True,
                                      bias=None, dx=None, dw=None, db=None, workspace=None, stream=None):
    """(dx [M, K], dw [N, K], db [N]) of linear_f16_cross_entropy from dloss and, where lse enters the objective
    too, dlse (float32 [M]); lse is the forward call's.  Those not wanted are None; db is wanted with b and dw
    unless bias says otherwise.  workspace: a uint8 device tensor of at least
    cross_entropy_backward_workspace_bytes(M, N, K, aligned) bytes (allocated per call when None)."""
    return _cross_entropy_backward_call("f16", torch.float16, False, dloss, x, weight, target, lse, b, dlse, need_dx, need_dw,
                                        bias, False, dx, dw, db, workspace, stream)


def linear_bf16_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                                       lse: torch.Tensor, b=None, dlse=None, need_dx: bool = True, need_dw: bool = True,
                                       bias=None, dx=None, dw=None, db=None, workspace=None, stream=None):
    """linear_f16_cross_entropy_backward on bfloat16 operands and outputs."""
    return _cross_entropy_backward_call("bf16", torch.bfloat16, False, dloss, x, weight, target, lse, b, dlse, need_dx,
                                        need_dw, bias, False, dx, dw, db, workspace, stream)


def linear_f16_cross_entropy_backward_f32out(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                                             lse: torch.Tensor, b=None, dlse=None, need_dx: bool = True, need_dw: bool = True,
                                             bias=None, accumulate: bool = False, dx=None, dw=None, db=None, workspace=None,
                                             stream=None):
    """linear_f16_cross_entropy_backward with dw and db as unrounded FP32 sums; accumulate: added to what dw (and
    db) hold."""
    return _cross_entropy_backward_call("f16", torch.float16, True, dloss, x, weight, target, lse, b, dlse, need_dx, need_dw,
                                        bias, accumulate, dx, dw, db, workspace, stream)


def linear_bf16_cross_entropy_backward_f32out(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                              target: torch.Tensor, lse: torch.Tensor, b=None, dlse=None,
                                              need_dx: bool = True, need_dw: bool = True, bias=None, accumulate: bool = False,
                                              dx=None, dw=None, db=None, workspace=None, stream=None):
    """linear_f16_cross_entropy_backward_f32out on bfloat16 operands."""
    return _cross_entropy_backward_call("bf16", torch.bfloat16, True, dloss, x, weight, target, lse, b, dlse, need_dx,
                                        need_dw, bias, accumulate, dx, dw, db, workspace, stream)


# linear_tensor.type (include/linear_amd.h, LINEAR_TYPE_*)
_TENSOR_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_dtype_of = operator.attrgetter("dtype")
GRAD_MAX_TENSORS = 65536


@functools.lru_cache(maxsize=256)
def grad_workspace_bytes(count: int) -> int:
    """Bytes of device workspace a norm over `count` tensors needs."""
    n = _lib().linear_grad_workspace_bytes(count)
    if n < 0:
        raise ValueError("at most %d tensors" % GRAD_MAX_TENSORS)
    return n


def _tensor_table(tensors, name):
    """The tensors as an array of linear_tensor (five 64-bit fields each): contiguous ones of any
    shape, as one row, and matrices with unit inner stride."""
    n = len(tensors)
    types = list(map(_dtype_of, tensors))
    try:
        if n and types.count(types[0]) == n:          # (the usual case, at less host time)
            kinds = array.array("q", (_TENSOR_TYPES[types[0]],)) * n
        else:
            kinds = array.array("q", map(_TENSOR_TYPES.__getitem__, types))
    except KeyError as e:
        raise TypeError("%s must be float16, bfloat16 or float32, got %s" % (name, e)) from None
    sizes = array.array("q", map(torch.Tensor.numel, tensors))
    table = array.array("q", (0, 1, 0, 0, 0)) * n
    table[0::5] = array.array("q", map(torch.Tensor.data_ptr, tensors))
    table[2::5] = sizes
    table[3::5] = sizes
    table[4::5] = kinds
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        for i, t in enumerate(tensors):
            if not t.is_contiguous():
                if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < t.shape[1]:
                    raise ValueError("%s must be contiguous, or matrices with unit inner stride" % name)
                _by_rows(table, i, t)
    return table


def _by_rows(table, i, t):
    table[5 * i + 1:5 * i + 4] = array.array("q", (t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]))


def linear_grad_norm(grads, out=None, workspace=None, stream=None) -> torch.Tensor:
    """The global 2-norm of the gradients (a sequence of float16, bfloat16 and float32 tensors), as a
    float32 [1] tensor.  workspace: a uint8 device tensor of at least grad_workspace_bytes(len(grads))
    bytes (allocated per call when None)."""
    grads = list(grads)
    table = _tensor_table(grads, "grads")
    if not grads and out is None:
        raise ValueError("no gradients and no out: the device is not known")
    handle = _launch_stream(stream, *grads, out, workspace)
    device = (grads[0] if grads else out).device
    with _on(stream, device):
        if out is None:
            out = torch.empty(1, dtype=torch.float32, device=device)
        workspace, wsp, wsn = _scratch(workspace, grad_workspace_bytes(len(grads)), device)
    if out.dtype != torch.float32 or out.numel() != 1:
        raise ValueError("out must be a float32 tensor of one value")
    rc = _lib().linear_grad_norm(table.buffer_info()[0], len(grads), out.data_ptr(), wsp, wsn, handle)
    _check(rc, "linear_grad_norm")
    return out


def linear_grad_clip(grads, norm: torch.Tensor, max_norm: float, out=None, stream=None):
    """The gradients times min(1, max_norm / (norm + 1e-6)), rounded to their types: into the tensors
    of out (the same sizes and types), or in place.  norm: the float32 tensor of linear_grad_norm."""
    grads = list(grads)
    table = _tensor_table(grads, "grads")
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be a float32 tensor of one value")
    outs = None
    if out is not None:
        out = list(out)
        outs = _tensor_table(out, "out")
        if len(out) != len(grads) or outs[4::5] != table[4::5]:
            raise ValueError("out must have as many tensors as grads, of the same types")
        if outs[1::5] != table[1::5] or outs[2::5] != table[2::5]:
            if any(a.shape != b.shape for a, b in zip(out, grads)):
                raise ValueError("out must have the gradients' shapes")
            # a matrix with padded rows on one side is described by its rows on both
            for i, (a, b) in enumerate(zip(grads, out)):
                if outs[5 * i + 1] != table[5 * i + 1]:
                    _by_rows(table, i, a)
                    _by_rows(outs, i, b)
    handle = _launch_stream(stream, *grads, norm, *(out or ()))
    rc = _lib().linear_grad_clip(table.buffer_info()[0], outs.buffer_info()[0] if outs else None, len(grads),
                                 norm.data_ptr(), float(max_norm), handle)
    _check(rc, "linear_grad_clip")
    return out if out is not None else grads


ADAMW_BLOCK = 32


def adamw_state(param: torch.Tensor, bits: int = 32) -> torch.Tensor:
    """A first or second moment of zeros for linear_adamw: float32 of the parameter's shape, or, with
    bits 8, a uint8 vector of its codes and its blocks' powers of two."""
    if bits == 32:
        return torch.zeros(param.shape, dtype=torch.float32, device=param.device)
    n = _lib().linear_adamw_state_bytes(param.numel(), bits)
    if n < 0:
        raise ValueError("bits must be 8 or 32")
    return torch.zeros(n, dtype=torch.uint8, device=param.device)


def _same_sizes(tables, tensors, names):
    """The tables describe tensors of the first one's shapes; a matrix with padded rows in one is
    described by its rows in all."""
    if any(len(t) != len(tables[0]) for t in tables):
        raise ValueError("%s must have as many tensors as %s" % (" and ".join(names[1:]), names[0]))
    first = tables[0]
    for ts, name in zip(tensors[1:], names[1:]):
        if not all(map(torch.Tensor.is_same_size, ts, tensors[0])):
            raise ValueError("%s must have the shapes of %s" % (name, names[0]))
    if all(t[1::5] == first[1::5] for t in tables):
        return
    for i in range(len(tensors[0])):
        if any(t[5 * i + 1] != first[5 * i + 1] for t in tables):
            for t, ts in zip(tables, tensors):
                if t[5 * i + 1] == 1:
                    _by_rows(t, i, ts[i])


def _state_pointers(states, sizes, eight, name):
    """The states' addresses, after a check of their types and sizes."""
    want = torch.uint8 if eight else torch.float32
    if len(states) != len(sizes) or set(map(_dtype_of, states)) - {want}:
        raise ValueError("%s must have a state for each tensor, all float32 or all uint8" % name)
    held = [n + -(-n // ADAMW_BLOCK) for n in sizes] if eight else sizes
    if list(map(torch.Tensor.numel, states)) != list(held) or not all(map(torch.Tensor.is_contiguous, states)):
        raise ValueError("%s must be contiguous, of adamw_state's sizes" % name)
    return array.array("q", map(torch.Tensor.data_ptr, states))


def _device_scalar(t, name, dtype):
    if t.dtype != dtype or t.numel() != 1:
        raise ValueError("%s must be a %s tensor of one value" % (name, dtype))
    return t.data_ptr()


def _adamw_tables(params, grads, m, v, copies):
    """The tables of an AdamW call's tensors, after checks that say what is wrong."""
    tensors, names = [params, grads], ["params", "grads"]
    if copies is not None:
        tensors.append(copies)
        names.append("copies")
    tables = [_tensor_table(t, n) for t, n in zip(tensors, names)]
    _same_sizes(tables, tensors, names)
    eight = bool(m) and m[0].dtype == torch.uint8
    sizes = list(map(torch.Tensor.numel, params))
    mp, vp = _state_pointers(m, sizes, eight, "m"), _state_pointers(v, sizes, eight, "v")
    return (*(t.tobytes() for t in tables), *(() if copies is not None else (None,)), mp.tobytes(), vp.tobytes(), eight)


def linear_adamw(params, grads, m, v, *, lr, step, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01, norm=None, max_norm=None, copies=None, stream=None):
    """One AdamW step, in place, over a sequence of parameters (float16, bfloat16, float32) and their gradients (of any
    of these types).  m, v: the moments of each (adamw_state: all float32 or all 8-bit).  step: 1 for the first update.
    norm, max_norm: linear_grad_norm's tensor and the norm that gradients are clipped to, within the same pass.
    copies: 16-bit tensors that the new parameters are also rounded into.  lr and step may be device tensors of one
    value (float32, int64), read when the step runs: a captured step then follows them.  Returns params."""
    params, grads, m, v = list(params), list(grads), list(m), list(v)
    copies = None if copies is None else list(copies)
    scalars = [t for t in (norm, lr, step) if isinstance(t, torch.Tensor)]
    packed = _marshal().adamw(params, grads, m, v, copies)    # None: not the plain case
    if packed is not None:
        pt, gt, ct, mp, vp, eight, device = packed
        if stream is None and all(t.get_device() == device for t in scalars):
            handle = _current_stream({device})
        else:
            handle = None
    else:
        pt, gt, ct, mp, vp, eight = _adamw_tables(params, grads, m, v, copies)
        handle = None
    if handle is None:
        handle = _many_launch_stream(stream, params, grads, m, v, scalars, copies or ())
    if (norm is None) != (max_norm is None):
        raise ValueError("norm and max_norm belong together")
    o = _AdamwOptions(beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, state_bits=8 if eight else 32)
    if norm is not None:
        o.norm, o.max_norm = _device_scalar(norm, "norm", torch.float32), max_norm
    if isinstance(lr, torch.Tensor):
        o.device_lr = _device_scalar(lr, "lr", torch.float32)
    else:
        o.lr = lr
    if isinstance(step, torch.Tensor):
        o.device_step = _device_scalar(step, "step", torch.int64)
    else:
        o.step = step
    rc = _lib().linear_adamw(pt, gt, mp, vp, ct, len(params), ctypes.byref(o), handle)
    _check(rc, "linear_adamw")
    return params


def linear_adamw_values(states, second: bool, out=None, like=None, stream=None):
    """The numbers that 8-bit moments stand for (second: second moments), exactly: into the bfloat16 or float32 tensors
    of out, or into new bfloat16 tensors of the shapes of `like` (the parameters)."""
    states = list(states)
    if out is None:
        if like is None:
            raise ValueError("give out, or like: a state does not know its parameter's shape")
        like = list(like)
        with _on(stream, like[0].device if like else torch.device("cpu")):
            out = [torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) for t in like]
    out = list(out)
    packed = _marshal().states(out, states)
    handle = None
    if packed is not None:
        table, sp, device = packed
        handle = _current_stream({device}) if stream is None else None
    else:
        table = _tensor_table(out, "out").tobytes()
        sp = _state_pointers(states, list(map(torch.Tensor.numel, out)), True, "states").tobytes()
    if handle is None:
        handle = _many_launch_stream(stream, states, out)
    rc = _lib().linear_adamw_values(table, sp, int(bool(second)), len(out), handle)
    _check(rc, "linear_adamw_values")
    return out


def linear_f16_plan(x: torch.Tensor, weight: torch.Tensor, b: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, path: int = PATH_AUTO) -> dict:
    """The kernel and tile a call would use (host only): path, tile_m/tile_n/tile_k,
    threads, vector_io, grid; for a GEMM split by columns into two launches also
    split_n (the second launch's first column), tile_m2/tile_n2 and grid2."""
    if out is None:
        out = torch.empty((x.shape[0], weight.shape[0]), dtype=torch.float16, device="meta")
        yp, ldy = 0x100000000, max(weight.shape[0], 1)
    else:
        yp, ldy = _mat(out, "out", out.dtype)
    xp, ldx = _mat(x, "x", x.dtype)
    wp, ldw = _mat(weight, "weight", weight.dtype)
    p = _Plan()
    rc = _lib().linear_f16_plan(xp, ldx, wp, ldw, None if b is None else b.data_ptr(), yp, ldy,
                                x.shape[0], weight.shape[0], x.shape[1], int(path), ctypes.byref(p))
    _check(rc, "linear_f16_plan")
    return {f: getattr(p, f) for f, _ in _Plan._fields_}


def linear_gated_backward_plan(M: int, N: int, K: int) -> dict:
    """How a gated backward call of these sizes forms its products (host only, aligned layouts):
    dx and dw, each with tile_m, tile_n, stages, sets, splits and, where the columns from split_c
    on are a second launch, tile_m2 and tile_n2; joint: both in one launch; two_words: dg and du
    are kept as two words."""
    p = _GatedPlan()
    _check(_lib().linear_gated_backward_plan(M, N, K, ctypes.byref(p)), "linear_gated_backward_plan")
    parts = {n: {f: getattr(getattr(p, n), f) for f, _ in _ProductPlan._fields_} for n in ("dx", "dw")}
    return {**parts, "joint": bool(p.joint), "two_words": bool(p.two_words)}


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """Convenience: the bias call when a bias is given, the projection alone otherwise;
    float16 or bfloat16 by x's dtype."""
    if x.dtype == torch.bfloat16:
        if bias is None:
            return linear_bf16_nobias(x, weight, out=out)
        return linear_bf16(x, weight, bias, out=out)
    if bias is None:
        return linear_f16_nobias(x, weight, out=out)
    return linear_f16(x, weight, bias, out=out)
