"""GB300 linear layer: Y = act(X . W^T + bias), W stored out x in.

A thin ctypes binding over the C ABI in ``include/lin.h`` (library
``_build/liblin.so``, built by :func:`build`). The binding only marshals
arguments: torch supplies device memory and the current CUDA stream, and every
step of the multiply runs in this package's CUDA kernels. There is no CPU path:
if the library is missing or the GPU call fails, an exception is raised.

Calls run on the current stream, or on ``stream`` (a stream object or a raw handle): their
results are then that stream's memory, as if made with it as the current one, and may be
used on the current stream too once it waits for them.

    import torch, transformer_linear_layer_gb300 as tll
    y = tll.forward(x_bf16, w_bf16, bias_fp32, epilogue="gelu")   # -> bf16
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

from .build import LIB as _LIB_PATH
from .build import TIMELINE_LIB as _TIMELINE_LIB_PATH
from .build import build

__all__ = [
    "LinError", "Context", "Plan", "forward", "forward_plan", "plan_query", "plan_make", "build",
    "backward_data", "backward_weight", "gelu_backward", "attention_forward", "attention_backward",
    "TokenLogprobs", "token_logprobs", "distill_forward", "distill_backward", "distill_forward_backward",
    "Rotary", "rotary_forward", "rotary_backward", "KVCache", "KVBatch", "cache_append", "paged_attention",
    "library", "PREC_FP32", "PREC_TF32", "PREC_BF16", "EPI_NONE", "EPI_GELU_TANH",
    "KERNEL_NONE", "KERNEL_FILL", "KERNEL_SKINNY", "KERNEL_FFMA", "KERNEL_TC", "KERNEL_GEMV",
]

PREC_FP32, PREC_TF32, PREC_BF16 = 0, 1, 2
EPI_NONE, EPI_GELU_TANH = 0, 1
KERNEL_NONE, KERNEL_FILL, KERNEL_SKINNY, KERNEL_FFMA, KERNEL_TC, KERNEL_GEMV = 0, 1, 2, 3, 4, 5
KERNEL_NAMES = {0: "none", 1: "fill", 2: "skinny", 3: "ffma", 4: "tc", 5: "gemv"}
OPT_EARLY_START = 1
OPT_ADAPTIVE_PLANS = 2
OPT_PROGRAMMATIC_LAUNCH = 3
# LIN_OPT_EARLY_START levels: nothing before the previous kernel finishes (the
# default); W and bias may be read early; X too (only when no other work on the
# stream writes a call's inputs between library calls).
EARLY_NONE, EARLY_WEIGHTS, EARLY_ALL = 0, 1, 2
OK, ERR_ARG, ERR_ALIGN, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
# lin_dtype
TYPE_FP32, TYPE_BF16, TYPE_INT32, TYPE_INT64 = 0, 1, 2, 3
# lin_rotary_layout
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
# LIN_STATIC_SCRATCH_BYTES: the fixed device array behind lin_forward_fp32_static.
STATIC_SCRATCH_BYTES = 8 << 20

_PREC_NAMES = {"fp32": PREC_FP32, "tf32": PREC_TF32, "bf16": PREC_BF16}
_EPI_NAMES = {"none": EPI_NONE, None: EPI_NONE, "gelu": EPI_GELU_TANH, "gelu_tanh": EPI_GELU_TANH}


class Plan(ctypes.Structure):
    """Mirror of ``lin_plan``."""

    _fields_ = [
        ("kernel", ctypes.c_int), ("variant", ctypes.c_int), ("bm", ctypes.c_int), ("bn", ctypes.c_int),
        ("bk", ctypes.c_int), ("splits", ctypes.c_int), ("stages", ctypes.c_int), ("grid_x", ctypes.c_int),
        ("grid_y", ctypes.c_int), ("grid_z", ctypes.c_int), ("threads", ctypes.c_int),
        ("workspace_bytes", ctypes.c_longlong),
    ]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["kernel_name"] = KERNEL_NAMES.get(self.kernel, "?")
        return d

    def __repr__(self):
        return f"Plan({self.as_dict()})"


class RotaryPlan(ctypes.Structure):
    """Mirror of ``lin_rotary``."""

    _fields_ = [("dim", ctypes.c_int), ("layout", ctypes.c_int), ("scale", ctypes.c_float),
                ("turns", ctypes.c_void_p)]


class KVCachePlan(ctypes.Structure):
    """Mirror of ``lin_kv_cache``."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong)]


class KVBatchPlan(ctypes.Structure):
    """Mirror of ``lin_kv_batch``."""

    _fields_ = [("sequences", ctypes.c_int), ("tokens", ctypes.c_int), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("table_pages", ctypes.c_int),
                ("table_stride", ctypes.c_longlong)]


class LinError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = library().lin_strerror(status).decode()
        super().__init__(f"{what}: status {status} ({msg})" if what else f"status {status} ({msg})")


_lock = threading.Lock()
_lib = None


def library() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"CUDA library not built ({_LIB_PATH} missing); run "
                    "`python -m transformer_linear_layer_gb300.build` or __graft_entry__.build()")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            PP = ctypes.POINTER(Plan)
            L, F = ctypes.c_longlong, ctypes.c_float
            sig = {
                "lin_create": ([ctypes.POINTER(P), I, Z], I),
                "lin_destroy": ([P], I),
                "lin_forward": ([P, I, I, I, P, P, P, P, I, I, P], I),
                "lin_forward_plan": ([P, PP, I, I, I, P, P, P, P, I, I, P], I),
                "lin_plan_query": ([I, I, I, I, I, I, Z, PP], I),
                "lin_plan_make": ([I, I, I, I, I, I, I, I, PP], I),
                "lin_check_device": ([P, P], I),
                "lin_ctx_info": ([P, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(Z)], I),
                "lin_set_option": ([P, I, ctypes.c_longlong], I),
                "lin_ctx_last_plan": ([P, PP], I),
                "lin_forward_fp32_static": ([I, I, I, P, P, P, P, I, P], I),
                "lin_backward_data": ([P, I, I, I, P, P, P, I, P], I),
                "lin_backward_weight": ([P, I, I, I, P, P, P, P, I, P], I),
                "lin_gelu_backward": ([P, ctypes.c_longlong, P, P, P, I, P], I),
                "lin_forward_residual": ([P, I, I, I, P, P, P, P, P, I, I, P], I),
                "lin_plan_check": ([PP, I, I, I, I, ctypes.c_size_t], I),
                "lin_backward_data_gelu": ([P, I, I, I, P, P, P, P, I, P], I),
                "lin_fold_layernorm": ([P, I, I, P, P, P, P, P, P, I, P], I),
                "lin_set_plan_override": ([P, I, I, I, I, I, PP], I),
                "lin_clear_plan_overrides": ([P], I),
                "lin_probe_ffma": ([P, I, P, ctypes.POINTER(ctypes.c_double), P], I),
                "lin_timeline": ([I, P, Z, I], I),
                "lin_attention_forward": ([P, I, I, I, I, P, P, P, I, ctypes.c_float, P], I),
                "lin_attention_backward": ([P, I, I, I, I, P, P, P, P, P, I, F, P], I),
                "lin_token_logprobs": ([P, I, I, P, L, I, P, I, F, I, P, P, P, P, P, P], I),
                "lin_distill_forward": ([P, I, I, I, P, L, I, P, I, P, I, F, P, P, P], I),
                "lin_distill_backward": ([P, I, I, I, P, L, I, P, I, P, I, F, P, P, P, L, P], I),
                "lin_distill_forward_backward": ([P, I, I, I, P, L, I, P, I, P, I, F, P, P, P, L, P], I),
                "lin_rotary_turns": ([P, I, P], I),
                "lin_rotary_forward": ([P, I, I, I, P, L, P, L, I, P, I, P, P], I),
                "lin_rotary_backward": ([P, I, I, I, P, L, P, L, I, P, I, P, P], I),
                "lin_cache_append": ([P, P, P, I, P, L, P, L, P, L, P, L, P, I, P, P], I),
                "lin_paged_attention": ([P, P, P, I, P, L, P, L, P, I, F, I, P, Z, P], I),
                "lin_paged_attention_workspace": ([P, P, P, I, I, ctypes.POINTER(Z)], I),
                "lin_strerror": ([I], ctypes.c_char_p),
                "lin_abi_version": ([], I),
            }
            for name, (args, res) in sig.items():
                f = getattr(lib, name)
                f.argtypes = args
                f.restype = res
            _lib = lib
    return _lib


# Shape of a kernel timeline array (LIN_TIMELINE_CTAS x LIN_TIMELINE_SLOTS),
# and the timeline id of the attention kernel (LIN_TIMELINE_ATTENTION).
TIMELINE_CTAS, TIMELINE_SLOTS = 1024, 192
TIMELINE_ATTENTION = 16


def use_timeline_build() -> str:
    """Build (if stale) the timeline library (kernels compiled with
    -DLIN_TIMELINE) and load it instead of the library build. Call before the
    first library call of the process; returns the library path."""
    global _LIB_PATH
    path = build(timeline=True)
    with _lock:
        if _lib is not None and _LIB_PATH != path:
            raise RuntimeError("the library build is already loaded in this process")
        _LIB_PATH = path
    return path


def timeline(kernel: int, clear: bool = True):
    """The stamp array of ``kernel`` (KERNEL_TC, KERNEL_SKINNY or
    TIMELINE_ATTENTION) as an int64
    numpy array of TIMELINE_CTAS x TIMELINE_SLOTS nanoseconds (0 = not
    reached), synchronously; zeroes it afterwards if ``clear``. Needs the
    timeline build (:func:`use_timeline_build`)."""
    import numpy as np

    buf = np.zeros(TIMELINE_CTAS * TIMELINE_SLOTS, dtype=np.uint64)
    rc = library().lin_timeline(kernel, buf.ctypes.data, buf.nbytes, 1 if clear else 0)
    if rc != OK:
        raise LinError(rc, "lin_timeline")
    return buf.reshape(TIMELINE_CTAS, TIMELINE_SLOTS).astype(np.int64)


def timeline_clear(kernel: int):
    """Zero a kernel's stamp array (timeline build only)."""
    rc = library().lin_timeline(kernel, None, 0, 1)
    if rc != OK:
        raise LinError(rc, "lin_timeline")


def _prec(p) -> int:
    return _PREC_NAMES[p] if isinstance(p, str) else int(p)


def _epi(e) -> int:
    return _EPI_NAMES[e] if (e is None or isinstance(e, str)) else int(e)


def plan_query(sm_count: int, M: int, N: int, K: int, precision="bf16", epilogue="none",
               workspace_bytes: int = 64 << 20) -> Plan:
    """The dispatch table's plan for a shape (host only, no GPU needed)."""
    p = Plan()
    rc = library().lin_plan_query(sm_count, M, N, K, _prec(precision), _epi(epilogue), workspace_bytes,
                                  ctypes.byref(p))
    if rc != OK:
        raise LinError(rc, "lin_plan_query")
    return p


def plan_make(sm_count: int, kernel: int, variant: int, splits: int, M: int, N: int, K: int,
              precision="bf16") -> Plan:
    """A plan for one kernel family / tile configuration (host only)."""
    p = Plan()
    rc = library().lin_plan_make(sm_count, kernel, variant, splits, M, N, K, _prec(precision), ctypes.byref(p))
    if rc != OK:
        raise LinError(rc, "lin_plan_make")
    return p


def plan_check(plan: Plan, M: int, N: int, K: int, precision="bf16", workspace_bytes: int = 64 << 20) -> int:
    """Status lin_forward_plan would return for this plan and shape (host only;
    0 = accepted)."""
    return library().lin_plan_check(ctypes.byref(plan), M, N, K, _prec(precision), workspace_bytes)


class Context:
    """Owns a ``lin_ctx``: device, split-K workspace and the device status word."""

    def __init__(self, device: int = 0, workspace_bytes: int = 0):
        self._h = ctypes.c_void_p()
        rc = library().lin_create(ctypes.byref(self._h), int(device), int(workspace_bytes))
        if rc != OK:
            raise LinError(rc, "lin_create")
        dev, sms, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
        library().lin_ctx_info(self._h, ctypes.byref(dev), ctypes.byref(sms), ctypes.byref(ws))
        self.device, self.sm_count, self.workspace_bytes = dev.value, sms.value, ws.value

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            library().lin_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def check(self, stream=None):
        """Synchronise and raise if a kernel reported a timeout (status word)."""
        rc = library().lin_check_device(self._h, _stream_ptr(stream, self.device))
        if rc != OK:
            raise LinError(rc, "lin_check_device")

    def set_option(self, option: int, value: int):
        rc = library().lin_set_option(self._h, int(option), int(value))
        if rc != OK:
            raise LinError(rc, "lin_set_option")

    def last_plan(self) -> Plan:
        """The plan of the last call launched through this context."""
        p = Plan()
        rc = library().lin_ctx_last_plan(self._h, ctypes.byref(p))
        if rc != OK:
            raise LinError(rc, "lin_ctx_last_plan")
        return p

    def plan(self, M, N, K, precision="bf16", epilogue="none") -> Plan:
        """The built-in table's plan (installed overrides are not consulted)."""
        return plan_query(self.sm_count, M, N, K, precision, epilogue, self.workspace_bytes)

    def set_override(self, M, N, K, precision, epilogue, plan: Plan | None):
        """Install (or, with None, remove) the plan lin_forward uses for this call signature."""
        rc = library().lin_set_plan_override(self._h, M, N, K, _prec(precision), _epi(epilogue),
                                             None if plan is None else ctypes.byref(plan))
        if rc != OK:
            raise LinError(rc, "lin_set_plan_override")

    def clear_overrides(self):
        rc = library().lin_clear_plan_overrides(self._h)
        if rc != OK:
            raise LinError(rc, "lin_clear_plan_overrides")

    # raw-pointer calls (the C ABI, one to one) ---------------------------------
    def forward_ptr(self, M, N, K, X, W, bias, Y, epilogue, precision, stream) -> int:
        return library().lin_forward(self._h, M, N, K, X, W, bias, Y, _epi(epilogue), _prec(precision), stream)

    def probe_ffma_ptr(self, iters: int, out, stream) -> float:
        """Launch the fp32 FMA throughput probe (lin_probe_ffma) on `stream`;
        returns the FLOPs launched. The caller times it."""
        flops = ctypes.c_double()
        rc = library().lin_probe_ffma(self._h, int(iters), out, ctypes.byref(flops), stream)
        if rc != OK:
            raise LinError(rc, "lin_probe_ffma")
        return flops.value

    def forward_plan_ptr(self, plan: Plan, M, N, K, X, W, bias, Y, epilogue, precision, stream) -> int:
        return library().lin_forward_plan(self._h, ctypes.byref(plan), M, N, K, X, W, bias, Y, _epi(epilogue),
                                          _prec(precision), stream)


def _stream_ptr(stream, device):
    import torch

    if stream is None:
        # the current stream's handle without the Stream object around it (a call's
        # host time counts for single tokens)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return ctypes.c_void_p(raw(device))
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _torch_stream(stream, device):
    """torch's stream of a stream object or a raw handle. 0 and 1 are the default stream's (to torch, external streams of
    these handles are ones of its own)."""
    import torch

    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.ExternalStream(raw, device=device) if raw > 1 else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, stream):
    """A call's result: memory taken on the stream that its kernels run on (a block freed on another may still be in use
    there), and not given back before what the current stream does with it is done."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


_contexts: dict = {}


def default_context(device: int) -> Context:
    with _lock:
        ctx = _contexts.get(device)
    if ctx is None:
        ctx = Context(device)
        with _lock:
            _contexts.setdefault(device, ctx)
            ctx = _contexts[device]
    return ctx


def _marshal(x, w, bias, out, precision, stream):
    import torch

    prec = precision
    if prec is None:
        prec = "bf16" if x.dtype == torch.bfloat16 else "fp32"
    prec = _prec(prec)
    want = torch.bfloat16 if prec == PREC_BF16 else torch.float32
    if x.dtype != want or w.dtype != want:
        raise TypeError(f"precision {prec} needs {want} X and W, got {x.dtype} and {w.dtype}")
    if not (x.is_cuda and w.is_cuda):
        raise ValueError("X and W must be CUDA tensors")
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"need X (M x K) and W (N x K), got {tuple(x.shape)} and {tuple(w.shape)}")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("X and W must be contiguous row-major")
    M, K = x.shape
    N = w.shape[0]
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_cuda or bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous fp32 CUDA vector of length N")
    if out is None:
        out = _empty((M, N), want, x.device, stream)
    elif out.dtype != want or out.shape != (M, N) or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous M x N CUDA tensor of the output dtype")
    return prec, M, N, K, out


def forward(x, w, bias=None, epilogue="none", precision=None, out=None, ctx: Context | None = None, stream=None):
    """Y = act(x . w^T + bias) on x's device, asynchronously on the current stream.

    x: M x K, w: N x K (bf16 for precision "bf16", fp32 for "fp32"/"tf32"),
    bias: fp32 length N or None, epilogue: "none" | "gelu". Returns Y (M x N).
    """
    prec, M, N, K, out = _marshal(x, w, bias, out, precision, stream)
    dev = x.device.index if x.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = ctx.forward_ptr(M, N, K, x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
                         out.data_ptr(), epilogue, prec, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_forward")
    return out


def forward_residual(x, w, residual, bias=None, epilogue="none", precision=None, out=None,
                     ctx: Context | None = None, stream=None):
    """Y = act(x . w^T + bias) + residual, the add in the GEMM's store.
    ``out`` may be ``residual`` itself (x = x + layer(h) in place); by
    default Y is a new tensor."""
    prec, M, N, K, out = _marshal(x, w, bias, out, precision, stream)
    _check(residual, out.dtype, (M, N), "residual")
    dev = x.device.index if x.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_forward_residual(ctx._h, M, N, K, x.data_ptr(), w.data_ptr(),
                                        None if bias is None else bias.data_ptr(), residual.data_ptr(),
                                        out.data_ptr(), _epi(epilogue), prec, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_forward_residual")
    return out


def fold_layernorm(w, gamma, beta=None, bias=None, precision="fp32", w_out=None, bias_out=None,
                   ctx: Context | None = None, stream=None):
    """The next layer's (W, bias) with a LayerNorm's scale and shift folded in,
    computed on the device in double: W_out = w diag(gamma), bias_out =
    bias + w beta. ``w`` (N x K), ``gamma``, ``beta`` and ``bias`` are fp32;
    W_out has the storage type of ``precision``. Returns (W_out, bias_out)."""
    import torch

    N, K = w.shape
    _check(w, torch.float32, (N, K), "w")
    _check(gamma, torch.float32, (K,), "gamma")
    if beta is not None:
        _check(beta, torch.float32, (K,), "beta")
    if bias is not None:
        _check(bias, torch.float32, (N,), "bias")
    prec = _prec(precision)
    wdt = torch.bfloat16 if prec == PREC_BF16 else torch.float32
    if w_out is None:
        w_out = _empty((N, K), wdt, w.device, stream)
    _check(w_out, wdt, (N, K), "w_out")
    if bias_out is None:
        bias_out = _empty((N,), torch.float32, w.device, stream)
    _check(bias_out, torch.float32, (N,), "bias_out")
    dev = w.device.index if w.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_fold_layernorm(ctx._h, N, K, w.data_ptr(), None if bias is None else bias.data_ptr(),
                                      gamma.data_ptr(), None if beta is None else beta.data_ptr(), w_out.data_ptr(),
                                      bias_out.data_ptr(), prec, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_fold_layernorm")
    return w_out, bias_out


def forward_plan(plan: Plan, x, w, bias=None, epilogue="none", precision=None, out=None,
                 ctx: Context | None = None, stream=None):
    """As :func:`forward` with an explicit launch configuration."""
    prec, M, N, K, out = _marshal(x, w, bias, out, precision, stream)
    dev = x.device.index if x.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = ctx.forward_plan_ptr(plan, M, N, K, x.data_ptr(), w.data_ptr(),
                              None if bias is None else bias.data_ptr(), out.data_ptr(), epilogue, prec,
                              _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_forward_plan")
    return out


# ---------------------------------------------------------------- backward

def _bwd_dtype(t, precision):
    import torch

    prec = precision
    if prec is None:
        prec = "bf16" if t.dtype == torch.bfloat16 else "fp32"
    prec = _prec(prec)
    return prec, (torch.bfloat16 if prec == PREC_BF16 else torch.float32)


def _check(t, want, shape, what):
    if t.dtype != want or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be a contiguous {want} CUDA tensor of shape {tuple(shape)}")


def backward_data(dz, w, out=None, precision=None, ctx: Context | None = None, stream=None):
    """dX (M x K) = dz (M x N) . w (N x K): the input gradient of the layer
    (dz = dY times the activation's slope)."""
    import torch

    prec, want = _bwd_dtype(dz, precision)
    M, N = dz.shape
    K = w.shape[1]
    _check(dz, want, (M, N), "dz")
    _check(w, want, (N, K), "w")
    if out is None:
        out = _empty((M, K), want, dz.device, stream)
    _check(out, want, (M, K), "out")
    dev = dz.device.index if dz.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_backward_data(ctx._h, M, N, K, dz.data_ptr(), w.data_ptr(), out.data_ptr(), prec,
                                     _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_backward_data")
    return out


def backward_data_gelu(dz, w, zp, out=None, precision=None, ctx: Context | None = None, stream=None):
    """dZp (M x K) = (dz . w) * gelu'(zp): the input gradient carried through
    the GELU that made this layer's input from the previous layer's
    pre-activation ``zp`` (M x K), in one pass. ``out`` may be ``zp``."""
    import torch

    prec, want = _bwd_dtype(dz, precision)
    M, N = dz.shape
    K = w.shape[1]
    _check(dz, want, (M, N), "dz")
    _check(w, want, (N, K), "w")
    _check(zp, want, (M, K), "zp")
    if out is None:
        out = _empty((M, K), want, dz.device, stream)
    _check(out, want, (M, K), "out")
    dev = dz.device.index if dz.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_backward_data_gelu(ctx._h, M, N, K, dz.data_ptr(), w.data_ptr(), zp.data_ptr(),
                                          out.data_ptr(), prec, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_backward_data_gelu")
    return out


def backward_weight(dz, x, out=None, db=None, precision=None, ctx: Context | None = None, stream=None):
    """dW (N x K) = dz^T . x (dz: M x N, x: M x K) and, when ``db`` is True or
    an fp32 tensor of length N, db = the column sums of dz. Returns (dW, db)."""
    import torch

    prec, want = _bwd_dtype(dz, precision)
    M, N = dz.shape
    K = x.shape[1]
    _check(dz, want, (M, N), "dz")
    _check(x, want, (M, K), "x")
    if out is None:
        out = _empty((N, K), want, dz.device, stream)
    _check(out, want, (N, K), "out")
    if db is True:
        db = _empty((N,), torch.float32, dz.device, stream)
    if db is not None and db is not False:
        _check(db, torch.float32, (N,), "db")
    else:
        db = None
    dev = dz.device.index if dz.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_backward_weight(ctx._h, M, N, K, dz.data_ptr(), x.data_ptr(), out.data_ptr(),
                                       None if db is None else db.data_ptr(), prec, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_backward_weight")
    return out, db


def gelu_backward(dy, z, out=None, precision=None, ctx: Context | None = None, stream=None):
    """dZ = dy * gelu'(z) (z: the forward's pre-activation), elementwise."""
    import torch

    prec, want = _bwd_dtype(dy, precision)
    _check(dy, want, tuple(dy.shape), "dy")
    _check(z, want, tuple(dy.shape), "z")
    if out is None:
        out = _empty(dy.shape, dy.dtype, dy.device, stream)
    _check(out, want, tuple(dy.shape), "out")
    dev = dy.device.index if dy.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_gelu_backward(ctx._h, dy.numel(), dy.data_ptr(), z.data_ptr(), out.data_ptr(), prec,
                                     _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_gelu_backward")
    return out


# ---------------------------------------------------------------- attention

def attention_forward(qkv, B: int, T: int, H: int, causal: bool = True, scale: float | None = None, out=None,
                      lse=None, with_lse: bool = False, ctx: Context | None = None, stream=None):
    """Fused self-attention forward from the qkv projection's output.

    qkv: contiguous bf16 CUDA tensor of (B*T) x 3C (C = 64 H; q, k, v at
    column offsets 0, C, 2C, head h at 64 h within each). Returns out
    ((B*T) x C bf16), or (out, lse) with lse (B, H, T) fp32 when ``with_lse``
    or an lse tensor is given. scale defaults to 1/sqrt(64)."""
    import torch

    D = 64
    C = H * D
    _check(qkv, torch.bfloat16, (B * T, 3 * C), "qkv")
    if out is None:
        out = _empty((B * T, C), torch.bfloat16, qkv.device, stream)
    _check(out, torch.bfloat16, (B * T, C), "out")
    if lse is None and with_lse:
        lse = _empty((B, H, T), torch.float32, qkv.device, stream)
    if lse is not None:
        _check(lse, torch.float32, (B, H, T), "lse")
    dev = qkv.device.index if qkv.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_attention_forward(ctx._h, B, T, H, D, qkv.data_ptr(), out.data_ptr(),
                                         None if lse is None else lse.data_ptr(), int(bool(causal)),
                                         0.0 if scale is None else float(scale), _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_attention_forward")
    return (out, lse) if lse is not None else out


def attention_backward(qkv, out, lse, dout, B: int, T: int, H: int, causal: bool = True, scale: float | None = None,
                       dqkv=None, ctx: Context | None = None, stream=None):
    """Gradient of :func:`attention_forward` with respect to qkv.

    qkv ((B*T) x 3C), out ((B*T) x C) and lse (B, H, T) are the forward's input
    and outputs (``with_lse=True``), dout ((B*T) x C bf16) the gradient of out.
    Returns dqkv ((B*T) x 3C bf16). Uses the context's workspace."""
    import torch

    D = 64
    C = H * D
    _check(qkv, torch.bfloat16, (B * T, 3 * C), "qkv")
    _check(out, torch.bfloat16, (B * T, C), "out")
    _check(lse, torch.float32, (B, H, T), "lse")
    _check(dout, torch.bfloat16, (B * T, C), "dout")
    if dqkv is None:
        dqkv = _empty(qkv.shape, qkv.dtype, qkv.device, stream)
    _check(dqkv, torch.bfloat16, (B * T, 3 * C), "dqkv")
    _same_device(qkv, out, lse, dout, dqkv)
    dev = qkv.device.index if qkv.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_attention_backward(ctx._h, B, T, H, D, qkv.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                          dout.data_ptr(), dqkv.data_ptr(), int(bool(causal)),
                                          0.0 if scale is None else float(scale), _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_attention_backward")
    return dqkv


# ---------------------------------------------------------------- logits

class TokenLogprobs(NamedTuple):
    """Result of :func:`token_logprobs` (fp32, ids int32)."""

    logprob: object       # R, or None without tokens
    entropy: object       # R
    lse: object           # R
    top_logprob: object   # R x top
    top_ids: object       # R x top


def _float_type(t, what):
    import torch

    if t.dtype == torch.float32:
        return TYPE_FP32
    if t.dtype == torch.bfloat16:
        return TYPE_BF16
    raise TypeError(f"{what} must be fp32 or bf16, got {t.dtype}")


def _index_type(t, what):
    import torch

    if t.dtype == torch.int32:
        return TYPE_INT32
    if t.dtype == torch.int64:
        return TYPE_INT64
    raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")


def _check_logits(t, what="logits"):
    """(rows, V, row stride) of an R x V tensor whose rows are contiguous."""
    if not t.is_cuda or t.dim() != 2 or t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be an R x V CUDA tensor (V >= 1) with contiguous rows")
    R, V = t.shape
    ld = t.stride(0) if R > 1 else V
    if ld < V:
        raise ValueError(f"{what}: rows overlap")
    return R, V, ld


def _same_device(first, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"all tensors must be on {first.device}, got one on {t.device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def token_logprobs(logits, tokens=None, top: int = 0, temperature: float = 1.0, ctx: Context | None = None,
                   stream=None) -> TokenLogprobs:
    """Log probability of ``tokens[r]`` under softmax(logits[r] / temperature),
    the distribution's entropy (nats), and its ``top`` (at most 64) most likely
    tokens in order, equal logits by the lowest index.

    logits: R x V, fp32 or bf16, rows contiguous (any row stride, so a padded
    vocabulary is passed as ``buffer[:, :V]``). tokens: R, int32 or int64; a
    negative token has log probability 0, one past the vocabulary NaN."""
    import torch

    R, V, ld = _check_logits(logits)
    ztype = _float_type(logits, "logits")
    if not 0 <= top <= min(64, V):
        raise ValueError(f"top must be between 0 and {min(64, V)}, got {top}")
    _same_device(logits, tokens)
    ttype = TYPE_INT64
    if tokens is not None:
        ttype = _index_type(tokens, "tokens")
        _check(tokens, tokens.dtype, (R,), "tokens")
    logprob = None if tokens is None else _empty(R, torch.float32, logits.device, stream)
    entropy = _empty(R, torch.float32, logits.device, stream)
    lse = _empty(R, torch.float32, logits.device, stream)
    top_logprob = _empty((R, top), torch.float32, logits.device, stream)
    top_ids = _empty((R, top), torch.int32, logits.device, stream)
    dev = logits.device.index if logits.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_token_logprobs(ctx._h, R, V, logits.data_ptr(), ld, ztype, _ptr(tokens), ttype,
                                      float(temperature), int(top), _ptr(logprob), entropy.data_ptr(),
                                      lse.data_ptr(), top_logprob.data_ptr(), top_ids.data_ptr(),
                                      _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, top_logprob, top_ids)


def _distill_args(logits, ids, teacher, lse=None, weight=None):
    import torch

    R, V, ld = _check_logits(logits)
    if ids.dim() != 2 or ids.shape[0] != R:
        raise ValueError(f"ids must be R x K with R = {R}, got {tuple(ids.shape)}")
    K = ids.shape[1]
    itype, ttype = _index_type(ids, "ids"), _float_type(teacher, "teacher")
    _check(ids, ids.dtype, (R, K), "ids")
    _check(teacher, teacher.dtype, (R, K), "teacher")
    for what, t in (("lse", lse), ("the rows' weight", weight)):
        if t is not None:
            _check(t, torch.float32, (R,), what)
    _same_device(logits, ids, teacher, lse, weight)
    return (R, V, K, logits.data_ptr(), ld, _float_type(logits, "logits"), ids.data_ptr(), itype,
            teacher.data_ptr(), ttype)


def _dlogits(logits, out, args, stream):
    """The gradient's tensor and row stride: ``out``, or a new one whose rows
    lie like the logits' (padding included, so that both move in whole units)."""
    import torch

    R, V, ld = args[0], args[1], args[4]
    if out is None:
        pitch = ld if ld <= V + 1024 else V
        out = _empty((R, pitch), logits.dtype, logits.device, stream)
        return (out if pitch == V else out[:, :V]), pitch
    if out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have the logits' shape and type")
    _same_device(logits, out)
    return out, _check_logits(out, "out")[2]


def distill_forward(logits, ids, teacher, temperature: float = 1.0, ctx: Context | None = None, stream=None):
    """Distillation loss of each row towards a teacher's top logits:
    tau^2 KL(softmax(teacher / tau) over the row's entries || softmax(logits / tau)).

    logits: R x V (fp32 or bf16, any row stride). ids, teacher: R x K token ids
    (int32 or int64, negative = padding) and the teacher's logits or log
    probabilities for them (fp32 or bf16). Returns (loss, lse), R fp32 each;
    lse is what :func:`distill_backward` needs."""
    import torch

    args = _distill_args(logits, ids, teacher)
    loss = _empty(args[0], torch.float32, logits.device, stream)
    lse = _empty(args[0], torch.float32, logits.device, stream)
    dev = logits.device.index if logits.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_distill_forward(ctx._h, *args, float(temperature), loss.data_ptr(), lse.data_ptr(),
                                       _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_distill_forward")
    return loss, lse


def distill_backward(logits, ids, teacher, lse, grad_loss, temperature: float = 1.0, out=None,
                     ctx: Context | None = None, stream=None):
    """The logits' gradient, from :func:`distill_forward`'s lse (of the same
    logits and temperature) and the gradient of each row's loss (R fp32).
    ``out`` may be ``logits``. Rows whose lse is too large to carry the
    probabilities' digits (above 512 for bf16 logits, 64 for fp32) are summed
    again."""
    args = _distill_args(logits, ids, teacher, lse, grad_loss)
    out, ldd = _dlogits(logits, out, args, stream)
    dev = logits.device.index if logits.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_distill_backward(ctx._h, *args, float(temperature), lse.data_ptr(), grad_loss.data_ptr(),
                                        out.data_ptr(), ldd, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_distill_backward")
    return out


def distill_forward_backward(logits, ids, teacher, weight=None, temperature: float = 1.0, out=None,
                             ctx: Context | None = None, stream=None):
    """(loss, dlogits) in one pass over the logits: the rows' losses and the
    gradient of sum_r weight[r] * loss[r] (weight: R fp32, default 1).
    ``out`` may be ``logits``: the gradient then replaces them."""
    import torch

    args = _distill_args(logits, ids, teacher, None, weight)
    out, ldd = _dlogits(logits, out, args, stream)
    loss = _empty(args[0], torch.float32, logits.device, stream)
    dev = logits.device.index if logits.device.index is not None else 0
    ctx = ctx or default_context(dev)
    rc = library().lin_distill_forward_backward(ctx._h, *args, float(temperature), _ptr(weight), loss.data_ptr(),
                                                out.data_ptr(), ldd, _stream_ptr(stream, dev))
    if rc != OK:
        raise LinError(rc, "lin_distill_forward_backward")
    return loss, out


# ---------------------------------------------------------------- rotary positions

class _Fixed:
    """A plan whose public attributes cannot be set anew: the library was given their addresses
    and sizes once. (What their tensors hold may change, ``batch.kv_len += 1`` for instance.)"""

    def __setattr__(self, name, value):
        held = self.__dict__
        if not name.startswith("_") and name in held and held[name] is not value:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be set anew: write into it, or make another")
        held[name] = value


class Rotary(_Fixed):
    """The plan of rotary positions: which elements of a head turn, and how fast.

    dim: elements of each head that rotate (even; the rest of the head does not).
    interleaved: pairs are neighbours (2i, 2i + 1) instead of halves (i, i + dim/2).
    Pair i turns by base ** (-2 i / dim) radians per position, scaled for longer
    contexts by ``scaling``:

      None      as trained
      "linear"  all frequencies divided by ``factor``
      "ntk"     the base times factor ** (dim / (dim - 2)): the slowest pair is
                divided by the factor, the fastest kept
      "yarn"    by parts: pairs that turn at most ``slow`` times in
                ``original_length`` positions are divided by the factor, those that
                turn ``fast`` times or more are kept, with a ramp between that is linear
                in the number of turns; the rotated elements are multiplied by
                0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window Extension
                of Large Language Models", whose text defines it so)

    or by ``frequencies`` (dim/2 radians per position) in place of all of these. Many
    checkpoints that name YaRN were made with another ramp, linear in the pair's
    index i from the pair that turns ``fast`` times to the one that turns ``slow`` times, and
    a model has to be served with the one that it was trained with: the two differ by up to a
    factor of 2.3 (dim 128, base 10000, original_length 4096, factor 8). For that one, pass::

        place = lambda turns: dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = math.floor(place(fast)), math.ceil(place(slow))
        keep = [1 - min(1, max(0, (i - low) / (high - low))) for i in range(dim // 2)]
        plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
        Rotary(dim, frequencies=[f * (k + (1 - k) / factor) for f, k in zip(plain, keep)],
               scale=0.1 * math.log(factor) + 1)

    (without floor and ceil where the model's configuration says so).
    ``scale`` replaces the factor on the rotated elements. The plan holds its
    table on ``device``; positions p may be any 64-bit integers (the angle is that of the
    frequencies to |p| 2^-62 radians)."""

    def __init__(self, dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str | None = None,
                 factor: float = 1.0, original_length: int | None = None, fast: float = 32.0, slow: float = 1.0,
                 frequencies=None, scale: float | None = None, device="cuda"):
        import math

        import torch

        if dim < 0 or dim % 2:
            raise ValueError(f"dim must be even and not negative, got {dim}")
        if scaling not in (None, "linear", "ntk", "yarn"):
            raise ValueError(f"unknown scaling {scaling!r}")
        if not (math.isfinite(factor) and factor >= 1.0):
            raise ValueError(f"factor must be at least 1, got {factor}")
        if not (math.isfinite(base) and base > 0):
            raise ValueError(f"base must be positive, got {base}")
        own_scale = 1.0
        if frequencies is None:
            if scaling == "ntk" and dim > 2:
                base = base * factor ** (dim / (dim - 2))
            frequencies = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
            if scaling == "linear":
                frequencies = [f / factor for f in frequencies]
            elif scaling == "yarn":
                if not original_length or original_length < 1 or not fast > slow:
                    raise ValueError("yarn needs original_length, and fast above slow")
                held = []
                for f in frequencies:
                    keep = (original_length * f / (2 * math.pi) - slow) / (fast - slow)
                    keep = min(1.0, max(0.0, keep))
                    held.append(f * keep + f / factor * (1.0 - keep))
                frequencies = held
                own_scale = 0.1 * math.log(factor) + 1.0
        self.frequencies = [float(f) for f in frequencies]
        n = dim // 2
        if len(self.frequencies) != n:
            raise ValueError(f"{n} frequencies are needed, got {len(self.frequencies)}")
        self.dim, self.interleaved = dim, bool(interleaved)
        self.scale = own_scale if scale is None else float(scale)
        turns = (ctypes.c_ulonglong * max(n, 1))()
        rc = library().lin_rotary_turns((ctypes.c_double * max(n, 1))(*self.frequencies), n, turns)
        if rc != OK:
            raise LinError(rc, "lin_rotary_turns")
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(signed[:n] or [0], dtype=torch.int64, device=device)
        self.index = self.turns.get_device()
        self._plan = RotaryPlan(dim, ROTARY_INTERLEAVED if self.interleaved else ROTARY_HALF, self.scale,
                                self.turns.data_ptr())
        self._ref = ctypes.byref(self._plan)


# A single token's call is bound by its time on the host: the entries below ask for the
# library, the context and the stream without a lock or an object each.

def _loaded():
    return _lib if _lib is not None else library()


def _context(index):
    return _contexts.get(index) or default_context(index)


def _on_device(ctx, index):
    if ctx.device != index:
        raise ValueError(f"the tensors are on cuda:{index}, the context is of cuda:{ctx.device}")
    return ctx


def _raw_stream(stream, index):
    import torch

    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_MOST = 2 ** 31 - 1  # sizes are ints


def _check_sizes(t, what):
    if max(t.shape) > _MOST:
        raise ValueError(f"{what}: sizes are 32 bits, got {tuple(t.shape)}")


def _check_heads(t, dtype, what, index=None):
    """(rows, heads, width, row stride) of an N x H x D tensor (of ``dtype``, on CUDA
    device ``index``) whose rows hold their heads one after the other, any distance apart."""
    if t.dim() != 3 or (dtype is not None and t.dtype != dtype) or not t.is_cuda:
        raise ValueError(f"{what} must be an N x heads x width CUDA tensor" + (f" of {dtype}" if dtype else ""))
    if index is not None and t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}, got {t.device}")
    N, H, D = t.shape
    if N > _MOST or H > _MOST or D > _MOST:
        _check_sizes(t, what)
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        raise ValueError(f"{what}: a row must hold its heads one after the other")
    ld = s0 if N > 1 else H * D
    if ld < H * D:
        raise ValueError(f"{what}: rows overlap")
    return N, H, D, ld


def _check_positions(t, N, index):
    if t.shape != (N,) or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"positions must be a contiguous tensor of {N} on cuda:{index}, got {tuple(t.shape)} on {t.device}")
    return _index_type(t, "positions")


def _rotary(call, x, positions, rotary, out, ctx, stream):
    import torch

    N, H, D, ldx = _check_heads(x, None, "x")
    index = x.get_device()
    kind = _float_type(x, "x")
    ptype = _check_positions(positions, N, index)
    if rotary.index != index:
        raise ValueError(f"the rotary plan must be on cuda:{index}, got cuda:{rotary.index}")
    if out is None:
        out, ldy = _empty((N, H, D), x.dtype, x.device, stream), H * D
    else:
        No, Ho, Do, ldy = _check_heads(out, x.dtype, "out", index)
        if (No, Ho, Do) != (N, H, D):
            raise ValueError(f"out must have shape {(N, H, D)}, got {tuple(out.shape)}")
    ctx = _context(index) if ctx is None else _on_device(ctx, index)
    rc = getattr(_loaded(), call)(ctx._h, N, H, D, x.data_ptr(), ldx, out.data_ptr(), ldy, kind,
                                  positions.data_ptr(), ptype, rotary._ref, _raw_stream(stream, index))
    if rc != OK:
        raise LinError(rc, call)
    return out


def rotary_forward(x, positions, rotary: Rotary, out=None, ctx: Context | None = None, stream=None):
    """Heads turned by their row's position.

    x: N x H x D, fp32 or bf16, the heads of a row one after the other and rows any
    distance apart: the query and key heads of a qkv projection's output are
    ``qkv[:, :2 * C].unflatten(1, (2 * H, D))``. positions: N, int32 or int64.
    Returns N x H x D; ``out`` may be ``x`` (in place)."""
    return _rotary("lin_rotary_forward", x, positions, rotary, out, ctx, stream)


def rotary_backward(dy, positions, rotary: Rotary, out=None, ctx: Context | None = None, stream=None):
    """The gradient of :func:`rotary_forward`'s input from its output's (``out`` may be ``dy``)."""
    return _rotary("lin_rotary_backward", dy, positions, rotary, out, ctx, stream)


# ---------------------------------------------------------------- paged cache

class KVCache(_Fixed):
    """A paged cache of keys and values: ``k`` and ``v`` bf16 of pages x heads x
    page_size x head width (64 or 128; page_size a power of two from 8 to 4096), of the same
    strides. The last dimension is contiguous, the others may have any
    strides (multiples of 8): token-major pages are passed as
    ``pages.transpose(1, 2)``, halves of one tensor as ``kv[:, 0]``, ``kv[:, 1]``."""

    def __init__(self, k, v):
        import torch

        for what, t in (("k", k), ("v", v)):
            if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{what} must be a bf16 CUDA tensor of pages x heads x page_size x width")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must have the same shape and strides")
        _check_sizes(k, "k")
        _same_device(k, v)
        self.k, self.v = k, v
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.device, self.index = k.device, k.get_device()
        self._sizes: dict = {}  # workspace bytes by query heads and tokens
        self._plan = KVCachePlan(k.data_ptr(), v.data_ptr(), *(k.shape[i] for i in (0, 2, 1, 3)), *k.stride()[:3])
        self._ref = ctypes.byref(self._plan)

    @property
    def _workspace(self):
        return _default_stream(self.index).workspace


class KVBatch(_Fixed):
    """Sequences whose new tokens are rows of packed tensors (int32, on the GPU; the
    kernels read them when they run).

    q_start: B + 1, sequence b's new tokens are rows q_start[b] to q_start[b + 1] - 1.
    kv_len: B, tokens of each sequence in the cache, the new ones included.
    block_table: B x pages of a sequence, rows contiguous: its tokens i * page_size
    and on lie in page block_table[b, i]."""

    def __init__(self, q_start, kv_len, block_table):
        import torch

        B = kv_len.shape[0] if kv_len.dim() == 1 else -1
        _check(kv_len, torch.int32, (B,), "kv_len")
        _check(q_start, torch.int32, (B + 1,), "q_start")
        if (not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 or
                block_table.shape[0] != B or (block_table.shape[1] > 1 and block_table.stride(1) != 1)):
            raise ValueError(f"block_table must be an int32 CUDA tensor of {B} rows, each contiguous")
        _check_sizes(block_table, "block_table")
        _same_device(kv_len, q_start, block_table)
        self.q_start, self.kv_len, self.block_table = q_start, kv_len, block_table
        self.sequences = B
        self.device, self.index = kv_len.device, kv_len.get_device()
        self._plans: dict = {}

    def _ref(self, tokens: int):
        ref = self._plans.get(tokens)
        if ref is None:
            t = self.block_table
            ref = ctypes.byref(KVBatchPlan(self.sequences, tokens, self.q_start.data_ptr(), self.kv_len.data_ptr(),
                                           t.data_ptr(), t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]))
            if len(self._plans) > 64:
                self._plans.clear()
            self._plans[tokens] = ref
        return ref


def cache_append(q, k, v, cache: KVCache, batch: KVBatch, rotary: Rotary | None = None, positions=None, q_out=None,
                 ctx: Context | None = None, stream=None):
    """Write new keys and values (tokens x heads x width, bf16) into the cache's pages, row by
    row to the places that ``batch`` gives them.

    With ``rotary``, keys are rotated on the way by their place in the sequence (or by
    ``positions``, one per row), and so is ``q`` (tokens x query heads x width, or None):
    returns it rotated, in ``q_out`` or a new tensor (``q_out`` may be ``q``). Without ``rotary`` q must be None.
    Rows that belong to no sequence are left out."""
    import torch

    D, index, bf16 = cache.head_dim, cache.index, torch.bfloat16
    N, Hk, Dk, ldk = _check_heads(k, bf16, "k", index)
    Nv, Hv, Dv, ldv = _check_heads(v, bf16, "v", index)
    if (Hk, Dk) != (cache.heads, D) or (Nv, Hv, Dv) != (N, Hk, Dk):
        raise ValueError(f"k and v must be tokens x {cache.heads} x {D}, got {tuple(k.shape)} and {tuple(v.shape)}")
    if batch.index != index or (rotary is not None and rotary.index != index):
        raise ValueError(f"the batch and the rotary plan must be on cuda:{index}, like the cache")
    H = ldq = ldo = 0
    if q is not None:
        Nq, H, Dq, ldq = _check_heads(q, bf16, "q", index)
        if (Nq, Dq) != (N, D):
            raise ValueError(f"q must be {N} x heads x {D}, got {tuple(q.shape)}")
        if rotary is None:
            raise ValueError("q is only rotated: without a rotary plan it must be None")
        if q_out is None:
            q_out, ldo = _empty((N, H, D), bf16, cache.device, stream), H * D
        else:
            No, Ho, Do, ldo = _check_heads(q_out, bf16, "q_out", index)
            if (No, Ho, Do) != (N, H, D):
                raise ValueError(f"q_out must have shape {(N, H, D)}, got {tuple(q_out.shape)}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    ptype = TYPE_INT64 if positions is None else _check_positions(positions, N, index)
    ctx = _context(index) if ctx is None else _on_device(ctx, index)
    rc = _loaded().lin_cache_append(ctx._h, cache._ref, batch._ref(N), H, _ptr(q), ldq, _ptr(q_out), ldo,
                                    k.data_ptr(), ldk, v.data_ptr(), ldv, _ptr(positions), ptype,
                                    None if rotary is None else rotary._ref, _raw_stream(stream, index))
    if rc != OK:
        raise LinError(rc, "lin_cache_append")
    return q_out


def paged_attention(q, cache: KVCache, batch: KVBatch, causal: bool = True, scale: float | None = None,
                    max_new: int | None = None, out=None, lse=None, with_lse: bool = False, workspace=None,
                    ctx: Context | None = None, stream=None):
    """Attention of the batch's new tokens over the cache, which holds their own keys and values already
    (:func:`cache_append`).

    q: tokens x query heads x width, bf16, rows any multiple of 8 elements apart; query heads a multiple
    (at most 128) of the cache's. scale: of the scores, default (or 0) 1/sqrt(width). causal: each token sees the keys up
    to its own place; otherwise all of its sequence's (a cross attention over an encoder's states).

    max_new: about how many new tokens the longest sequence has (default: the average), which picks the kernel; any
    value is right, but the average misjudges a long prompt among single tokens (63 of them and a prompt of 900, 12
    heads of 64: 161 us instead of 138).

    Returns out (like q, contiguous), or (out, lse) with lse tokens x heads fp32 when ``with_lse`` or an lse tensor is
    given. Rows that belong to no sequence are not written.

    workspace: a uint8 tensor of :func:`paged_attention_workspace` bytes, for one call at a time. By default, calls on
    the default stream share one that is kept for the device (up to 40 MB on a GB300), and any other call has its own
    from torch's allocator."""
    import torch

    index = cache.index
    N, H, D, ldq = _check_heads(q, torch.bfloat16, "q", index)
    if D != cache.head_dim:
        raise ValueError(f"q must be tokens x heads x {cache.head_dim}, got {tuple(q.shape)}")
    if batch.index != index:
        raise ValueError(f"the batch must be on cuda:{index}, like the cache")
    if out is None:
        out, ldo = _empty((N, H, D), torch.bfloat16, cache.device, stream), H * D
    else:
        No, Ho, Do, ldo = _check_heads(out, torch.bfloat16, "out", index)
        if (No, Ho, Do) != (N, H, D):
            raise ValueError(f"out must have shape {(N, H, D)}, got {tuple(out.shape)}")
    if lse is None and with_lse:
        lse = _empty((N, H), torch.float32, cache.device, stream)
    elif lse is not None:
        _check(lse, torch.float32, (N, H), "lse")
        _same_device(q, lse)
    ctx = _context(index) if ctx is None else _on_device(ctx, index)
    hint = 0 if max_new is None else int(max_new)
    raw = _raw_stream(stream, index)
    call = _loaded().lin_paged_attention
    args = (ctx._h, cache._ref, batch._ref(N), H, q.data_ptr(), ldq, out.data_ptr(), ldo, _ptr(lse), int(bool(causal)),
            0.0 if scale is None else float(scale), hint)
    if workspace is None:
        # (the size goes by the device too, and all contexts of a cache are on its own)
        key = (H, hint, N if hint == 0 else 0, batch.sequences if hint == 0 else 0)
        size = cache._sizes.get(key)
        if size is None:
            size = paged_attention_workspace(cache, batch, N, H, hint, ctx)
            if len(cache._sizes) > 64:
                cache._sizes.clear()
            cache._sizes[key] = size
        if raw == 0 and stream is None:
            # The default stream: its kernels run one after the other, and none is captured. The rest
            # of the time (an allocation takes 3 us of a call's 15) a call's workspace is its own.
            # One thread at a time, since a call's two kernels have to follow one another on the stream.
            shared = _default_stream(index)
            with shared.turn:
                if shared.workspace is None or shared.workspace.numel() < size:
                    shared.workspace = _scratch(cache.device, size, None)
                rc = call(*args, shared.workspace.data_ptr(), size, raw)
        else:
            workspace = _scratch(cache.device, size, stream)
            rc = call(*args, workspace.data_ptr(), size, raw)
    else:
        _same_device(q, workspace)
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        rc = call(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw)
    if rc != OK:
        raise LinError(rc, "lin_paged_attention")
    return (out, lse) if lse is not None else out


class _DefaultStream:
    """The workspace of paged attention's calls on a device's default stream, and whose turn it is to enqueue with it."""

    def __init__(self):
        self.turn, self.workspace = threading.RLock(), None


_default_streams: dict = {}


def _default_stream(index) -> _DefaultStream:
    shared = _default_streams.get(index)
    return shared if shared is not None else _default_streams.setdefault(index, _DefaultStream())


def paged_attention_workspace(cache: KVCache, batch: KVBatch, tokens: int, heads: int, max_new: int = 0,
                              ctx: Context | None = None) -> int:
    """Bytes of workspace that :func:`paged_attention` needs for such a call."""
    ctx = default_context(cache.index) if ctx is None else _on_device(ctx, cache.index)
    size = ctypes.c_size_t()
    rc = library().lin_paged_attention_workspace(ctx._h, cache._ref, batch._ref(tokens), heads, max_new,
                                                 ctypes.byref(size))
    if rc != OK:
        raise LinError(rc, "lin_paged_attention_workspace")
    return size.value


def _scratch(device, size, stream):
    """Bytes from torch's allocator for one call's kernels, taken on the stream that they run on."""
    import torch

    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.empty(size, dtype=torch.uint8, device=device)
