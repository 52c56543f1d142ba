"""Thin ctypes binding of libflce.so (the C ABI in include/flce.h).

Argument marshalling only: torch tensors supply device memory and the current CUDA stream;
every step of the computation runs in the library's kernels. If the library has not been
built the first call raises, there is no fallback.

Calls run on the current stream, or on the one given as ``stream``: then it also owns the
tensors that the call makes, and it must already wait for what made the inputs; a stream that
reads the results waits for it.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflce.so")

FLCE_OK, FLCE_ERR_INVALID_ARG, FLCE_ERR_UNSUPPORTED, FLCE_ERR_TARGET_RANGE = 0, 1, 2, 3
FLCE_ERR_WORKSPACE, FLCE_ERR_CUDA, FLCE_ERR_TIMEOUT, FLCE_ERR_SCRATCH_LIMIT = 4, 5, 6, 7
NOALLOC_SCRATCH_BYTES = 128 << 20
REDUCTIONS = {"mean": 0, "sum": 1, "none": 2}
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
FLAG_FORCE_SIMT = 0x1
FLAG_NO_ROW_REF = 0x2
FLAG_DW_OVERWRITE = 0x4
FLAG_SEPARATE_BWD = 0x8
FLAG_DEBUG_STALL = 0x100
FLAG_DEBUG_STALL_BWD = 0x200
EXPORTED = ("flce_workspace_size", "flce_chunk_rows", "flce_fwd_bwd", "flce_fwd_bwd_noalloc",
            "flce_get_status",
            "flce_profile_create", "flce_profile_reset", "flce_profile_destroy",
            "flce_profile_read", "flce_last_cuda_error", "flce_status_string", "flce_abi_version",
            "flce_jsd_workspace_size", "flce_fused_linear_jsd", "flce_scale_by",
            "flce_plan_describe",
            "flce_embed_fwd", "flce_embed_bwd", "flce_embed_workspace_size",
            "flce_rmsnorm_fwd", "flce_rmsnorm_bwd", "flce_rmsnorm_workspace_size",
            "flce_ckpt8_pack", "flce_ckpt8_dw", "flce_ckpt8_dw_workspace_size")
Q_BLOCK = 128  # columns of an 8-bit row that share a scale
STAGES = ("prologue", "gather", "fwd", "finalize", "gpass", "dx", "dw", "reduce", "bwd")


class FlceArgs(ctypes.Structure):
    """Mirror of ``flce_args`` (field order and C types must match include/flce.h)."""
    _fields_ = [
        ("BT", ctypes.c_int64), ("H", ctypes.c_int64), ("V", ctypes.c_int64),
        ("in_dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("targets", ctypes.c_void_p), ("ignore_index", ctypes.c_int64),
        ("z_loss_scale", ctypes.c_float), ("grad_out", ctypes.c_void_p),
        ("want_dX", ctypes.c_int32), ("want_dW", ctypes.c_int32), ("dW_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("loss", ctypes.c_void_p), ("z_loss", ctypes.c_void_p), ("acc", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("pred", ctypes.c_void_p), ("n_labelled", ctypes.c_void_p),
        ("dX", ctypes.c_void_p), ("dW", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_uint32),
        ("profile", ctypes.c_void_p),
    ]


class FlceJsdArgs(ctypes.Structure):
    """Mirror of ``flce_jsd_args`` (field order and C types must match include/flce.h)."""
    _fields_ = [
        ("BT", ctypes.c_int64), ("Hs", ctypes.c_int64), ("Ht", ctypes.c_int64), ("V", ctypes.c_int64),
        ("in_dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("Xs", ctypes.c_void_p), ("Ws", ctypes.c_void_p), ("Xt", ctypes.c_void_p), ("Wt", ctypes.c_void_p),
        ("labels", ctypes.c_void_p), ("ignore_index", ctypes.c_int64),
        ("beta", ctypes.c_float), ("temperature", ctypes.c_float), ("grad_out", ctypes.c_void_p),
        ("want_dX", ctypes.c_int32), ("want_dW", ctypes.c_int32), ("dW_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("loss", ctypes.c_void_p), ("n_labelled", ctypes.c_void_p), ("dX", ctypes.c_void_p),
        ("dW", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_uint32),
        ("profile", ctypes.c_void_p),
    ]


class FlceEmbedArgs(ctypes.Structure):
    """Mirror of ``flce_embed_args``."""
    _fields_ = [
        ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("V", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("dE_dtype", ctypes.c_int32),
        ("tokens", ctypes.c_void_p), ("ignore_index", ctypes.c_int64),
        ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
        ("E", ctypes.c_void_p), ("ldE", ctypes.c_int64), ("out", ctypes.c_void_p), ("ldout", ctypes.c_int64),
        ("dout", ctypes.c_void_p), ("lddout", ctypes.c_int64), ("dE", ctypes.c_void_p), ("lddE", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
    ]


class FlceRmsnormArgs(ctypes.Structure):
    """Mirror of ``flce_rmsnorm_args``."""
    _fields_ = [
        ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float), ("flags", ctypes.c_uint32),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("residual", ctypes.c_void_p), ("ldres", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("rstd", ctypes.c_void_p),
        ("y8", ctypes.c_void_p), ("ldy8", ctypes.c_int64), ("y8_scale", ctypes.c_void_p),
        ("h8", ctypes.c_void_p), ("ldh8", ctypes.c_int64), ("h8_scale", ctypes.c_void_p),
    ]


class FlceRmsnormBwdArgs(ctypes.Structure):
    """Mirror of ``flce_rmsnorm_bwd_args``."""
    _fields_ = [
        ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("dweight_dtype", ctypes.c_int32),
        ("weight_offset", ctypes.c_float), ("flags", ctypes.c_uint32),
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
        ("h8", ctypes.c_void_p), ("ldh8", ctypes.c_int64), ("h8_scale", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dweight", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class FlceCkpt8Args(ctypes.Structure):
    """Mirror of ``flce_ckpt8_args``."""
    _fields_ = [
        ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64),
        ("scale", ctypes.c_void_p),
    ]


class FlceCkpt8DwArgs(ctypes.Structure):
    """Mirror of ``flce_ckpt8_dw_args``."""
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("dW_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("wait_timeout_ms", ctypes.c_uint32),
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64),
        ("scale", ctypes.c_void_p), ("dW", ctypes.c_void_p), ("lddW", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
    ]


_lib = None


def load(path: str | None = None):
    """Load libflce.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with linear_cross_entropy_logits_gb300.build.build()")
    lib = ctypes.CDLL(p)
    lib.flce_workspace_size.restype = ctypes.c_size_t
    lib.flce_workspace_size.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_size_t]
    lib.flce_chunk_rows.restype = ctypes.c_int64
    lib.flce_chunk_rows.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_size_t]
    lib.flce_plan_describe.restype = ctypes.c_int64
    lib.flce_plan_describe.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_size_t,
                                                              ctypes.c_char_p, ctypes.c_size_t]
    lib.flce_fwd_bwd.restype = ctypes.c_int32
    lib.flce_fwd_bwd.argtypes = [ctypes.POINTER(FlceArgs), ctypes.c_void_p]
    lib.flce_fwd_bwd_noalloc.restype = ctypes.c_int32
    lib.flce_fwd_bwd_noalloc.argtypes = [ctypes.POINTER(FlceArgs), ctypes.c_void_p]
    lib.flce_get_status.restype = ctypes.c_int32
    lib.flce_get_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.flce_status_string.restype = ctypes.c_char_p
    lib.flce_status_string.argtypes = [ctypes.c_int32]
    lib.flce_abi_version.restype = ctypes.c_int32
    lib.flce_last_cuda_error.restype = ctypes.c_char_p
    lib.flce_last_cuda_error.argtypes = []
    lib.flce_scale_by.restype = ctypes.c_int32
    lib.flce_scale_by.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                  ctypes.c_void_p]
    lib.flce_jsd_workspace_size.restype = ctypes.c_size_t
    lib.flce_jsd_workspace_size.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int32, ctypes.c_size_t]
    lib.flce_fused_linear_jsd.restype = ctypes.c_int32
    lib.flce_fused_linear_jsd.argtypes = [ctypes.POINTER(FlceJsdArgs), ctypes.c_void_p]
    for name, args in (("embed_fwd", FlceEmbedArgs), ("embed_bwd", FlceEmbedArgs),
                       ("rmsnorm_fwd", FlceRmsnormArgs), ("rmsnorm_bwd", FlceRmsnormBwdArgs),
                       ("ckpt8_pack", FlceCkpt8Args), ("ckpt8_dw", FlceCkpt8DwArgs)):
        fn = getattr(lib, "flce_" + name)
        fn.restype = ctypes.c_int32
        fn.argtypes = [ctypes.POINTER(args), ctypes.c_void_p]
    lib.flce_embed_workspace_size.restype = ctypes.c_size_t
    lib.flce_embed_workspace_size.argtypes = [ctypes.c_int64] * 3
    lib.flce_rmsnorm_workspace_size.restype = ctypes.c_size_t
    lib.flce_rmsnorm_workspace_size.argtypes = [ctypes.c_int64] * 2
    lib.flce_ckpt8_dw_workspace_size.restype = ctypes.c_size_t
    lib.flce_ckpt8_dw_workspace_size.argtypes = [ctypes.POINTER(FlceCkpt8DwArgs)]
    lib.flce_profile_create.restype = ctypes.c_void_p
    lib.flce_profile_create.argtypes = []
    lib.flce_profile_reset.restype = None
    lib.flce_profile_reset.argtypes = [ctypes.c_void_p]
    lib.flce_profile_destroy.restype = None
    lib.flce_profile_destroy.argtypes = [ctypes.c_void_p]
    lib.flce_profile_read.restype = ctypes.c_int32
    lib.flce_profile_read.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_float),
                                      ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]
    _lib = lib
    return lib


class FlceError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = f"{where}: {status_string(code)}"
        if code == FLCE_ERR_CUDA:
            msg += f" ({load().flce_last_cuda_error().decode()})"
        super().__init__(msg)


def status_string(code: int) -> str:
    return load().flce_status_string(int(code)).decode()


def workspace_size(BT, H, V, dtype=torch.bfloat16, budget_bytes=0) -> int:
    return int(load().flce_workspace_size(BT, H, V, DTYPES[dtype], budget_bytes))


def chunk_rows(BT, H, V, dtype, workspace_bytes) -> int:
    return int(load().flce_chunk_rows(BT, H, V, DTYPES[dtype], workspace_bytes))


def describe_plan(BT, H, V, dtype=torch.bfloat16, workspace_bytes=None, budget_bytes=0) -> str:
    """The library's text plan of a call (chunk rows, workspace regions, GEMM tiles) for a
    workspace of ``workspace_bytes`` (default: the planner's size for ``budget_bytes``)."""
    lib = load()
    wb = workspace_size(BT, H, V, dtype, budget_bytes) if workspace_bytes is None else workspace_bytes
    n = int(lib.flce_plan_describe(BT, H, V, DTYPES[dtype], wb, None, 0))
    if n < 0:
        raise FlceError(FLCE_ERR_INVALID_ARG, "flce_plan_describe")
    buf = ctypes.create_string_buffer(n + 1)
    lib.flce_plan_describe(BT, H, V, DTYPES[dtype], wb, buf, n + 1)
    return buf.value.decode()


class Profiler:
    """Per-stage device time of the calls that are given this profiler (CUDA events
    recorded by the library on the launching stream)."""

    def __init__(self):
        self._lib = load()
        self.handle = self._lib.flce_profile_create()
        if not self.handle:
            raise MemoryError("flce_profile_create")

    def reset(self):
        self._lib.flce_profile_reset(self.handle)

    def read(self):
        n = len(STAGES)
        ms = (ctypes.c_float * n)()
        cnt = (ctypes.c_int32 * n)()
        rc = self._lib.flce_profile_read(self.handle, ms, cnt, n)
        if rc != FLCE_OK:
            raise FlceError(rc, "flce_profile_read")
        return {s: (float(ms[i]), int(cnt[i])) for i, s in enumerate(STAGES)}

    def close(self):
        if self.handle:
            self._lib.flce_profile_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(stream, fn, kw):
    """fn(**kw) with `stream` as the current one: what the call allocates and fills comes from that
    stream's memory and is ordered with its kernels. Tensors of the caller's are recorded on
    `stream`, those that the call makes on the stream that was current, so that neither is handed
    out again before the other stream is done with it."""
    given = [t for v in kw.values() for t in (v.values() if isinstance(v, dict) else (v,)) if torch.is_tensor(t)]
    if any(t.device != stream.device for t in given):
        raise ValueError(f"stream is on {stream.device}, not every tensor is")
    kw["stream"] = None
    caller = torch.cuda.current_stream(stream.device)
    if caller == stream:
        return fn(**kw)
    with torch.cuda.stream(stream):
        o = fn(**kw)
    for t in given:
        t.record_stream(stream)
    for t in o.values():
        if torch.is_tensor(t) and not any(t is g for g in given):
            t.record_stream(caller)
    return o


def fwd_bwd(X, W, targets, bias=None, *, ignore_index=-100, reduction="mean",
            z_loss_scale=0.0, grad_out=None, want_dX=True, want_dW=True, dW=None, dbias=None,
            workspace=None, workspace_bytes=None, budget_bytes=0, outputs=None, flags=0,
            wait_timeout_ms=0, check=True, stream=None, profiler=None):
    """Fused linear cross entropy forward + backward on X's device.

    X [BT,H] and W [V,H] share a dtype (fp32, bf16 or fp16); targets int64 [BT]. dW/dbias
    are accumulated into when given (fp32, or X's dtype for same-dtype accumulation), else
    allocated as fp32 zeros. Returns a dict of
    tensors: loss, z_loss, acc (reduced per ``reduction``), lse, pred, n_labelled, dX, dW,
    dbias, and the status code when ``check`` is set (which synchronises the stream).
    ``outputs`` may carry preallocated output tensors under the same keys.
    """
    if stream is not None:
        return _on(stream, fwd_bwd, locals())
    lib = load()
    if X.device.type != "cuda":
        raise ValueError("X must be a CUDA tensor")
    BT, H = X.shape
    V = W.shape[0]
    dev = X.device
    red = REDUCTIONS[reduction]
    o = dict(outputs or {})
    nl = BT if reduction == "none" else 1
    if o.get("loss") is None:
        o["loss"] = torch.empty(nl, dtype=torch.float32, device=dev)
    if o.get("z_loss") is None:
        o["z_loss"] = torch.empty(nl, dtype=torch.float32, device=dev)
    if o.get("acc") is None:
        o["acc"] = torch.empty(nl, dtype=torch.float32, device=dev)
    if o.get("lse") is None:
        o["lse"] = torch.empty(BT, dtype=torch.float32, device=dev)
    if o.get("pred") is None:
        o["pred"] = torch.empty(BT, dtype=torch.int64, device=dev)
    if o.get("n_labelled") is None:
        o["n_labelled"] = torch.empty(1, dtype=torch.int32, device=dev)
    if o.get("status") is None:
        o["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if want_dX and o.get("dX") is None:
        o["dX"] = torch.empty_like(X)
    dW_dt = torch.float32 if dW is None else dW.dtype
    if want_dW and dW is None:
        dW = torch.zeros(V, H, dtype=dW_dt, device=dev)
    if want_dW and bias is not None and dbias is None:
        dbias = torch.zeros(V, dtype=dW_dt, device=dev)
    if workspace is None:
        nbytes = workspace_bytes or workspace_size(BT, H, V, X.dtype, budget_bytes)
        if nbytes == 0:
            raise FlceError(FLCE_ERR_WORKSPACE, "workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    if grad_out is not None and not torch.is_tensor(grad_out):
        grad_out = torch.tensor([float(grad_out)], dtype=torch.float32, device=dev)

    a = FlceArgs()
    a.BT, a.H, a.V = BT, H, V
    a.in_dtype = DTYPES[X.dtype]
    a.reduction = red
    a.X, a.W, a.bias = _ptr(X), _ptr(W), _ptr(bias)
    a.targets = _ptr(targets)
    a.ignore_index = ignore_index
    a.z_loss_scale = z_loss_scale
    a.grad_out = _ptr(grad_out)
    a.want_dX, a.want_dW = int(bool(want_dX)), int(bool(want_dW))
    a.dW_dtype = DTYPES[dW_dt]
    a.flags = flags
    a.loss, a.z_loss, a.acc = _ptr(o["loss"]), _ptr(o["z_loss"]), _ptr(o["acc"])
    a.lse, a.pred, a.n_labelled = _ptr(o["lse"]), _ptr(o["pred"]), _ptr(o["n_labelled"])
    a.dX = _ptr(o.get("dX")) if want_dX else None
    a.dW = _ptr(dW) if want_dW else None
    a.dbias = _ptr(dbias) if (want_dW and bias is not None) else None
    a.workspace, a.workspace_bytes = _ptr(workspace), wbytes
    a.status = _ptr(o["status"])
    a.wait_timeout_ms = wait_timeout_ms
    a.profile = profiler.handle if profiler is not None else None
    s = torch.cuda.current_stream(dev)
    rc = lib.flce_fwd_bwd(ctypes.byref(a), ctypes.c_void_p(s.cuda_stream))
    if rc != FLCE_OK:
        raise FlceError(rc, "flce_fwd_bwd")
    o["dW"], o["dbias"] = dW, dbias
    o["workspace"] = workspace
    if check:
        o["status_code"] = int(lib.flce_get_status(ctypes.c_void_p(_ptr(o["status"])), None,
                                                   ctypes.c_void_p(s.cuda_stream)))
    return o


def jsd_workspace_size(BT, Hs, Ht, V, dtype=torch.bfloat16, budget_bytes=0) -> int:
    return int(load().flce_jsd_workspace_size(BT, Hs, Ht, V, DTYPES[dtype], budget_bytes))


def fused_linear_jsd(Xs, Ws, Xt, Wt, labels=None, *, beta=0.5, temperature=1.0, ignore_index=-100,
                     reduction="mean", grad_out=None, want_dX=True, want_dW=True, dW=None,
                     workspace=None, budget_bytes=0, flags=0, check=True, stream=None, profiler=None,
                     outputs=None):
    """Fused linear JSD / KL distillation forward + backward (student gradients only).
    Returns a dict with loss, n_labelled, dX, dW (and status_code when ``check``)."""
    if stream is not None:
        return _on(stream, fused_linear_jsd, locals())
    lib = load()
    BT, Hs = Xs.shape
    Ht = Xt.shape[1]
    V = Ws.shape[0]
    dev = Xs.device
    nl = BT if reduction == "none" else 1
    o = dict(outputs or {})
    if o.get("loss") is None:
        o["loss"] = torch.empty(nl, dtype=torch.float32, device=dev)
    if o.get("n_labelled") is None:
        o["n_labelled"] = torch.empty(1, dtype=torch.int32, device=dev)
    if o.get("status") is None:
        o["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if want_dX and o.get("dX") is None:
        o["dX"] = torch.empty_like(Xs)
    if want_dW and dW is None:
        dW = torch.zeros(V, Hs, dtype=torch.float32, device=dev)
    if workspace is None:
        nbytes = jsd_workspace_size(BT, Hs, Ht, V, Xs.dtype, budget_bytes)
        if nbytes == 0:
            raise FlceError(FLCE_ERR_WORKSPACE, "jsd_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if grad_out is not None and not torch.is_tensor(grad_out):
        grad_out = torch.tensor([float(grad_out)], dtype=torch.float32, device=dev)
    a = FlceJsdArgs()
    a.BT, a.Hs, a.Ht, a.V = BT, Hs, Ht, V
    a.in_dtype = DTYPES[Xs.dtype]
    a.reduction = REDUCTIONS[reduction]
    a.Xs, a.Ws, a.Xt, a.Wt = _ptr(Xs), _ptr(Ws), _ptr(Xt), _ptr(Wt)
    a.labels = _ptr(labels)
    a.ignore_index = ignore_index
    a.beta, a.temperature = beta, temperature
    a.grad_out = _ptr(grad_out)
    a.want_dX, a.want_dW = int(bool(want_dX)), int(bool(want_dW))
    a.dW_dtype = DTYPES[dW.dtype] if dW is not None else 0
    a.flags = flags
    a.loss, a.n_labelled = _ptr(o["loss"]), _ptr(o["n_labelled"])
    a.dX = _ptr(o.get("dX")) if want_dX else None
    a.dW = _ptr(dW) if want_dW else None
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    a.status = _ptr(o["status"])
    a.profile = profiler.handle if profiler is not None else None
    s = torch.cuda.current_stream(dev)
    rc = lib.flce_fused_linear_jsd(ctypes.byref(a), ctypes.c_void_p(s.cuda_stream))
    if rc != FLCE_OK:
        raise FlceError(rc, "flce_fused_linear_jsd")
    o["dW"] = dW
    if check:
        o["status_code"] = int(lib.flce_get_status(ctypes.c_void_p(_ptr(o["status"])), None,
                                                   ctypes.c_void_p(s.cuda_stream)))
    return o


def scale_by(x, g, stream=None):
    """x *= g in place (x: contiguous CUDA tensor, fp32/bf16/fp16; g: one-element fp32 CUDA
    tensor), skipped on the device when g == 1."""
    s = torch.cuda.current_stream(x.device)
    if stream is not None and stream != s:
        x.record_stream(stream)
        g.record_stream(stream)
        s = stream
    rc = load().flce_scale_by(ctypes.c_void_p(x.data_ptr()), x.numel(), DTYPES[x.dtype],
                              ctypes.c_void_p(g.data_ptr()), ctypes.c_void_p(s.cuda_stream))
    if rc != FLCE_OK:
        raise FlceError(rc, "flce_scale_by")
    return x


def raw_call(args: FlceArgs, stream_handle: int) -> int:
    """Call flce_fwd_bwd with a prepared FlceArgs (for callers that manage every buffer)."""
    return int(load().flce_fwd_bwd(ctypes.byref(args), ctypes.c_void_p(stream_handle)))


# ---------------------------------------------------------------------------------------
# Operators around the head: embedding, residual RMS norm, 8-bit checkpoints
# ---------------------------------------------------------------------------------------

def _matrix(name, t, rows, cols, dtype, dev):
    """Checks a [rows, cols] CUDA matrix of unit column stride; returns (pointer, row pitch)."""
    if t.dtype is dtype and t.device == dev and t.shape == (rows, cols):
        if t.is_contiguous():
            return t.data_ptr(), cols
        ld, inner = t.stride()
        if rows <= 1:
            ld = max(ld, cols)
        if (inner == 1 or cols == 1) and ld >= cols:
            return t.data_ptr(), ld
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap, got strides {t.stride()}")
    raise ValueError(f"{name} must be {dtype} [{rows}, {cols}] on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _dense(name, t, shape, dtype, dev):
    """Checks a dense tensor; returns its pointer."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a dense {dtype} tensor {shape} on {dev}, got {t.dtype} {tuple(t.shape)} "
                     f"strides {t.stride()} on {t.device}")


def _cuda_2d(name, t):
    """Checks the operand that decides device and dtype; returns (device, shape, flce_dtype)."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    dt = DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    return dev, shape, dt


def _grad_dtype(name, t):
    dt = DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    return dt


def empty_rows8(N, H, device):
    """An [N, H] e4m3 tensor whose rows start at multiples of 16 bytes."""
    return torch.empty_strided((N, H), ((H + 15) & ~15, 1), dtype=torch.float8_e4m3fn, device=device)


def _workspace(ws, nbytes, dev):
    """The caller's byte workspace, or a new one."""
    if ws is not None:
        if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != dev:
            raise ValueError(f"workspace must be a dense uint8 tensor on {dev}")
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _launch(fn, where, args, dev):
    """Enqueue on the current stream; returns its handle."""
    index = dev.index
    handle = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        rc = fn(args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(args, handle)
    if rc != FLCE_OK:
        raise FlceError(rc, where)
    return handle


def _status(o, status, check, dev):
    """Pointer of the status word: the caller's, a new one when the status is to be checked."""
    if status is None:
        if not check:
            return None
        status = torch.empty(1, dtype=torch.int32, device=dev)
    o["status"] = status
    return _dense("status", status, (1,), torch.int32, dev)


def _finish(o, lib, check, handle):
    if check:
        o["status_code"] = int(lib.flce_get_status(o["status"].data_ptr(), None, handle))
    return o


def embed_fwd(tokens, E, *, scale=1.0, ignore_index=-100, out=None, status=None, check=True, stream=None):
    """out[i] = scale * E[tokens[i]], a zero row where tokens[i] == ignore_index.

    tokens int64 [N], E [V, H] (fp32, bf16 or fp16; unit column stride). Returns a dict with
    out and, when ``check`` is set (which synchronises the stream), status_code: a token
    outside [0, V) gives a zero row and FLCE_ERR_TARGET_RANGE. ``status`` (int32 [1]) receives
    the device status word without a check.
    """
    if stream is not None:
        return _on(stream, embed_fwd, locals())
    lib = _lib or load()
    dev, (V, H), dt = _cuda_2d("E", E)
    N = tokens.shape[0]
    if out is None:
        out = torch.empty((N, H), dtype=E.dtype, device=dev)
    o = {"out": out}
    pE, ldE = _matrix("E", E, V, H, E.dtype, dev)
    po, ldo = _matrix("out", out, N, H, E.dtype, dev)
    a = FlceEmbedArgs(N, H, V, dt, 0, _dense("tokens", tokens, (N,), torch.int64, dev), ignore_index, scale, 0,
                      pE, ldE, po, ldo, None, 0, None, 0, None, 0, _status(o, status, check, dev))
    h = _launch(lib.flce_embed_fwd, "flce_embed_fwd", a, dev)
    return _finish(o, lib, check, h)


def embed_bwd(tokens, dout, *, V=None, dE=None, scale=1.0, ignore_index=-100, workspace=None, flags=0, status=None,
              check=True, stream=None):
    """dE[v] += scale * sum of the rows of dout whose token is v, in fp32 and in a fixed order.

    dout [N, H]; dE [V, H] in fp32 or dout's dtype, accumulated into (FLAG_DW_OVERWRITE: all of
    it is written), for instance the head's own dW of a tied embedding. Without dE a new fp32
    one of ``V`` rows is written. Returns a dict with dE (and status_code when ``check``).
    """
    if stream is not None:
        return _on(stream, embed_bwd, locals())
    lib = _lib or load()
    dev, (N, H), dt = _cuda_2d("dout", dout)
    if dE is None:
        if V is None:
            raise ValueError("embed_bwd needs V or dE")
        dE = torch.empty((V, H), dtype=torch.float32, device=dev)
        flags |= FLAG_DW_OVERWRITE
    V = dE.shape[0]
    workspace = _workspace(workspace, lib.flce_embed_workspace_size(N, H, V), dev)
    o = {"dE": dE, "workspace": workspace}
    pd, ldd = _matrix("dout", dout, N, H, dout.dtype, dev)
    pE, ldE = _matrix("dE", dE, V, H, dE.dtype, dev)
    a = FlceEmbedArgs(N, H, V, dt, _grad_dtype("dE", dE), _dense("tokens", tokens, (N,), torch.int64, dev),
                      ignore_index, scale, flags, None, 0, None, 0, pd, ldd, pE, ldE, workspace.data_ptr(),
                      workspace.numel(), _status(o, status, check, dev))
    h = _launch(lib.flce_embed_bwd, "flce_embed_bwd", a, dev)
    return _finish(o, lib, check, h)


def rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, weight_offset=0.0, want_y=True, want_h=None, want_y8=False,
                want_h8=False, outputs=None, stream=None):
    """h = x + residual, y = h * rstd * (weight + weight_offset), rstd = 1/sqrt(mean(h^2) + eps).

    x and residual [N, H], weight [H], one dtype (fp32, bf16 or fp16). Returns a dict with rstd
    and, as wanted: y; h (default: when a residual is given); y8, y8_scale (the 8-bit output);
    h8, h8_scale (8-bit checkpoint of h for ``rmsnorm_bwd``). ``outputs`` may carry preallocated
    tensors under the same keys; h may be x or residual itself.
    """
    if stream is not None:
        return _on(stream, rmsnorm_fwd, locals())
    lib = _lib or load()
    dev, (N, H), dt = _cuda_2d("x", x)
    dtype = x.dtype
    if want_h is None:
        want_h = residual is not None
    o = {} if outputs is None else _wanted(outputs, rstd=True, y=want_y, h=want_h, y8=want_y8, y8_scale=want_y8,
                                           h8=want_h8, h8_scale=want_h8)
    given = o.get
    px, ldx = _matrix("x", x, N, H, dtype, dev)
    pr, ldr = (None, 0) if residual is None else _matrix("residual", residual, N, H, dtype, dev)
    rstd = given("rstd")
    if rstd is None:
        rstd = o["rstd"] = torch.empty(N, dtype=torch.float32, device=dev)
        prstd = rstd.data_ptr()
    else:
        prstd = _dense("rstd", rstd, (N,), torch.float32, dev)
    (py, ldy) = _row_output(o, "y", x, N, H, dtype, dev) if want_y else (None, 0)
    (ph, ldh) = _row_output(o, "h", x, N, H, dtype, dev) if want_h else (None, 0)
    (py8, ldy8, psy) = _rows8(o, "y8", "y8_scale", N, H, dev) if want_y8 else (None, 0, None)
    (ph8, ldh8, psh) = _rows8(o, "h8", "h8_scale", N, H, dev) if want_h8 else (None, 0, None)
    a = FlceRmsnormArgs(N, H, dt, eps, weight_offset, 0, px, ldx, pr, ldr, _dense("weight", weight, (H,), dtype, dev),
                        ph, ldh, py, ldy, prstd, py8, ldy8, psy, ph8, ldh8, psh)
    _launch(lib.flce_rmsnorm_fwd, "flce_rmsnorm_fwd", a, dev)
    return o


def _wanted(outputs, **wanted):
    """The given outputs that the call writes; others (of an earlier call, say) are not passed on."""
    return {k: t for k, t in outputs.items() if wanted.get(k)}


def _row_output(o, key, like, N, H, dtype, dev):
    """Pointer and pitch of the output matrix o[key], made as `like` if absent."""
    t = o.get(key)
    if t is None:
        t = o[key] = torch.empty_like(like, memory_format=torch.contiguous_format)
        return t.data_ptr(), H
    return _matrix(key, t, N, H, dtype, dev)


def _rows8(o, key, scale_key, N, H, dev):
    """Pointer and pitch of the 8-bit rows o[key] and the pointer of their scales, made if absent."""
    t, s = o.get(key), o.get(scale_key)
    shape = (N, (H + Q_BLOCK - 1) // Q_BLOCK)
    if t is None:
        t = o[key] = empty_rows8(N, H, dev)
        p, ld = t.data_ptr(), (H + 15) & ~15
    else:
        p, ld = _matrix(key, t, N, H, torch.float8_e4m3fn, dev)
    if s is None:
        s = o[scale_key] = torch.empty(shape, dtype=torch.float32, device=dev)
        return p, ld, s.data_ptr()
    return p, ld, _dense(scale_key, s, shape, torch.float32, dev)


def rmsnorm_bwd(dy, weight, rstd, h=None, *, h8=None, h8_scale=None, dh=None, weight_offset=0.0, want_dx=True,
                want_dweight=True, dweight=None, workspace=None, outputs=None, flags=0, stream=None):
    """Gradient of ``rmsnorm_fwd``: dx (of x and residual alike; with ``dh``, the residual
    stream's own gradient, added) and dweight, accumulated into when given (fp32 or dy's dtype;
    FLAG_DW_OVERWRITE: written), else a new fp32 vector. The norm's input is ``h`` or its 8-bit
    checkpoint ``h8, h8_scale``. Returns a dict with dx and dweight."""
    if stream is not None:
        return _on(stream, rmsnorm_bwd, locals())
    lib = _lib or load()
    dev, (N, H), dt = _cuda_2d("dy", dy)
    dtype = dy.dtype
    if (h is None) == (h8 is None) or (h8 is not None and h8_scale is None):
        raise ValueError("rmsnorm_bwd takes h, or h8 with h8_scale")
    o = {} if outputs is None else _wanted(outputs, dx=want_dx)
    (pdx, lddx) = _row_output(o, "dx", dy, N, H, dtype, dev) if want_dx else (None, 0)
    pw = pws = None
    wbytes, wdt = 0, 0
    if want_dweight:
        if dweight is None:
            dweight = torch.empty(H, dtype=torch.float32, device=dev)
            flags |= FLAG_DW_OVERWRITE
        wdt = _grad_dtype("dweight", dweight)
        pw = _dense("dweight", dweight, (H,), dweight.dtype, dev)
        workspace = _workspace(workspace, lib.flce_rmsnorm_workspace_size(N, H), dev)
        pws, wbytes = workspace.data_ptr(), workspace.numel()
        o["dweight"], o["workspace"] = dweight, workspace
    (ph, ldh) = (None, 0) if h is None else _matrix("h", h, N, H, dtype, dev)
    p8 = ps8 = None
    ld8 = 0
    if h8 is not None:
        p8, ld8 = _matrix("h8", h8, N, H, torch.float8_e4m3fn, dev)
        ps8 = _dense("h8_scale", h8_scale, (N, (H + Q_BLOCK - 1) // Q_BLOCK), torch.float32, dev)
    (pdh, lddh) = (None, 0) if dh is None else _matrix("dh", dh, N, H, dtype, dev)
    pdy, lddy = _matrix("dy", dy, N, H, dtype, dev)
    a = FlceRmsnormBwdArgs(N, H, dt, wdt, weight_offset, flags, pdy, lddy, ph, ldh, p8, ld8, ps8,
                           _dense("rstd", rstd, (N,), torch.float32, dev),
                           _dense("weight", weight, (H,), dtype, dev), pdh, lddh, pdx, lddx, pw, pws, wbytes)
    _launch(lib.flce_rmsnorm_bwd, "flce_rmsnorm_bwd", a, dev)
    return o


def ckpt8_pack(x, *, outputs=None, stream=None):
    """8-bit checkpoint of x [N, H]: a dict with q (e4m3 [N, H], rows at multiples of 16 bytes)
    and scale (fp32 [N, ceil(H/128)], powers of two); the value kept is q * scale."""
    if stream is not None:
        return _on(stream, ckpt8_pack, locals())
    lib = _lib or load()
    dev, (N, H), dt = _cuda_2d("x", x)
    o = {} if outputs is None else _wanted(outputs, q=True, scale=True)
    px, ldx = _matrix("x", x, N, H, x.dtype, dev)
    pq, ldq, ps = _rows8(o, "q", "scale", N, H, dev)
    _launch(lib.flce_ckpt8_pack, "flce_ckpt8_pack", FlceCkpt8Args(N, H, dt, 0, px, ldx, pq, ldq, ps), dev)
    return o


def ckpt8_dw(dy, q, scale, *, dW=None, workspace=None, flags=0, wait_timeout_ms=0, status=None, check=True,
             stream=None):
    """Weight gradient of y = x W^T from the 8-bit checkpoint of x: dW += dy^T (q * scale).

    dy [M, N] (fp32, bf16 or fp16), q e4m3 [M, K], scale fp32 [M, ceil(K/128)]; dW [N, K] in
    fp32 or dy's dtype, accumulated into (FLAG_DW_OVERWRITE: written), else a new fp32 one.
    Returns a dict with dW (and status_code when ``check``, which synchronises the stream).
    """
    if stream is not None:
        return _on(stream, ckpt8_dw, locals())
    lib = _lib or load()
    dev, (M, N), dt = _cuda_2d("dy", dy)
    if q.dim() != 2:
        raise ValueError(f"q must be 2-D, got {tuple(q.shape)}")
    K = q.shape[1]
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=dev)
        flags |= FLAG_DW_OVERWRITE
    o = {"dW": dW}
    pdy, lddy = _matrix("dy", dy, M, N, dy.dtype, dev)
    pq, ldq = _matrix("q", q, M, K, torch.float8_e4m3fn, dev)
    pW, ldW = _matrix("dW", dW, N, K, dW.dtype, dev)
    a = FlceCkpt8DwArgs(M, N, K, dt, _grad_dtype("dW", dW), flags, wait_timeout_ms, pdy, lddy, pq, ldq,
                        _dense("scale", scale, (M, (K + Q_BLOCK - 1) // Q_BLOCK), torch.float32, dev), pW, ldW,
                        None, 0, _status(o, status, check, dev))
    workspace = o["workspace"] = _workspace(workspace, lib.flce_ckpt8_dw_workspace_size(a), dev)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    h = _launch(lib.flce_ckpt8_dw, "flce_ckpt8_dw", a, dev)
    return _finish(o, lib, check, h)
