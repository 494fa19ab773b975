"""Thin Python binding of the C ABI in include/rmsnorm.h (ctypes).

Argument marshalling only: every step of the RMSNorm forward runs in the CUDA
library. The raw functions keep the C names and take integer device
addresses; ``fwd`` is a convenience over torch tensors (torch supplies device
memory and the current stream, nothing else). There is no fallback: if the
library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

BF16, FP16, FP32 = 0, 1, 2
VARIANTS = {"auto": 0, "warp": 1, "cta": 2, "tma": 3, "generic": 4, "cluster": 5}
VARIANT_NAMES = {v: k for k, v in VARIANTS.items()}
STATUS = {
    0: "RMSNORM_OK", -1: "RMSNORM_ERR_NULL", -2: "RMSNORM_ERR_SHAPE", -3: "RMSNORM_ERR_DTYPE",
    -4: "RMSNORM_ERR_SCALAR", -5: "RMSNORM_ERR_OVERLAP", -6: "RMSNORM_ERR_CUDA",
    -7: "RMSNORM_ERR_DEVICE_TIMEOUT", -8: "RMSNORM_ERR_UNSUPPORTED", -9: "RMSNORM_ERR_OPTIONS",
    -10: "RMSNORM_ERR_ALIGN", -11: "RMSNORM_ERR_WORKSPACE", -12: "RMSNORM_ERR_DEVICE_INDEX",
}
# Every function include/rmsnorm.h declares.
EXPORTS = ("rmsnorm_fwd", "rmsnorm_fwd_ex", "rmsnorm_fwd_strided", "rmsnorm_fwd_host",
           "rmsnorm_fwd_host_workspace_size", "rmsnorm_bwd", "rmsnorm_bwd_noalloc",
           "rmsnorm_bwd_workspace_size", "rmsnorm_plan_info", "rmsnorm_bwd_plan_info",
           "rmsnorm_block_fwd", "rmsnorm_block_bwd", "rmsnorm_block_bwd_workspace_size",
           "rmsnorm_rope_fwd", "rmsnorm_rope_bwd", "rmsnorm_rope_bwd_workspace_size",
           "rmsnorm_rope_steps", "rmsnorm_cache_write", "rmsnorm_cache_read",
           "rmsnorm_check_device_status",
           "rmsnorm_strerror", "rmsnorm_last_error", "rmsnorm_version")


class RMSNormError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class Options(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("max_ctas", ctypes.c_int32), ("lanes_per_row", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("rows_per_stage", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("cluster_size", ctypes.c_int32),
                ("wait_limit_ns", ctypes.c_int64), ("l2_prefetch", ctypes.c_int32),
                ("prewait_prefetch", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "variant", "threads", "grid", "lanes_per_row", "vecs_per_lane", "rows_per_stage",
        "stages", "smem_bytes", "ctas_per_sm", "sm_count", "cluster_size", "l2_prefetch",
        "prewait_prefetch")]

    def as_dict(self) -> dict:
        d = {n: getattr(self, n) for n, _ in self._fields_}
        d["variant"] = VARIANT_NAMES.get(d["variant"], d["variant"])
        return d


# Argument structs of the block, rope and cache operators (field names and order
# of include/rmsnorm.h).
_I, _Q, _F, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class BlockArgs(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("dtype", _I), ("M", _Q), ("N", _Q), ("gate_rows", _Q)]
                + [(n, _P) for n in ("h", "r", "w_post", "gate", "w_pre", "s", "y", "rstd_post",
                                     "rstd_pre")]
                + [(n, _Q) for n in ("ldh", "ldr", "ldg", "lds", "ldy")]
                + [(n, _F) for n in ("eps", "offset", "alpha", "beta")])


class BlockGrads(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("reserved", _I)]
                + [(n, _P) for n in ("dy", "ds", "dh", "dr", "dgate", "dw_post", "dw_pre")]
                + [(n, _Q) for n in ("lddy", "ldds", "lddh", "lddr", "lddg")])


class Heads(ctypes.Structure):
    _fields_ = [("ptr", _P), ("batch_stride", _Q), ("token_stride", _Q), ("head_stride", _Q)]


class RopeArgs(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("dtype", _I), ("batch", _Q), ("seq", _Q)]
                + [(n, _I) for n in ("heads_q", "heads_k", "head_dim", "rotary_dim", "interleaved",
                                     "reserved")]
                + [("positions", _P), ("positions_stride", _Q)]
                + [(n, _P) for n in ("steps", "w_q", "w_k", "rstd_q", "rstd_k")]
                + [(n, _F) for n in ("eps", "offset", "magnitude", "reserved_f")]
                + [(n, Heads) for n in ("q", "k", "out_q", "out_k")])


class RopeGrads(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("reserved", _I)]
                + [(n, Heads) for n in ("dout_q", "dout_k", "dq", "dk")]
                + [("dw_q", _P), ("dw_k", _P)])


class RopeScaling(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("kind", _I)]
                + [(n, ctypes.c_double) for n in ("factor", "length", "beta_fast", "beta_slow")])


class CacheArgs(ctypes.Structure):
    _fields_ = ([("struct_size", _I), ("format", _I), ("pages", _Q)]
                + [(n, _I) for n in ("page_size", "heads", "head_dim", "heads_first")]
                + [(n, _P) for n in ("k_codes", "k_scales", "v_codes", "v_scales")])


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded CUDA library. Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(
                    f"RMSNorm CUDA library not built ({path} missing); run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(path)
            vp, i64, f32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
            L.rmsnorm_fwd.argtypes = [vp, vp, vp, vp, i64, i64, f32, f32, i32, vp]
            L.rmsnorm_fwd.restype = i32
            L.rmsnorm_fwd_ex.argtypes = [vp, vp, vp, vp, i64, i64, f32, f32, i32,
                                         ctypes.POINTER(Options), vp]
            L.rmsnorm_fwd_ex.restype = i32
            L.rmsnorm_fwd_strided.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, f32, f32, i32,
                                              ctypes.POINTER(Options), vp]
            L.rmsnorm_fwd_strided.restype = i32
            L.rmsnorm_fwd_host.argtypes = [vp, vp, vp, vp, i64, i64, f32, f32, i32, i64, vp, i64,
                                           ctypes.POINTER(Options), vp]
            L.rmsnorm_fwd_host.restype = i32
            L.rmsnorm_fwd_host_workspace_size.argtypes = [i64, i64, i32, i64,
                                                          ctypes.POINTER(ctypes.c_int64)]
            L.rmsnorm_fwd_host_workspace_size.restype = i32
            L.rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, f32, i32, vp, i64,
                                      ctypes.POINTER(Options), vp]
            L.rmsnorm_bwd.restype = i32
            L.rmsnorm_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, f32, i32,
                                              ctypes.POINTER(Options), vp]
            L.rmsnorm_bwd_noalloc.restype = i32
            L.rmsnorm_bwd_workspace_size.argtypes = [i64, i64, i32, ctypes.POINTER(Options),
                                                     ctypes.POINTER(ctypes.c_int64)]
            L.rmsnorm_bwd_workspace_size.restype = i32
            L.rmsnorm_plan_info.argtypes = [i64, i64, i32, vp, vp, vp, ctypes.POINTER(Options),
                                            ctypes.POINTER(Plan)]
            L.rmsnorm_plan_info.restype = i32
            L.rmsnorm_bwd_plan_info.argtypes = [i64, i64, i32, ctypes.POINTER(Options),
                                                ctypes.POINTER(Plan)]
            L.rmsnorm_bwd_plan_info.restype = i32
            # Argument structs: a ctypes structure by reference, or its packed bytes.
            L.rmsnorm_block_fwd.argtypes = [vp, ctypes.POINTER(Options), vp]
            L.rmsnorm_block_bwd.argtypes = [vp, vp, vp, i64, ctypes.POINTER(Options), vp]
            L.rmsnorm_block_bwd_workspace_size.argtypes = [i64, i64, i32,
                                                           ctypes.POINTER(ctypes.c_int64)]
            L.rmsnorm_rope_fwd.argtypes = [vp, ctypes.POINTER(Options), vp]
            L.rmsnorm_rope_bwd.argtypes = [vp, vp, vp, i64, ctypes.POINTER(Options), vp]
            L.rmsnorm_rope_bwd_workspace_size.argtypes = [i32, ctypes.POINTER(ctypes.c_int64)]
            L.rmsnorm_rope_steps.argtypes = [i32, ctypes.c_double, vp, vp, vp]
            L.rmsnorm_cache_write.argtypes = [vp, vp, vp, vp, i64, i32, ctypes.POINTER(Options), vp]
            L.rmsnorm_cache_read.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, i32,
                                             ctypes.POINTER(Options), vp]
            for name in EXPORTS:
                if name.startswith(("rmsnorm_block", "rmsnorm_rope", "rmsnorm_cache")):
                    getattr(L, name).restype = i32
            L.rmsnorm_check_device_status.argtypes = [vp]
            L.rmsnorm_check_device_status.restype = i32
            L.rmsnorm_strerror.argtypes = [i32]
            L.rmsnorm_strerror.restype = ctypes.c_char_p
            L.rmsnorm_last_error.argtypes = []
            L.rmsnorm_last_error.restype = ctypes.c_char_p
            L.rmsnorm_version.argtypes = []
            L.rmsnorm_version.restype = i32
            _lib = L
    return _lib


def _check(rc: int) -> int:
    if rc != 0:
        raise RMSNormError(rc, lib().rmsnorm_last_error().decode())
    return rc


FLAG_NO_PDL = 1
FLAG_BLOCKED_ROWS = 2
FLAG_EARLY_LOADS = 4
FLAG_HOST_DIRECT = 8
FLAG_EARLY_WEIGHTS = 16
FLAG_BULK_STORE = 32


def make_options(variant: str | int = "auto", max_ctas: int = 0, lanes_per_row: int = 0,
                 stages: int = 0, rows_per_stage: int = 0, wait_limit_ns: int = 0,
                 pdl: bool = True, blocked: bool = False, early_loads: bool = False,
                 cluster_size: int = 0, host_direct: bool = False,
                 early_weights: bool = False, bulk_store: bool = False,
                 l2_prefetch: int = 0, prewait_prefetch: int = 0) -> Options:
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    flags = ((0 if pdl else FLAG_NO_PDL) | (FLAG_BLOCKED_ROWS if blocked else 0)
             | (FLAG_EARLY_LOADS if early_loads else 0) | (FLAG_HOST_DIRECT if host_direct else 0)
             | (FLAG_EARLY_WEIGHTS if early_weights else 0) | (FLAG_BULK_STORE if bulk_store else 0))
    return Options(ctypes.sizeof(Options), v, max_ctas, lanes_per_row, stages, rows_per_stage,
                   flags, cluster_size, wait_limit_ns, l2_prefetch, prewait_prefetch)


# ---- raw C ABI (integer device addresses) --------------------------------

def rmsnorm_fwd(x: int, w: int, y: int, rstd: int, M: int, N: int, eps: float, offset: float,
                dtype: int, stream: int) -> int:
    return lib().rmsnorm_fwd(x, w, y, rstd, M, N, eps, offset, dtype, stream)


def rmsnorm_fwd_ex(x: int, w: int, y: int, rstd: int, M: int, N: int, eps: float, offset: float,
                   dtype: int, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_fwd_ex(x, w, y, rstd, M, N, eps, offset, dtype,
                                ctypes.byref(opts) if opts is not None else None, stream)


def rmsnorm_fwd_strided(x: int, ldx: int, w: int, y: int, ldy: int, rstd: int, M: int, N: int,
                        eps: float, offset: float, dtype: int, opts: Options | None,
                        stream: int) -> int:
    return lib().rmsnorm_fwd_strided(x, ldx, w, y, ldy, rstd, M, N, eps, offset, dtype,
                                     ctypes.byref(opts) if opts is not None else None, stream)


def rmsnorm_fwd_host(x_host: int, w: int, y_host: int, rstd_host: int, M: int, N: int,
                     eps: float, offset: float, dtype: int, chunk_rows: int, workspace: int,
                     workspace_bytes: int, opts: Options | None, stream: int) -> int:
    """The forward over host-resident x/y/rstd (w and the workspace on the device)."""
    return lib().rmsnorm_fwd_host(x_host, w, y_host, rstd_host, M, N, eps, offset, dtype,
                                  chunk_rows, workspace, workspace_bytes,
                                  ctypes.byref(opts) if opts is not None else None, stream)


def rmsnorm_fwd_host_workspace_size(M: int, N: int, dtype: int, chunk_rows: int = 0) -> int:
    out = ctypes.c_int64(0)
    _check(lib().rmsnorm_fwd_host_workspace_size(M, N, dtype, chunk_rows, ctypes.byref(out)))
    return out.value


def rmsnorm_bwd(x: int, w: int, rstd: int, dy: int, dx: int, dw: int, M: int, N: int,
                offset: float, dtype: int, workspace: int, workspace_bytes: int,
                opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_bwd(x, w, rstd, dy, dx, dw, M, N, offset, dtype, workspace,
                             workspace_bytes, ctypes.byref(opts) if opts is not None else None,
                             stream)


def rmsnorm_bwd_noalloc(x: int, w: int, rstd: int, dy: int, dx: int, dw: int, M: int, N: int,
                        offset: float, dtype: int, opts: Options | None, stream: int) -> int:
    """rmsnorm_bwd with the library's built-in scratch instead of a workspace
    (for callers that cannot allocate device memory at the call)."""
    return lib().rmsnorm_bwd_noalloc(x, w, rstd, dy, dx, dw, M, N, offset, dtype,
                                     ctypes.byref(opts) if opts is not None else None, stream)


def rmsnorm_bwd_workspace_size(M: int, N: int, dtype: int, opts: Options | None = None) -> int:
    out = ctypes.c_int64(0)
    _check(lib().rmsnorm_bwd_workspace_size(M, N, dtype,
                                            ctypes.byref(opts) if opts is not None else None,
                                            ctypes.byref(out)))
    return out.value


def rmsnorm_plan_info(M: int, N: int, dtype: int, x: int = 0, w: int = 0, y: int = 0,
                      opts: Options | None = None) -> dict:
    out = Plan()
    _check(lib().rmsnorm_plan_info(M, N, dtype, x, w, y,
                                   ctypes.byref(opts) if opts is not None else None,
                                   ctypes.byref(out)))
    return out.as_dict()


def rmsnorm_bwd_plan_info(M: int, N: int, dtype: int, opts: Options | None = None) -> dict:
    """The backward row kernel's launch for aligned buffers (no launch)."""
    out = Plan()
    _check(lib().rmsnorm_bwd_plan_info(M, N, dtype, ctypes.byref(opts) if opts is not None else None,
                                       ctypes.byref(out)))
    return out.as_dict()


def _arg(s):
    """An argument struct as the library takes it: packed bytes as they are."""
    return s if s is None or isinstance(s, bytes) else ctypes.byref(s)


def _opt(opts: Options | None):
    return ctypes.byref(opts) if opts is not None else None


def rmsnorm_block_fwd(args: BlockArgs | bytes, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_block_fwd(_arg(args), _opt(opts), stream)


def rmsnorm_block_bwd(args: BlockArgs | bytes, grads: BlockGrads | bytes, workspace: int,
                      workspace_bytes: int, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_block_bwd(_arg(args), _arg(grads), workspace, workspace_bytes, _opt(opts),
                                   stream)


def rmsnorm_block_bwd_workspace_size(M: int, N: int, dtype: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().rmsnorm_block_bwd_workspace_size(M, N, dtype, ctypes.byref(out)))
    return out.value


def rmsnorm_rope_fwd(args: RopeArgs | bytes, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_rope_fwd(_arg(args), _opt(opts), stream)


def rmsnorm_rope_bwd(args: RopeArgs | bytes, grads: RopeGrads | bytes, workspace: int,
                     workspace_bytes: int, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_rope_bwd(_arg(args), _arg(grads), workspace, workspace_bytes, _opt(opts),
                                  stream)


def rmsnorm_rope_bwd_workspace_size(head_dim: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().rmsnorm_rope_bwd_workspace_size(head_dim, ctypes.byref(out)))
    return out.value


def rmsnorm_rope_steps(rotary_dim: int, base: float, scaling: RopeScaling | None, steps: int,
                       magnitude: int = 0) -> int:
    """Steps into host memory at the address `steps` (rotary_dim / 2 64-bit
    values) and the magnitude into the float at `magnitude` (0: not wanted)."""
    return lib().rmsnorm_rope_steps(rotary_dim, base, _arg(scaling), steps, magnitude or None)


def rmsnorm_cache_write(cache: CacheArgs | bytes, k: Heads | bytes | None, v: Heads | bytes | None,
                        slots: int, T: int, dtype: int, opts: Options | None, stream: int) -> int:
    return lib().rmsnorm_cache_write(_arg(cache), _arg(k), _arg(v), slots, T, dtype, _opt(opts),
                                     stream)


def rmsnorm_cache_read(cache: CacheArgs | bytes, table: int, table_width: int, cu_rows: int,
                       starts: int, sequences: int, rows: int, k_out: Heads | bytes | None,
                       v_out: Heads | bytes | None, dtype: int, opts: Options | None,
                       stream: int) -> int:
    return lib().rmsnorm_cache_read(_arg(cache), table, table_width, cu_rows, starts, sequences,
                                    rows, _arg(k_out), _arg(v_out), dtype, _opt(opts), stream)


def rmsnorm_check_device_status(stream: int = 0) -> int:
    return lib().rmsnorm_check_device_status(stream)


def rmsnorm_strerror(status: int) -> str:
    return lib().rmsnorm_strerror(status).decode()


def rmsnorm_last_error() -> str:
    return lib().rmsnorm_last_error().decode()


def rmsnorm_version() -> int:
    return lib().rmsnorm_version()


# ---- torch convenience ---------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"RMSNorm takes bf16, fp16 or fp32 activations, got {t.dtype}")


def fwd(x, w, eps: float = 1e-6, offset: float = 0.0, y=None, rstd=None, stream=None,
        **options):
    """y, rstd = fwd(x, w): RMSNorm forward of a contiguous CUDA tensor x[..., N].

    ``y`` and ``rstd`` may be passed to write in place (y may be x itself);
    ``rstd=False`` skips storing rstd (inference). 2-D ``x``/``y`` views with unit
    column stride (rows of wider tensors) go through ``rmsnorm_fwd_strided``.
    Keyword ``options`` go to :func:`make_options` (variant, max_ctas, ...).
    Runs on ``stream`` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    if not (x.is_cuda and w.is_cuda):
        raise ValueError("x and w must be CUDA tensors")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    N = x.shape[-1]
    if w.dtype != x.dtype or w.numel() != N:
        raise ValueError("w must have x's dtype and N elements")
    if x.is_contiguous():
        M, ldx = (x.numel() // N if N else 0), N
    elif x.dim() == 2 and x.stride(1) == 1:
        M, ldx = x.shape[0], x.stride(0)  # rows of a wider tensor
    else:
        raise ValueError("x must be contiguous, or 2-D with unit column stride")
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    ldy = y.stride(0) if (y.dim() == 2 and not y.is_contiguous()) else N
    if y.shape != x.shape or (ldy == N and not y.is_contiguous()):
        raise ValueError("y must have x's shape, contiguous or 2-D with unit column stride")
    if rstd is None:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    r_ptr = 0 if rstd is False else rstd.data_ptr()
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    opts = make_options(**options) if options else None
    with torch.cuda.device(x.device):
        _check(rmsnorm_fwd_strided(x.data_ptr(), ldx, w.data_ptr(), y.data_ptr(), ldy, r_ptr, M,
                                   N, eps, offset, _dtype_code(x), opts, s.cuda_stream))
    return y, (None if rstd is False else rstd)


def fwd_host(x, w, eps: float = 1e-6, offset: float = 0.0, y=None, rstd=None,
             chunk_rows: int = 0, workspace=None, stream=None, **options):
    """y, rstd = fwd_host(x, w): the forward of a contiguous CPU tensor x[..., N]
    (pinned for overlapped copies) with w on the GPU, through rmsnorm_fwd_host.

    ``y`` and ``rstd`` are CPU tensors (allocated pinned when not given; y may be
    x itself); ``rstd=False`` skips rstd. The device ``workspace`` (a CUDA tensor)
    is allocated here with torch when not given (none with ``host_direct=True``:
    the kernel then reads and writes the pinned host buffers itself). The call
    is asynchronous on
    ``stream`` (or the current stream of w's device): synchronise before reading.
    """
    import torch
    if x.is_cuda or not w.is_cuda:
        raise ValueError("x must be a CPU tensor and w a CUDA tensor")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    N = x.shape[-1]
    if w.dtype != x.dtype or w.numel() != N:
        raise ValueError("w must have x's dtype and N elements")
    M = x.numel() // N if N else 0
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype).pin_memory()
    if y.shape != x.shape or y.dtype != x.dtype or y.is_cuda or not y.is_contiguous():
        raise ValueError("y must be a contiguous CPU tensor like x")
    if rstd is None:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32).pin_memory()
    r_ptr = 0 if rstd is False else rstd.data_ptr()
    code = _dtype_code(x)
    opts = make_options(**options) if options else None
    with torch.cuda.device(w.device):
        need = rmsnorm_fwd_host_workspace_size(M, N, code, chunk_rows)
        if workspace is None and not options.get("host_direct"):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=w.device)
        s = stream if stream is not None else torch.cuda.current_stream(w.device)
        ws_ptr = 0 if workspace is None else workspace.data_ptr()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(rmsnorm_fwd_host(x.data_ptr(), w.data_ptr(), y.data_ptr(), r_ptr, M, N, eps,
                                offset, code, chunk_rows, ws_ptr, ws_bytes, opts, s.cuda_stream))
    return y, (None if rstd is False else rstd)


def bwd(x, w, rstd, dy, offset: float = 0.0, dx=None, stream=None, **options):
    """dx, dw = bwd(x, w, rstd, dy): backward of ``fwd`` for contiguous CUDA tensors.

    The fp32 workspace for the dw partials is allocated here with torch (the C
    library never allocates); dw comes back in fp32.
    """
    import torch
    N = x.shape[-1]
    M = x.numel() // N if N else 0
    if dx is None:
        dx = torch.empty_like(x)
    dw = torch.empty(N, dtype=torch.float32, device=x.device)
    opts = make_options(**options) if options else None
    with torch.cuda.device(x.device):
        nbytes = rmsnorm_bwd_workspace_size(M, N, _dtype_code(x), opts)
        ws = torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=x.device)
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        _check(rmsnorm_bwd(x.data_ptr(), w.data_ptr(), rstd.data_ptr(), dy.data_ptr(),
                           dx.data_ptr(), dw.data_ptr(), M, N, offset, _dtype_code(x),
                           ws.data_ptr(), ws.numel() * 4, opts, s.cuda_stream))
        # The workspace was allocated on the current stream; keep it from being
        # reused before the work on `s` is done.
        ws.record_stream(s)
    return dx, dw


# ---- the operators between a block's matrix products -----------------------
#
# Calls of a decoding step are host-bound, so these pack their argument structs
# with struct.Struct, check a tensor in one expression and make no context managers
# unless the tensors' device or the stream is not the current one.

_BLOCK = struct.Struct("=2i3q9Q5q4f")
_BLOCK_GRADS = struct.Struct("=2i7Q5q")
_ROPE = struct.Struct("=2i2q6iQq5Q4f" + "Q3q" * 4)
_ROPE_GRADS = struct.Struct("=2i" + "Q3q" * 4 + "2Q")
_CACHE = struct.Struct("=2iq4i4Q")
_HEADS = struct.Struct("=Q3q")
CACHE_FORMATS = {"e4m3": 0, "e2m1": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_CODES: dict = {}
_sizes: dict = {}  # workspace bytes by device and sizes


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        import torch
        _CODES.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
        if dtype not in _CODES:
            raise TypeError(f"RMSNorm takes bf16, fp16 or fp32 activations, got {dtype}")
        code = _CODES[dtype]
    return code


def _elsewhere(t, stream):
    """None where `t` is on the current device and no stream is given; else a
    context in which both are current (outputs and workspaces made there belong
    to that stream)."""
    import torch
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        return None if t.get_device() == torch.cuda.current_device() else torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _stream_ptr(device: int) -> int:
    """The current stream of a device (torch's own accessor of the address where it
    has one: 0.1 us against 2.9 for a Stream object)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _workspace(t, size, *key):
    """A workspace of size(*key) bytes on t's device, the current one."""
    import torch
    n = _sizes.get((size, t.get_device(), key))
    if n is None:
        if len(_sizes) >= 4096:  # ragged batches: as many sizes as lengths
            _sizes.clear()
        n = _sizes[(size, t.get_device(), key)] = size(*key)
    return t.new_empty(n, dtype=torch.uint8)


def _given(workspace, device):
    """(address, bytes) of a workspace, which may be a caller's: all of its bytes and no
    others."""
    if workspace.get_device() != device:
        raise ValueError(f"workspace must be on cuda:{device}, got {workspace.device}")
    if not workspace.is_contiguous():  # a view's bytes are not numel * element size from its start
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _refuse(t, name, shape, dtype, device):
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, shape, dtype, device, N):
    """(address, row stride) of a matrix of rows given as [..., N]."""
    if t is None:
        return 0, 0
    if t.shape == shape and t.dtype is dtype and t.get_device() == device:
        if t.is_contiguous():
            return t.data_ptr(), N
        if t.dim() == 2 and (t.stride(1) == 1 or N == 1):
            return t.data_ptr(), t.stride(0)
    _refuse(t, name, shape, dtype, device)
    raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")


def _vector(t, name, n, dtype, device):
    """The address of n contiguous elements (0 for None)."""
    if t is None:
        return 0
    if t.numel() == n and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, None, dtype, device)
    raise ValueError(f"{name} must be contiguous with {n} elements")


def _gate(gate, gate_rows, dtype, device, M, N):
    """(address, row stride, rows of h per gate row) of a gate [N] or [..., N]."""
    if gate is None:
        if gate_rows:
            raise ValueError("gate_rows without a gate")
        return 0, 0, 0
    _refuse(gate, "gate", None, dtype, device)
    if gate.shape[-1] != N:
        raise ValueError(f"gate must have {N} columns, got {tuple(gate.shape)}")
    G = gate.numel() // N if N else 0
    if not gate_rows:
        if gate.dim() == 1 or G == 1 or M == 0:
            gate_rows = max(M, 1)
        else:
            gate_rows = M // G if G and M % G == 0 else 0
    if gate_rows < 1 or -(-M // gate_rows) != G and M > 0:
        raise ValueError(f"{G} gate rows do not divide {M} rows: give gate_rows, the rows per gate row")
    if gate.is_contiguous() or G <= 1 and gate.stride(-1) == 1:
        return gate.data_ptr(), N, gate_rows
    if gate.dim() == 3 and gate.shape[1] == 1:
        gate = gate[:, 0]
    if gate.dim() == 2 and (gate.stride(1) == 1 or N == 1):
        return gate.data_ptr(), gate.stride(0), gate_rows
    raise ValueError("gate must be contiguous, or 2-D with unit column stride")


def block_fwd(h, r, w_post=None, w_pre=None, gate=None, gate_rows=None, eps: float = 1e-6,
              offset: float = 0.0, alpha: float = 1.0, beta: float = 1.0, s=None, y=None,
              rstd: bool = True, stream=None, **options):
    """s, y, rstd_post, rstd_pre = block_fwd(h, r, w_post, w_pre): the norm after a
    block, its gate, the scaled residual and the norm before the next block.

        n = h * rstd_post * (offset + w_post);  s = beta * r + alpha * gate * n
        y = s * rstd_pre * (offset + w_pre)

    h, r: CUDA tensors [..., N] (contiguous, or 2-D with unit column stride).
    Without w_post there is no norm of h, without w_pre no y (None). ``gate`` is
    [N] (a gate per channel), h's shape (per element), or [G, N] or [G, 1, N]
    with ``gate_rows`` consecutive rows of h per gate row (default M / G). ``s`` and
    ``y`` may be passed to write into (each may be h or r); ``rstd=False`` keeps no
    rstd. Options as for :func:`make_options` (variant, max_ctas, pdl).
    """
    import torch
    ctx = _elsewhere(h, stream)
    if ctx is not None:
        with ctx:
            return block_fwd(h, r, w_post, w_pre, gate, gate_rows, eps, offset, alpha, beta, s, y,
                             rstd, **options)
    shape, dtype, dev = h.shape, h.dtype, h.get_device()
    N = shape[-1]
    M = h.numel() // N if N else 0
    code = _code(dtype)
    hp, ldh = _rows(h, "h", shape, dtype, dev, N)
    rp, ldr = _rows(r, "r", shape, dtype, dev, N)
    gp, ldg, gate_rows = _gate(gate, gate_rows, dtype, dev, M, N)
    wpost = _vector(w_post, "w_post", N, dtype, dev)
    wpre = _vector(w_pre, "w_pre", N, dtype, dev)
    lds = ldy = N
    if s is None:
        s = h.new_empty(shape)
        sp = s.data_ptr()
    else:
        sp, lds = _rows(s, "s", shape, dtype, dev, N)
    yp = 0
    if y is not None:
        if not wpre:
            raise ValueError("y without w_pre")
        yp, ldy = _rows(y, "y", shape, dtype, dev, N)
    elif wpre:
        y = h.new_empty(shape)
        yp = y.data_ptr()
    a = b = None
    ap = bp = 0
    if rstd:
        if wpost:
            a = h.new_empty(shape[:-1], dtype=torch.float32)
            ap = a.data_ptr()
        if wpre:
            b = h.new_empty(shape[:-1], dtype=torch.float32)
            bp = b.data_ptr()
    args = _BLOCK.pack(160, code, M, N, gate_rows, hp, rp, wpost, gp, wpre, sp, yp, ap, bp,
                       ldh, ldr, ldg, lds, ldy, eps, offset, alpha, beta)
    rc = (_lib or lib()).rmsnorm_block_fwd(args, _opt(make_options(**options)) if options else None,
                                           _stream_ptr(dev))
    if rc:
        _check(rc)
    return s, y, a, b


def block_bwd(h, s, rstd_post, rstd_pre, dy=None, ds=None, w_post=None, w_pre=None, gate=None,
              gate_rows=None, offset: float = 0.0, alpha: float = 1.0, beta: float = 1.0, dh=None,
              dr=None, workspace=None, stream=None, **options):
    """dh, dr, dgate, dw_post, dw_pre = block_bwd(h, s, rstd_post, rstd_pre, dy, ds, ...):
    backward of :func:`block_fwd` from the gradients dy of y and ds of s (None:
    zero), the s and rstd that the forward returned and its other arguments.

    dgate is in the gate's shape and dtype, dw_post and dw_pre in fp32 (None
    without gate, w_post, w_pre; zeros where there are no rows). ``workspace`` is a
    contiguous CUDA tensor of at least rmsnorm_block_bwd_workspace_size() bytes;
    allocated here when not given.
    """
    import torch
    ctx = _elsewhere(h, stream)
    if ctx is not None:
        with ctx:
            return block_bwd(h, s, rstd_post, rstd_pre, dy, ds, w_post, w_pre, gate, gate_rows,
                             offset, alpha, beta, dh, dr, workspace, **options)
    shape, dtype, dev = h.shape, h.dtype, h.get_device()
    N = shape[-1]
    M = h.numel() // N if N else 0
    code, f32 = _code(dtype), torch.float32
    hp, ldh = _rows(h, "h", shape, dtype, dev, N)
    sp, lds = _rows(s, "s", shape, dtype, dev, N)
    dyp, lddy = _rows(dy, "dy", shape, dtype, dev, N)
    dsp, ldds = _rows(ds, "ds", shape, dtype, dev, N)
    gp, ldg, gate_rows = _gate(gate, gate_rows, dtype, dev, M, N)
    wpost = _vector(w_post, "w_post", N, dtype, dev)
    wpre = _vector(w_pre, "w_pre", N, dtype, dev)
    ap = _vector(rstd_post, "rstd_post", M, f32, dev) if wpost else 0
    bp = _vector(rstd_pre, "rstd_pre", M, f32, dev) if wpre else 0
    lddh = lddr = N
    if dh is None:
        dh = h.new_empty(shape)
        dhp = dh.data_ptr()
    else:
        dhp, lddh = _rows(dh, "dh", shape, dtype, dev, N)
    if dr is None:
        dr = h.new_empty(shape)
        drp = dr.data_ptr()
    else:
        drp, lddr = _rows(dr, "dr", shape, dtype, dev, N)
    dgate = dwa = dwb = None
    dgp = dwap = dwbp = lddg = 0
    if gate is not None:
        # no row: the sum of nothing, which no kernel writes
        dgate = h.new_empty(gate.shape) if M else h.new_zeros(gate.shape)
        dgp, lddg = dgate.data_ptr(), N
    if wpost:
        dwa = h.new_empty(N, dtype=f32)
        dwap = dwa.data_ptr()
    if wpre:
        dwb = h.new_empty(N, dtype=f32)
        dwbp = dwb.data_ptr()
    if workspace is None:
        workspace = _workspace(h, rmsnorm_block_bwd_workspace_size, M, N, code)
    ws_ptr, ws_bytes = _given(workspace, dev)
    args = _BLOCK.pack(160, code, M, N, gate_rows, hp, 0, wpost, gp, wpre, sp, 0, ap, bp,
                       ldh, 0, ldg, lds, 0, 0.0, offset, alpha, beta)
    grads = _BLOCK_GRADS.pack(104, 0, dyp, dsp, dhp, drp, dgp, dwap, dwbp, lddy, ldds, lddh, lddr,
                              lddg)
    rc = (_lib or lib()).rmsnorm_block_bwd(args, grads, ws_ptr, ws_bytes,
                                           _opt(make_options(**options)) if options else None,
                                           _stream_ptr(dev))
    if rc:
        _check(rc)
    return dh, dr, dgate, dwa, dwb


def rope_steps(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None, device="cuda"):
    """steps, magnitude = rope_steps(rotary_dim): the frequencies of rotary positions
    as rope_fwd and rope_bwd take them (int64 [rotary_dim / 2] on the device: turns
    per position times 2^64), and the factor on cos and sin that belongs to them.

    ``scaling``: None or a dict with "kind" ("linear", "ntk", "yarn" or "bands"),
    "factor", and for "yarn" and "bands" the original "length" and optionally
    "beta_fast" (32 for yarn, 4 for bands) and "beta_slow" (1).
    """
    import torch
    steps = torch.empty(max(rotary_dim // 2, 1), dtype=torch.int64)
    sc = None
    if scaling:
        extra = set(scaling) - {"kind", "factor", "length", "beta_fast", "beta_slow"}
        if extra or scaling.get("kind") not in ROPE_SCALINGS:
            raise ValueError(f"not a scaling of rotary positions: {scaling}")
        kind = scaling["kind"]
        sc = RopeScaling(ctypes.sizeof(RopeScaling), ROPE_SCALINGS[kind], scaling.get("factor", 1.0),
                         scaling.get("length", 0.0),
                         scaling.get("beta_fast", 32.0 if kind == "yarn" else 4.0),
                         scaling.get("beta_slow", 1.0))
    mag = ctypes.c_float(1.0)
    _check(rmsnorm_rope_steps(rotary_dim, base, sc, steps.data_ptr(), ctypes.addressof(mag)))
    return steps.to(device), mag.value


def _heads(t, name, shape, dtype, device):
    """A heads tensor [T, H, D] or [B, S, H, D] as the struct's four values."""
    if t is None:
        return _NO_HEADS
    if t.shape == shape and t.dtype is dtype and t.get_device() == device:
        st = t.stride()
        if st[-1] == 1 or shape[-1] == 1:
            return (t.data_ptr(), 0, st[0], st[1]) if len(st) == 3 else (t.data_ptr(), *st[:3])
    _refuse(t, name, shape, dtype, device)
    raise ValueError(f"{name} must have unit stride within a head")


_NO_HEADS = (0, 0, 0, 0)


def _new_heads(like, shape):
    """A new contiguous heads tensor and its struct values."""
    t = like.new_empty(shape)
    if len(shape) == 3:
        H, D = shape[1], shape[2]
        return t, (t.data_ptr(), 0, H * D, D)
    S, H, D = shape[1], shape[2], shape[3]
    return t, (t.data_ptr(), S * H * D, H * D, D)


def _rope_common(q, k, steps, positions, w_q, w_k, interleaved):
    """The fields of the rope struct up to the weights."""
    import torch
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    if len(shape) == 3:
        B, (S, hq, D) = 1, shape
    elif len(shape) == 4:
        B, S, hq, D = shape
    else:
        raise ValueError("q must be [tokens, heads, head_dim] or [batch, seq, heads, head_dim]")
    hk = 0
    if k is not None:
        ks = k.shape
        if len(ks) != len(shape) or ks[:-2] != shape[:-2] or ks[-1] != D:
            raise ValueError(f"k must be like q but for its heads, got {tuple(ks)}")
        hk = ks[-2]
    half = steps.numel()
    sp = _vector(steps, "steps", half, torch.int64, dev)
    pp = ps = 0
    if positions is not None:
        if positions.dtype is not torch.int64 or positions.get_device() != dev:
            _refuse(positions, "positions", None, torch.int64, dev)
        ps = positions.shape
        if (ps != shape[:-2] and ps != (S,)) or (S > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be [seq] or [batch, seq], the last contiguous")
        pp, ps = positions.data_ptr(), positions.stride(0) if len(ps) == 2 and B > 1 else 0
    return (248, _code(dtype), B, S, hq, hk, D, 2 * half, 1 if interleaved else 0, 0, pp, ps, sp,
            _vector(w_q, "w_q", D, dtype, dev), _vector(w_k, "w_k", D, dtype, dev))


def rope_fwd(q, k, steps, positions=None, w_q=None, w_k=None, interleaved: bool = False,
             eps: float = 1e-6, offset: float = 0.0, magnitude: float = 1.0, q_out=None, k_out=None,
             rstd: bool = True, stream=None, **options):
    """q_out, k_out, rstd_q, rstd_k = rope_fwd(q, k, steps, positions): rotary positions
    on the first 2 * len(steps) values of every head, after the head's RMSNorm where
    w_q or w_k is given.

    q, k (k may be None): CUDA tensors [T, heads, head_dim] or [batch, seq, heads,
    head_dim] with unit stride within a head, any other strides (slices of a
    projection, transposed [batch, heads, seq, head_dim]). ``steps`` and ``magnitude``
    come from :func:`rope_steps`; ``positions`` is int64 [T], [seq] or [batch, seq]
    (default: the index). Pairs are (i, i + half), or (2i, 2i + 1) when
    ``interleaved``. ``q_out`` and ``k_out`` may be passed (q and k themselves to work in
    place). rstd_q and rstd_k are None without weights or with ``rstd=False``.
    """
    import torch
    ctx = _elsewhere(q, stream)
    if ctx is not None:
        with ctx:
            return rope_fwd(q, k, steps, positions, w_q, w_k, interleaved, eps, offset, magnitude,
                            q_out, k_out, rstd, **options)
    head = _rope_common(q, k, steps, positions, w_q, w_k, interleaved)
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    qh = _heads(q, "q", shape, dtype, dev)
    if q_out is None:
        q_out, qo = _new_heads(q, shape)
    else:
        qo = _heads(q_out, "q_out", shape, dtype, dev)
    kh = ko = _NO_HEADS
    a = b = None
    ap = bp = 0
    if k is not None:
        kshape = k.shape
        kh = _heads(k, "k", kshape, dtype, dev)
        if k_out is None:
            k_out, ko = _new_heads(k, kshape)
        else:
            ko = _heads(k_out, "k_out", kshape, dtype, dev)
        if rstd and w_k is not None:
            b = k.new_empty(kshape[:-1], dtype=torch.float32)
            bp = b.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if rstd and w_q is not None:
        a = q.new_empty(shape[:-1], dtype=torch.float32)
        ap = a.data_ptr()
    args = _ROPE.pack(*head, ap, bp, eps, offset, magnitude, 0.0, *qh, *kh, *qo, *ko)
    rc = (_lib or lib()).rmsnorm_rope_fwd(args, _opt(make_options(**options)) if options else None,
                                          _stream_ptr(dev))
    if rc:
        _check(rc)
    return q_out, k_out, a, b


def rope_bwd(dq_out, dk_out, steps, positions=None, q=None, k=None, rstd_q=None, rstd_k=None,
             w_q=None, w_k=None, interleaved: bool = False, offset: float = 0.0,
             magnitude: float = 1.0, dq=None, dk=None, workspace=None, stream=None, **options):
    """dq, dk, dw_q, dw_k = rope_bwd(dq_out, dk_out, steps, positions, ...): backward of
    :func:`rope_fwd` from the gradients of its outputs. With w_q (w_k) it needs the
    forward's q (k) and the rstd_q (rstd_k) it returned. dw_q and dw_k are fp32
    (None without weights). ``dq`` and ``dk`` may be passed (dq_out and dk_out
    themselves to work in place); ``workspace`` as in :func:`block_bwd`
    (rmsnorm_rope_bwd_workspace_size() bytes, needed with weights only).
    """
    import torch
    ctx = _elsewhere(dq_out, stream)
    if ctx is not None:
        with ctx:
            return rope_bwd(dq_out, dk_out, steps, positions, q, k, rstd_q, rstd_k, w_q, w_k,
                            interleaved, offset, magnitude, dq, dk, workspace, **options)
    head = _rope_common(dq_out, dk_out, steps, positions, w_q, w_k, interleaved)
    shape, dtype, dev, f32 = dq_out.shape, dq_out.dtype, dq_out.get_device(), torch.float32
    D = shape[-1]
    gq = _heads(dq_out, "dq_out", shape, dtype, dev)
    if dq is None:
        dq, oq = _new_heads(dq_out, shape)
    else:
        oq = _heads(dq, "dq", shape, dtype, dev)
    qh = kh = gk = ok = _NO_HEADS
    dwq = dwk = None
    ap = bp = wqp = wkp = 0
    if w_q is not None:
        ap = _vector(rstd_q, "rstd_q", shape[:-1].numel(), f32, dev)
        qh = _heads(q, "q", shape, dtype, dev)
        dwq = dq_out.new_empty(D, dtype=f32)
        wqp = dwq.data_ptr()
    if dk_out is not None:
        kshape = dk_out.shape
        gk = _heads(dk_out, "dk_out", kshape, dtype, dev)
        if dk is None:
            dk, ok = _new_heads(dk_out, kshape)
        else:
            ok = _heads(dk, "dk", kshape, dtype, dev)
        if w_k is not None:
            bp = _vector(rstd_k, "rstd_k", kshape[:-1].numel(), f32, dev)
            kh = _heads(k, "k", kshape, dtype, dev)
            dwk = dq_out.new_empty(D, dtype=f32)
            wkp = dwk.data_ptr()
    elif dk is not None:
        raise ValueError("dk without dk_out")
    if workspace is None and (wqp or wkp):
        workspace = _workspace(dq_out, rmsnorm_rope_bwd_workspace_size, D)
    args = _ROPE.pack(*head, ap, bp, 0.0, offset, magnitude, 0.0, *qh, *kh, *_NO_HEADS, *_NO_HEADS)
    grads = _ROPE_GRADS.pack(152, 0, *gq, *gk, *oq, *ok, wqp, wkp)
    ws_ptr = ws_bytes = 0
    if workspace is not None:
        ws_ptr, ws_bytes = _given(workspace, dev)
    rc = (_lib or lib()).rmsnorm_rope_bwd(args, grads, ws_ptr, ws_bytes,
                                          _opt(make_options(**options)) if options else None,
                                          _stream_ptr(dev))
    if rc:
        _check(rc)
    return dq, dk, dwq, dwk


class Cache:
    """A paged cache of k and v in 8 ("e4m3") or 4 ("e2m1") bits per value, one
    power-of-two scale byte for 32 values of a head: ``k_codes`` and ``v_codes``
    [pages, page_size, heads, code bytes], ``k_scales`` and ``v_scales`` [pages,
    page_size, heads, ceil(head_dim / 32)] (heads before page_size with
    ``heads_first``), zero at the start. ``values=False`` holds k alone;
    ``tensors`` = (k_codes, k_scales, v_codes, v_scales) takes existing memory.
    """

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, fmt: str = "e4m3",
                 device="cuda", heads_first: bool = False, values: bool = True, tensors=None):
        import torch
        if fmt not in CACHE_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(CACHE_FORMATS)}, got {fmt!r}")
        self.pages, self.page_size, self.heads, self.head_dim = pages, page_size, heads, head_dim
        self.fmt, self.heads_first = fmt, bool(heads_first)
        lead = (pages, heads, page_size) if heads_first else (pages, page_size, heads)
        shapes = [(*lead, head_dim if fmt == "e4m3" else (head_dim + 1) // 2),
                  (*lead, (head_dim + 31) // 32)]
        shapes = shapes * 2 if values else shapes
        if tensors is None:
            tensors = [torch.zeros(s, dtype=torch.uint8, device=device) for s in shapes]
        if len(tensors) != len(shapes):
            raise ValueError(f"the cache is made of {len(shapes)} tensors, got {len(tensors)}")
        for t, s in zip(tensors, shapes):
            if tuple(t.shape) != s or t.dtype != torch.uint8 or not t.is_contiguous() or \
                    t.device != tensors[0].device or not t.is_cuda:
                raise ValueError(f"cache tensors must be contiguous uint8 CUDA tensors {s} on one "
                                 f"device, got {t.dtype} {tuple(t.shape)} on {t.device}")
        self.k_codes, self.k_scales = tensors[:2]
        self.v_codes, self.v_scales = tensors[2:] if values else (None, None)
        self._args = _CACHE.pack(64, CACHE_FORMATS[fmt], pages, page_size, heads, head_dim,
                                 int(self.heads_first), *(t.data_ptr() for t in tensors),
                                 *(() if values else (0, 0)))


def _tokens(t, name, shape, dtype, device):
    if t.shape == shape and t.dtype is dtype and t.get_device() == device:
        st = t.stride()
        if st[2] == 1 or shape[2] == 1:
            return _HEADS.pack(t.data_ptr(), 0, st[0], st[1])
    _refuse(t, name, shape, dtype, device)
    raise ValueError(f"{name} must have unit stride within a head")


def cache_write(cache: Cache, k, v, slots, stream=None, **options) -> None:
    """Quantises k and v ([T, heads, head_dim], unit stride within a head; v None: k
    alone) into ``cache``: token t into slot slots[t] (int64: page * page_size +
    index; negative: padding, skipped). Slots must be distinct."""
    import torch
    ctx = _elsewhere(cache.k_codes, stream)
    if ctx is not None:
        with ctx:
            return cache_write(cache, k, v, slots, **options)
    dev, dtype = cache.k_codes.get_device(), k.dtype
    T = k.shape[0] if k.dim() == 3 else -1
    shape = (T, cache.heads, cache.head_dim)
    code = _code(dtype)
    kh = _tokens(k, "k", shape, dtype, dev)
    vh = None if v is None else _tokens(v, "v", shape, dtype, dev)
    sp = _vector(slots, "slots", T, torch.int64, dev)
    rc = (_lib or lib()).rmsnorm_cache_write(cache._args, kh, vh, sp, T, code,
                                             _opt(make_options(**options)) if options else None,
                                             _stream_ptr(dev))
    if rc:
        _check(rc)


def cache_read(cache: Cache, table, cu_rows, rows: int, starts=None, dtype=None, k_out=None,
               v_out=None, stream=None, **options):
    """k, v = cache_read(cache, table, cu_rows, rows): a ragged batch read back. Rows
    cu_rows[b] to cu_rows[b + 1] of the outputs [rows, heads, head_dim] are the
    tokens of sequence b from starts[b] (default 0) on, by its row of ``table``.

    ``table`` int32 [sequences, pages per sequence], ``cu_rows`` int32 [sequences + 1],
    ``starts`` int32 [sequences]. Outputs are ``dtype`` (default bf16) and are
    allocated here, or passed as ``k_out`` and ``v_out`` (unit stride within a head);
    rows behind cu_rows[-1] are not written. v is None in a cache without v.
    """
    import torch
    like = cache.k_codes
    ctx = _elsewhere(like, stream)
    if ctx is not None:
        with ctx:
            return cache_read(cache, table, cu_rows, rows, starts, dtype, k_out, v_out, **options)
    dev, i32 = like.get_device(), torch.int32
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else torch.bfloat16
    code = _code(dtype)
    shape = (rows, cache.heads, cache.head_dim)
    if table.dim() != 2:
        raise ValueError("table must be [sequences, pages per sequence]")
    n, width = table.shape
    tp = _vector(table, "table", n * width, i32, dev)
    cp = _vector(cu_rows, "cu_rows", n + 1, i32, dev)
    sp = _vector(starts, "starts", n, i32, dev)
    if k_out is None:
        k_out = like.new_empty(shape, dtype=dtype)
    kh, vh = _tokens(k_out, "k_out", shape, dtype, dev), None
    if cache.v_codes is not None:
        if v_out is None:
            v_out = like.new_empty(shape, dtype=dtype)
    if v_out is not None:
        vh = _tokens(v_out, "v_out", shape, dtype, dev)
    rc = (_lib or lib()).rmsnorm_cache_read(cache._args, tp, width, cp, sp, n, rows, kh, vh, code,
                                            _opt(make_options(**options)) if options else None,
                                            _stream_ptr(dev))
    if rc:
        _check(rc)
    return k_out, v_out
