"""MI355X-native MoE prompt (prefill) FFN layer, the same layer for a few tokens, the MXFP4
operators, and those of 16-bit experts and low-rank adapters -- Python binding.

A thin ctypes binding of ``libmoe_prefill.so`` (C ABI in
``include/moe_prefill.h``).  It only marshals arguments: routing, grouping,
quantisation, both grouped GEMMs, SwiGLU, requantisation, the combine and the
slot pool's copies all run in the library (HIP kernels for gfx950 and its C++
host runtime).  PyTorch supplies device memory, pinned host memory and
streams; there is no CPU fallback -- if the library is missing, importing the
binding's entry points raises.

The function names are the C entry points' names.
"""
from __future__ import annotations

import ctypes
import os
from concurrent.futures import ThreadPoolExecutor
from typing import Callable, Dict, Optional, Sequence

import numpy as np
import torch  # loaded first so the library binds to the same HIP runtime as torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_prefill.so")

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_EHIP, MOE_EUNSUPPORTED, MOE_ESTATE, MOE_ETIMEOUT = 0, -1, -2, -3, -4, -5, -6
MOE_WARN_SLOT_OVER_BUDGET, MOE_WARN_POOL_DEGRADED, MOE_WARN_DEPTH_REDUCED = 1, 2, 4
_NAMES = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_ENOMEM", -3: "MOE_EHIP", -4: "MOE_EUNSUPPORTED",
          -5: "MOE_ESTATE", -6: "MOE_ETIMEOUT"}


class MoePrefillError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_NAMES.get(code, code)}: {msg}")
        self.code = code


_u32, _i32, _i64, _u64, _vp = ctypes.c_uint32, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p


class moe_prefill_params_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("d_model", _i32), ("d_ff", _i32), ("n_experts", _i32),
                ("top_k", _i32), ("max_tokens", _i32), ("device", _i32), ("reserved0", _i32),
                ("workspace", _vp), ("workspace_bytes", _u64)]


class moe_layer_io_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("layer", _i32), ("weights_dev", _vp), ("n_tokens", _i32),
                ("reserved0", _i32), ("x", _vp), ("logits", _vp), ("y", _vp),
                ("eidx", _vp), ("weights", _vp), ("counts", _vp), ("bounds", _vp), ("rows", _vp),
                ("pos", _vp), ("xq", _vp), ("dx", _vp), ("gu", _vp), ("h", _vp), ("hq", _vp),
                ("dh", _vp), ("dm", _vp), ("combine", _i32), ("reserved1", _i32)]


class moe_decode_io_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("layer", _i32), ("weights_dev", _vp), ("n_tokens", _i32),
                ("dtype", _i32), ("x", _vp), ("x_stride", _i64), ("logits", _vp), ("logits_stride", _i64),
                ("y", _vp), ("y_stride", _i64), ("workspace", _vp), ("workspace_bytes", _u64),
                ("eidx", _vp), ("weights", _vp)]


class moe_mxfp4_matrix_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("dtype", _i32), ("K", _i32), ("M", _i64),
                ("values", _vp), ("stride", _i64), ("codes", _vp), ("scales", _vp)]


class moe_mxfp4_gemm_args_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("a_codes", _vp), ("a_scales", _vp), ("a_rows", _i64),
                ("b_codes", _vp), ("b_scales", _vp), ("bounds", _vp), ("rows", _vp), ("n_groups", _i32),
                ("top_k", _i32), ("M", _i64), ("N", _i32), ("K", _i32), ("swiglu", _i32), ("dtype", _i32),
                ("out", _vp), ("out_stride", _i64)]


class moe_group_args_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("eidx", _vp), ("n_pairs", _i64), ("n_groups", _i32),
                ("reserved0", _i32), ("bounds", _vp), ("rows", _vp), ("pos", _vp), ("counts", _vp),
                ("workspace", _vp), ("workspace_bytes", _u64)]


class moe_grouped_gemm_args_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("a", _vp), ("a_stride", _i64), ("a_rows", _i64),
                ("b", _vp), ("b_stride", _i64), ("b_group_stride", _i64), ("bounds", _vp), ("rows", _vp),
                ("n_groups", _i32), ("top_k", _i32), ("M", _i64), ("N", _i32), ("K", _i32), ("swiglu", _i32),
                ("dtype", _i32), ("out_dtype", _i32), ("reserved0", _i32), ("out", _vp), ("out_stride", _i64)]


class moe_combine_args_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("d", _vp), ("d_stride", _i64), ("d_rows", _i64),
                ("weights", _vp), ("pos", _vp), ("base", _vp), ("base_stride", _i64), ("y", _vp), ("y_stride", _i64),
                ("n_tokens", _i64), ("N", _i32), ("top_k", _i32), ("d_dtype", _i32), ("base_dtype", _i32),
                ("y_dtype", _i32), ("reserved0", _i32)]


class moe_lora_args_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("device", _i32), ("x", _vp), ("x_stride", _i64), ("a", _vp), ("b", _vp),
                ("adapters", _vp), ("scales", _vp), ("base", _vp), ("base_stride", _i64), ("out", _vp),
                ("out_stride", _i64), ("M", _i64), ("N", _i32), ("K", _i32), ("rank", _i32), ("n_adapters", _i32),
                ("dtype", _i32), ("base_dtype", _i32), ("out_dtype", _i32), ("reserved0", _i32),
                ("workspace", _vp), ("workspace_bytes", _u64)]


_DECODE_IO_SIZE = ctypes.sizeof(moe_decode_io_t)
_MX_MATRIX_SIZE = ctypes.sizeof(moe_mxfp4_matrix_t)
_MX_GEMM_SIZE = ctypes.sizeof(moe_mxfp4_gemm_args_t)
_GROUP_SIZE = ctypes.sizeof(moe_group_args_t)
_GROUPED_GEMM_SIZE = ctypes.sizeof(moe_grouped_gemm_args_t)
_COMBINE_SIZE = ctypes.sizeof(moe_combine_args_t)
_LORA_SIZE = ctypes.sizeof(moe_lora_args_t)

MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
_DTYPE_ID = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
MOE_DECODE_MAX_PAIRS = 1024

COMBINE_MODES = {"gather": 0, "atomic": 1}   # MOE_COMBINE_GATHER, MOE_COMBINE_ATOMIC


class stream_pool_params_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("n_layers", _i32), ("host_blobs", ctypes.POINTER(_vp)),
                ("layer_bytes", _u64), ("prefetch_depth", _i32), ("resident_layers", _i32),
                ("max_vram_bytes", _i64), ("requested_slots", _i32), ("eff_slots", _i32),
                ("eff_depth", _i32), ("eff_residents", _i32), ("warnings", _i32), ("reserved0", _i32),
                ("active_only", _i32), ("reserved1", _i32), ("reserve_bytes", _i64)]


class stream_pool_budget_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("reserved0", _i32), ("max_vram_bytes", _i64),
                ("eff_slots", _i32), ("eff_depth", _i32), ("eff_residents", _i32), ("warnings", _i32),
                ("released_bytes", _u64)]


class moe_pool_trim_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("n_layers", _i32), ("residents", _i32), ("streaming", _i32),
                ("budget_slots", _i64), ("new_residents", _i32), ("new_streaming", _i32),
                ("evicted", _i32), ("converted", _i32), ("released", _i32), ("warnings", _i32)]


class moe_pool_plan_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("n_layers", _i32), ("slot_bytes", _u64),
                ("prefetch_depth", _i32), ("resident_layers", _i32), ("max_vram_bytes", _i64),
                ("requested_slots", _i32), ("max_alloc_slots", _i32), ("slots", _i32),
                ("depth", _i32), ("residents", _i32), ("warnings", _i32)]


class moe_stats_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("reserved0", _i32), ("layers_run", _u64),
                ("prefetch_queued", _u64), ("prefetch_activated", _u64), ("sync_loads", _u64),
                ("prefetch_failed", _u64), ("bytes_h2d", _u64), ("eff_slots", _i32),
                ("eff_depth", _i32), ("eff_residents", _i32), ("warnings", _i32),
                ("sparse_loads", _u64), ("experts_loaded", _u64), ("bytes_sparse", _u64),
                ("evicted_residents", _u64), ("released_bytes", _u64), ("pressure_trims", _u64)]


MOE_N_KERNELS = 7
MOE_LOG_ERROR, MOE_LOG_WARN, MOE_LOG_INFO = 0, 1, 2
_LOG_FN = ctypes.CFUNCTYPE(None, _i32, ctypes.c_char_p, _vp)


class moe_kernel_times_t(ctypes.Structure):
    _fields_ = [("struct_size", _u32), ("n_kernels", _i32), ("launches", _u64 * MOE_N_KERNELS),
                ("total_ms", ctypes.c_double * MOE_N_KERNELS)]


EXPORTED_SYMBOLS = [
    "moe_prefill_workspace_size", "moe_prefill_create", "moe_prefill_destroy",
    "moe_prefill_last_error", "moe_prefill_expert_bytes", "moe_prefill_layer_bytes",
    "moe_prefill_pack_expert", "moe_prefill_run_layer", "stream_pool_configure",
    "moe_prefill_plan_pool", "moe_prefill_plan_trim", "stream_pool_set_budget",
    "moe_prefill_get_stats", "moe_prefill_set_log", "moe_prefill_set_timing",
    "moe_prefill_kernel_times", "moe_prefill_kernel_name",
    "moe_prefill_exp_host", "moe_prefill_exp_device", "moe_prefill_run_layer_noalloc",
    "moe_decode_workspace_size", "moe_decode_run_layer",
    "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_gemm",
    "moe_group_workspace_size", "moe_group_rows", "moe_grouped_gemm", "moe_combine_rows",
    "moe_lora_workspace_size", "moe_lora_add",
]

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python moe_prefill_ffn_amd/build.py` "
                          "(or __graft_entry__.build()); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    L.moe_prefill_workspace_size.argtypes = [ctypes.POINTER(moe_prefill_params_t), ctypes.POINTER(_u64)]
    L.moe_prefill_create.argtypes = [ctypes.POINTER(moe_prefill_params_t), ctypes.POINTER(_vp)]
    L.moe_prefill_destroy.argtypes = [_vp]
    L.moe_prefill_destroy.restype = None
    L.moe_prefill_last_error.argtypes = [_vp]
    L.moe_prefill_last_error.restype = ctypes.c_char_p
    L.moe_prefill_expert_bytes.argtypes = [_i32, _i32]
    L.moe_prefill_expert_bytes.restype = _u64
    L.moe_prefill_layer_bytes.argtypes = [_i32, _i32, _i32]
    L.moe_prefill_layer_bytes.restype = _u64
    L.moe_prefill_pack_expert.argtypes = [_i32, _i32, _vp, _vp, _vp, _vp, _vp]
    L.moe_prefill_run_layer.argtypes = [_vp, ctypes.POINTER(moe_layer_io_t), _vp]
    L.stream_pool_configure.argtypes = [_vp, ctypes.POINTER(stream_pool_params_t)]
    L.moe_prefill_plan_pool.argtypes = [ctypes.POINTER(moe_pool_plan_t)]
    L.moe_prefill_plan_trim.argtypes = [ctypes.POINTER(moe_pool_trim_t)]
    L.stream_pool_set_budget.argtypes = [_vp, ctypes.POINTER(stream_pool_budget_t)]
    L.moe_prefill_get_stats.argtypes = [_vp, ctypes.POINTER(moe_stats_t)]
    L.moe_prefill_set_log.argtypes = [_vp, _LOG_FN, _vp, _i32]
    L.moe_prefill_set_timing.argtypes = [_vp, _i32]
    L.moe_prefill_kernel_times.argtypes = [_vp, ctypes.POINTER(moe_kernel_times_t), _i32]
    L.moe_prefill_kernel_name.argtypes = [_i32]
    L.moe_prefill_kernel_name.restype = ctypes.c_char_p
    L.moe_prefill_run_layer_noalloc.argtypes = [ctypes.POINTER(moe_prefill_params_t),
                                                ctypes.POINTER(moe_layer_io_t), _vp]
    L.moe_prefill_exp_host.argtypes = [_u32, _u64, _vp]
    L.moe_prefill_exp_device.argtypes = [_u32, _u64, _vp, _vp]
    L.moe_decode_workspace_size.argtypes = [ctypes.POINTER(moe_prefill_params_t), ctypes.POINTER(_u64)]
    L.moe_decode_run_layer.argtypes = [_vp, ctypes.POINTER(moe_decode_io_t), _vp]
    L.moe_mxfp4_quantize.argtypes = [ctypes.POINTER(moe_mxfp4_matrix_t), _vp]
    L.moe_mxfp4_dequantize.argtypes = [ctypes.POINTER(moe_mxfp4_matrix_t), _vp]
    L.moe_mxfp4_gemm.argtypes = [ctypes.POINTER(moe_mxfp4_gemm_args_t), _vp]
    L.moe_group_workspace_size.argtypes = [_i64, _i32, ctypes.POINTER(_u64)]
    L.moe_group_rows.argtypes = [ctypes.POINTER(moe_group_args_t), _vp]
    L.moe_grouped_gemm.argtypes = [ctypes.POINTER(moe_grouped_gemm_args_t), _vp]
    L.moe_combine_rows.argtypes = [ctypes.POINTER(moe_combine_args_t), _vp]
    L.moe_lora_workspace_size.argtypes = [_i64, _i32, _i32, ctypes.POINTER(_u64)]
    L.moe_lora_add.argtypes = [ctypes.POINTER(moe_lora_args_t), _vp]
    _lib = L
    return L


def _check(rc: int, handle=None):
    if rc != MOE_OK:
        msg = lib().moe_prefill_last_error(handle).decode(errors="replace")
        raise MoePrefillError(rc, msg)


def moe_prefill_last_error(handle=None) -> str:
    return lib().moe_prefill_last_error(handle.ptr if handle else None).decode(errors="replace")


# ---------------------------------------------------------------- handle ---

class Handle:
    """Owner of a ``moe_prefill_t*`` plus references that must outlive it."""

    def __init__(self, ptr: int, params: dict, keep=()):
        self.ptr = ptr
        self.params = params
        self.layer_bytes = moe_prefill_layer_bytes(params["d_model"], params["d_ff"], params["n_experts"])
        self._keep = list(keep)
        self._pool_keep = []
        self._log_cb = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def close(self):
        if self.ptr:
            lib().moe_prefill_destroy(self.ptr)
            self.ptr = None
        self._pool_keep = []

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


def _params(d_model, d_ff, n_experts, top_k, max_tokens, device=0, workspace=None):
    p = moe_prefill_params_t()
    p.struct_size = ctypes.sizeof(p)
    p.d_model, p.d_ff, p.n_experts, p.top_k, p.max_tokens, p.device = (
        d_model, d_ff, n_experts, top_k, max_tokens, device)
    if workspace is not None:
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    return p


def moe_prefill_workspace_size(d_model: int, d_ff: int, n_experts: int, top_k: int, max_tokens: int) -> int:
    p = _params(d_model, d_ff, n_experts, top_k, max_tokens)
    out = _u64()
    _check(lib().moe_prefill_workspace_size(ctypes.byref(p), ctypes.byref(out)))
    return int(out.value)


def moe_prefill_create(d_model: int, d_ff: int, n_experts: int, top_k: int, max_tokens: int,
                       device: int = 0, workspace: Optional[torch.Tensor] = None) -> Handle:
    """Create a handle.  ``workspace``: optional lent device uint8 tensor."""
    p = _params(d_model, d_ff, n_experts, top_k, max_tokens, device, workspace)
    out = _vp()
    _check(lib().moe_prefill_create(ctypes.byref(p), ctypes.byref(out)))
    return Handle(out.value, dict(d_model=d_model, d_ff=d_ff, n_experts=n_experts, top_k=top_k,
                                  max_tokens=max_tokens, device=device),
                  keep=[workspace] if workspace is not None else [])


def moe_prefill_destroy(handle: Handle):
    handle.close()


# ----------------------------------------------------------------- blobs ---

def moe_prefill_expert_bytes(d_model: int, d_ff: int) -> int:
    return int(lib().moe_prefill_expert_bytes(d_model, d_ff))


def moe_prefill_layer_bytes(d_model: int, d_ff: int, n_experts: int) -> int:
    return int(lib().moe_prefill_layer_bytes(d_model, d_ff, n_experts))


def _np_ptr(a: np.ndarray, dtype) -> int:
    if a.dtype != dtype or not a.flags["C_CONTIGUOUS"]:
        raise TypeError(f"expected a C-contiguous {np.dtype(dtype)} array")
    return a.ctypes.data


def moe_prefill_pack_expert(d_model: int, d_ff: int, wgu_q: np.ndarray, wgu_s: np.ndarray,
                            wd_q: np.ndarray, wd_s: np.ndarray, dst_ptr: int) -> None:
    """Pack one expert's canonical weights into host memory at ``dst_ptr``."""
    for a, shp in ((wgu_q, (2 * d_ff, d_model)), (wgu_s, (2 * d_ff, d_model // 32)),
                   (wd_q, (d_model, d_ff)), (wd_s, (d_model, d_ff // 32))):
        if tuple(a.shape) != shp:
            raise ValueError(f"shape {a.shape} != {shp}")
    rc = lib().moe_prefill_pack_expert(
        d_model, d_ff, _np_ptr(wgu_q, np.int8), _np_ptr(wgu_s, np.uint16), _np_ptr(wd_q, np.int8),
        _np_ptr(wd_s, np.uint16), dst_ptr)
    _check(rc)


def pack_layer(d_model: int, d_ff: int, n_experts: int, expert_fn: Callable, out: torch.Tensor,
               threads: int = 8) -> torch.Tensor:
    """Pack a whole layer blob into ``out`` (a host uint8 tensor, e.g. pinned).

    ``expert_fn(e)`` returns an object with ``wgu_q, wgu_s, wd_q, wd_s``.
    """
    eb = moe_prefill_expert_bytes(d_model, d_ff)
    if out.device.type != "cpu" or out.dtype != torch.uint8 or out.numel() < eb * n_experts:
        raise ValueError("out must be a host uint8 tensor of at least layer_bytes")
    base = out.data_ptr()

    def one(e):
        w = expert_fn(e)
        moe_prefill_pack_expert(d_model, d_ff, w.wgu_q, w.wgu_s, w.wd_q, w.wd_s, base + e * eb)

    with ThreadPoolExecutor(max_workers=max(1, threads)) as ex:
        list(ex.map(one, range(n_experts)))
    return out


# ------------------------------------------------------------- one layer ---

_EXPORTS = ("eidx", "weights", "counts", "bounds", "rows", "pos", "xq", "dx", "gu", "h", "hq", "dh", "dm")


def _dev_ptr(t: Optional[torch.Tensor], dtype, name: str, numel: Optional[int] = None) -> int:
    if t is None:
        return 0
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} device tensor")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements")
    return t.data_ptr()


def _layer_io(P: dict, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor, layer: int,
              weights: Optional[torch.Tensor], exports: Optional[Dict[str, torch.Tensor]],
              combine: str = "gather") -> moe_layer_io_t:
    T = x.shape[0]
    io = moe_layer_io_t()
    io.struct_size = ctypes.sizeof(io)
    io.layer = layer
    io.n_tokens = T
    if combine not in COMBINE_MODES:
        raise ValueError(f"combine must be one of {sorted(COMBINE_MODES)}")
    io.combine = COMBINE_MODES[combine]
    io.x = _dev_ptr(x, torch.float32, "x", T * P["d_model"])
    io.logits = _dev_ptr(logits, torch.float32, "logits", T * P["n_experts"])
    io.y = _dev_ptr(y, torch.float32, "y", T * P["d_model"])
    if layer < 0:
        if weights is None:
            raise ValueError("layer=-1 needs a resident weight blob")
        io.weights_dev = _dev_ptr(weights, torch.uint8, "weights",
                                  moe_prefill_layer_bytes(P["d_model"], P["d_ff"], P["n_experts"]))
    dt = dict(eidx=torch.int32, weights=torch.float32, counts=torch.int32, bounds=torch.int32,
              rows=torch.int32, pos=torch.int32, xq=torch.int8, dx=torch.float32, gu=torch.float32,
              h=torch.float32, hq=torch.int8, dh=torch.float32, dm=torch.float32)
    R, d, f, E = T * P["top_k"], P["d_model"], P["d_ff"], P["n_experts"]
    need = dict(eidx=R, weights=R, counts=E, bounds=E + 1, rows=R, pos=R, xq=T * d, dx=T * d // 32,
                gu=R * 2 * f, h=R * f, hq=R * f, dh=R * f // 32, dm=R * d)
    for name, t in (exports or {}).items():
        if name not in _EXPORTS:
            raise KeyError(name)
        setattr(io, name, _dev_ptr(t, dt[name], name, need[name]))
    return io


def moe_prefill_run_layer(handle: Handle, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor,
                          layer: int = -1, weights: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None,
                          exports: Optional[Dict[str, torch.Tensor]] = None,
                          combine: str = "gather") -> None:
    """Enqueue one MoE prefill FFN layer on ``stream`` (default: torch's current stream).
    combine: "gather" (deterministic, default) or "atomic" (the down GEMM adds into y)."""
    io = _layer_io(handle.params, x, logits, y, layer, weights, exports, combine)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    _check(lib().moe_prefill_run_layer(handle.ptr, ctypes.byref(io), _vp(s.cuda_stream)), handle.ptr)


def moe_prefill_run_layer_noalloc(d_model: int, d_ff: int, n_experts: int, top_k: int, x: torch.Tensor,
                                  logits: torch.Tensor, y: torch.Tensor, weights: torch.Tensor,
                                  device: int = 0, stream: Optional[torch.cuda.Stream] = None,
                                  exports: Optional[Dict[str, torch.Tensor]] = None,
                                  combine: str = "gather") -> None:
    """One resident layer with no handle and no device allocation: the library's static
    per-device scratch array is the workspace (calls on one device must not overlap)."""
    T = x.shape[0]
    P = dict(d_model=d_model, d_ff=d_ff, n_experts=n_experts, top_k=top_k, max_tokens=max(T, 1))
    io = _layer_io(P, x, logits, y, -1, weights, exports, combine)
    p = _params(d_model, d_ff, n_experts, top_k, max(T, 1), device)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    _check(lib().moe_prefill_run_layer_noalloc(ctypes.byref(p), ctypes.byref(io), _vp(s.cuda_stream)))


# ---------------------------------------------------- a few tokens' layer ---

# the raw handle of torch's current stream, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(stream: Optional[torch.cuda.Stream], index: int) -> int:
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors are on device {index}")
    return stream.cuda_stream


def _scratch(shape, dtype, index: int, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Memory for work on ``stream``, from that stream's own pool: a block of the current stream's may
    have been freed under kernels that are still queued there, and ``stream`` does not wait for them."""
    device = torch.device("cuda", index)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype, index: int, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """_scratch() that is handed to the caller, who goes on with it on the current stream: freed there,
    it is not used again before that stream's work on it is done."""
    t = _scratch(shape, dtype, index, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(index))
    return t


def _rows_of(t: torch.Tensor, name: str, rows: int, cols: int, index: int) -> int:
    """Row stride of a [rows, cols] matrix on device `index` whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    if t.get_device() != index:
        raise TypeError(f"{name}: expected a tensor on device {index}, got {t.device}")
    stride, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows <= 1:
        return cols
    if stride < cols:
        raise ValueError(f"{name}: rows overlap")
    return stride


def moe_decode_workspace_size(d_model: int, d_ff: int, n_experts: int, top_k: int, max_tokens: int) -> int:
    """Bytes of moe_decode_run_layer's workspace for up to max_tokens tokens."""
    p = _params(d_model, d_ff, n_experts, top_k, max_tokens)
    out = _u64()
    _check(lib().moe_decode_workspace_size(ctypes.byref(p), ctypes.byref(out)))
    return int(out.value)


def moe_decode_run_layer(handle: Handle, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor,
                         layer: int = -1, weights: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None,
                         exports: Optional[Dict[str, torch.Tensor]] = None) -> None:
    """Enqueue the MoE FFN layer for a few tokens (x.shape[0] * top_k <= 1024) on ``stream``.

    x, y: [T, d_model] fp32, bf16 or fp16, the same type (rows may be strided, 16-byte aligned);
    logits: [T, n_experts] fp32, -inf where an expert is not available.  ``workspace``: device
    uint8 scratch of moe_decode_workspace_size() bytes that no other call in flight uses;
    without one the call takes it from torch's allocator, on ``stream``.  exports: "eidx" int32 and
    "weights" fp32, [T, top_k] each."""
    P = handle.params
    d, E, k, index = P["d_model"], P["n_experts"], P["top_k"], P["device"]
    T = x.shape[0]
    dtype = _DTYPE_ID.get(x.dtype)
    if dtype is None or y.dtype != x.dtype:
        raise TypeError("x and y: expected the same of float32, bfloat16, float16")
    if logits.dtype != torch.float32:
        raise TypeError("logits: expected float32")
    if x.get_device() != index:
        raise TypeError(f"x: expected a tensor on the handle's device cuda:{index}")
    x_stride = _rows_of(x, "x", T, d, index)
    l_stride = _rows_of(logits, "logits", T, E, index)
    y_stride = _rows_of(y, "y", T, d, index)
    blob = None
    if layer < 0:
        if weights is None:
            raise ValueError("layer=-1 needs a resident weight blob")
        if weights.get_device() != index:
            raise TypeError(f"weights: expected a tensor on device {index}")
        blob = _dev_ptr(weights, torch.uint8, "weights", handle.layer_bytes)
    raw = _stream_of(stream, index)
    if workspace is None:
        if 0 < T * k <= MOE_DECODE_MAX_PAIRS:
            workspace = _scratch(moe_decode_workspace_size(d, P["d_ff"], E, k, T), torch.uint8, index, stream)
    elif workspace.get_device() != index:
        raise TypeError(f"workspace: expected a tensor on device {index}")
    ws, ws_bytes = (_dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel()) if workspace is not None else (None, 0)
    io = moe_decode_io_t(_DECODE_IO_SIZE, layer, blob, T, dtype, x.data_ptr(), x_stride, logits.data_ptr(), l_stride,
                         y.data_ptr(), y_stride, ws, ws_bytes)
    if exports:
        for name, t in exports.items():
            if name not in ("eidx", "weights"):
                raise KeyError(name)
            if t.get_device() != index:
                raise TypeError(f"{name}: expected a tensor on device {index}")
            setattr(io, name, _dev_ptr(t, torch.int32 if name == "eidx" else torch.float32, name, T * k))
    rc = lib().moe_decode_run_layer(handle.ptr, io, raw)
    if rc:
        _check(rc, handle.ptr)


# ----------------------------------------------------------------- MXFP4 ---

def _mx_device(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    return index


def _mx_bytes(t: torch.Tensor, name: str, shape, index: int) -> int:
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != torch.uint8 or t.get_device() != index or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous uint8 tensor on device {index}")
    return t.data_ptr()


def _mx_matrix(values, codes, scales, M, K, index) -> moe_mxfp4_matrix_t:
    dtype = _DTYPE_ID.get(values.dtype)
    if dtype is None:
        raise TypeError("expected float32, bfloat16 or float16 values")
    return moe_mxfp4_matrix_t(_MX_MATRIX_SIZE, index, dtype, K, M, values.data_ptr(), _rows_of(values, "values", M, K, index),
                              _mx_bytes(codes, "codes", (M, K // 2), index), _mx_bytes(scales, "scales", (M, K // 32), index))


def moe_mxfp4_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """x [M, K] (fp32, bf16 or fp16; K a multiple of 32) -> MXFP4 (codes [M, K/2] uint8, scales [M, K/32] uint8)."""
    index = _mx_device(x, "x")
    if x.dim() != 2:
        raise ValueError("x: expected a matrix")
    M, K = x.shape
    raw = _stream_of(stream, index)
    if codes is None:
        codes = _result((M, K // 2), torch.uint8, index, stream)
    if scales is None:
        scales = _result((M, K // 32), torch.uint8, index, stream)
    rc = lib().moe_mxfp4_quantize(_mx_matrix(x, codes, scales, M, K, index), raw)
    if rc:
        _check(rc)
    return codes, scales


def moe_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.float32,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """MXFP4 (codes [M, K/2], scales [M, K/32]) -> values [M, K] in ``out`` (or a new tensor of ``dtype``)."""
    index = _mx_device(codes, "codes")
    if codes.dim() != 2:
        raise ValueError("codes: expected a matrix")
    M, K = codes.shape
    K *= 2
    raw = _stream_of(stream, index)
    if out is None:
        out = _result((M, K), dtype, index, stream)
    rc = lib().moe_mxfp4_dequantize(_mx_matrix(out, codes, scales, M, K, index), raw)
    if rc:
        _check(rc)
    return out


def moe_mxfp4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                   out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
                   bounds: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                   top_k: int = 1, swiglu: bool = False,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[r] = A[src(r)] B[g(r)]^T of two MXFP4 matrices (fp32 sums, one rounding to out's type).

    a_codes [A, K/2], b_codes [N, K/2] or [G, N, K/2] (their scales with K/32); with swiglu B has
    2N rows a group, gate then up.  bounds: int32 [G + 1], group g's rows of out; rows: int32 [M],
    src(r) = rows[r] // top_k (the row table moe_prefill_run_layer exports); without rows
    src(r) = r // top_k and M = A * top_k.  Rows of out in no group are left as they were."""
    index = _mx_device(a_codes, "a_codes")
    b_shape = b_codes.shape
    if a_codes.dim() != 2 or len(b_shape) not in (2, 3):
        raise ValueError("a_codes: expected a matrix; b_codes: a matrix, or one per group")
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    A, K2 = a_codes.shape
    K = K2 * 2
    G = b_shape[0] if len(b_shape) == 3 else 1
    NB = b_shape[-2]
    if swiglu and NB % 2:
        raise ValueError("b_codes: swiglu needs gate and up rows, an even number")
    N = NB // 2 if swiglu else NB
    M = rows.shape[0] if rows is not None else A * top_k
    raw = _stream_of(stream, index)
    if out is None:
        out = _result((M, N), dtype, index, stream)
    out_dtype = _DTYPE_ID.get(out.dtype)
    if out_dtype is None:
        raise TypeError("out: expected float32, bfloat16 or float16")
    if bounds is None and G != 1:
        raise ValueError("b_codes of several groups need bounds")
    if bounds is not None and bounds.shape != (G + 1,):
        raise ValueError(f"bounds: expected shape ({G + 1},)")
    if rows is not None and rows.dim() != 1:
        raise ValueError("rows: expected a vector")
    for name, t in (("bounds", bounds), ("rows", rows)):
        if t is not None and (t.get_device() != index or t.dtype != torch.int32 or not t.is_contiguous()):
            raise TypeError(f"{name}: expected a contiguous int32 tensor on device {index}")
    a = moe_mxfp4_gemm_args_t(
        _MX_GEMM_SIZE, index, _mx_bytes(a_codes, "a_codes", (A, K2), index), _mx_bytes(a_scales, "a_scales", (A, K // 32), index),
        A, _mx_bytes(b_codes, "b_codes", (*b_shape[:-1], K2), index), _mx_bytes(b_scales, "b_scales", (*b_shape[:-1], K // 32), index),
        bounds.data_ptr() if bounds is not None else None, rows.data_ptr() if rows is not None else None, G, top_k, M, N, K,
        1 if swiglu else 0, out_dtype, out.data_ptr(), _rows_of(out, "out", M, N, index))
    rc = lib().moe_mxfp4_gemm(a, raw)
    if rc:
        _check(rc)
    return out


# ---------------------------------------------------- experts in 16 bits ---

def _vector(t: torch.Tensor, name: str, shape, dtype, index: int) -> int:
    """Address of a contiguous tensor of that shape and type on device `index`."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} tensor on device {index}")
    return t.data_ptr()


def _workspace(workspace: Optional[torch.Tensor], nbytes: Callable[[], int], index: int,
               stream: Optional[torch.cuda.Stream]):
    """(tensor to keep until the call is enqueued, address, bytes) of a caller's workspace, or of one of
    nbytes() from torch's allocator."""
    if workspace is None:
        n = nbytes()
        if n == 0:
            return None, None, 0
        workspace = _scratch(n, torch.uint8, index, stream)
    elif workspace.get_device() != index:
        raise TypeError(f"workspace: expected a tensor on device {index}")
    return workspace, _dev_ptr(workspace, torch.uint8, "workspace") if workspace.numel() else None, workspace.numel()


def moe_group_workspace_size(n_pairs: int, n_groups: int) -> int:
    """Bytes of moe_group_rows' workspace (0: it needs none)."""
    out = _u64()
    _check(lib().moe_group_workspace_size(n_pairs, n_groups, ctypes.byref(out)))
    return int(out.value)


def moe_group_rows(eidx: torch.Tensor, n_groups: int, bounds: Optional[torch.Tensor] = None,
                   rows: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """The row table of the experts that a router chose: (bounds, rows, pos).

    eidx: int32, contiguous, [T, k] or any shape; pair p is its p-th element, in no group where it is
    outside [0, n_groups).  bounds int32 [n_groups + 1]; rows int32 [P], the pairs in group order, ascending
    inside a group, untouched behind bounds[n_groups]; pos int32 like eidx, each pair's row, -1: none.
    counts: int32 [n_groups], filled if given.  workspace: device uint8 scratch of
    moe_group_workspace_size() bytes that no other call in flight uses."""
    index = _mx_device(eidx, "eidx")
    P = eidx.numel()
    at = _vector(eidx, "eidx", eidx.shape, torch.int32, index)
    raw = _stream_of(stream, index)
    keep, ws, ws_bytes = _workspace(workspace, lambda: moe_group_workspace_size(P, n_groups), index, stream)
    if bounds is None:
        bounds = _result((n_groups + 1,), torch.int32, index, stream)
    if rows is None:
        rows = _result((P,), torch.int32, index, stream)
    if pos is None:
        pos = _result(tuple(eidx.shape), torch.int32, index, stream)
    a = moe_group_args_t(_GROUP_SIZE, index, at, P, n_groups, 0, _vector(bounds, "bounds", (n_groups + 1,), torch.int32, index),
                         _vector(rows, "rows", (P,), torch.int32, index), _vector(pos, "pos", eidx.shape, torch.int32, index),
                         _vector(counts, "counts", (n_groups,), torch.int32, index) if counts is not None else None, ws, ws_bytes)
    rc = lib().moe_group_rows(a, raw)
    if rc:
        _check(rc)
    return bounds, rows, pos


def moe_grouped_gemm(a: torch.Tensor, b: torch.Tensor, out: Optional[torch.Tensor] = None,
                     dtype: Optional[torch.dtype] = None, bounds: Optional[torch.Tensor] = None,
                     rows: Optional[torch.Tensor] = None, top_k: int = 1, swiglu: bool = False,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[r] = A[src(r)] B[g(r)]^T of bf16 or fp16 matrices (fp32 sums, one rounding to out's type).

    a [A, K] (rows may be strided), b [N, K] or [G, N, K] (its rows and groups too; K a multiple of 8, rows
    16-byte aligned); with swiglu B has 2N rows a group, gate then up.  bounds: int32 [G + 1], group g's rows
    of out; rows: int32 [M], src(r) = rows[r] // top_k; without rows src(r) = r // top_k and M = A * top_k.
    out (or a new tensor of ``dtype``): a's type (the default) or float32.  Rows of out in no group are left as
    they were."""
    index = _mx_device(a, "a")
    b_shape = b.shape
    if a.dim() != 2 or len(b_shape) not in (2, 3):
        raise ValueError("a: expected a matrix; b: a matrix, or one per group")
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    A, K = a.shape
    G = b_shape[0] if len(b_shape) == 3 else 1
    NB = b_shape[-2]
    if swiglu and NB % 2:
        raise ValueError("b: swiglu needs gate and up rows, an even number")
    in_dtype = _DTYPE_ID.get(a.dtype)
    if in_dtype not in (MOE_BF16, MOE_F16) or b.dtype != a.dtype or b.get_device() != index:
        raise TypeError(f"a and b: expected the same of bfloat16, float16, on device {index}")
    if b_shape[-1] != K:
        raise ValueError(f"b: expected rows of {K}")
    N = NB // 2 if swiglu else NB
    M = rows.shape[0] if rows is not None else A * top_k
    if b.stride(-1) != 1 and K > 1:
        raise ValueError("b: rows must be contiguous")
    b_stride = b.stride(-2) if NB > 1 else K
    if b_stride < K:
        raise ValueError("b: rows overlap")
    raw = _stream_of(stream, index)
    if bounds is None and G != 1:
        raise ValueError("b of several groups needs bounds")
    bounds_at = _vector(bounds, "bounds", (G + 1,), torch.int32, index) if bounds is not None else None
    rows_at = _vector(rows, "rows", (M,), torch.int32, index) if rows is not None else None
    if out is None:
        out = _result((M, N), a.dtype if dtype is None else dtype, index, stream)
    out_dtype = _DTYPE_ID.get(out.dtype)
    if out_dtype not in (MOE_F32, in_dtype):
        raise TypeError("out: expected float32 or the type of a")
    args = moe_grouped_gemm_args_t(
        _GROUPED_GEMM_SIZE, index, a.data_ptr(), _rows_of(a, "a", A, K, index), A, b.data_ptr(), b_stride,
        b.stride(0) if G > 1 else 0, bounds_at, rows_at, G, top_k, M, N, K, 1 if swiglu else 0, in_dtype, out_dtype, 0,
        out.data_ptr(), _rows_of(out, "out", M, N, index))
    rc = lib().moe_grouped_gemm(args, raw)
    if rc:
        _check(rc)
    return out


def moe_combine_rows(d: torch.Tensor, weights: torch.Tensor, pos: torch.Tensor, y: Optional[torch.Tensor] = None,
                     base: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y[t] = base[t] + sum_j weights[t, j] * d[pos[t, j]], summed in slot order in fp32, rounded once.

    d [R, N], base [T, N] (None: 0; may be y itself) and y (or a new tensor of ``dtype``, by default d's type): fp32, bf16
    or fp16 each, rows may be strided.  weights fp32, pos int32, [T, k]; a slot whose pos is outside [0, R)
    is left out."""
    index = _mx_device(d, "d")
    if d.dim() != 2 or pos.dim() != 2:
        raise ValueError("d and pos: expected matrices")
    R, N = d.shape
    T, k = pos.shape
    raw = _stream_of(stream, index)
    weights_at = _vector(weights, "weights", (T, k), torch.float32, index)
    pos_at = _vector(pos, "pos", (T, k), torch.int32, index)
    if y is None:
        y = _result((T, N), d.dtype if dtype is None else dtype, index, stream)
    types = [_DTYPE_ID.get(t.dtype) if t is not None else MOE_F32 for t in (d, base, y)]
    if None in types:
        raise TypeError("d, base and y: expected float32, bfloat16 or float16")
    args = moe_combine_args_t(
        _COMBINE_SIZE, index, d.data_ptr(), _rows_of(d, "d", R, N, index), R, weights_at, pos_at,
        base.data_ptr() if base is not None else None, _rows_of(base, "base", T, N, index) if base is not None else 0,
        y.data_ptr(), _rows_of(y, "y", T, N, index), T, N, k, *types, 0)
    rc = lib().moe_combine_rows(args, raw)
    if rc:
        _check(rc)
    return y


# ----------------------------------------------------- low-rank adapters ---

def moe_lora_workspace_size(M: int, K: int, rank: int) -> int:
    """Bytes of moe_lora_add's workspace for M rows or fewer."""
    out = _u64()
    _check(lib().moe_lora_workspace_size(M, K, rank, ctypes.byref(out)))
    return int(out.value)


def moe_lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapters: torch.Tensor,
                 base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[t] = base[t] + scales[i] * (x[t] A_i^T) B_i^T with i = adapters[t]; a row whose adapter is outside
    [0, n) (-1) gets base[t].  Returns out.

    x [M, K], a [n, rank, K] and b [n, N, rank]: the same of bf16, fp16 (K and rank multiples of 8, rank up to
    256); adapters int32 [M]; scales fp32 [n] (None: 1); base [M, N] (None: 0; may be out itself) and out (or a new
    tensor of ``dtype``, by default x's type): fp32, bf16 or fp16 each.  Rows of x, base and out may be
    strided.  workspace: device uint8 scratch of moe_lora_workspace_size() bytes that no other call in flight
    uses; without one the call takes it from torch's allocator, on ``stream``."""
    index = _mx_device(x, "x")
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x: expected a matrix; a and b: one per adapter")
    M, K = x.shape
    n, r = a.shape[:2]
    N = b.shape[1]
    in_dtype = _DTYPE_ID.get(x.dtype)
    if in_dtype not in (MOE_BF16, MOE_F16):
        raise TypeError("x: expected bfloat16 or float16")
    a_at, b_at = _vector(a, "a", (n, r, K), x.dtype, index), _vector(b, "b", (n, N, r), x.dtype, index)
    adapters_at = _vector(adapters, "adapters", (M,), torch.int32, index)
    scales_at = _vector(scales, "scales", (n,), torch.float32, index) if scales is not None else None
    raw = _stream_of(stream, index)
    keep, ws, ws_bytes = _workspace(workspace, lambda: moe_lora_workspace_size(M, K, r), index, stream)
    if out is None:
        out = _result((M, N), x.dtype if dtype is None else dtype, index, stream)
    types = [_DTYPE_ID.get(t.dtype) if t is not None else MOE_F32 for t in (base, out)]
    if None in types:
        raise TypeError("base and out: expected float32, bfloat16 or float16")
    args = moe_lora_args_t(
        _LORA_SIZE, index, x.data_ptr(), _rows_of(x, "x", M, K, index), a_at, b_at, adapters_at, scales_at,
        base.data_ptr() if base is not None else None, _rows_of(base, "base", M, N, index) if base is not None else 0,
        out.data_ptr(), _rows_of(out, "out", M, N, index), M, N, K, r, n, in_dtype, *types, 0, ws, ws_bytes)
    rc = lib().moe_lora_add(args, raw)
    if rc:
        _check(rc)
    return out


# ----------------------------------------------------------- stream pool ---

def stream_pool_configure(handle: Handle, host_blobs: Sequence[torch.Tensor], prefetch_depth: int = 1,
                          resident_layers: int = 0, max_vram_bytes: int = 0,
                          requested_slots: int = 0, active_only: bool = False,
                          reserve_bytes: int = 0) -> dict:
    """Plan + allocate the slot pool over pinned host blobs (one per layer).
    active_only: streamed layers are loaded after their routing, only the experts with rows.
    reserve_bytes: device memory to keep free; checked when a pass starts (layer 0)."""
    p = stream_pool_params_t()
    p.struct_size = ctypes.sizeof(p)
    n = len(host_blobs)
    arr = (_vp * max(n, 1))()
    for i, b in enumerate(host_blobs):
        if b.device.type != "cpu" or b.dtype != torch.uint8 or not b.is_contiguous():
            raise TypeError("host blobs must be contiguous host uint8 tensors")
        if not b.is_pinned():
            raise TypeError("host blobs must be pinned (torch.empty(..., pin_memory=True))")
        arr[i] = b.data_ptr()
    p.n_layers = n
    p.host_blobs = ctypes.cast(arr, ctypes.POINTER(_vp))
    p.layer_bytes = host_blobs[0].numel() if n else 0
    p.prefetch_depth = prefetch_depth
    p.resident_layers = resident_layers
    p.max_vram_bytes = max_vram_bytes
    p.requested_slots = requested_slots
    p.active_only = 1 if active_only else 0
    p.reserve_bytes = reserve_bytes
    _check(lib().stream_pool_configure(handle.ptr, ctypes.byref(p)), handle.ptr)
    handle._pool_keep = list(host_blobs)
    return dict(slots=p.eff_slots, depth=p.eff_depth, residents=p.eff_residents, warnings=p.warnings)


def stream_pool_set_budget(handle: Handle, max_vram_bytes: int) -> dict:
    """Shrink the live pool to max_vram_bytes (memory pressure); returns the effective shape
    and the device bytes released."""
    p = stream_pool_budget_t()
    p.struct_size = ctypes.sizeof(p)
    p.max_vram_bytes = max_vram_bytes
    _check(lib().stream_pool_set_budget(handle.ptr, ctypes.byref(p)), handle.ptr)
    return dict(slots=p.eff_slots, depth=p.eff_depth, residents=p.eff_residents, warnings=p.warnings,
                released_bytes=p.released_bytes)


def moe_prefill_plan_trim(n_layers: int, residents: int, streaming: int, budget_slots: int) -> dict:
    p = moe_pool_trim_t()
    p.struct_size = ctypes.sizeof(p)
    p.n_layers, p.residents, p.streaming, p.budget_slots = n_layers, residents, streaming, budget_slots
    rc = lib().moe_prefill_plan_trim(ctypes.byref(p))
    return dict(rc=rc, residents=p.new_residents, streaming=p.new_streaming, evicted=p.evicted,
                converted=p.converted, released=p.released, warnings=p.warnings)


def moe_prefill_plan_pool(n_layers: int, slot_bytes: int, prefetch_depth: int, resident_layers: int,
                          max_vram_bytes: int = 0, requested_slots: int = 0,
                          max_alloc_slots: int = 0) -> dict:
    p = moe_pool_plan_t()
    p.struct_size = ctypes.sizeof(p)
    p.n_layers, p.slot_bytes, p.prefetch_depth, p.resident_layers = n_layers, slot_bytes, prefetch_depth, resident_layers
    p.max_vram_bytes, p.requested_slots, p.max_alloc_slots = max_vram_bytes, requested_slots, max_alloc_slots
    rc = lib().moe_prefill_plan_pool(ctypes.byref(p))
    out = dict(rc=rc, slots=p.slots, depth=p.depth, residents=p.residents, warnings=p.warnings)
    return out


def moe_prefill_get_stats(handle: Handle) -> dict:
    s = moe_stats_t()
    s.struct_size = ctypes.sizeof(s)
    _check(lib().moe_prefill_get_stats(handle.ptr, ctypes.byref(s)), handle.ptr)
    return {name: getattr(s, name) for name, _ in moe_stats_t._fields_ if name not in ("struct_size", "reserved0")}


# --------------------------------------------------------------- logging ---

def moe_prefill_set_log(handle: Handle, fn: Optional[Callable[[int, str], None]], level: int = MOE_LOG_WARN) -> None:
    """Route the handle's messages of level <= `level` to fn(level, text); fn=None removes the sink."""
    if fn is None:
        cb = ctypes.cast(None, _LOG_FN)
    else:
        cb = _LOG_FN(lambda lv, msg, user: fn(int(lv), msg.decode(errors="replace")))
    handle._log_cb = cb                    # the library keeps the pointer: keep the callback alive
    _check(lib().moe_prefill_set_log(handle.ptr, cb, None, level), handle.ptr)


# --------------------------------------------------------------- tracing ---

def moe_prefill_kernel_name(kernel_id: int) -> str:
    return lib().moe_prefill_kernel_name(kernel_id).decode()


def moe_prefill_set_timing(handle: Handle, enable: bool = True) -> None:
    _check(lib().moe_prefill_set_timing(handle.ptr, 1 if enable else 0), handle.ptr)


def moe_prefill_kernel_times(handle: Handle, reset: bool = True) -> dict:
    """{kernel name: (launches, total device ms)} of the timed launches so far."""
    t = moe_kernel_times_t()
    t.struct_size = ctypes.sizeof(t)
    _check(lib().moe_prefill_kernel_times(handle.ptr, ctypes.byref(t), 1 if reset else 0), handle.ptr)
    return {moe_prefill_kernel_name(i): (int(t.launches[i]), float(t.total_ms[i])) for i in range(t.n_kernels)}


def moe_prefill_exp_host(first_bits: int, out: np.ndarray) -> np.ndarray:
    """The library's fp32 exponential (host build) of the inputs with bit patterns
    first_bits .. first_bits + out.size - 1, written into out (float32, contiguous)."""
    assert out.dtype == np.float32 and out.flags["C_CONTIGUOUS"]
    _check(lib().moe_prefill_exp_host(first_bits, out.size, out.ctypes.data))
    return out


def moe_prefill_exp_device(first_bits: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """The kernels' fp32 exponential of the inputs with bit patterns first_bits ..
    first_bits + out.numel() - 1, enqueued on `stream` into the device tensor out."""
    assert out.dtype == torch.float32 and out.is_cuda and out.is_contiguous()
    st = stream if stream is not None else torch.cuda.current_stream(out.device)
    _check(lib().moe_prefill_exp_device(first_bits, out.numel(), out.data_ptr(), st.cuda_stream))
    return out
