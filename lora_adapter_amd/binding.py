"""Thin ctypes binding of liblora (the C ABI in include/lora.h).

Argument marshalling only: every step of the layer runs in the HIP library.
Tensors are torch tensors on the GPU (PyTorch serves as the device allocator
and stream provider); their data pointers are handed to the C entry points
with the current torch stream.  If liblora.so is missing, loading fails loudly:
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
# LORA_ADAPTER_LIB names another build of the same library (the host-sanitized
# one that the CPU tests load under the address sanitizer runtime)
LIB_PATH = os.environ.get("LORA_ADAPTER_LIB") or os.path.join(PKG, "liblora.so")

LORA_OK, LORA_ERR_INVALID_ARG, LORA_ERR_UNSUPPORTED, LORA_ERR_CAPACITY, LORA_ERR_DEVICE = range(5)
LORA_F32, LORA_BF16 = 0, 1
LORA_MAX_RANK = 1024
LORA_MAX_K = 8
DEVERR_BAD_ID, DEVERR_BAD_RANK, DEVERR_BAD_POOL, DEVERR_CAPACITY = 1, 2, 4, 8
PH_PAIRS, PH_SEGS, PH_ERR, PH_RPAIRS, PH_RUSED, PH_T, PH_K, PH_N = range(8)

EXPORTS = (
    "lora_abi_version", "lora_status_string", "lora_plan_bytes", "lora_plan_layout", "lora_plan",
    "lora_plan_header",
    "lora_apply_workspace_bytes", "lora_apply_u_offset", "lora_shrink", "lora_base_expand",
    "lora_base_gemm", "lora_expand_epilogue", "lora_shrink_gemm", "lora_apply",
    "lora_forward_gemm", "lora_forward_finish", "lora_forward", "lora_forward_noalloc_bytes",
    "lora_forward_noalloc", "lora_merge_delta", "lora_grad_workspace_bytes", "lora_grad",
    "lora_grad_x_workspace_bytes", "lora_grad_x", "lora_transpose", "lora_merge_delta_layers",
    "lora_page_table_create", "lora_page_table_destroy", "lora_page_table_admit",
    "lora_page_table_tables", "lora_residency_table_ints", "lora_residency_create",
    "lora_residency_destroy", "lora_residency_prepare", "lora_residency_finish",
    "lora_residency_stats", "lora_residency_page_table", "lora_tsqr_workspace_bytes", "lora_tsqr",
    "lora_compress_workspace_bytes", "lora_compress",
    "lora_quantised_row_bytes", "lora_quantised_scale_bytes", "lora_quantise_rows",
    "lora_quantise_weight", "lora_apply_quantised_workspace_bytes", "lora_apply_quantised",
    "lora_forward_quantised", "lora_grad_x_quantised_workspace_bytes", "lora_grad_x_quantised",
    "lora_orthogonalise_workspace_bytes", "lora_orthogonalise",
    "lora_orthogonal_step_workspace_bytes", "lora_orthogonal_step",
    "lora_gated_apply", "lora_gated_forward", "lora_gated_grad_workspace_bytes", "lora_gated_grad",
    "lora_cross_entropy_workspace_bytes", "lora_cross_entropy", "lora_clip_grad_workspace_bytes",
    "lora_clip_grad",
)


class LoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


class PoolDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
        ("n_adapters", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("n_page_ids", ctypes.c_int64),
        ("a_pages", ctypes.c_void_p), ("b_pages", ctypes.c_void_p), ("rank", ctypes.c_void_p),
        ("page_start", ctypes.c_void_p), ("page_ids", ctypes.c_void_p), ("scale", ctypes.c_void_p),
    ]


class LayerDesc(ctypes.Structure):
    _fields_ = [("W_t", ctypes.c_void_p), ("pool", PoolDesc)]


class PageCopy(ctypes.Structure):
    _fields_ = [("adapter", ctypes.c_int32), ("row", ctypes.c_int32), ("page", ctypes.c_int32),
                ("count", ctypes.c_int32)]


class QuantisedWeightDesc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("q_t", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("q", ctypes.c_void_p), ("scale_t", ctypes.c_void_p)]


class FactorUpdateDesc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("lr", ctypes.c_float), ("decay", ctypes.c_float)]


class GradDesc(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("dA_pages", ctypes.c_void_p), ("dB_pages", ctypes.c_void_p),
                ("dA_out", ctypes.c_void_p), ("dB_out", ctypes.c_void_p)]


class ResidencyConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("n_adapters", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("rank", ctypes.c_void_p), ("store_row", ctypes.c_void_p),
                ("store_a", ctypes.c_void_p), ("store_b", ctypes.c_void_p),
                ("a_pages", ctypes.c_void_p), ("b_pages", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("staging", ctypes.c_void_p)]


_lib = None
_I32, _I64, _SZ, _VP, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_PD = ctypes.POINTER(PoolDesc)
_QW = ctypes.POINTER(QuantisedWeightDesc)

_PROTOS = {
    "lora_abi_version": (_I32, []),
    "lora_status_string": (ctypes.c_char_p, [_I32]),
    "lora_plan_bytes": (_SZ, [_I32, _I32, _I32]),
    "lora_plan_layout": (_I32, [_I32, _I32, _I32, ctypes.POINTER(_I64)]),
    "lora_plan": (_I32, [_VP, _VP, _I32, _I32, _PD, _VP, _SZ, _VP]),
    "lora_plan_header": (_I32, [_VP, ctypes.POINTER(_I32), _VP]),
    "lora_apply_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "lora_apply_u_offset": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "lora_shrink": (_I32, [_VP, _VP, _F32, _I32, _I32, _VP, _PD, _VP, _VP, _SZ, _VP]),
    "lora_base_expand": (_I32, [_VP, _VP, _VP, _I32, _I32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_base_gemm": (_I32, [_VP, _VP, _VP, _I32, _I32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_expand_epilogue": (_I32, [_VP, _VP, _VP, _I32, _I32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_shrink_gemm": (_I32, [_VP, _VP, _VP, _I32, _I32, _VP, _VP, _F32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_apply": (_I32, [_VP, _VP, _VP, _I32, _I32, _VP, _VP, _F32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_forward_gemm": (_I32, [_VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _F32, _PD, _VP, _SZ,
                                 _VP, _SZ, _VP]),
    "lora_forward_finish": (_I32, [_VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _F32, _PD, _VP, _SZ,
                                   _VP, _SZ, _VP]),
    "lora_forward": (_I32, [_VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _F32, _PD, _VP, _SZ, _VP,
                            _SZ, _VP]),
    "lora_forward_noalloc_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "lora_forward_noalloc": (_I32, [_VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _F32, _PD, _I32,
                                    _VP]),
    "lora_merge_delta": (_I32, [_VP, _PD, _VP, _VP, _I32, _VP]),
    "lora_grad_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "lora_grad": (_I32, [_VP, _VP, _F32, _VP, _I32, _I32, _VP, _PD, _VP, _VP, _SZ, _VP, _VP,
                         _I32, _VP, _SZ, _VP]),
    "lora_grad_x_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "lora_grad_x": (_I32, [_VP, _VP, _VP, _I32, _I32, _PD, _VP, _VP, _SZ, _I32, _VP, _VP, _SZ,
                           _VP]),
    "lora_transpose": (_I32, [_VP, _VP, _I32, _I32, _I32, _VP]),
    "lora_merge_delta_layers": (_I32, [ctypes.POINTER(LayerDesc), _I32, _VP, _VP, _I32, _VP]),
    "lora_page_table_create": (_I32, [_VP, _I32, _I64, ctypes.POINTER(_VP)]),
    "lora_page_table_destroy": (None, [_VP]),
    "lora_page_table_admit": (_I32, [_VP, _VP, _I64, ctypes.POINTER(PageCopy), _I64,
                                     ctypes.POINTER(_I64), ctypes.POINTER(_I32), _I64,
                                     ctypes.POINTER(_I64)]),
    "lora_page_table_tables": (_I32, [_VP, ctypes.POINTER(_I32), ctypes.POINTER(_I32),
                                      ctypes.POINTER(_I32), ctypes.POINTER(_I64)]),
    "lora_residency_table_ints": (_SZ, [_I32, _I64]),
    "lora_residency_create": (_I32, [ctypes.POINTER(ResidencyConfig), ctypes.POINTER(_VP)]),
    "lora_residency_destroy": (None, [_VP]),
    "lora_residency_prepare": (_I32, [_VP, _VP, _I64, _VP, _VP, _PD]),
    "lora_residency_finish": (_I32, [_VP, _VP]),
    "lora_residency_stats": (_I32, [_VP, ctypes.POINTER(_I64)]),
    "lora_residency_page_table": (_VP, [_VP]),
    "lora_tsqr_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "lora_tsqr": (_I32, [_VP, _I32, _VP, _I32, _I32, _I32, _VP, _VP, _VP, _SZ, _VP]),
    "lora_compress_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "lora_compress": (_I32, [_PD, _VP, _I32, _I32, _I32, _F32, _F32, _I32, _VP, _VP, _VP, _VP, _VP,
                             _SZ, _VP]),
    "lora_quantised_row_bytes": (_I64, [_I32]),
    "lora_quantised_scale_bytes": (_I64, [_I32]),
    "lora_quantise_rows": (_I32, [_VP, _I32, _I32, _I32, _VP, _VP, _VP]),
    "lora_quantise_weight": (_I32, [_VP, _I32, _QW, _VP]),
    "lora_apply_quantised_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "lora_apply_quantised": (_I32, [_VP, _QW, _VP, _I32, _I32, _VP, _VP, _F32, _PD, _VP, _VP, _SZ, _VP]),
    "lora_forward_quantised": (_I32, [_VP, _VP, _I32, _I32, _VP, _QW, _VP, _VP, _F32, _PD, _VP, _SZ,
                                      _VP, _SZ, _VP]),
    "lora_grad_x_quantised_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "lora_grad_x_quantised": (_I32, [_VP, _QW, _VP, _I32, _I32, _PD, _VP, _VP, _SZ, _I32, _VP, _VP,
                                     _SZ, _VP]),
    "lora_orthogonalise_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "lora_orthogonalise": (_I32, [_PD, _VP, _I32, _I32, _VP, _VP, _I32, _I32, ctypes.POINTER(_F32),
                                  _F32, _VP, _VP, _SZ, _VP]),
    "lora_orthogonal_step_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "lora_orthogonal_step": (_I32, [_PD, _VP, _I32, _I32, ctypes.POINTER(FactorUpdateDesc),
                                    ctypes.POINTER(FactorUpdateDesc), _F32, _I32, _I32,
                                    ctypes.POINTER(_F32), _F32, _VP, _VP, _SZ, _VP]),
    "lora_gated_apply": (_I32, [_VP, _VP, _VP, _I32, _VP, _VP, _VP, _I32, _I32, _VP, _VP, _F32, _PD, _PD,
                                _VP, _VP, _SZ, _VP, _SZ, _VP]),
    "lora_gated_forward": (_I32, [_VP, _VP, _I32, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _F32,
                                  _PD, _PD, _VP, _SZ, _VP, _SZ, _VP, _SZ, _VP]),
    "lora_gated_grad_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "lora_gated_grad": (_I32, [_VP, _VP, _VP, _I32, _VP, _VP, _VP, _F32, _I32, _I32, _VP, _PD, _PD, _VP,
                               _I32, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_cross_entropy_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "lora_cross_entropy": (_I32, [_VP, _VP, _I32, _I32, _I32, _I32, _VP, _VP, _F32, _VP, _VP, _VP, _SZ, _VP]),
    "lora_clip_grad_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "lora_clip_grad": (_I32, [ctypes.POINTER(GradDesc), _I32, _VP, _I32, _I32, _F32, _I32, _VP, _VP, _SZ, _VP]),
}


def lib() -> ctypes.CDLL:
    """Load liblora.so (built in-tree); raise if it is not there."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m lora_adapter_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _PROTOS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lora_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != LORA_OK:
        raise LoraError(fn, status)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


# ---------------------------------------------------------------- pool

class Pool:
    """Device tensors of one adapter pool and the matching C descriptor."""

    def __init__(self, dtype: int, d_in: int, d_out: int, a_pages, b_pages, rank, page_start,
                 page_ids, scale):
        self.tensors = (a_pages, b_pages, rank, page_start, page_ids, scale)
        self.dtype, self.d_in, self.d_out = dtype, d_in, d_out
        self.n_adapters = int(rank.numel())
        self.desc = PoolDesc(dtype, d_in, d_out, self.n_adapters, int(a_pages.shape[0]),
                             int(page_ids.numel()), _ptr(a_pages), _ptr(b_pages), _ptr(rank),
                             _ptr(page_start), _ptr(page_ids) if page_ids.numel() else None,
                             _ptr(scale))

    @property
    def ref(self):
        return ctypes.byref(self.desc)


# ---------------------------------------------------------------- entry points

def lora_abi_version() -> int:
    return int(lib().lora_abi_version())


def lora_plan_bytes(T: int, K: int, n_adapters: int) -> int:
    return int(lib().lora_plan_bytes(T, K, n_adapters))


def lora_plan_layout(T: int, K: int, n_adapters: int):
    out = (_I64 * 9)()
    _check("lora_plan_layout", lib().lora_plan_layout(T, K, n_adapters, out))
    return [int(v) for v in out]


def lora_plan(ids, gates, T: int, K: int, pool: Pool, plan, stream=None):
    _check("lora_plan", lib().lora_plan(_ptr(ids), _ptr(gates), T, K, pool.ref, _ptr(plan),
                                        plan.numel() * plan.element_size(), _stream(stream)))


def lora_plan_header(plan, stream=None):
    """The plan's 16 header words (waits for the work queued on the stream)."""
    out = (_I32 * 16)()
    _check("lora_plan_header", lib().lora_plan_header(_ptr(plan), out, _stream(stream)))
    return [int(v) for v in out]


def lora_apply_workspace_bytes(T: int, K: int, d_in: int, d_out: int, max_rank: int, dtype: int) -> int:
    return int(lib().lora_apply_workspace_bytes(T, K, d_in, d_out, max_rank, dtype))


def lora_apply_u_offset(T: int, K: int, d_in: int, d_out: int, dtype: int) -> int:
    return int(lib().lora_apply_u_offset(T, K, d_in, d_out, dtype))


def lora_shrink(X, keep_mask, keep_scale: float, T: int, K: int, gates, pool: Pool, plan, ws,
                stream=None):
    _check("lora_shrink", lib().lora_shrink(_ptr(X), _ptr(keep_mask), float(keep_scale), T, K,
                                            _ptr(gates), pool.ref, _ptr(plan), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)))


def lora_base_expand(X, W_t, Y, T: int, K: int, pool: Pool, plan, ws, stream=None):
    _check("lora_base_expand", lib().lora_base_expand(_ptr(X), _ptr(W_t), _ptr(Y), T, K,
                                                      pool.ref, _ptr(plan), _ptr(ws),
                                                      ws.numel() * ws.element_size(), _stream(stream)))


def lora_base_gemm(X, W_t, Y, T: int, K: int, pool: Pool, plan, ws, stream=None):
    _check("lora_base_gemm", lib().lora_base_gemm(_ptr(X), _ptr(W_t), _ptr(Y), T, K,
                                                  pool.ref, _ptr(plan), _ptr(ws),
                                                  ws.numel() * ws.element_size(), _stream(stream)))


def lora_expand_epilogue(X, W_t, Y, T: int, K: int, pool: Pool, plan, ws, stream=None):
    _check("lora_expand_epilogue", lib().lora_expand_epilogue(
        _ptr(X), _ptr(W_t), _ptr(Y), T, K, pool.ref, _ptr(plan), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def lora_shrink_gemm(X, W_t, Y, T: int, K: int, gates, keep_mask, keep_scale: float, pool: Pool,
                     plan, ws, stream=None):
    _check("lora_shrink_gemm",
           lib().lora_shrink_gemm(_ptr(X), _ptr(W_t), _ptr(Y), T, K, _ptr(gates), _ptr(keep_mask),
                                  float(keep_scale), pool.ref, _ptr(plan), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)))


def lora_apply(X, W_t, Y, T: int, K: int, gates, keep_mask, keep_scale: float, pool: Pool,
               plan, ws, stream=None):
    _check("lora_apply", lib().lora_apply(_ptr(X), _ptr(W_t), _ptr(Y), T, K, _ptr(gates),
                                          _ptr(keep_mask), float(keep_scale), pool.ref, _ptr(plan),
                                          _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def _forward_call(name, ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool, plan, ws, stream):
    _check(name, getattr(lib(), name)(
        _ptr(ids), _ptr(gates), T, K, _ptr(X), _ptr(W_t), _ptr(Y), _ptr(keep_mask),
        float(keep_scale), pool.ref, _ptr(plan), plan.numel() * plan.element_size(), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def lora_forward_gemm(ids, gates, T: int, K: int, X, W_t, Y, keep_mask, keep_scale: float,
                      pool: Pool, plan, ws, stream=None):
    _forward_call("lora_forward_gemm", ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool,
                  plan, ws, stream)


def lora_forward_finish(ids, gates, T: int, K: int, X, W_t, Y, keep_mask, keep_scale: float,
                        pool: Pool, plan, ws, stream=None):
    _forward_call("lora_forward_finish", ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool,
                  plan, ws, stream)


def lora_forward(ids, gates, T: int, K: int, X, W_t, Y, keep_mask, keep_scale: float, pool: Pool,
                 plan, ws, stream=None):
    _forward_call("lora_forward", ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool, plan,
                  ws, stream)


def lora_forward_noalloc_bytes(T: int, K: int, n_adapters: int, d_in: int, d_out: int,
                               max_rank: int, dtype: int) -> int:
    return int(lib().lora_forward_noalloc_bytes(T, K, n_adapters, d_in, d_out, max_rank, dtype))


def lora_forward_noalloc(ids, gates, T: int, K: int, X, W_t, Y, keep_mask, keep_scale: float,
                         pool: Pool, max_rank: int, stream=None):
    _check("lora_forward_noalloc", lib().lora_forward_noalloc(
        _ptr(ids), _ptr(gates), T, K, _ptr(X), _ptr(W_t), _ptr(Y), _ptr(keep_mask),
        float(keep_scale), pool.ref, int(max_rank), _stream(stream)))


def lora_merge_delta(W_t, pool: Pool, merge_ids, coeffs, m: int, stream=None):
    _check("lora_merge_delta", lib().lora_merge_delta(_ptr(W_t), pool.ref, _ptr(merge_ids),
                                                      _ptr(coeffs), m, _stream(stream)))


def lora_grad_workspace_bytes(T: int, K: int, n_adapters: int, d_in: int, d_out: int, max_rank: int,
                              dtype: int) -> int:
    return int(lib().lora_grad_workspace_bytes(T, K, n_adapters, d_in, d_out, max_rank, dtype))


def lora_grad(X, keep_mask, keep_scale: float, dY, T: int, K: int, gates, pool: Pool, plan,
              apply_ws, dA_pages, dB_pages, max_rank: int, ws, stream=None):
    _check("lora_grad", lib().lora_grad(_ptr(X), _ptr(keep_mask), float(keep_scale), _ptr(dY), T, K,
                                        _ptr(gates), pool.ref, _ptr(plan), _ptr(apply_ws),
                                        apply_ws.numel() * apply_ws.element_size(), _ptr(dA_pages),
                                        _ptr(dB_pages), max_rank, _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)))


def lora_grad_x_workspace_bytes(T: int, d_in: int, d_out: int, dtype: int) -> int:
    return int(lib().lora_grad_x_workspace_bytes(T, d_in, d_out, dtype))


def lora_grad_x(dY, W, keep_mask, T: int, K: int, pool: Pool, plan, grad_ws, max_rank: int, dX,
                ws, stream=None):
    _check("lora_grad_x", lib().lora_grad_x(
        _ptr(dY), _ptr(W), _ptr(keep_mask), T, K, pool.ref, _ptr(plan), _ptr(grad_ws),
        grad_ws.numel() * grad_ws.element_size(), int(max_rank), _ptr(dX), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def lora_transpose(src, dst, rows: int, cols: int, dtype: int, stream=None):
    _check("lora_transpose", lib().lora_transpose(_ptr(src), _ptr(dst), rows, cols, dtype,
                                                  _stream(stream)))


def lora_merge_delta_layers(Ws, pools, merge_ids, coeffs, m: int, stream=None):
    """The same signed merge on every (W_t, pool) pair (one launch per up to
    16 layers of the MFMA form)."""
    n = len(Ws)
    arr = (LayerDesc * max(n, 1))()
    for i, (W, p) in enumerate(zip(Ws, pools)):
        arr[i].W_t = _ptr(W)
        arr[i].pool = p.desc
    _check("lora_merge_delta_layers", lib().lora_merge_delta_layers(
        arr, n, _ptr(merge_ids), _ptr(coeffs), m, _stream(stream)))


# ---------------------------------------------------------------- pool residency

def _host_i32(a):
    import numpy as np
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


class PageTable:
    """The residency policy alone (host object, no GPU)."""

    def __init__(self, rank, n_pages: int, handle=None):
        self._rank = _host_i32(rank)
        self.N, self.n_pages = int(self._rank.size), int(n_pages)
        self._own = handle is None
        if handle is None:
            h = _VP()
            _check("lora_page_table_create", lib().lora_page_table_create(
                self._rank.ctypes.data, self.N, self.n_pages, ctypes.byref(h)))
            handle = h.value
        self.h = handle

    def admit(self, ids):
        """{"copies": [(adapter, row, page, count)], "evicted": [...]} or
        {"error": "capacity"}."""
        ids = _host_i32(ids).reshape(-1)
        cp = (PageCopy * max(self.n_pages, 1))()
        ev = (_I32 * max(self.N, 1))()
        nc, ne = _I64(), _I64()
        st = lib().lora_page_table_admit(self.h, ids.ctypes.data if ids.size else None, ids.size,
                                         cp, self.n_pages, ctypes.byref(nc), ev, self.N,
                                         ctypes.byref(ne))
        if st == LORA_ERR_CAPACITY:
            return {"error": "capacity"}
        _check("lora_page_table_admit", st)
        return {"copies": [(c.adapter, c.row, c.page, c.count) for c in cp[:nc.value]],
                "evicted": [int(v) for v in ev[:ne.value]]}

    def tables(self):
        import numpy as np
        rk = np.zeros(self.N, np.int32)
        ps = np.zeros(self.N + 1, np.int32)
        pid = np.zeros(max(self.n_pages, 1), np.int32)
        n = _I64()
        _check("lora_page_table_tables", lib().lora_page_table_tables(
            self.h, rk.ctypes.data_as(ctypes.POINTER(_I32)), ps.ctypes.data_as(ctypes.POINTER(_I32)),
            pid.ctypes.data_as(ctypes.POINTER(_I32)), ctypes.byref(n)))
        return rk, ps, pid[:n.value].copy()

    def close(self):
        if self._own and self.h:
            lib().lora_page_table_destroy(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Residency:
    """The GPU pool of one projection, filled from a pinned host store on a
    copy stream (lora_residency_*).  `store_a`/`store_b` are pinned CPU torch
    tensors [rows][d]; `a_pages`/`b_pages` device tensors [n_pages][d]."""

    def __init__(self, dtype, d_in, d_out, rank, store_row, store_a, store_b, a_pages, b_pages,
                 scale):
        import numpy as np
        import torch
        self._rank = _host_i32(rank)
        self._row = np.ascontiguousarray(np.asarray(store_row, dtype=np.int64))
        self.N, self.n_pages = int(self._rank.size), int(a_pages.shape[0])
        nt = int(lib().lora_residency_table_ints(self.N, self.n_pages))
        self.tables = torch.zeros(nt, dtype=torch.int32, device=a_pages.device)
        self.staging = torch.zeros(nt, dtype=torch.int32).pin_memory()
        self._keep = (store_a, store_b, a_pages, b_pages, scale)
        self.cfg = ResidencyConfig(dtype, d_in, d_out, self.N, self.n_pages, self._rank.ctypes.data,
                                   self._row.ctypes.data, _ptr(store_a), _ptr(store_b),
                                   _ptr(a_pages), _ptr(b_pages), _ptr(scale), _ptr(self.tables),
                                   _ptr(self.staging))
        h = _VP()
        _check("lora_residency_create", lib().lora_residency_create(ctypes.byref(self.cfg),
                                                                    ctypes.byref(h)))
        self.h = h.value
        self.dtype, self.d_in, self.d_out = dtype, d_in, d_out

    def prepare(self, ids, copy_stream, compute_stream=None):
        """Returns a Pool (descriptor of the batch's tables) for the batch."""
        ids = _host_i32(ids).reshape(-1)
        desc = PoolDesc()
        st = lib().lora_residency_prepare(self.h, ids.ctypes.data if ids.size else None, ids.size,
                                          _stream(copy_stream), _stream(compute_stream),
                                          ctypes.byref(desc))
        _check("lora_residency_prepare", st)
        p = Pool.__new__(Pool)
        p.tensors = self._keep + (self.tables,)
        p.dtype, p.d_in, p.d_out, p.n_adapters = self.dtype, self.d_in, self.d_out, self.N
        p.desc = desc
        return p

    def finish(self, compute_stream=None):
        _check("lora_residency_finish", lib().lora_residency_finish(self.h, _stream(compute_stream)))

    def stats(self):
        out = (_I64 * 4)()
        _check("lora_residency_stats", lib().lora_residency_stats(self.h, out))
        return {"batches": out[0], "rows_copied": out[1], "evictions": out[2], "bytes": out[3]}

    def page_table(self):
        return PageTable(self._rank, self.n_pages, handle=lib().lora_residency_page_table(self.h))

    def close(self):
        if self.h:
            lib().lora_residency_destroy(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- tall-skinny QR

def lora_tsqr_workspace_bytes(M: int, m: int, n: int) -> int:
    return int(lib().lora_tsqr_workspace_bytes(M, m, n))


def lora_tsqr(src, dtype: int, cols, M: int, m: int, n: int, Qt, R, ws, stream=None):
    _check("lora_tsqr", lib().lora_tsqr(_ptr(src), dtype, _ptr(cols), M, m, n, _ptr(Qt), _ptr(R),
                                        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def lora_compress_workspace_bytes(M: int, d_in: int, d_out: int, n: int) -> int:
    return int(lib().lora_compress_workspace_bytes(M, d_in, d_out, n))


def lora_compress(pool: Pool, adapters, M: int, n: int, policy: int, ratio: float, energy: float,
                  floor_rank: int, out_a, out_b, out_rank, out_sigma, ws, stream=None):
    _check("lora_compress", lib().lora_compress(
        pool.ref, _ptr(adapters), M, n, policy, float(ratio), float(energy), floor_rank,
        _ptr(out_a), _ptr(out_b), _ptr(out_rank), _ptr(out_sigma), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------- 8-bit base weight

def lora_quantised_row_bytes(d: int) -> int:
    return int(lib().lora_quantised_row_bytes(d))


def lora_quantised_scale_bytes(d: int) -> int:
    return int(lib().lora_quantised_scale_bytes(d))


class QuantisedWeight:
    """Device tensors of one weight's e4m3 codes and scale bytes (layouts in
    include/lora.h) and the matching C descriptor.  `q` and `scale_t` (the
    codes of W for the input gradient) may be None."""

    def __init__(self, d_out: int, d_in: int, q_t, scale, q=None, scale_t=None):
        rb, sb, nb = lora_quantised_row_bytes, lora_quantised_scale_bytes, lambda d: (d + 127) // 128
        for t, rows, row in ((q_t, d_out, rb(d_in)), (scale, nb(d_out), sb(d_in)),
                             (q, d_in, rb(d_out)), (scale_t, nb(d_in), sb(d_out))):
            if t is not None and (tuple(t.shape) != (rows, row) or t.element_size() != 1
                                  or not t.is_contiguous()):
                raise ValueError(f"expected a contiguous 1-byte tensor [{rows}][{row}], got {tuple(t.shape)}")
        self.d_out, self.d_in = d_out, d_in
        self.q_t, self.scale, self.q, self.scale_t = q_t, scale, q, scale_t
        self.desc = QuantisedWeightDesc(d_in, d_out, _ptr(q_t), _ptr(scale), _ptr(q), _ptr(scale_t))

    @classmethod
    def empty(cls, d_out: int, d_in: int, device="cuda", both: bool = True):
        """Unfilled buffers for lora_quantise_weight (`both`: W too)."""
        import torch
        rb, sb, nb = lora_quantised_row_bytes, lora_quantised_scale_bytes, lambda d: (d + 127) // 128
        e = lambda *s: torch.empty(s, dtype=torch.uint8, device=device)
        return cls(d_out, d_in, e(d_out, rb(d_in)), e(nb(d_out), sb(d_in)),
                   e(d_in, rb(d_out)) if both else None, e(nb(d_in), sb(d_out)) if both else None)

    @property
    def ref(self):
        return ctypes.byref(self.desc)


def lora_quantise_rows(X, dtype: int, T: int, d: int, codes, scale, stream=None):
    _check("lora_quantise_rows", lib().lora_quantise_rows(_ptr(X), dtype, T, d, _ptr(codes),
                                                          _ptr(scale), _stream(stream)))


def lora_quantise_weight(W_t, dtype: int, w: QuantisedWeight, stream=None):
    _check("lora_quantise_weight", lib().lora_quantise_weight(_ptr(W_t), dtype, w.ref, _stream(stream)))


def lora_apply_quantised_workspace_bytes(T: int, K: int, d_in: int, d_out: int, max_rank: int,
                                         dtype: int) -> int:
    return int(lib().lora_apply_quantised_workspace_bytes(T, K, d_in, d_out, max_rank, dtype))


def lora_apply_quantised(X, W: QuantisedWeight, Y, T: int, K: int, gates, keep_mask,
                         keep_scale: float, pool: Pool, plan, ws, stream=None):
    _check("lora_apply_quantised", lib().lora_apply_quantised(
        _ptr(X), W.ref, _ptr(Y), T, K, _ptr(gates), _ptr(keep_mask), float(keep_scale), pool.ref,
        _ptr(plan), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def lora_forward_quantised(ids, gates, T: int, K: int, X, W: QuantisedWeight, Y, keep_mask,
                           keep_scale: float, pool: Pool, plan, ws, stream=None):
    _check("lora_forward_quantised", lib().lora_forward_quantised(
        _ptr(ids), _ptr(gates), T, K, _ptr(X), W.ref, _ptr(Y), _ptr(keep_mask), float(keep_scale),
        pool.ref, _ptr(plan), plan.numel() * plan.element_size(), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def lora_grad_x_quantised_workspace_bytes(T: int, d_in: int, d_out: int, dtype: int) -> int:
    return int(lib().lora_grad_x_quantised_workspace_bytes(T, d_in, d_out, dtype))


def lora_grad_x_quantised(dY, W: QuantisedWeight, keep_mask, T: int, K: int, pool: Pool, plan,
                          grad_ws, max_rank: int, dX, ws, stream=None):
    _check("lora_grad_x_quantised", lib().lora_grad_x_quantised(
        _ptr(dY), W.ref, _ptr(keep_mask), T, K, pool.ref, _ptr(plan), _ptr(grad_ws),
        grad_ws.numel() * grad_ws.element_size(), int(max_rank), _ptr(dX), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------- orthogonalised updates

NS_COEF = (3.4445, -4.7750, 2.0315)     # quintic coefficients whose slope at 0 is largest


def _check_pages(pool: Pool, t, d: int, size: int):
    """Pages that a call takes as [n_pages][d] elements of `size` bytes."""
    n = int(pool.desc.n_pages)
    if tuple(t.shape) != (n, d) or t.element_size() != size or not t.is_contiguous():
        raise ValueError(f"expected contiguous pages [{n}][{d}] of {size}-byte elements, got {tuple(t.shape)}")


class FactorUpdate:
    """One factor's buffers of lora_orthogonal_step: its pages (the pool's own
    a_pages or b_pages), float32 gradient, momentum and (or None) master pages."""

    def __init__(self, pages, grad, momentum, master, lr: float, decay: float = 0.0):
        if not pages.is_contiguous():
            raise ValueError("expected contiguous pages")
        for t in (grad, momentum, master):
            if t is not None and (t.shape != pages.shape or t.element_size() != 4 or not t.is_contiguous()):
                raise ValueError(f"expected contiguous float32 pages {tuple(pages.shape)}, got {tuple(t.shape)}")
        self.tensors = (pages, grad, momentum, master)
        self.desc = FactorUpdateDesc(_ptr(pages), _ptr(master), _ptr(momentum), _ptr(grad), float(lr),
                                     float(decay))

    @property
    def ref(self):
        return ctypes.byref(self.desc)


def lora_orthogonalise_workspace_bytes(M: int, max_rank: int, d: int) -> int:
    return int(lib().lora_orthogonalise_workspace_bytes(M, max_rank, d))


def lora_orthogonalise(pool: Pool, adapters, M: int, max_rank: int, src_pages, out_pages, d: int,
                       steps: int, coef, eps: float, ws, out_rank=None, stream=None):
    for t in (src_pages, out_pages):
        _check_pages(pool, t, d, 4)
    _check("lora_orthogonalise", lib().lora_orthogonalise(
        pool.ref, _ptr(adapters), M, max_rank, _ptr(src_pages), _ptr(out_pages), d, steps,
        (_F32 * 3)(*coef), float(eps), _ptr(out_rank), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def lora_orthogonal_step_workspace_bytes(M: int, max_rank: int, d_in: int, d_out: int) -> int:
    return int(lib().lora_orthogonal_step_workspace_bytes(M, max_rank, d_in, d_out))


def lora_orthogonal_step(pool: Pool, adapters, M: int, max_rank: int, a: FactorUpdate,
                         b: FactorUpdate, momentum: float, nesterov: bool, steps: int, coef,
                         eps: float, ws, out_rank=None, stream=None):
    for f, d in ((a, pool.d_in), (b, pool.d_out)):
        _check_pages(pool, f.tensors[0], d, 2 if pool.dtype == LORA_BF16 else 4)
    _check("lora_orthogonal_step", lib().lora_orthogonal_step(
        pool.ref, _ptr(adapters), M, max_rank, a.ref, b.ref, float(momentum), int(nesterov), steps,
        (_F32 * 3)(*coef), float(eps), _ptr(out_rank), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


# ---------------------------------------------------------------- gated feed-forward

LORA_ACT_SILU, LORA_ACT_GELU, LORA_ACT_GELU_TANH = range(3)


def _size(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _check_rows(pool: Pool, T: int, **tensors):
    """Contiguous rows [T][width] of the pool's dtype: name=(tensor or None, width)."""
    size = 2 if pool.dtype == LORA_BF16 else 4
    for name, (t, width) in tensors.items():
        if t is not None and (tuple(t.shape) != (T, width) or t.element_size() != size or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous [{T}][{width}] of {size}-byte elements, got {tuple(t.shape)}")


def _check_values(size: int, n: int, **tensors):
    """Contiguous, n elements of `size` bytes or more: name=tensor or None."""
    for name, t in tensors.items():
        if t is not None and (t.numel() < n or t.element_size() != size or not t.is_contiguous()):
            raise ValueError(f"{name}: expected {n} contiguous elements of {size} bytes, got {tuple(t.shape)} of {t.dtype}")


def _check_routing(pool: Pool, T: int, K: int, gates, keep_mask, ids=None):
    _check_values(4, T * K, ids=ids, gates=gates)
    _check_values(1, T * pool.d_in, keep_mask=keep_mask)


def lora_gated_apply(X, W_gate_t, W_up_t, activation: int, H, pre_gate, pre_up, T: int, K: int, gates,
                     keep_mask, keep_scale: float, gate: Pool, up: Pool, plan, ws_gate, ws_up, stream=None):
    F = gate.d_out
    _check_rows(gate, T, X=(X, gate.d_in), H=(H, F), pre_gate=(pre_gate, F), pre_up=(pre_up, F))
    _check_rows(gate, F, W_gate_t=(W_gate_t, gate.d_in), W_up_t=(W_up_t, gate.d_in))
    _check_routing(gate, T, K, gates, keep_mask)
    _check("lora_gated_apply", lib().lora_gated_apply(
        _ptr(X), _ptr(W_gate_t), _ptr(W_up_t), activation, _ptr(H), _ptr(pre_gate), _ptr(pre_up), T, K,
        _ptr(gates), _ptr(keep_mask), float(keep_scale), gate.ref, up.ref, _ptr(plan), _ptr(ws_gate),
        _size(ws_gate), _ptr(ws_up), _size(ws_up), _stream(stream)))


def lora_gated_forward(ids, gates, T: int, K: int, X, W_gate_t, W_up_t, activation: int, H, pre_gate, pre_up,
                       keep_mask, keep_scale: float, gate: Pool, up: Pool, plan, ws_gate, ws_up, stream=None):
    F = gate.d_out
    _check_rows(gate, T, X=(X, gate.d_in), H=(H, F), pre_gate=(pre_gate, F), pre_up=(pre_up, F))
    _check_rows(gate, F, W_gate_t=(W_gate_t, gate.d_in), W_up_t=(W_up_t, gate.d_in))
    _check_routing(gate, T, K, gates, keep_mask, ids)
    _check("lora_gated_forward", lib().lora_gated_forward(
        _ptr(ids), _ptr(gates), T, K, _ptr(X), _ptr(W_gate_t), _ptr(W_up_t), activation, _ptr(H),
        _ptr(pre_gate), _ptr(pre_up), _ptr(keep_mask), float(keep_scale), gate.ref, up.ref, _ptr(plan),
        _size(plan), _ptr(ws_gate), _size(ws_gate), _ptr(ws_up), _size(ws_up), _stream(stream)))


def lora_gated_grad_workspace_bytes(T: int, K: int, d_in: int, d_out: int, max_rank: int, dtype: int) -> int:
    return int(lib().lora_gated_grad_workspace_bytes(T, K, d_in, d_out, max_rank, dtype))


def lora_gated_grad(dH, pre_gate, pre_up, activation: int, W_gate, W_up, keep_mask, keep_scale: float, T: int,
                    K: int, gates, gate: Pool, up: Pool, plan, max_rank: int, d_gate, d_up, dX, ws, stream=None):
    F = gate.d_out
    _check_rows(gate, T, dH=(dH, F), pre_gate=(pre_gate, F), pre_up=(pre_up, F), d_gate=(d_gate, F),
                d_up=(d_up, F), dX=(dX, gate.d_in))
    _check_rows(gate, gate.d_in, W_gate=(W_gate, F), W_up=(W_up, F))
    _check_routing(gate, T, K, gates, keep_mask)
    _check("lora_gated_grad", lib().lora_gated_grad(
        _ptr(dH), _ptr(pre_gate), _ptr(pre_up), activation, _ptr(W_gate), _ptr(W_up), _ptr(keep_mask),
        float(keep_scale), T, K, _ptr(gates), gate.ref, up.ref, _ptr(plan), max_rank, _ptr(d_gate),
        _ptr(d_up), _ptr(dX), _ptr(ws), _size(ws), _stream(stream)))


# ---------------------------------------------------------------- cross entropy

def lora_cross_entropy_workspace_bytes(T: int, V: int, d: int, dtype: int, with_grad: bool = True) -> int:
    return int(lib().lora_cross_entropy_workspace_bytes(T, V, d, dtype, int(with_grad)))


def lora_cross_entropy(X, W_t, dtype: int, T: int, V: int, d: int, targets, weights, logit_scale: float, loss,
                       dX, ws, stream=None):
    """weights and dX may be None (1 for each token; the loss alone)."""
    size = 2 if dtype == LORA_BF16 else 4
    for name, t, shape, n in (("X", X, (T, d), size), ("W_t", W_t, (V, d), size), ("targets", targets, (T,), 4),
                              ("weights", weights, (T,), 4), ("loss", loss, (T,), 4), ("dX", dX, (T, d), size)):
        if t is not None and (tuple(t.shape) != shape or t.element_size() != n or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {list(shape)} of {n}-byte elements, got {tuple(t.shape)}")
    _check("lora_cross_entropy", lib().lora_cross_entropy(
        _ptr(X), _ptr(W_t), dtype, T, V, d, _ptr(targets), _ptr(weights), float(logit_scale), _ptr(loss),
        _ptr(dX), _ptr(ws), _size(ws), _stream(stream)))


# ---------------------------------------------------------------- gradient clipping

class GradLayers:
    """The gradient pages of many layers for lora_clip_grad: entries (pool, dA,
    dB) to clip in place, or (pool, dA, dB, dA_out, dB_out)."""

    def __init__(self, layers):
        self.layers = [tuple(e) if len(e) == 5 else (e[0], e[1], e[2], e[1], e[2]) for e in layers]
        self.n = len(self.layers)
        self.desc = (GradDesc * max(self.n, 1))()
        for d, (pool, a, b, oa, ob) in zip(self.desc, self.layers):
            for t, width in ((a, pool.d_in), (b, pool.d_out), (oa, pool.d_in), (ob, pool.d_out)):
                _check_pages(pool, t, width, 4)
            d.pool = pool.desc
            d.dA_pages, d.dB_pages, d.dA_out, d.dB_out = _ptr(a), _ptr(b), _ptr(oa), _ptr(ob)


def lora_clip_grad_workspace_bytes(layers: GradLayers, M: int, max_rank: int) -> int:
    return int(lib().lora_clip_grad_workspace_bytes(layers.n, M, max_rank))


def lora_clip_grad(layers: GradLayers, adapters, M: int, max_rank: int, max_norm: float, together: bool, norm,
                   ws, stream=None):
    if norm.numel() != M + 1 or norm.element_size() != 4 or not norm.is_contiguous():
        raise ValueError(f"norm: expected {M + 1} contiguous float32, got {tuple(norm.shape)}")
    _check_values(4, M, adapters=adapters)
    _check("lora_clip_grad", lib().lora_clip_grad(
        layers.desc, layers.n, _ptr(adapters), M, max_rank, float(max_norm), int(together), _ptr(norm), _ptr(ws),
        _size(ws), _stream(stream)))
