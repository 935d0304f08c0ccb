"""Python binding of the GB300 embedding-step library (include/emb_gb300.h).

Argument marshalling only: every function forwards to the C entry point of the
same name in ``_build/libemb_gb300.so``, passing tensor data pointers, sizes
and the current CUDA stream.  All computation happens in the library's
sm_103a kernels; there is no fallback path.  If the library has not been
built, importing succeeds but the first call raises ``LibraryNotBuilt``.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import re
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from .build import HEADER, LIB_PATH, build

__all__ = [
    "EmbError", "LibraryNotBuilt", "Table", "lib", "declared_symbols",
    "emb_table_create", "emb_table_create_device", "emb_table_destroy", "emb_table_get_stats", "emb_table_plan",
    "emb_lookup_fwd", "emb_lookup_fwd_record", "emb_lookup_fwd_dedup", "emb_bwd_adagrad_recorded", "emb_bwd_workspace_size", "emb_bwd_adagrad", "emb_bwd_adagrad_noalloc",
    "emb_bwd_ftrl", "emb_bwd_ftrl_recorded", "emb_table_export_z", "emb_table_import_z",
    "emb_debug_fail_device_alloc", "emb_debug_live_device_allocs", "emb_debug_set_probe_bound", "emb_debug_lose_op_wait",
    "emb_debug_fp8_matmul_plan", "Pipeline",
    "emb_bwd_unique_keys", "emb_bwd_phase_events", "EMB_NOALLOC_SCRATCH_BYTES", "EMB_SORT_DIGIT_BITS", "BWD_PHASES",
    "emb_resolve", "emb_table_export", "emb_table_export_rows", "emb_table_slots", "emb_check_device_flag",
    "emb_status_string", "emb_last_error",
    "EMB_FLAG_PROBE_BOUND", "EMB_FLAG_BAD_OFFSETS", "EMB_FLAG_SLOT_MISMATCH", "EMB_FLAG_BAD_ROW",
    "emb_fp8_quantize", "emb_fp8_matmul", "emb_fp8_matmul_workspace_size", "emb_norm_gate_fwd", "emb_norm_gate_bwd",
    "emb_norm_gate_bwd_workspace_size", "emb_adamw_step", "AdamW", "emb_check_op_flag",
    "EMB_FLAG_OP_TIMEOUT", "EMB_FP8_BLOCK", "EMB_ADAM_BLOCK", "EMB_NORM_MAX_DIM",
]

EMB_OK = 0
STATUS = {0: "EMB_OK", 1: "EMB_ERR_INVALID_ARG", 2: "EMB_ERR_CUDA", 3: "EMB_ERR_OOM", 4: "EMB_ERR_DUP_KEY",
          5: "EMB_ERR_RESERVED_KEY", 6: "EMB_ERR_LOAD_FACTOR", 7: "EMB_ERR_WORKSPACE",
          8: "EMB_ERR_DEVICE_FLAG", 9: "EMB_ERR_UNSUPPORTED"}
EMB_FLAG_PROBE_BOUND, EMB_FLAG_BAD_OFFSETS, EMB_FLAG_SLOT_MISMATCH, EMB_FLAG_BAD_ROW = 1, 2, 4, 8
EMB_NOALLOC_SCRATCH_BYTES = 64 << 20
EMB_SORT_DIGIT_BITS = 7
EMB_FLAG_OP_TIMEOUT = 16
EMB_FP8_BLOCK = 128
EMB_ADAM_BLOCK = 256
EMB_NORM_MAX_DIM = 8192
BWD_PHASES = ("expand", "sort", "reduce", "fixup")
_DTYPE = {"f32": 0, "f16": 1, "f16m": 2}   # f16m: f32 master rows + the f16 copy the forward reads
_POOL = {"sum": 0, "mean": 1}
_OPT = {"adagrad": 0, "ftrl": 1, "rowwise_adagrad": 2}
_FTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_NORM = {"rms": 0, "layer": 1}
_ACT = {"identity": 0, "sigmoid": 1}
_ADAM_STATE = {"f32": 0, "q8": 1}


class LibraryNotBuilt(ImportError):
    pass


class EmbError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS.get(status, str(status))
        self.message = message


class _Desc(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("slot_dim", ctypes.POINTER(ctypes.c_int32)),
                ("wdtype", ctypes.c_int), ("capacity", ctypes.c_int64), ("acc_init", ctypes.c_float),
                ("optimizer", ctypes.c_int)]


class _Ftrl(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("lambda1", ctypes.c_float),
                ("lambda2", ctypes.c_float)]


class _Stats(ctypes.Structure):
    _fields_ = [("n_keys", ctypes.c_int64), ("capacity", ctypes.c_int64), ("n_elems", ctypes.c_int64),
                ("n_slots", ctypes.c_int32), ("sum_dims", ctypes.c_int32), ("max_dim", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("max_probe", ctypes.c_int64), ("sum_probe", ctypes.c_int64),
                ("max_cluster", ctypes.c_int64), ("probe_bound", ctypes.c_int64),
                ("load_factor", ctypes.c_double), ("device_bytes", ctypes.c_uint64),
                ("max_slot_keys", ctypes.c_int64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class _NormGate(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("stream_t", ctypes.c_int), ("block_t", ctypes.c_int),
                ("norm", ctypes.c_int), ("gate", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float)]


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("first", ctypes.c_int64), ("param_t", ctypes.c_int), ("grad_t", ctypes.c_int), ("copy_t", ctypes.c_int)]


class _AdamwParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("state", ctypes.c_int),
                ("seed", ctypes.c_uint32), ("grad_scale", ctypes.c_void_p)]


_lib = None
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


def lib():
    """The loaded library (ctypes.CDLL); raises LibraryNotBuilt if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LibraryNotBuilt(f"{LIB_PATH} is missing: run `python -c 'import sparse_ctr_embedding_gb300 as E; E.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "emb_table_create": [ctypes.POINTER(_Desc), _vp, _i64, _vp, _vp, _vp, ctypes.POINTER(_vp)],
            "emb_table_destroy": [_vp],
            "emb_table_create_device": [ctypes.POINTER(_Desc), _vp, _i64, _vp, _vp, _vp, ctypes.POINTER(_vp)],
            "emb_table_get_stats": [_vp, ctypes.POINTER(_Stats)],
            "emb_table_plan": [ctypes.POINTER(_Desc), _vp, _i64, ctypes.POINTER(_Stats), _vp, _vp],
            "emb_lookup_fwd": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _vp],
            "emb_bwd_workspace_size": [_vp, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)],
            "emb_bwd_adagrad": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, ctypes.c_float, ctypes.c_float,
                                _vp, ctypes.c_size_t, _vp],
            "emb_bwd_unique_keys": [_vp, _vp, ctypes.c_size_t, _vp, _vp, _vp],
            "emb_bwd_phase_events": [_vp, ctypes.POINTER(_vp), ctypes.c_int],
            "emb_lookup_fwd_record": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp],
            "emb_lookup_fwd_dedup": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp],
            "emb_bwd_adagrad_recorded": [_vp, _i64, _i64, ctypes.c_int, _vp, ctypes.c_float, ctypes.c_float, _vp,
                                         ctypes.c_size_t, _vp],
            "emb_bwd_adagrad_noalloc": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, ctypes.c_float,
                                        ctypes.c_float, _vp],
            "emb_bwd_ftrl": [_vp, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, ctypes.POINTER(_Ftrl), _vp,
                             ctypes.c_size_t, _vp],
            "emb_bwd_ftrl_recorded": [_vp, _i64, _i64, ctypes.c_int, _vp, ctypes.POINTER(_Ftrl), _vp,
                                      ctypes.c_size_t, _vp],
            "emb_table_export_z": [_vp, _vp, _vp],
            "emb_debug_fail_device_alloc": [_i64],
            "emb_pipeline_create": [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, ctypes.POINTER(_vp)],
            "emb_pipeline_destroy": [_vp],
            "emb_pipeline_submit": [_vp, _vp, _i64, _vp, _i64, _vp, ctypes.POINTER(_i64)],
            "emb_pipeline_forward": [_vp, _i64, ctypes.c_int, _vp, _vp, ctypes.POINTER(_vp)],
            "emb_pipeline_backward_adagrad": [_vp, _i64, _vp, ctypes.c_float, ctypes.c_float],
            "emb_pipeline_backward_ftrl": [_vp, _i64, _vp, ctypes.POINTER(_Ftrl)],
            "emb_pipeline_release": [_vp, _i64],
            "emb_pipeline_wait": [_vp, _i64],
            "emb_debug_set_probe_bound": [_vp, _i64],
            "emb_debug_lose_op_wait": [ctypes.c_int32, _i64],
            "emb_debug_fp8_matmul_plan": [_i64, _i64, _i64, ctypes.POINTER(_i64)],
            "emb_table_import_z": [_vp, _vp, _vp],
            "emb_resolve": [_vp, _vp, _i64, _vp, _vp, _vp],
            "emb_table_export": [_vp, _vp, _vp, _vp, _vp],
            "emb_table_slots": [_vp, _vp, _vp, _vp],
            "emb_table_export_rows": [_vp, _vp, _i64, _vp, _vp, _vp],
            "emb_check_device_flag": [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)],
            "emb_fp8_quantize": [_vp, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int32, _vp, _i64, _vp, _vp, _i64, _vp, _vp],
            "emb_fp8_matmul_workspace_size": [_i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)],
            "emb_fp8_matmul": [_vp, _i64, _vp, ctypes.c_int32, _vp, _i64, _vp, ctypes.c_int32, _i64, _i64, _i64, _vp,
                               _vp, ctypes.c_int, _i64, _vp, ctypes.c_size_t, _vp],
            "emb_norm_gate_fwd": [ctypes.POINTER(_NormGate)] + [_vp] * 11,
            "emb_norm_gate_bwd_workspace_size": [ctypes.POINTER(_NormGate), ctypes.POINTER(ctypes.c_size_t)],
            "emb_norm_gate_bwd": [ctypes.POINTER(_NormGate)] + [_vp] * 17 + [ctypes.c_size_t, _vp],
            "emb_adamw_step": [_vp, _vp, ctypes.c_int32, ctypes.POINTER(_AdamwParams), _vp],
            "emb_check_op_flag": [_vp, ctypes.POINTER(ctypes.c_uint32)],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.emb_status_string.argtypes = [ctypes.c_int]
        L.emb_status_string.restype = ctypes.c_char_p
        L.emb_last_error.argtypes = []
        L.emb_last_error.restype = ctypes.c_char_p
        L.emb_debug_live_device_allocs.argtypes = []
        L.emb_debug_live_device_allocs.restype = ctypes.c_int64
        _lib = L
    return _lib


def declared_symbols() -> Sequence[str]:
    """Entry points declared in include/emb_gb300.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^EMB_API [^(]*?\b(emb_\w+)\(", text, flags=re.M)))


def emb_status_string(status: int) -> str:
    return lib().emb_status_string(status).decode()


def emb_last_error() -> str:
    return lib().emb_last_error().decode()


def _check(rc: int):
    if rc != EMB_OK:
        raise EmbError(rc, emb_last_error())


def _stream(stream) -> _vp:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return _vp(stream.cuda_stream)
    return _vp(int(stream))


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _ptr(t, dtype, name)


def _desc(dims, wdtype, capacity, acc_init, optimizer="adagrad"):
    dims_arr = (ctypes.c_int32 * len(dims))(*[int(d) for d in dims])
    d = _Desc(len(dims), dims_arr, _DTYPE[wdtype], int(capacity), float(acc_init), _OPT[optimizer])
    return d, dims_arr


class Table:
    """Owner of one emb_table handle."""

    def __init__(self, handle: int, dims, wdtype: str, optimizer: str = "adagrad"):
        self._h = _vp(handle)
        self.dims = tuple(int(d) for d in dims)
        self.wdtype = wdtype
        self.optimizer = optimizer
        self.stats = emb_table_get_stats(self)

    @property
    def handle(self):
        return self._h

    @property
    def n_slots(self):
        return len(self.dims)

    def close(self):
        if self._h:
            lib().emb_table_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def emb_table_create(dims, wdtype: str, keys: torch.Tensor, values: Optional[torch.Tensor] = None,
                     acc: Optional[torch.Tensor] = None, capacity: int = 0, acc_init: float = 0.0,
                     stream=None, optimizer: str = "adagrad") -> Table:
    """keys: CPU int64; values/acc: CPU or CUDA, ragged rows in keys order.
    optimizer: "adagrad", "ftrl" (acc is then FTRL's n; z starts at 0) or
    "rowwise_adagrad" (acc holds one value per key, in keys order)."""
    if keys.is_cuda:
        raise ValueError("keys must be host memory (the table is prepared on the host)")
    wt = torch.float16 if wdtype == "f16" else torch.float32
    d, _keep = _desc(dims, wdtype, capacity, acc_init, optimizer)
    h = _vp()
    _check(lib().emb_table_create(ctypes.byref(d), _ptr(keys, torch.int64, "keys"), keys.numel(),
                                  _ptr(values, wt, "values"), _ptr(acc, torch.float32, "acc"), _stream(stream),
                                  ctypes.byref(h)))
    return Table(h.value, dims, wdtype, optimizer)


def emb_table_create_device(dims, wdtype: str, keys: torch.Tensor, values: Optional[torch.Tensor] = None,
                            acc: Optional[torch.Tensor] = None, capacity: int = 0, acc_init: float = 0.0,
                            stream=None, optimizer: str = "adagrad") -> Table:
    """The table of emb_table_create, prepared on the GPU: keys is a CUDA int64 tensor."""
    if not keys.is_cuda:
        raise ValueError("keys must be device memory (emb_table_create takes host keys)")
    wt = torch.float16 if wdtype == "f16" else torch.float32
    d, _keep = _desc(dims, wdtype, capacity, acc_init, optimizer)
    h = _vp()
    _check(lib().emb_table_create_device(ctypes.byref(d), _cuda(keys, torch.int64, "keys"), keys.numel(),
                                         _ptr(values, wt, "values"), _ptr(acc, torch.float32, "acc"),
                                         _stream(stream), ctypes.byref(h)))
    return Table(h.value, dims, wdtype, optimizer)


def emb_table_destroy(table: Table):
    table.close()


def emb_table_get_stats(table: Table) -> dict:
    s = _Stats()
    _check(lib().emb_table_get_stats(table.handle, ctypes.byref(s)))
    return s.as_dict()


def emb_table_plan(dims, wdtype: str, keys, capacity: int = 0, layout: bool = False, optimizer: str = "adagrad"):
    """Host-only validation/statistics; with layout=True also the slot layout (numpy)."""
    keys = np.ascontiguousarray(keys, dtype=np.int64)
    d, _keep = _desc(dims, wdtype, capacity, 0.0, optimizer)
    s = _Stats()
    sk = sr = None
    if layout:
        cap = capacity
        if cap == 0:
            cap = 2
            while cap < 2 * keys.size:
                cap <<= 1
        sk = np.empty(cap, dtype=np.int64)
        sr = np.empty(cap, dtype=np.int64)
    _check(lib().emb_table_plan(ctypes.byref(d), keys.ctypes.data, keys.size, ctypes.byref(s),
                                None if sk is None else sk.ctypes.data, None if sr is None else sr.ctypes.data))
    return s.as_dict(), sk, sr


def emb_lookup_fwd(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    n_bags = offsets.numel() - 1
    if out is None:
        out = torch.empty((n_bags // table.n_slots, sum(table.dims)), dtype=torch.float32, device=offsets.device)
    _check(lib().emb_lookup_fwd(table.handle, _cuda(offsets, torch.int64, "offsets"), n_bags,
                                _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                                _cuda(out, torch.float32, "out"), _stream(stream)))
    return out


def emb_lookup_fwd_record(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str, workspace: torch.Tensor,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """emb_lookup_fwd that also records the resolved (row, bag) pairs into
    `workspace` for emb_bwd_adagrad_recorded."""
    n_bags = offsets.numel() - 1
    if out is None:
        out = torch.empty((n_bags // table.n_slots, sum(table.dims)), dtype=torch.float32, device=offsets.device)
    _check(lib().emb_lookup_fwd_record(table.handle, _cuda(offsets, torch.int64, "offsets"), n_bags,
                                       _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                                       _cuda(out, torch.float32, "out"), _cuda(workspace, None, "workspace"),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def emb_lookup_fwd_dedup(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str, workspace: torch.Tensor,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The forward with a within-batch dedupe: pairs placed and sorted by row,
    each unique row read once; the recorded backward that follows skips its sort."""
    n_bags = offsets.numel() - 1
    if out is None:
        out = torch.empty((n_bags // table.n_slots, sum(table.dims)), dtype=torch.float32, device=offsets.device)
    _check(lib().emb_lookup_fwd_dedup(table.handle, _cuda(offsets, torch.int64, "offsets"), n_bags,
                                      _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                                      _cuda(out, torch.float32, "out"), _cuda(workspace, None, "workspace"),
                                      workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def emb_bwd_adagrad_recorded(table: Table, n_bags: int, nnz: int, pool: str, grad_out: torch.Tensor, lr: float,
                             eps: float, workspace: torch.Tensor, stream=None) -> None:
    _check(lib().emb_bwd_adagrad_recorded(table.handle, n_bags, nnz, _POOL[pool],
                                          _cuda(grad_out, torch.float32, "grad_out"), ctypes.c_float(lr),
                                          ctypes.c_float(eps), _cuda(workspace, None, "workspace"),
                                          workspace.numel() * workspace.element_size(), _stream(stream)))


def emb_bwd_workspace_size(table: Table, n_bags: int, nnz: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().emb_bwd_workspace_size(table.handle, n_bags, nnz, ctypes.byref(b)))
    return b.value


def emb_bwd_adagrad(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str, grad_out: torch.Tensor,
                    lr: float, eps: float, workspace: torch.Tensor, stream=None) -> None:
    _check(lib().emb_bwd_adagrad(table.handle, _cuda(offsets, torch.int64, "offsets"), offsets.numel() - 1,
                                 _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                                 _cuda(grad_out, torch.float32, "grad_out"), ctypes.c_float(lr),
                                 ctypes.c_float(eps), _cuda(workspace, None, "workspace"),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def emb_bwd_adagrad_noalloc(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str,
                            grad_out: torch.Tensor, lr: float, eps: float, stream=None) -> None:
    """emb_bwd_adagrad without a workspace: for callers that cannot allocate
    device memory, it uses the library's fixed EMB_NOALLOC_SCRATCH_BYTES scratch
    (shared by every call on the device: order overlapping calls)."""
    _check(lib().emb_bwd_adagrad_noalloc(table.handle, _cuda(offsets, torch.int64, "offsets"), offsets.numel() - 1,
                                         _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                                         _cuda(grad_out, torch.float32, "grad_out"), ctypes.c_float(lr),
                                         ctypes.c_float(eps), _stream(stream)))


def _ftrl(alpha, beta, lambda1, lambda2):
    return _Ftrl(float(alpha), float(beta), float(lambda1), float(lambda2))


def emb_bwd_ftrl(table: Table, offsets: torch.Tensor, keys: torch.Tensor, pool: str, grad_out: torch.Tensor,
                 alpha: float, beta: float, lambda1: float, lambda2: float, workspace: torch.Tensor,
                 stream=None) -> None:
    """The backward with the FTRL-Proximal update (tables created with optimizer="ftrl")."""
    p = _ftrl(alpha, beta, lambda1, lambda2)
    _check(lib().emb_bwd_ftrl(table.handle, _cuda(offsets, torch.int64, "offsets"), offsets.numel() - 1,
                              _cuda(keys, torch.int64, "keys"), keys.numel(), _POOL[pool],
                              _cuda(grad_out, torch.float32, "grad_out"), ctypes.byref(p),
                              _cuda(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                              _stream(stream)))


def emb_bwd_ftrl_recorded(table: Table, n_bags: int, nnz: int, pool: str, grad_out: torch.Tensor, alpha: float,
                          beta: float, lambda1: float, lambda2: float, workspace: torch.Tensor, stream=None) -> None:
    p = _ftrl(alpha, beta, lambda1, lambda2)
    _check(lib().emb_bwd_ftrl_recorded(table.handle, n_bags, nnz, _POOL[pool],
                                       _cuda(grad_out, torch.float32, "grad_out"), ctypes.byref(p),
                                       _cuda(workspace, None, "workspace"),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def emb_table_export_z(table: Table, z_out: torch.Tensor, stream=None) -> None:
    _check(lib().emb_table_export_z(table.handle, _ptr(z_out, torch.float32, "z_out"), _stream(stream)))


def emb_table_import_z(table: Table, z_in: torch.Tensor, stream=None) -> None:
    _check(lib().emb_table_import_z(table.handle, _ptr(z_in, torch.float32, "z_in"), _stream(stream)))


def emb_bwd_phase_events(table: Table, events) -> None:
    """Register torch.cuda.Event objects (timing enabled) that each later
    emb_bwd_adagrad records after its expand, sort, reduce and fixup phases."""
    if any(not e.cuda_event for e in events):
        raise ValueError("record each event once (torch creates CUDA events lazily) before registering it")
    arr = (_vp * max(1, len(events)))(*[_vp(e.cuda_event) for e in events])
    _check(lib().emb_bwd_phase_events(table.handle, arr, len(events)))


def emb_bwd_unique_keys(table: Table, workspace: torch.Tensor, keys_out: torch.Tensor, n_unique_out: torch.Tensor,
                        stream=None) -> None:
    _check(lib().emb_bwd_unique_keys(table.handle, _cuda(workspace, None, "workspace"),
                                     workspace.numel() * workspace.element_size(),
                                     _cuda(keys_out, torch.int64, "keys_out"),
                                     _cuda(n_unique_out, torch.int64, "n_unique_out"), _stream(stream)))


def emb_resolve(table: Table, keys: torch.Tensor, slot_out: Optional[torch.Tensor] = None,
                row_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    if slot_out is None:
        slot_out = torch.empty_like(keys)
    if row_out is None:
        row_out = torch.empty_like(keys)
    _check(lib().emb_resolve(table.handle, _cuda(keys, torch.int64, "keys"), keys.numel(),
                             _cuda(slot_out, torch.int64, "slot_out"), _cuda(row_out, torch.int64, "row_out"),
                             _stream(stream)))
    return slot_out, row_out


def emb_table_export(table: Table, keys_out: Optional[torch.Tensor], values_out: Optional[torch.Tensor],
                     acc_out: Optional[torch.Tensor], stream=None) -> None:
    wt = torch.float16 if table.wdtype == "f16" else torch.float32
    _check(lib().emb_table_export(table.handle, _ptr(keys_out, torch.int64, "keys_out"),
                                  _ptr(values_out, wt, "values_out"), _ptr(acc_out, torch.float32, "acc_out"),
                                  _stream(stream)))


def emb_table_export_rows(table: Table, rows: torch.Tensor, values_out: Optional[torch.Tensor] = None,
                          acc_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Weights/accumulators of keys-array rows as [n, max_dim] device tensors (zero padded);
    a row-wise Adagrad table's accumulators come as [n]."""
    n, md = rows.numel(), max(table.dims)
    wt = torch.float16 if table.wdtype == "f16" else torch.float32
    if values_out is None:
        values_out = torch.empty((n, md), dtype=wt, device=rows.device)
    if acc_out is None:
        shape = (n,) if table.optimizer == "rowwise_adagrad" else (n, md)
        acc_out = torch.empty(shape, dtype=torch.float32, device=rows.device)
    _check(lib().emb_table_export_rows(table.handle, _cuda(rows, torch.int64, "rows"), n,
                                       _cuda(values_out, wt, "values_out"), _cuda(acc_out, torch.float32, "acc_out"),
                                       _stream(stream)))
    return values_out, acc_out


def emb_table_slots(table: Table, slot_key_out: Optional[torch.Tensor], slot_row_out: Optional[torch.Tensor],
                    stream=None) -> None:
    _check(lib().emb_table_slots(table.handle, _ptr(slot_key_out, torch.int64, "slot_key_out"),
                                 _ptr(slot_row_out, torch.int64, "slot_row_out"), _stream(stream)))


def emb_check_device_flag(table: Table, stream=None) -> int:
    """Synchronise, read and clear the device flag word; returns the flag bits (0 = clean)."""
    f = ctypes.c_uint32()
    rc = lib().emb_check_device_flag(table.handle, _stream(stream), ctypes.byref(f))
    if rc not in (EMB_OK, 8):
        raise EmbError(rc, emb_last_error())
    return f.value


def emb_debug_fail_device_alloc(after: int) -> None:
    """Fault injection: the next `after` device allocations succeed, later ones fail (negative: never)."""
    _check(lib().emb_debug_fail_device_alloc(int(after)))


def emb_debug_live_device_allocs() -> int:
    return int(lib().emb_debug_live_device_allocs())


def emb_debug_set_probe_bound(table: Table, bound: int) -> None:
    """Fault injection: lower the table's probe bound (as a corrupted table would)."""
    _check(lib().emb_debug_set_probe_bound(table.handle, int(bound)))
    table.stats = emb_table_get_stats(table)


def emb_debug_lose_op_wait(role: Optional[str], step: int = 0) -> None:
    """From now on the wait of this role ("load", "product", "scales", "other") at this step of a tiled
    emb_fp8_matmul counts as run out (None: none, the default)."""
    _check(lib().emb_debug_lose_op_wait(-1 if role is None else ("load", "product", "scales", "other").index(role), int(step)))


def emb_debug_fp8_matmul_plan(m: int, n: int, k: int) -> Tuple[int, int, int, int]:
    """(columns of a tile or 0, tiles, blocks, steps of a block or 0 for whole tiles) of an emb_fp8_matmul."""
    plan = (_i64 * 4)()
    _check(lib().emb_debug_fp8_matmul_plan(m, n, k, plan))
    return tuple(plan)


class Pipeline:
    """emb_pipeline: overlaps the next batch's host-to-device copy (and the
    pooled output's copy back) with the current step.  Host tensors should be
    pinned.  Per batch: submit -> forward -> backward_adagrad/ftrl (or
    release) -> wait; submit may run up to depth - 1 batches ahead."""

    def __init__(self, table: Table, max_bags: int, max_nnz: int, depth: int = 2, upload_grad: bool = False,
                 stream=None):
        self.table = table
        self._keep = []
        h = _vp()
        _check(lib().emb_pipeline_create(table.handle, int(max_bags), int(max_nnz), int(depth), int(upload_grad),
                                         _stream(stream), ctypes.byref(h)))
        self._h = h

    def submit(self, offsets_h: torch.Tensor, keys_h: torch.Tensor, grad_h: Optional[torch.Tensor] = None) -> int:
        for t, n in ((offsets_h, "offsets"), (keys_h, "keys"), (grad_h, "grad_out")):
            if t is not None and t.is_cuda:
                raise ValueError(f"{n} must be host memory")
        tk = ctypes.c_int64()
        _check(lib().emb_pipeline_submit(self._h, _ptr(offsets_h, torch.int64, "offsets"), offsets_h.numel() - 1,
                                         _ptr(keys_h, torch.int64, "keys"), keys_h.numel(),
                                         _ptr(grad_h, torch.float32, "grad_out"), ctypes.byref(tk)))
        self._keep.append((offsets_h, keys_h, grad_h))   # host memory must outlive the copy
        self._keep = self._keep[-8:]
        return tk.value

    def forward(self, ticket: int, pool: str, out: Optional[torch.Tensor] = None,
                out_h: Optional[torch.Tensor] = None) -> int:
        """Returns the device address of the pooled output (out, or the set's own buffer)."""
        used = _vp()
        _check(lib().emb_pipeline_forward(self._h, int(ticket), _POOL[pool], _ptr(out, torch.float32, "out"),
                                          _ptr(out_h, torch.float32, "out_h"), ctypes.byref(used)))
        return used.value

    def backward_adagrad(self, ticket: int, lr: float, eps: float, grad_out: Optional[torch.Tensor] = None):
        _check(lib().emb_pipeline_backward_adagrad(self._h, int(ticket), _ptr(grad_out, torch.float32, "grad_out"),
                                                   ctypes.c_float(lr), ctypes.c_float(eps)))

    def backward_ftrl(self, ticket: int, alpha, beta, lambda1, lambda2, grad_out: Optional[torch.Tensor] = None):
        p = _ftrl(alpha, beta, lambda1, lambda2)
        _check(lib().emb_pipeline_backward_ftrl(self._h, int(ticket), _ptr(grad_out, torch.float32, "grad_out"),
                                                ctypes.byref(p)))

    def release(self, ticket: int):
        _check(lib().emb_pipeline_release(self._h, int(ticket)))

    def wait(self, ticket: int):
        _check(lib().emb_pipeline_wait(self._h, int(ticket)))

    def close(self):
        if self._h:
            lib().emb_pipeline_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ the dense tower's operators
#
# These run as often as a layer does, some for microseconds: one condition per
# tensor finds the usual case, and only a call that fails it is looked at again
# for its message.  The current stream is read as its raw handle.  A kernel runs
# on the current device, so every tensor of a call has to be there.

_F8, _F32, _U8 = torch.float8_e4m3fn, torch.float32, torch.uint8
_new = torch.empty


_current_device = getattr(torch._C, "_cuda_getDevice", None)   # absent where torch has no CUDA


def _launch_device(t: torch.Tensor, name: str) -> int:
    """The current device, which has to be this tensor's."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _raw_stream(stream, dev: Optional[int] = None) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(_current_device() if dev is None else dev)
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    if dev is not None and stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _empty(stream, like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """A tensor for use on `stream`: torch's allocator then reuses its memory in that stream's order."""
    if stream is None:
        return _new(shape, dtype=dtype, device=like.device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return _new(shape, dtype=dtype, device=like.device)


def _dense(t: Optional[torch.Tensor], dtype, name: str, dev: int) -> Optional[int]:
    """The address of a contiguous tensor of this type on the launch's device."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others are on cuda:{dev}")
    raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _ftype(dtype, name: str) -> int:
    code = _FTYPE.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _row_stride(t: torch.Tensor, name: str, dev: int) -> int:
    """Checks a matrix with neighbouring columns on the launch's device; returns the distance of its rows."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{dev}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if rows > 1 else max(ld, cols)


def _code_stride(t: torch.Tensor, name: str, dev: int) -> int:
    if t.dtype is not _F8:
        raise TypeError(f"{name} must be {_F8}, got {t.dtype}")
    ld = _row_stride(t, name, dev)
    return -(-ld // 16) * 16 if ld % 16 and (t.shape[0] <= 1 or t.shape[1] == 0) else ld


def emb_fp8_quantize(x: torch.Tensor, block_rows: int = 1, transpose: bool = False, stream=None):
    """e4m3 codes and scales of x[rows, cols] (float32, bfloat16 or float16; rows
    may be strided): (q, s), with q[rows, cols] and s[ceil(cols/128),
    ceil(rows/block_rows)]; with transpose=True (q, s, qt, st), the codes of
    x.T in blocks along x's rows as well, from the same pass."""
    dev = _launch_device(x, "x")
    ldx = _row_stride(x, "x", dev)
    if block_rows not in (1, EMB_FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    r, c = x.shape
    rb, cb, ldq, ldqt = (r + 127) >> 7, (c + 127) >> 7, (c + 15) & ~15, (r + 15) & ~15
    rows, cols = (r, c) if block_rows == 1 else (rb, cb)
    q, s = _empty(stream, x, (r, ldq), _F8), _empty(stream, x, (cb, rows), _F32)
    if not transpose:
        _check(lib().emb_fp8_quantize(x.data_ptr(), _ftype(x.dtype, "x"), r, c, ldx, block_rows, q.data_ptr(), ldq, s.data_ptr(),
                                      None, 0, None, _raw_stream(stream, dev)))
        return (q if ldq == c else q[:, :c]), s
    qt, st = _empty(stream, x, (c, ldqt), _F8), _empty(stream, x, (rb, cols), _F32)
    _check(lib().emb_fp8_quantize(x.data_ptr(), _ftype(x.dtype, "x"), r, c, ldx, block_rows, q.data_ptr(), ldq, s.data_ptr(),
                                  qt.data_ptr(), ldqt, st.data_ptr(), _raw_stream(stream, dev)))
    return (q if ldq == c else q[:, :c]), s, (qt if ldqt == r else qt[:, :r]), st


def emb_fp8_matmul_workspace_size(m: int, n: int, k: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().emb_fp8_matmul_workspace_size(m, n, k, ctypes.byref(b)))
    return b.value


def _block_rows(s: torch.Tensor, rows: int, k_blocks: int, name: str) -> int:
    shape = s.shape
    if shape == (k_blocks, rows):
        return 1
    if shape == (k_blocks, (rows + 127) >> 7):
        return EMB_FP8_BLOCK
    raise ValueError(f"{name} must be [ceil(k/128), rows] or [ceil(k/128), ceil(rows/128)], got {tuple(shape)}")


def emb_fp8_matmul(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                   out_dtype: torch.dtype = torch.bfloat16, bias: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """a[m, k] @ b[n, k].T of codes and scales from emb_fp8_quantize (+ bias[n]).
    workspace: emb_fp8_matmul_workspace_size bytes that the caller keeps; made
    for the call if None."""
    dev = _launch_device(a, "a")
    lda, ldb = _code_stride(a, "a", dev), _code_stride(b, "b", dev)
    (m, k), (n, kb) = a.shape, b.shape
    if kb != k:
        raise ValueError(f"a and b must have the same columns, got {k} and {kb}")
    if bias is not None and bias.numel() != n:
        raise ValueError(f"bias must have {n} elements")
    blocks = (k + 127) >> 7
    a_rows, b_rows = _block_rows(sa, m, blocks, "sa"), _block_rows(sb, n, blocks, "sb")
    if out is None:
        out, ldo = _empty(stream, a, (m, n), out_dtype), n
    else:
        if out.shape != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
        ldo = _row_stride(out, "out", dev)
    wp, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = emb_fp8_matmul_workspace_size(m, n, k)
        if ws_bytes:
            workspace = _empty(stream, a, ws_bytes, _U8)
            wp = workspace.data_ptr()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
    else:
        wp, ws_bytes = workspace.data_ptr(), workspace.nbytes
    _check(lib().emb_fp8_matmul(a.data_ptr(), lda, _dense(sa, _F32, "sa", dev), a_rows, b.data_ptr(), ldb, _dense(sb, _F32, "sb", dev),
                                b_rows, m, n, k, None if bias is None else _dense(bias, _F32, "bias", dev),
                                out.data_ptr(), _ftype(out.dtype, "out"), ldo, wp, ws_bytes, _raw_stream(stream, dev)))
    return out


def _norm_gate(x: torch.Tensor, block_dtype: torch.dtype, gate, norm: str, act: str, eps: float,
               res_scale: float) -> _NormGate:
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x, f, y, h and their gradients must be matrices of one shape")
    r, d = shape
    kind = 0
    if gate is not None:
        gs = gate.shape
        kind = 1 if gs == shape else 2 if gs == (r, 1) else 3 if gs == (d,) else 0
        if kind == 0:
            raise ValueError(f"gate must be [{r}, {d}], [{r}, 1] or [{d}], got {tuple(gs)}")
        if gate.dtype is not (_F32 if kind == 3 else block_dtype):
            raise TypeError("a gate per element or row has f's type, a gate per channel is float32")
    return _NormGate(r, d, _ftype(x.dtype, "x"), _ftype(block_dtype, "f"), _NORM[norm], kind, _ACT[act], eps, res_scale)


def _vector(t: Optional[torch.Tensor], dim: int, name: str, dev: int):
    if t is None:
        return None
    if t.numel() != dim:
        raise ValueError(f"{name} must have {dim} elements")
    return _dense(t, _F32, name, dev)


def _same(t: Optional[torch.Tensor], shape, dtype, name: str, dev: int):
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return _dense(t, dtype, name, dev)


def emb_norm_gate_fwd(x: torch.Tensor, f: Optional[torch.Tensor], gate: Optional[torch.Tensor] = None, *,
                      w_post: Optional[torch.Tensor] = None, b_post: Optional[torch.Tensor] = None,
                      w_pre: Optional[torch.Tensor] = None, b_pre: Optional[torch.Tensor] = None, norm: str = "rms",
                      act: str = "sigmoid", eps: float = 1e-6, res_scale: float = 1.0, pre: bool = True,
                      stats: bool = True, block_dtype: Optional[torch.dtype] = None, stream=None):
    """y = res_scale * x + act(gate) * (norm(f) * w_post + b_post) and h = norm(y) *
    w_pre + b_pre: (y, h, stats).  f=None: y is x (None is returned for it).
    pre=False: no norm follows (h is None).  gate: [rows, dim] or [rows, 1] in f's
    type, or float32 [dim].  stats: float32 [rows, 4] for the backward, or None
    with stats=False.  block_dtype: h's type where f is None (default x's)."""
    shape, st_type = x.shape, x.dtype
    block_dtype = f.dtype if f is not None else block_dtype or st_type
    d = _norm_gate(x, block_dtype, gate, norm, act, eps, res_scale)
    dim = d.dim
    dev = _launch_device(x, "x")
    xp, fp = _dense(x, st_type, "x", dev), _same(f, shape, block_dtype, "f", dev)
    gp = None if gate is None else _dense(gate, gate.dtype, "gate", dev)
    wp = None if w_post is None else _vector(w_post, dim, "w_post", dev)
    bp = None if b_post is None else _vector(b_post, dim, "b_post", dev)
    wq = None if w_pre is None else _vector(w_pre, dim, "w_pre", dev)
    bq = None if b_pre is None else _vector(b_pre, dim, "b_pre", dev)
    y = h = st = yp = hp = sp = None
    if f is not None:
        y = _empty(stream, x, shape, st_type)
        yp = y.data_ptr()
    if pre:
        h = _empty(stream, x, shape, block_dtype)
        hp = h.data_ptr()
    if stats:
        st = _empty(stream, x, (shape[0], 4), _F32)
        sp = st.data_ptr()
    _check(lib().emb_norm_gate_fwd(ctypes.byref(d), xp, fp, gp, wp, bp, wq, bq, yp, hp, sp, _raw_stream(stream, dev)))
    return y, h, st


def emb_norm_gate_bwd_workspace_size(rows: int, dim: int) -> int:
    b = ctypes.c_size_t()
    d = _NormGate(rows, dim, 0, 0, 0, 0, 0, 1.0, 1.0)
    _check(lib().emb_norm_gate_bwd_workspace_size(ctypes.byref(d), ctypes.byref(b)))
    return b.value


def emb_norm_gate_bwd(dy: Optional[torch.Tensor], dh: Optional[torch.Tensor], y: torch.Tensor,
                      f: Optional[torch.Tensor], gate: Optional[torch.Tensor], stats: torch.Tensor, *,
                      w_post: Optional[torch.Tensor] = None, b_post: Optional[torch.Tensor] = None,
                      w_pre: Optional[torch.Tensor] = None, b_pre: Optional[torch.Tensor] = None, norm: str = "rms",
                      act: str = "sigmoid", eps: float = 1e-6, res_scale: float = 1.0,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of emb_norm_gate_fwd from dy (of y, along the residual stream) and
    dh (of h), either None if absent: {"dx", "df", "dgate", "dw_post", "db_post",
    "dw_pre", "db_pre"}, None for those of an input that is absent.  y: the
    forward's y (its x where f is None)."""
    if f is None and dh is None:
        raise ValueError("f and dh are both None")
    shape, st_type = y.shape, y.dtype
    bt = f.dtype if f is not None else dh.dtype
    d = _norm_gate(y, bt, gate, norm, act, eps, res_scale)
    r, dim = shape
    f32 = _F32
    dev = _launch_device(y, "y")
    ins = (_same(dy, shape, st_type, "dy", dev), _same(dh, shape, bt, "dh", dev), _dense(y, st_type, "y", dev),
           _same(f, shape, bt, "f", dev), None if gate is None else _dense(gate, gate.dtype, "gate", dev),
           _same(stats, (r, 4), f32, "stats", dev), _vector(w_post, dim, "w_post", dev), _vector(b_post, dim, "b_post", dev),
           _vector(w_pre, dim, "w_pre", dev))
    _vector(b_pre, dim, "b_pre", dev)
    out = {"dx": _empty(stream, y, shape, st_type), "df": None if f is None else _empty(stream, y, shape, bt),
           "dgate": None if gate is None else _empty(stream, y, gate.shape, gate.dtype)}
    for name, v in (("dw_post", w_post), ("db_post", b_post), ("dw_pre", w_pre), ("db_pre", b_pre)):
        out[name] = None if v is None else _empty(stream, y, (dim,), f32)
    if workspace is None:
        workspace = _empty(stream, y, emb_norm_gate_bwd_workspace_size(r, dim), torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
    _check(lib().emb_norm_gate_bwd(ctypes.byref(d), *ins, *[None if v is None else v.data_ptr() for v in out.values()],
                                   workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev)))
    return out


def emb_adamw_step(tensors, grads, params: _AdamwParams, stream=None, dev: Optional[int] = None) -> None:
    """One step over a ctypes array of _AdamwTensor and the address of an array of gradient pointers (AdamW makes both)."""
    _check(lib().emb_adamw_step(tensors, grads, len(tensors), ctypes.byref(params), _raw_stream(stream, dev)))


_dtype_of = operator.attrgetter("dtype")


class AdamW:
    """AdamW over a list of tensors, one launch a step (per 380 tensors).  params:
    contiguous CUDA tensors (float32, bfloat16 or float16), updated in place.
    copies: for each float32 parameter a bfloat16 or float16 tensor (or None) that
    receives the updated weights, as the "f16m" tables keep them.  state "f32", or
    "q8": m and sqrt(v) as e4m3 codes with a scale per 256 elements,
    stochastically rounded from `seed`.  The states live in `arena` (m, v, m_scale,
    v_scale: all tensors one after another, each from a multiple of 256 elements),
    which with `step_count` is the checkpoint; load_state takes per-tensor lists.
    A parameter, copy or state that is given other storage (p.data = ..., half(),
    set_()) is found by its address at the next step and described anew (the old
    storage is held until then); its size and device must stay.  A CUDA
    graph replays the step number, the rates and the addresses it was captured with."""

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: float = 0.01, state: str = "f32", seed: int = 0,
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None):
        self.params = list(params)
        if not self.params:
            raise ValueError("params is empty")
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, betas, eps, weight_decay, seed
        self.state, self.step_count, self.device = state, 0, self.params[0].device
        self._copies = list(copies) if copies is not None else [None] * len(self.params)
        if len(self._copies) != len(self.params):
            raise ValueError("copies must have one entry per parameter")
        self._state = _ADAM_STATE[state]
        q8 = self._state == 1
        block = EMB_ADAM_BLOCK
        self._n = [p.numel() for p in self.params]
        self._dev = self.params[0].get_device()
        if self._dev < 0:
            raise ValueError("param must be a contiguous CUDA tensor")
        self._devs = [self._dev] * len(self.params)
        self._at = [0]
        for n in self._n:
            self._at.append(self._at[-1] + -(-n // block) * block)
        total = self._at[-1]
        st = torch.float8_e4m3fn if q8 else torch.float32
        zeros = lambda n, t: torch.zeros(n, dtype=torch.uint8 if t.itemsize == 1 else t, device=self.device).view(t)  # noqa: E731
        self.arena = {"m": zeros(total, st), "v": zeros(total, st),
                      "m_scale": zeros(total // block, torch.float32) if q8 else None,
                      "v_scale": zeros(total // block, torch.float32) if q8 else None}
        self._total, self._state_type = total, st
        self._params = self._hyper = None
        self._given = [c for c in self._copies if c is not None]
        self._states = [k for k, v in self.arena.items() if v is not None]
        self._grad_dtypes = [p.dtype for p in self.params]
        self._bind()

    def _used(self):
        """Every tensor whose address a step uses, the gradients apart."""
        return [*self.params, *self._given, *map(self.arena.__getitem__, self._states)]

    def _bind(self) -> None:
        """Describes parameters, copies and states to the library, as they are now.  The
        addresses are kept for the steps, and with them an alias of each tensor: as
        long as it lives no other tensor can come to lie there, so an address that is
        still the same is still the same memory."""
        q8, block = self._state == 1, EMB_ADAM_BLOCK
        base, size = {}, {"m": self._total, "v": self._total, "m_scale": self._total // block, "v_scale": self._total // block}
        for k, v in self.arena.items():
            if (v is None) != (k.endswith("scale") and not q8) or (v is not None and v.numel() != size[k]):
                raise ValueError(f"arena {k} does not match the state kind {self.state} and {self._total} elements")
            base[k] = 0 if v is None else _dense(v, torch.float32 if k.endswith("scale") else self._state_type, f"arena {k}", self._dev)
        if len(self.params) != len(self._n):
            raise ValueError("the number of parameters has changed")
        tensors = (_AdamwTensor * len(self.params))()
        st = self._state_type.itemsize
        for i, (p, c) in enumerate(zip(self.params, self._copies)):
            if p.numel() != self._n[i]:
                raise ValueError(f"parameter {i} had {self._n[i]} elements and has {p.numel()}")
            if c is not None and c.numel() != p.numel():
                raise ValueError("a copy must have its parameter's size")
            at = self._at[i]
            tensors[i] = _AdamwTensor(_dense(p, p.dtype, "param", self._dev), None if c is None else _dense(c, c.dtype, "copy", self._dev),
                                      base["m"] + at * st, base["v"] + at * st,
                                      base["m_scale"] + at // block * 4 if q8 else None,
                                      base["v_scale"] + at // block * 4 if q8 else None, self._n[i], at,
                                      _ftype(p.dtype, "param"), _ftype(self._grad_dtypes[i], "grad"),
                                      0 if c is None else _ftype(c.dtype, "copy"))
        used = self._used()
        for t in used:
            if (t.storage_offset() + t.numel()) * t.itemsize > t.untyped_storage().nbytes():
                raise ValueError("a parameter, copy or state has lost its storage")
        self._tensors, self._addresses, self._aliases = tensors, list(map(torch.Tensor.data_ptr, used)), [t.detach() for t in used]

    def load_state(self, step: int, m, v, m_scale=None, v_scale=None) -> None:
        """Sets the states from one tensor per parameter (the layout of `arena`, without its padding): all of them, or none if one does not fit."""
        to, of = [], []
        for key, parts in (("m", m), ("v", v), ("m_scale", m_scale), ("v_scale", v_scale)):
            whole = self.arena[key]
            if (parts is None) != (whole is None):
                raise ValueError(f"{key} does not match the state kind {self.state}")
            if parts is None:
                continue
            parts = list(parts)
            if len(parts) != len(self.params):
                raise ValueError(f"{key}: expected {len(self.params)} tensors")
            for part, at, n in zip(parts, self._at, self._n):
                if key.endswith("scale"):
                    at, n = at // EMB_ADAM_BLOCK, -(-n // EMB_ADAM_BLOCK)
                if part.numel() != n or part.dtype != whole.dtype:
                    raise ValueError(f"{key}: expected {n} elements of {whole.dtype}")
                to.append(whole[at:at + n].view(torch.uint8))
                of.append(part.reshape(-1).view(torch.uint8))
        torch._foreach_copy_(to, of)
        self.step_count = int(step)

    def step(self, grads: Sequence[torch.Tensor], grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
        """One step.  grads: one contiguous tensor per parameter (float32, bfloat16 or
        float16); grad_scale: device float32 scalar that multiplies them."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} gradients are needed, got {len(grads)}")
        T = torch.Tensor
        if list(map(T.numel, grads)) != self._n or not all(map(T.is_contiguous, grads)) or list(map(T.get_device, grads)) != self._devs:
            raise ValueError(f"each gradient must be a contiguous tensor on cuda:{self._dev} of its parameter's size")
        if _current_device() != self._dev:
            raise ValueError(f"the parameters are on cuda:{self._dev}, the current device is cuda:{_current_device()}")
        if list(map(T.data_ptr, self._used())) != self._addresses:
            self._bind()                    # a parameter, copy or state has moved
        dtypes = list(map(_dtype_of, grads))
        if dtypes != self._grad_dtypes:
            kinds = [_ftype(g, "grad") for g in dtypes]
            for t, kind in zip(self._tensors, kinds):
                t.grad_t = kind
            self._grad_dtypes = dtypes
        ptrs = array.array("Q", map(T.data_ptr, grads))
        hyper = (self.lr, *self.betas, self.eps, self.weight_decay, self.seed)
        if hyper != self._hyper:
            self._params = _AdamwParams(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, 0, self._state,
                                        self.seed & 0xFFFFFFFF, None)
            self._hyper = hyper
        if grad_scale is not None and grad_scale.numel() != 1:
            raise ValueError(f"grad_scale must have one element, got {grad_scale.numel()}")
        p = self._params
        p.step, p.grad_scale = self.step_count + 1, _dense(grad_scale, _F32, "grad_scale", self._dev)
        emb_adamw_step(self._tensors, ptrs.buffer_info()[0], p, stream, self._dev)
        self.step_count += 1


def emb_check_op_flag(stream=None) -> int:
    """Synchronise, read and clear the dense operators' flag word (0 = clean)."""
    f = ctypes.c_uint32()
    rc = lib().emb_check_op_flag(_raw_stream(stream), ctypes.byref(f))
    if rc not in (EMB_OK, 8):
        raise EmbError(rc, emb_last_error())
    return f.value
