"""ctypes binding of libbitsmoe (include/bitsmoe.h), same names as the C calls.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch tensors on the GPU (device pointers are taken with
``data_ptr()``); the stream defaults to torch's current stream.  If the shared
library is missing the import of any call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import numpy as np
import torch

# BITSMOE_CHECKED=1 selects the bounds-checked build (libbitsmoe_checked.so): every
# computed index of the expert kernels is checked, a violation sets ST_BOUNDS.
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libbitsmoe_checked.so" if os.environ.get("BITSMOE_CHECKED") == "1" else "libbitsmoe.so")

OK, EINVAL, EWIDTH, ESIZE, ECUDA, EFORMAT, ENOMEM = 0, -1, -2, -3, -4, -5, -6
ST_NONFINITE, ST_BADSCALE, ST_BADEXPERT, ST_TIMEOUT, ST_PLANMISMATCH, ST_BOUNDS = 1, 2, 4, 8, 16, 32
ST_NOCONVERGE = 64
ST_BADGROUP = 128
F32, F16, BF16 = 0, 1, 2  # element types
SCORING = {"softmax": 0, "sigmoid": 1}

# Every symbol include/bitsmoe.h declares.
EXPORTS = (
    "bitsmoe_pack_plan", "bitsmoe_plan_from_header", "bitsmoe_plan_free", "bitsmoe_plan_blob_bytes",
    "bitsmoe_plan_header_bytes", "bitsmoe_plan_get_dims", "bitsmoe_plan_write_header", "bitsmoe_compute_scales",
    "bitsmoe_pack", "bitsmoe_unpack_q", "bitsmoe_shared_proj", "bitsmoe_expert_workspace_bytes",
    "bitsmoe_expert_forward", "bitsmoe_layer_workspace_bytes", "bitsmoe_layer_launches", "bitsmoe_layer_forward",
    "bitsmoe_layer_forward_chained", "bitsmoe_layer_forward_t1_noalloc", "bitsmoe_ffn_down_workspace_bytes",
    "bitsmoe_ffn_down_launches", "bitsmoe_ffn_down", "bitsmoe_ffn_workspace_bytes", "bitsmoe_ffn_launches",
    "bitsmoe_ffn_forward", "bitsmoe_ssd_workspace_bytes", "bitsmoe_ssd_decompose", "bitsmoe_assign_widths",
    "bitsmoe_fqcm_eps", "bitsmoe_fqcm_beta", "bitsmoe_allocate_widths",
    "bitsmoe_norm_residual", "bitsmoe_topk_route_workspace_bytes", "bitsmoe_topk_route", "bitsmoe_q4_bytes",
    "bitsmoe_q4_pack", "bitsmoe_q4_unpack", "bitsmoe_ffn_down_q4_workspace_bytes", "bitsmoe_ffn_down_q4_launches",
    "bitsmoe_ffn_down_q4", "bitsmoe_grouped_matmul", "bitsmoe_dense_ffn_workspace_bytes", "bitsmoe_dense_ffn_forward",
    "bitsmoe_read_status", "bitsmoe_strerror", "bitsmoe_version",
)


class BitsMoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("top_k", ctypes.c_int32)]


class FfnDims(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32)]


class ProjIO(ctypes.Structure):
    _fields_ = [("plan", ctypes.c_void_p), ("blob", ctypes.c_void_p), ("phi_t", ctypes.c_void_p),
                ("Z", ctypes.c_void_p), ("Y_experts", ctypes.c_void_p), ("Y_sum", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with mixed_precision_decode_b200.build.build()"
                               f" (checked=True for the bounds-checked build)")
        L = ctypes.CDLL(_LIB_PATH)
        vp, u64, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32
        sig = {
            "bitsmoe_pack_plan": ([ctypes.POINTER(Dims), vp, ctypes.POINTER(vp)], ctypes.c_int),
            "bitsmoe_plan_from_header": ([vp, u64, i32, i32, ctypes.POINTER(vp)], ctypes.c_int),
            "bitsmoe_plan_free": ([vp], None),
            "bitsmoe_plan_blob_bytes": ([vp], u64),
            "bitsmoe_plan_header_bytes": ([vp], u64),
            "bitsmoe_plan_get_dims": ([vp, ctypes.POINTER(Dims)], ctypes.c_int),
            "bitsmoe_plan_write_header": ([vp, vp, u64], ctypes.c_int),
            "bitsmoe_compute_scales": ([vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "bitsmoe_pack": ([vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "bitsmoe_unpack_q": ([vp, vp, vp, vp], ctypes.c_int),
            "bitsmoe_shared_proj": ([vp, vp, vp, i32, i32, i32, vp], ctypes.c_int),
            "bitsmoe_expert_workspace_bytes": ([vp, i32], u64),
            "bitsmoe_expert_forward": ([vp, vp, vp, vp, vp, i32, vp, vp, vp, u64, vp, vp], ctypes.c_int),
            "bitsmoe_layer_workspace_bytes": ([vp, vp, i32], u64),
            "bitsmoe_layer_launches": ([vp, vp, i32], ctypes.c_int),
            "bitsmoe_layer_forward": ([ctypes.POINTER(ProjIO), ctypes.POINTER(ProjIO), vp, vp, vp, i32, vp, u64,
                                       vp, vp], ctypes.c_int),
            "bitsmoe_layer_forward_chained": ([ctypes.POINTER(ProjIO), ctypes.POINTER(ProjIO), vp, vp, vp, i32, vp,
                                               u64, vp, vp, vp, vp], ctypes.c_int),
            "bitsmoe_layer_forward_t1_noalloc": ([ctypes.POINTER(ProjIO), ctypes.POINTER(ProjIO), vp, vp, vp, vp,
                                                  vp], ctypes.c_int),
            "bitsmoe_ffn_down_workspace_bytes": ([ctypes.POINTER(FfnDims), i32], u64),
            "bitsmoe_ffn_down_launches": ([ctypes.POINTER(FfnDims), i32], ctypes.c_int),
            "bitsmoe_ffn_down": ([ctypes.POINTER(FfnDims), vp, vp, vp, vp, vp, i32, vp, vp, u64, vp, vp],
                                 ctypes.c_int),
            "bitsmoe_ffn_workspace_bytes": ([vp, vp, i32], u64),
            "bitsmoe_ffn_launches": ([vp, vp, i32], ctypes.c_int),
            "bitsmoe_ffn_forward": ([ctypes.POINTER(ProjIO), ctypes.POINTER(ProjIO), vp, vp, vp, vp, i32, vp, vp, u64,
                                     vp, vp], ctypes.c_int),
            "bitsmoe_ssd_workspace_bytes": ([i32, i32, i32, i32], u64),
            "bitsmoe_ssd_decompose": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, u64, vp, vp], ctypes.c_int),
            "bitsmoe_assign_widths": ([vp, i32, i32, vp, vp, i32, vp], ctypes.c_int),
            "bitsmoe_fqcm_eps": ([vp, i32, i32, i32, vp], ctypes.c_int),
            "bitsmoe_fqcm_beta": ([vp, vp, vp, i32, i32, i32, i32, vp], ctypes.c_int),
            "bitsmoe_allocate_widths": ([vp, vp, vp, i32, i32, i32, u64, vp, vp], ctypes.c_int),
            "bitsmoe_norm_residual": ([vp, vp], ctypes.c_int),
            "bitsmoe_topk_route_workspace_bytes": ([i32, i32, i32], u64),
            "bitsmoe_topk_route": ([vp, vp], ctypes.c_int),
            "bitsmoe_q4_bytes": ([i32, i32, i32, i32], u64),
            "bitsmoe_q4_pack": ([vp, i32, i32, i32, i32, i32, vp, vp, vp], ctypes.c_int),
            "bitsmoe_q4_unpack": ([vp, i32, i32, i32, i32, vp, vp], ctypes.c_int),
            "bitsmoe_ffn_down_q4_workspace_bytes": ([ctypes.POINTER(FfnDims), i32, i32], u64),
            "bitsmoe_ffn_down_q4_launches": ([ctypes.POINTER(FfnDims), i32, i32], ctypes.c_int),
            "bitsmoe_ffn_down_q4": ([vp, vp], ctypes.c_int),
            "bitsmoe_grouped_matmul": ([vp, vp], ctypes.c_int),
            "bitsmoe_dense_ffn_workspace_bytes": ([ctypes.POINTER(FfnDims), i32], u64),
            "bitsmoe_dense_ffn_forward": ([vp, vp], ctypes.c_int),
            "bitsmoe_read_status": ([vp, vp, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "bitsmoe_strerror": ([ctypes.c_int], ctypes.c_char_p),
            "bitsmoe_version": ([], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().bitsmoe_strerror(code).decode()


def version() -> int:
    return lib().bitsmoe_version()


def _check(rc: int, what: str):
    if rc != 0:
        raise BitsMoEError(rc, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return int(t)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class Plan:
    """Owns one bitsmoe_plan (host object describing one projection's blob)."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def __del__(self):
        if getattr(self, "_h", None) is not None and self._h.value and _lib is not None:
            _lib.bitsmoe_plan_free(self._h)
            self._h = None

    @property
    def blob_bytes(self) -> int:
        return int(lib().bitsmoe_plan_blob_bytes(self._h))

    @property
    def header_bytes(self) -> int:
        return int(lib().bitsmoe_plan_header_bytes(self._h))

    @property
    def dims(self) -> Dims:
        d = Dims()
        _check(lib().bitsmoe_plan_get_dims(self._h, ctypes.byref(d)), "plan_get_dims")
        return d

    def header(self) -> np.ndarray:
        out = np.zeros(self.header_bytes, np.uint8)
        _check(lib().bitsmoe_plan_write_header(self._h, out.ctypes.data, out.size), "plan_write_header")
        return out


def pack_plan(d_in: int, d_out: int, n_experts: int, rank: int, top_k: int, widths) -> Plan:
    w = np.ascontiguousarray(widths.cpu().numpy() if isinstance(widths, torch.Tensor) else widths, dtype=np.uint8)
    d = Dims(d_in, d_out, n_experts, rank, top_k)
    h = ctypes.c_void_p()
    _check(lib().bitsmoe_pack_plan(ctypes.byref(d), w.ctypes.data, ctypes.byref(h)), "pack_plan")
    return Plan(h.value)


def plan_from_header(header, d_in: int, top_k: int) -> Plan:
    hb = np.ascontiguousarray(header.cpu().numpy() if isinstance(header, torch.Tensor) else header, dtype=np.uint8)
    h = ctypes.c_void_p()
    _check(lib().bitsmoe_plan_from_header(hb.ctypes.data, hb.size, d_in, top_k, ctypes.byref(h)), "plan_from_header")
    return Plan(h.value)


def compute_scales(plan: Plan, comps, widths, scales, status=None, stream=None):
    _check(lib().bitsmoe_compute_scales(plan.handle, _ptr(comps), _ptr(widths), _ptr(scales), _ptr(status),
                                        _stream(stream)), "compute_scales")


def pack(plan: Plan, comps, widths, scales, amps, blob, status=None, stream=None):
    _check(lib().bitsmoe_pack(plan.handle, _ptr(comps), _ptr(widths), _ptr(scales), _ptr(amps), _ptr(blob),
                              _ptr(status), _stream(stream)), "pack")


def unpack_q(plan: Plan, blob, q, stream=None):
    _check(lib().bitsmoe_unpack_q(plan.handle, _ptr(blob), _ptr(q), _stream(stream)), "unpack_q")


def shared_proj(phi_t, X, Z, T: int, d_in: int, r: int, stream=None):
    _check(lib().bitsmoe_shared_proj(_ptr(phi_t), _ptr(X), _ptr(Z), T, d_in, r, _stream(stream)), "shared_proj")


def expert_workspace_bytes(plan: Plan, T: int) -> int:
    return int(lib().bitsmoe_expert_workspace_bytes(plan.handle, T))


def expert_forward(plan: Plan, blob, Z, topk_ids, gate_w, T: int, Y_experts, Y_sum, workspace, workspace_bytes: int,
                   status=None, stream=None):
    _check(lib().bitsmoe_expert_forward(plan.handle, _ptr(blob), _ptr(Z), _ptr(topk_ids), _ptr(gate_w), T,
                                        _ptr(Y_experts), _ptr(Y_sum), _ptr(workspace), workspace_bytes,
                                        _ptr(status), _stream(stream)), "expert_forward")


def layer_workspace_bytes(plan_gate: Plan, plan_up: Plan, T: int) -> int:
    return int(lib().bitsmoe_layer_workspace_bytes(plan_gate.handle, plan_up.handle, T))


def layer_launches(plan_gate: Plan, plan_up: Plan, T: int) -> int:
    n = int(lib().bitsmoe_layer_launches(plan_gate.handle, plan_up.handle, T))
    if n < 0:
        raise BitsMoEError(n, "layer_launches")
    return n


def proj_io(plan: Plan, blob, phi_t, Y_sum, Z=None, Y_experts=None) -> ProjIO:
    return ProjIO(plan.handle.value, _ptr(blob), _ptr(phi_t), _ptr(Z), _ptr(Y_experts), _ptr(Y_sum))


def layer_forward(gate: ProjIO, up: ProjIO, X, topk_ids, gate_w, T: int, workspace, workspace_bytes: int,
                  status=None, stream=None):
    _check(lib().bitsmoe_layer_forward(ctypes.byref(gate), ctypes.byref(up), _ptr(X), _ptr(topk_ids), _ptr(gate_w),
                                       T, _ptr(workspace), workspace_bytes, _ptr(status), _stream(stream)),
           "layer_forward")


def layer_forward_chained(gate: ProjIO, up: ProjIO, X, topk_ids, gate_w, T: int, workspace, workspace_bytes: int,
                          next_phi_t_gate, next_phi_t_up, status=None, stream=None):
    _check(lib().bitsmoe_layer_forward_chained(ctypes.byref(gate), ctypes.byref(up), _ptr(X), _ptr(topk_ids),
                                               _ptr(gate_w), T, _ptr(workspace), workspace_bytes,
                                               _ptr(next_phi_t_gate), _ptr(next_phi_t_up), _ptr(status),
                                               _stream(stream)),
           "layer_forward_chained")


def layer_forward_t1_noalloc(gate: ProjIO, up: ProjIO, X, topk_ids, gate_w, status=None, stream=None):
    _check(lib().bitsmoe_layer_forward_t1_noalloc(ctypes.byref(gate), ctypes.byref(up), _ptr(X), _ptr(topk_ids),
                                                  _ptr(gate_w), _ptr(status), _stream(stream)),
           "layer_forward_t1_noalloc")


def ffn_dims(d_model: int, d_ff: int, n_experts: int, top_k: int) -> FfnDims:
    return FfnDims(d_model, d_ff, n_experts, top_k)


def ffn_down_workspace_bytes(dims: FfnDims, T: int) -> int:
    return int(lib().bitsmoe_ffn_down_workspace_bytes(ctypes.byref(dims), T))


def ffn_down_launches(dims: FfnDims, T: int) -> int:
    n = int(lib().bitsmoe_ffn_down_launches(ctypes.byref(dims), T))
    if n < 0:
        raise BitsMoEError(n, "ffn_down_launches")
    return n


def ffn_down(dims: FfnDims, w_down, Y_gate, Y_up, topk_ids, gate_w, T: int, out, workspace=None,
             workspace_bytes: int = 0, status=None, stream=None):
    _check(lib().bitsmoe_ffn_down(ctypes.byref(dims), _ptr(w_down), _ptr(Y_gate), _ptr(Y_up), _ptr(topk_ids),
                                  _ptr(gate_w), T, _ptr(out), _ptr(workspace), workspace_bytes, _ptr(status),
                                  _stream(stream)), "ffn_down")


def ffn_workspace_bytes(plan_gate: Plan, plan_up: Plan, T: int) -> int:
    return int(lib().bitsmoe_ffn_workspace_bytes(plan_gate.handle, plan_up.handle, T))


def ffn_launches(plan_gate: Plan, plan_up: Plan, T: int) -> int:
    n = int(lib().bitsmoe_ffn_launches(plan_gate.handle, plan_up.handle, T))
    if n < 0:
        raise BitsMoEError(n, "ffn_launches")
    return n


def ffn_forward(gate: ProjIO, up: ProjIO, w_down, X, topk_ids, gate_w, T: int, out, workspace, workspace_bytes: int,
                status=None, stream=None):
    _check(lib().bitsmoe_ffn_forward(ctypes.byref(gate), ctypes.byref(up), _ptr(w_down), _ptr(X), _ptr(topk_ids),
                                     _ptr(gate_w), T, _ptr(out), _ptr(workspace), workspace_bytes, _ptr(status),
                                     _stream(stream)), "ffn_forward")


def ssd_workspace_bytes(n_experts: int, d_out: int, d_in: int, rank: int) -> int:
    return int(lib().bitsmoe_ssd_workspace_bytes(n_experts, d_out, d_in, rank))


def ssd_decompose(W, rank: int, phi_t, amps, comps, workspace, workspace_bytes: int, sigma=None, phi_t32=None,
                  status=None, stream=None):
    """W [E][d_out][d_in] f32 (GPU) -> phi_t [rank][d_in] fp16, amps [E][rank], comps [E][rank][d_out]."""
    E, d_out, d_in = W.shape
    _check(lib().bitsmoe_ssd_decompose(_ptr(W), E, d_out, d_in, rank, _ptr(phi_t), _ptr(phi_t32), _ptr(sigma),
                                       _ptr(amps), _ptr(comps), _ptr(workspace), workspace_bytes, _ptr(status),
                                       _stream(stream)),
           "ssd_decompose")


def assign_widths(amps_host, widths_in_order, counts) -> np.ndarray:
    """Widths [E][r] u8 by descending amplitude within each expert (host)."""
    a = np.ascontiguousarray(np.asarray(amps_host, dtype=np.float32))
    E, r = a.shape
    wo = np.ascontiguousarray(np.asarray(widths_in_order, dtype=np.uint8))
    ct = np.ascontiguousarray(np.asarray(counts, dtype=np.int32))
    out = np.zeros((E, r), np.uint8)
    _check(lib().bitsmoe_assign_widths(a.ctypes.data, E, r, wo.ctypes.data, ct.ctypes.data, len(wo), out.ctypes.data),
           "assign_widths")
    return out


WIDTH_SET = (0, 1, 2, 3, 4, 6, 8, 16)  # the width order of eps arrays


def _host(a, dtype):
    return np.ascontiguousarray(np.asarray(a, dtype=dtype))


def fqcm_eps(comps_host) -> np.ndarray:
    """eps [E][r][8] f64: squared error of each unit direction stored at each width."""
    c = _host(comps_host, np.float32)
    E, r, d_out = c.shape
    out = np.zeros((E, r, 8), np.float64)
    _check(lib().bitsmoe_fqcm_eps(c.ctypes.data, E, r, d_out, out.ctypes.data), "fqcm_eps")
    return out


def fqcm_beta(Z_host, topk_ids_host, gate_w_host, n_experts: int) -> np.ndarray:
    """beta [E][r] f64 from z = Phi^T x of calibration tokens and their routing."""
    Z = _host(Z_host, np.float32)
    ids = _host(topk_ids_host, np.int32)
    g = _host(gate_w_host, np.float32)
    T, r = Z.shape
    out = np.zeros((n_experts, r), np.float64)
    _check(lib().bitsmoe_fqcm_beta(Z.ctypes.data, ids.ctypes.data, g.ctypes.data, T, ids.shape[1], n_experts, r,
                                   out.ctypes.data), "fqcm_beta")
    return out


def allocate_widths(amps_host, beta_host, eps_host, d_out: int, budget_bits: int) -> tuple[np.ndarray, float]:
    """(widths [E][r] u8, total cost) under sum d_out b <= budget_bits."""
    a = _host(amps_host, np.float32)
    b = _host(beta_host, np.float64)
    e = _host(eps_host, np.float64)
    E, r = a.shape
    w = np.zeros((E, r), np.uint8)
    loss = ctypes.c_double(0.0)
    _check(lib().bitsmoe_allocate_widths(a.ctypes.data, b.ctypes.data, e.ctypes.data, E, r, d_out, int(budget_bits),
                                         w.ctypes.data, ctypes.byref(loss)), "allocate_widths")
    return w, float(loss.value)


# ---- the block around the routed experts ----
# These calls take one structure.  It is packed into a bytes object (one C call) instead
# of a ctypes structure or a long argument list, which cost more than the launch itself.
_TYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_NORM = struct.Struct("@7P5q6i2f")         # bitsmoe_norm_args
_ROUTE = struct.Struct("@7PQq6ifi")        # bitsmoe_route_args
_Q4 = struct.Struct("@6i8PQ")              # bitsmoe_q4_args
_GMM = struct.Struct("@7Pq10i")            # bitsmoe_gmm_args
_DENSE = struct.Struct("@6i11PQq")         # bitsmoe_dense_ffn_args


def _refuse(what: str, why: str):
    raise BitsMoEError(EINVAL, f"{what}: {why}")


def _matrix(what: str, name: str, t: torch.Tensor, shape: tuple, dev: int) -> tuple:
    """(pointer, type, row stride) of a 2-D operand with contiguous rows on GPU dev."""
    s = t.stride()
    kind = _TYPE.get(t.dtype)
    if t.shape != shape or (s[1] != 1 and shape[1] > 1):
        _refuse(what, f"{name} is not {list(shape)} with contiguous rows")
    if kind is None:
        _refuse(what, f"{name} is {t.dtype}, not float32, float16 or bfloat16")
    if t.get_device() != dev:
        _refuse(what, "the tensors are not on one GPU")
    return t.data_ptr(), kind, s[0]


def _dense(what: str, name: str, t: torch.Tensor, dtype, shape: tuple, dev: int) -> int:
    """Pointer of a contiguous operand on GPU dev."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(what, f"{name} is not a contiguous {dtype} tensor of shape {list(shape)}")
    if t.get_device() != dev:
        _refuse(what, "the tensors are not on one GPU")
    return t.data_ptr()


def _status(what: str, t, dev: int) -> int:
    """Pointer of an optional status word on GPU dev; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.numel() < 1:
        _refuse(what, "status is not an int32 tensor")
    if t.get_device() != dev:
        _refuse(what, "the tensors are not on one GPU")
    return t.data_ptr()


def _bytes(what: str, name: str, t, dev: int, need: int = 0) -> int:
    """Pointer of an optional buffer of at least `need` bytes on GPU dev; 0 for None."""
    if t is None:
        return 0
    if not t.is_contiguous():
        _refuse(what, f"{name} is not contiguous")
    if t.nbytes < need:
        raise BitsMoEError(ESIZE, f"{what}: {name} of {t.nbytes} bytes, {need} needed")
    if t.get_device() != dev:
        _refuse(what, "the tensors are not on one GPU")
    return t.data_ptr()


def _blob(what: str, t, need: int, dev: int) -> int:
    """Pointer of packed matrices (uint8, `need` bytes; 0: bad dimensions) on GPU dev."""
    if need == 0:
        _refuse(what, "the dimensions or the group (32, 64 or 128) are out of range")
    if t.dtype is not torch.uint8:
        _refuse(what, f"blob is {t.dtype}, not uint8")
    return _bytes(what, "blob", t, dev, need)


def _launch(what: str, call, dev: int, stream, *args):
    """Calls the library with GPU dev current; the stream defaults to torch's current one there."""
    if dev == torch._C._cuda_getDevice():
        rc = call(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            rc = call(*args, _stream(stream))
    if rc != 0:
        raise BitsMoEError(rc, what)


def norm_residual(h, y=None, w_pre=None, x=None, *, w_post=None, gate=None, alpha: float = 1.0, eps: float = 1e-6,
                  h_out=None, stream=None):
    """h' = h + alpha * gate * (y, or y normalised with w_post); x = h' normalised with w_pre.

    h, y, x [T][d] in float32, float16 or bfloat16, any row stride; gate float32 [T or 1][d or 1];
    w_pre, w_post [d] float32.  h' goes to h_out (default: h itself when y is given), x is written
    when given."""
    what = "norm_residual"
    shape = h.shape
    if len(shape) != 2:
        _refuse(what, "h is not [T][d]")
    T, d = shape
    dev = h.get_device()
    hp, ht, hs = _matrix(what, "h", h, shape, dev)
    yp = yt = ys = op = os_ = xp = xt = xs = gp = gs = gc = wo = wi = 0
    if y is not None:
        yp, yt, ys = _matrix(what, "y", y, shape, dev)
        if h_out is None:
            op, os_ = hp, hs
    if h_out is not None:
        op, ot, os_ = _matrix(what, "h_out", h_out, shape, dev)
        if ot != ht:
            _refuse(what, "h_out has another type than h")
    if x is not None:
        xp, xt, xs = _matrix(what, "x", x, shape, dev)
        if w_pre is None:
            _refuse(what, "x needs w_pre")
    if w_pre is not None:
        wi = _dense(what, "w_pre", w_pre, torch.float32, (d,), dev)
    if w_post is not None:
        wo = _dense(what, "w_post", w_post, torch.float32, (d,), dev)
    if gate is not None:
        if gate.dim() != 2 or gate.shape[0] not in (1, T) or gate.shape[1] not in (1, d):
            _refuse(what, "gate is not [T or 1][d or 1]")
        gp, gt, gs = _matrix(what, "gate", gate, gate.shape, dev)
        if gt != F32:
            _refuse(what, "gate is not float32")
        if gate.shape[0] == 1:
            gs = 0
        gc = gate.shape[1] > 1
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_norm_residual, dev, stream,
            _NORM.pack(hp, yp, wo, gp, op, wi, xp, hs, ys, gs, os_, xs, T, d, ht, yt, xt, gc, alpha, eps))


def topk_route_workspace_bytes(T: int, n_experts: int, top_k: int) -> int:
    return int(lib().bitsmoe_topk_route_workspace_bytes(T, n_experts, top_k))


def topk_route(logits, topk_ids, gate_w, offsets=None, order=None, *, scoring: str = "softmax",
               renormalise: bool = True, scale: float = 1.0, workspace=None, status=None, stream=None):
    """The top_k largest logits [T][E] of every token into topk_ids [T][top_k] int32 and their weights
    into gate_w [T][top_k] float32; with offsets [E+1] and order [T*top_k] (int32) also the pairs
    t*top_k + slot grouped by expert."""
    what = "topk_route"
    shape, kshape = logits.shape, topk_ids.shape
    if len(shape) != 2 or len(kshape) != 2 or kshape[0] != shape[0]:
        _refuse(what, "logits or topk_ids is not [T][*]")
    T, E = shape
    K = kshape[1]
    mode = SCORING.get(scoring)
    if mode is None:
        _refuse(what, f"scoring {scoring!r} is neither softmax nor sigmoid")
    dev = logits.get_device()
    lp, lt, ls = _matrix(what, "logits", logits, shape, dev)
    ids = _dense(what, "topk_ids", topk_ids, torch.int32, kshape, dev)
    gw = _dense(what, "gate_w", gate_w, torch.float32, kshape, dev)
    off = 0 if offsets is None else _dense(what, "offsets", offsets, torch.int32, (E + 1,), dev)
    od = 0 if order is None else _dense(what, "order", order, torch.int32, (T * K,), dev)
    ws = _bytes(what, "workspace", workspace, dev)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_topk_route, dev, stream,
            _ROUTE.pack(lp, ids, gw, off, od, ws, _status(what, status, dev), workspace.nbytes if ws else 0, ls, T, E, K,
                        lt, mode, renormalise, scale, 0))


@functools.lru_cache(maxsize=256)  # a call of the library took 0.8 us of every step's
def q4_bytes(n_experts: int, rows: int, cols: int, group: int) -> int:
    return int(lib().bitsmoe_q4_bytes(n_experts, rows, cols, group))


def q4_pack(W, group: int, blob, status=None, stream=None):
    """W [E][rows][cols] (float32, float16 or bfloat16) into 4 bits with a scale per `group` columns."""
    what = "q4_pack"
    if W.dim() != 3 or not W.is_contiguous() or W.dtype not in _TYPE:
        _refuse(what, "W is not a contiguous float32, float16 or bfloat16 [E][rows][cols]")
    E, rows, cols = W.shape
    n = q4_bytes(E, rows, cols, group)
    if n == 0:
        _refuse(what, f"group {group} is not 32, 64 or 128, or W is empty")
    dev = W.get_device()
    _blob(what, blob, n, dev)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_q4_pack, dev, stream, W.data_ptr(), _TYPE[W.dtype], E, rows, cols, group,
            blob.data_ptr(), _status(what, status, dev))


def q4_unpack(blob, group: int, W, stream=None):
    """The stored values of packed matrices into W [E][rows][cols] float32."""
    what = "q4_unpack"
    if W.dim() != 3:
        _refuse(what, "W is not [E][rows][cols]")
    E, rows, cols = W.shape
    dev = W.get_device()
    bp = _blob(what, blob, q4_bytes(E, rows, cols, group), dev)
    wp = _dense(what, "W", W, torch.float32, (E, rows, cols), dev)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_q4_unpack, dev, stream, bp, E, rows, cols, group, wp)


def ffn_down_q4_workspace_bytes(dims: FfnDims, group: int, T: int) -> int:
    return int(lib().bitsmoe_ffn_down_q4_workspace_bytes(ctypes.byref(dims), group, T))


def ffn_down_q4_launches(dims: FfnDims, group: int, T: int) -> int:
    n = int(lib().bitsmoe_ffn_down_q4_launches(ctypes.byref(dims), group, T))
    if n < 0:
        raise BitsMoEError(n, "ffn_down_q4_launches")
    return n


def ffn_down_q4(dims: FfnDims, blob, group: int, Y_gate, Y_up, topk_ids, gate_w, T: int, out, workspace=None,
                workspace_bytes: int = 0, status=None, stream=None):
    """ffn_down with the down matrices in 4 bits (q4_pack).  Y_up None: h = Y_gate, no activation."""
    what = "ffn_down_q4"
    d_model, d_ff, E, K = dims.d_model, dims.d_ff, dims.n_experts, dims.top_k
    dev = blob.get_device()
    shape = (T, K, d_ff)
    yg = _dense(what, "Y_gate", Y_gate, torch.float32, shape, dev)
    yu = 0 if Y_up is None else _dense(what, "Y_up", Y_up, torch.float32, shape, dev)
    ids = _dense(what, "topk_ids", topk_ids, torch.int32, (T, K), dev)
    gw = _dense(what, "gate_w", gate_w, torch.float32, (T, K), dev)
    op = _dense(what, "out", out, torch.float32, (T, d_model), dev)
    bp = _blob(what, blob, q4_bytes(E, d_model, d_ff, group), dev)
    ws = _bytes(what, "workspace", workspace, dev, workspace_bytes)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_ffn_down_q4, dev, stream,
            _Q4.pack(d_model, d_ff, E, K, group, T, bp, yg, yu, ids, gw, op, ws, _status(what, status, dev),
                     workspace_bytes))


def grouped_matmul(A, W, offsets, out, *, W_up=None, rows=None, rows_per_a: int = 1, scatter: bool = False, status=None,
                   stream=None):
    """Sorted rows times their expert's matrix: out row i = W[e] a_i for offsets[e] <= i < offsets[e+1],
    or SiLU(W[e] a_i) * (W_up[e] a_i) with W_up.

    A [*][K] and W, W_up [E][N][K] float16 or bfloat16; out [n][N] of the same type or float32.
    a_i is row i of A, or with rows [n] int32 row rows[i] // rows_per_a; with scatter the result
    goes to row rows[i] of out."""
    what = "grouped_matmul"
    wshape, ashape, oshape = W.shape, A.shape, out.shape
    if len(ashape) != 2 or len(wshape) != 3 or len(oshape) != 2:
        _refuse(what, "A, W and out are not [*][K], [E][N][K] and [n][N]")
    E, N, K = wshape
    n = oshape[0]
    dev = A.get_device()
    ap, it, lda = _matrix(what, "A", A, (ashape[0], K), dev)
    if ashape[0] <= 1:
        lda = K
    wp = _dense(what, "W", W, A.dtype, wshape, dev)
    up = 0 if W_up is None else _dense(what, "W_up", W_up, A.dtype, wshape, dev)
    ot = _TYPE.get(out.dtype, -1)
    op = _dense(what, "out", out, out.dtype, (n, N), dev)
    off = _dense(what, "offsets", offsets, torch.int32, (E + 1,), dev)
    rp = 0 if rows is None else _dense(what, "rows", rows, torch.int32, (n,), dev)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_grouped_matmul, dev, stream,
            _GMM.pack(ap, wp, up, off, rp, op, _status(what, status, dev), lda, n, ashape[0], N, K, E, it, ot, rows_per_a,
                      scatter, 0))


def dense_ffn_workspace_bytes(dims: FfnDims, T: int) -> int:
    return int(lib().bitsmoe_dense_ffn_workspace_bytes(ctypes.byref(dims), T))


def dense_ffn_forward(dims: FfnDims, w_gate, w_up, w_down, x, topk_ids, gate_w, offsets, order, out, workspace,
                      status=None, stream=None):
    """The routed FFN of dense experts: w_gate, w_up [E][d_ff][d_model], w_down [E][d_model][d_ff] and
    x [T][d_model] in float16 or bfloat16, the routing of topk_route, out [T][d_model] float32."""
    what = "dense_ffn_forward"
    d_model, d_ff, E, K = dims.d_model, dims.d_ff, dims.n_experts, dims.top_k
    T = x.shape[0]
    dev = x.get_device()
    xp, kind, xs = _matrix(what, "x", x, (T, d_model), dev)
    wg = _dense(what, "w_gate", w_gate, x.dtype, (E, d_ff, d_model), dev)
    wu = _dense(what, "w_up", w_up, x.dtype, (E, d_ff, d_model), dev)
    wd = _dense(what, "w_down", w_down, x.dtype, (E, d_model, d_ff), dev)
    ids = _dense(what, "topk_ids", topk_ids, torch.int32, (T, K), dev)
    gw = _dense(what, "gate_w", gate_w, torch.float32, (T, K), dev)
    off = _dense(what, "offsets", offsets, torch.int32, (E + 1,), dev)
    od = _dense(what, "order", order, torch.int32, (T * K,), dev)
    op = _dense(what, "out", out, torch.float32, (T, d_model), dev)
    ws = _bytes(what, "workspace", workspace, dev)
    if dev < 0:
        _refuse(what, "the tensors are not on one GPU")
    _launch(what, lib().bitsmoe_dense_ffn_forward, dev, stream,
            _DENSE.pack(d_model, d_ff, E, K, T, kind, xp, wg, wu, wd, ids, gw, off, od, op, ws, _status(what, status, dev),
                        workspace.nbytes if ws else 0, xs if T > 1 else d_model))


def read_status(status, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(lib().bitsmoe_read_status(_ptr(status), _stream(stream), ctypes.byref(out)), "read_status")
    return int(out.value)
