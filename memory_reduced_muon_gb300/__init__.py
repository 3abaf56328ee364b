"""Python binding of the qmuon C ABI (``include/qmuon.h``).

Argument marshalling only: every function below converts its arguments to
the C types of the entry point with the same name, calls ``libqmuon.so``
and raises :class:`QmuonError` on a non-OK status.  All arithmetic runs in
the library's CUDA kernels; there is no Python or CPU fallback, and calling
any entry point without the built library raises.

Device buffers are passed as torch tensors (their ``data_ptr()``) or as raw
integer addresses; the clipping, AdamW and RMS norm entries, which take a
model's own tensors, check the former.  ``stream`` is a ``torch.cuda.Stream``, a raw
``cudaStream_t`` integer, or ``None`` for torch's current stream.
"""

from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Iterable, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmuon.so")

QMUON_OK = 0
QMUON_ERR_INVALID_ARGUMENT = 1
QMUON_ERR_MISALIGNED_SEGMENT = 2
QMUON_ERR_UNSUPPORTED = 3
QMUON_ERR_WORKSPACE_TOO_SMALL = 4
QMUON_ERR_CUDA = 5
QMUON_ERR_TIMEOUT = 6
QMUON_ERR_OUT_OF_MEMORY = 7

QMUON_Q8_INT8, QMUON_Q8_UINT8 = 0, 1
QMUON_BF16, QMUON_FP16, QMUON_FP32 = 0, 1, 2
QMUON_WS_UPDATE, QMUON_WS_STEP = 0, 1
QMUON_NS_BF16, QMUON_NS_MXFP8 = 0, 1
QMUON_STATE_F32, QMUON_STATE_E4M3 = 0, 1

Q8_KINDS = {"int8": QMUON_Q8_INT8, "uint8": QMUON_Q8_UINT8}
DTYPES = {"bf16": QMUON_BF16, "f16": QMUON_FP16, "f32": QMUON_FP32}
STATE_KINDS = {"f32": QMUON_STATE_F32, "e4m3": QMUON_STATE_E4M3}


class QmuonError(RuntimeError):
    def __init__(self, status: int, where: str, detail: Optional[str] = None):
        self.status = int(status)
        if detail is None:
            detail = ""
            try:
                detail = lib().qmuon_last_error().decode()
            except Exception:
                pass
        super().__init__(f"{where}: {status_string(status)} (status {status})" + (f" -- {detail}" if detail else ""))


class qmuon_tensor(C.Structure):
    _fields_ = [("q8", C.c_void_p), ("absmax", C.c_void_p), ("grad", C.c_void_p),
                ("rows", C.c_int64), ("cols", C.c_int64)]


class qmuon_norm_segment(C.Structure):
    _fields_ = [("tensor_index", C.c_int32), ("group_id", C.c_int32),
                ("start", C.c_int64), ("length", C.c_int64)]


class qmuon_ns_problem(C.Structure):
    _fields_ = [("x", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64), ("ld", C.c_int64),
                ("inv_norm", C.c_void_p), ("input", C.c_int32), ("reserved", C.c_int32),
                ("payload", C.c_void_p), ("scale_inv", C.c_void_p)]


class qmuon_grasp_matrix(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("res", C.c_void_p), ("res_rmax", C.c_void_p),
                ("res_cmax", C.c_void_p), ("p", C.c_void_p), ("p_rmax", C.c_void_p), ("p_cmax", C.c_void_p),
                ("r", C.c_void_p), ("r_rmax", C.c_void_p), ("r_cmax", C.c_void_p), ("grad", C.c_void_p)]


class qmuon_grad(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("numel", C.c_int64), ("dtype", C.c_int32), ("reserved", C.c_int32)]


class qmuon_adamw_tensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("copy", C.c_void_p), ("m", C.c_void_p),
                ("v", C.c_void_p), ("m_absmax", C.c_void_p), ("v_absmax", C.c_void_p), ("numel", C.c_int64),
                ("lr_scale", C.c_float), ("weight_decay", C.c_float), ("grad_dtype", C.c_int32),
                ("copy_dtype", C.c_int32)]


class qmuon_rmsnorm(C.Structure):
    _fields_ = [("x", C.c_void_p), ("residual", C.c_void_p), ("gain", C.c_void_p), ("sum", C.c_void_p),
                ("y", C.c_void_p), ("payload", C.c_void_p), ("scale_inv", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64), ("ld_x", C.c_int64), ("ld_residual", C.c_int64), ("ld_sum", C.c_int64),
                ("ld_y", C.c_int64), ("eps", C.c_float), ("dtype", C.c_int32)]


class qmuon_rmsnorm_grad(C.Structure):
    _fields_ = [("dy", C.c_void_p), ("h", C.c_void_p), ("dsum", C.c_void_p), ("gain", C.c_void_p),
                ("dx", C.c_void_p), ("dgain", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("ld_dy", C.c_int64), ("ld_h", C.c_int64), ("ld_dsum", C.c_int64), ("ld_dx", C.c_int64),
                ("eps", C.c_float), ("dtype", C.c_int32)]


GRASP_RANK, GRASP_BLOCK = 8, 64

COUNTER_FIELDS = (
    "update_calls", "update_sr_calls", "carrier_calls", "ns_calls", "step_block_calls", "step_full_calls",
    "step_sr_calls", "step_host_fed_calls", "grasp_calls", "grad_bf16_tensors", "grad_fp16_tensors",
    "grad_fp32_tensors", "state_int8_tensors", "state_uint8_tensors", "carrier_payload_u8_tensors",
    "carrier_scale_u8_tensors", "carrier_inv_norm_f32_values", "ns_bf16_problems", "ns_mxfp8_problems",
    "ns_bf16_handoff_bytes", "weight_f32_tensors", "grasp_matrices", "host_pulled_bytes", "host_copied_bytes")


class qmuon_counters(C.Structure):
    _fields_ = [(f, C.c_uint64) for f in COUNTER_FIELDS]

_lib_handle = None


def lib() -> C.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"qmuon CUDA library not built ({LIB_PATH} missing); "
                           "run `python -m memory_reduced_muon_gb300.build`")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
    f64 = C.c_double
    sig = {
        "qmuon_plan_create": (i32, [C.POINTER(qmuon_tensor), i32, i32, i32, C.POINTER(qmuon_norm_segment),
                                    i32, i32, i32, i32, C.POINTER(vp)]),
        "qmuon_plan_destroy": (None, [vp]),
        "qmuon_plan_info": (i32, [vp, C.POINTER(i64), C.POINTER(i32), C.POINTER(i32), C.POINTER(i32)]),
        "qmuon_workspace_size": (sz, [vp, i32]),
        "qmuon_update_multi_normalize_groups": (i32, [vp, f32, i32, vp, vp, vp, sz, vp]),
        "qmuon_update_multi_normalize_groups_sr": (i32, [vp, f32, i32, C.c_uint64, i64, vp, vp, vp, sz, vp]),
        "qmuon_plan_set_stochastic_rounding": (i32, [vp, i32, C.c_uint64]),
        "qmuon_plan_set_host_ingest": (i32, [vp, i32]),
        "qmuon_grasp_workspace_size": (sz, [C.POINTER(qmuon_grasp_matrix), i32]),
        "qmuon_grasp_step": (i32, [C.POINTER(qmuon_grasp_matrix), i32, f32, vp, sz, vp]),
        "qmuon_carrier_workspace_size": (sz, [i64, i64]),
        "qmuon_update_mxfp8_carrier": (i32, [C.POINTER(qmuon_tensor), i32, i32, f32, vp, vp, vp, vp, sz, vp]),
        "qmuon_update_mxfp8_carrier_multi": (i32, [vp, f32, C.POINTER(vp), C.POINTER(vp), vp, vp, vp, sz, vp]),
        "qmuon_ns_workspace_size": (sz, [C.POINTER(qmuon_ns_problem), i32]),
        "qmuon_newton_schulz_batched": (i32, [C.POINTER(qmuon_ns_problem), i32, i32, C.POINTER(f32), vp, sz, vp]),
        "qmuon_step": (i32, [vp, i64, i32, f32, f32, f32, C.POINTER(vp), C.POINTER(f32), i32, vp, vp, sz, vp]),
        "qmuon_sync_status": (i32, [vp, vp]),
        "qmuon_status_string": (C.c_char_p, [i32]),
        "qmuon_version": (C.c_char_p, []),
        "qmuon_last_error": (C.c_char_p, []),
        "qmuon_update_normalize_noalloc": (i32, [C.POINTER(qmuon_tensor), i32, i32, f32, vp, vp, vp]),
        "qmuon_step_prepare": (i32, [vp, C.POINTER(vp), vp, sz]),
        "qmuon_step_from_host": (i32, [vp, i64, i32, f32, f32, f32, C.POINTER(vp), C.POINTER(f32), i32,
                                       C.POINTER(vp), vp, vp, vp, sz, vp, vp]),
        "qmuon_plan_set_nonfinite_counter": (i32, [vp, vp]),
        "qmuon_noalloc_sync_status": (i32, [vp]),
        "qmuon_noalloc_inject_status": (i32, [i32, C.c_uint32]),
        "qmuon_clip_plan_create": (i32, [C.POINTER(qmuon_grad), i32, C.POINTER(vp)]),
        "qmuon_clip_plan_destroy": (None, [vp]),
        "qmuon_clip_workspace_size": (sz, [vp]),
        "qmuon_grad_clip": (i32, [vp, f32, i32, vp, vp, sz, vp]),
        "qmuon_adamw_plan_create": (i32, [C.POINTER(qmuon_adamw_tensor), i32, i32, C.POINTER(vp)]),
        "qmuon_adamw_plan_destroy": (None, [vp]),
        "qmuon_adamw_step": (i32, [vp, i64, f64, f64, f64, f64, vp, vp]),
        "qmuon_adamw_step_sr": (i32, [vp, i64, f64, f64, f64, f64, C.c_uint64, vp, vp]),
        "qmuon_rmsnorm_forward": (i32, [C.POINTER(qmuon_rmsnorm), vp]),
        "qmuon_rmsnorm_workspace_size": (sz, [i64, i64]),
        "qmuon_rmsnorm_backward": (i32, [C.POINTER(qmuon_rmsnorm_grad), vp, sz, vp]),
        "qmuon_get_counters": (i32, [C.POINTER(qmuon_counters), sz]),
        "qmuon_reset_counters": (None, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib_handle = L
    return L


def exported_symbols() -> list:
    return ["qmuon_plan_create", "qmuon_plan_destroy", "qmuon_plan_info", "qmuon_workspace_size",
            "qmuon_update_multi_normalize_groups", "qmuon_carrier_workspace_size",
            "qmuon_update_mxfp8_carrier", "qmuon_ns_workspace_size", "qmuon_newton_schulz_batched",
            "qmuon_step", "qmuon_sync_status", "qmuon_status_string", "qmuon_version", "qmuon_last_error",
            "qmuon_update_normalize_noalloc", "qmuon_step_prepare", "qmuon_update_multi_normalize_groups_sr",
            "qmuon_plan_set_stochastic_rounding", "qmuon_update_mxfp8_carrier_multi",
            "qmuon_grasp_workspace_size", "qmuon_grasp_step", "qmuon_step_from_host",
            "qmuon_plan_set_nonfinite_counter", "qmuon_noalloc_sync_status", "qmuon_noalloc_inject_status",
            "qmuon_get_counters", "qmuon_reset_counters", "qmuon_plan_set_host_ingest",
            "qmuon_clip_plan_create", "qmuon_clip_plan_destroy", "qmuon_clip_workspace_size", "qmuon_grad_clip",
            "qmuon_adamw_plan_create", "qmuon_adamw_plan_destroy", "qmuon_adamw_step", "qmuon_adamw_step_sr",
            "qmuon_rmsnorm_forward", "qmuon_rmsnorm_workspace_size", "qmuon_rmsnorm_backward"]


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _ptr(x) -> Optional[int]:
    return x if x is None or isinstance(x, int) else x.data_ptr()


_raw_stream = None   # torch's current raw stream, without the Stream object (3 us of a small call)


def _current_stream() -> int:
    global _raw_stream
    if _raw_stream is None:
        import torch
        s = int(torch.cuda.current_stream().cuda_stream)   # initialises torch's CUDA state
        of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if of is None or device is None:
            return s
        _raw_stream = lambda: of(device())   # noqa: E731
    return _raw_stream()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _nbytes(x) -> int:
    return int(x.numel() * x.element_size())


def _check(status: int, where: str):
    if status != QMUON_OK:
        raise QmuonError(status, where)


def status_string(status: int) -> str:
    try:
        return lib().qmuon_status_string(int(status)).decode()
    except RuntimeError:
        return "library not built"


qmuon_status_string = status_string


def qmuon_version() -> str:
    return lib().qmuon_version().decode()


def qmuon_last_error() -> str:
    return lib().qmuon_last_error().decode()


class Plan:
    """An owned ``qmuon_plan*`` (destroyed with the object)."""

    def __init__(self, handle: int, keepalive):
        self.handle = handle
        self._keep = keepalive

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib_handle is not None:
            _lib_handle.qmuon_plan_destroy(h)


def tensor_desc(q8, absmax, grad, rows: int, cols: int) -> qmuon_tensor:
    return qmuon_tensor(_ptr(q8), _ptr(absmax), _ptr(grad), int(rows), int(cols))


def qmuon_plan_create(tensors: Sequence, q8_kind="int8", grad_dtype="bf16", segments=None,
                      n_groups: int = 0, tile=(1, 1)) -> Plan:
    """``tensors``: ``(q8, absmax, grad, rows, cols)`` tuples or ``qmuon_tensor``;
    ``segments``: ``(tensor_index, start, length, group_id)`` tuples."""
    descs = [t if isinstance(t, qmuon_tensor) else tensor_desc(*t) for t in tensors]
    arr = (qmuon_tensor * max(1, len(descs)))(*descs)
    segs = None
    nseg = 0
    if segments:
        nseg = len(segments)
        segs = (qmuon_norm_segment * nseg)(*[
            s if isinstance(s, qmuon_norm_segment) else
            qmuon_norm_segment(int(s[0]), int(s[3]), int(s[1]), int(s[2])) for s in segments])
    out = C.c_void_p()
    q = Q8_KINDS.get(q8_kind, q8_kind)
    d = DTYPES.get(grad_dtype, grad_dtype)
    st = lib().qmuon_plan_create(arr, len(descs), q, d, segs, nseg, int(n_groups), int(tile[0]), int(tile[1]),
                                 C.byref(out))
    _check(st, "qmuon_plan_create")
    return Plan(out.value, (tensors, segments))


def qmuon_plan_destroy(plan: Plan):
    if plan.handle:
        lib().qmuon_plan_destroy(plan.handle)
        plan.handle = None


def qmuon_plan_info(plan: Plan) -> dict:
    nb, g, gf, gb = C.c_int64(), C.c_int32(), C.c_int32(), C.c_int32()
    _check(lib().qmuon_plan_info(plan.handle, C.byref(nb), C.byref(g), C.byref(gf), C.byref(gb)),
           "qmuon_plan_info")
    return {"n_blocks": nb.value, "n_groups": g.value, "n_full_groups": gf.value, "n_block_groups": gb.value}


def qmuon_workspace_size(plan: Plan, which: int = QMUON_WS_UPDATE) -> int:
    return int(lib().qmuon_workspace_size(plan.handle, int(which)))


def qmuon_update_multi_normalize_groups(plan: Plan, beta: float, normalize_mode: int, group_sumsq, group_inv_norm,
                                        ws, ws_bytes: Optional[int] = None, stream=None):
    st = lib().qmuon_update_multi_normalize_groups(
        plan.handle, float(beta), int(normalize_mode), _ptr(group_sumsq), _ptr(group_inv_norm), _ptr(ws),
        _nbytes(ws) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "qmuon_update_multi_normalize_groups")


def qmuon_update_multi_normalize_groups_sr(plan: Plan, beta: float, normalize_mode: int, seed: int, step: int,
                                           group_sumsq, group_inv_norm, ws, ws_bytes: Optional[int] = None,
                                           stream=None):
    st = lib().qmuon_update_multi_normalize_groups_sr(
        plan.handle, float(beta), int(normalize_mode), int(seed) & 0xFFFFFFFFFFFFFFFF, int(step),
        _ptr(group_sumsq), _ptr(group_inv_norm), _ptr(ws), _nbytes(ws) if ws_bytes is None else int(ws_bytes),
        _stream(stream))
    _check(st, "qmuon_update_multi_normalize_groups_sr")


def qmuon_plan_set_nonfinite_counter(plan: Plan, counter):
    """``counter``: a device uint32/int32 tensor of one element, or None."""
    _check(lib().qmuon_plan_set_nonfinite_counter(plan.handle, _ptr(counter)), "qmuon_plan_set_nonfinite_counter")


QMUON_INGEST_PULL = 0
QMUON_INGEST_COPY = 1


def qmuon_plan_set_host_ingest(plan: Plan, mode: int):
    """QMUON_INGEST_PULL (default) or QMUON_INGEST_COPY for qmuon_step_from_host."""
    _check(lib().qmuon_plan_set_host_ingest(plan.handle, int(mode)), "qmuon_plan_set_host_ingest")


def qmuon_plan_set_stochastic_rounding(plan: Plan, enable: bool, seed: int = 0):
    _check(lib().qmuon_plan_set_stochastic_rounding(plan.handle, 1 if enable else 0,
                                                    int(seed) & 0xFFFFFFFFFFFFFFFF),
           "qmuon_plan_set_stochastic_rounding")


def qmuon_carrier_workspace_size(rows: int, cols: int) -> int:
    return int(lib().qmuon_carrier_workspace_size(int(rows), int(cols)))


def qmuon_update_mxfp8_carrier(q8, absmax, grad, rows: int, cols: int, q8_kind, grad_dtype, beta: float,
                               payload, scale_inv, inv_norm, ws, ws_bytes: Optional[int] = None, stream=None):
    t = tensor_desc(q8, absmax, grad, rows, cols)
    st = lib().qmuon_update_mxfp8_carrier(
        C.byref(t), Q8_KINDS.get(q8_kind, q8_kind), DTYPES.get(grad_dtype, grad_dtype), float(beta),
        _ptr(payload), _ptr(scale_inv), _ptr(inv_norm), _ptr(ws),
        _nbytes(ws) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "qmuon_update_mxfp8_carrier")


def qmuon_update_mxfp8_carrier_multi(plan: Plan, beta: float, payloads: Sequence, scale_invs: Sequence, inv_norms,
                                     ws, group_sumsq=None, ws_bytes: Optional[int] = None, stream=None):
    n = len(payloads)
    pp = (C.c_void_p * max(1, n))(*[_ptr(x) for x in payloads])
    sp = (C.c_void_p * max(1, n))(*[_ptr(x) for x in scale_invs])
    st = lib().qmuon_update_mxfp8_carrier_multi(plan.handle, float(beta), pp, sp, _ptr(inv_norms), _ptr(group_sumsq),
                                                _ptr(ws), _nbytes(ws) if ws_bytes is None else int(ws_bytes),
                                                _stream(stream))
    _check(st, "qmuon_update_mxfp8_carrier_multi")


def ns_problem(x, rows: int, cols: int, ld: Optional[int] = None, inv_norm=None, input_kind=QMUON_NS_BF16,
               payload=None, scale_inv=None) -> qmuon_ns_problem:
    return qmuon_ns_problem(_ptr(x), int(rows), int(cols), int(cols if ld is None else ld), _ptr(inv_norm),
                            int(input_kind), 0, _ptr(payload), _ptr(scale_inv))


def _problems(problems: Iterable):
    ps = [p if isinstance(p, qmuon_ns_problem) else ns_problem(*p) for p in problems]
    return (qmuon_ns_problem * max(1, len(ps)))(*ps), len(ps)


def qmuon_ns_workspace_size(problems) -> int:
    arr, n = _problems(problems)
    return int(lib().qmuon_ns_workspace_size(arr, n))


def qmuon_newton_schulz_batched(problems, iters: int, coeffs, ws, ws_bytes: Optional[int] = None, stream=None):
    arr, n = _problems(problems)
    cf = (C.c_float * 3)(*[float(c) for c in coeffs])
    st = lib().qmuon_newton_schulz_batched(arr, n, int(iters), cf, _ptr(ws),
                                           _nbytes(ws) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "qmuon_newton_schulz_batched")


def qmuon_step(plan: Plan, t: int, P: int, beta: float, eta_full: float, eta_block: float, weights,
               coeffs, iters: int, group_sumsq, ws, ws_bytes: Optional[int] = None, stream=None):
    wp = (C.c_void_p * max(1, len(weights)))(*[_ptr(w) for w in weights])
    cf = (C.c_float * 3)(*[float(c) for c in coeffs])
    st = lib().qmuon_step(plan.handle, int(t), int(P), float(beta), float(eta_full), float(eta_block), wp, cf,
                          int(iters), _ptr(group_sumsq), _ptr(ws),
                          _nbytes(ws) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "qmuon_step")


def qmuon_step_from_host(plan: Plan, t: int, P: int, beta: float, eta_full: float, eta_block: float, weights,
                         coeffs, iters: int, host_grads, host_group_sumsq, group_sumsq, ws,
                         ws_bytes: Optional[int] = None, stream=None, copy_stream=None):
    """``host_grads``: host tensors (page-locked for overlap) or raw host
    addresses, one per plan tensor; ``host_group_sumsq``: a host fp32 tensor
    or None."""
    wp = (C.c_void_p * max(1, len(weights)))(*[_ptr(w) for w in weights])
    hp = (C.c_void_p * max(1, len(host_grads)))(*[_ptr(h) for h in host_grads])
    cf = (C.c_float * 3)(*[float(c) for c in coeffs])
    st = lib().qmuon_step_from_host(plan.handle, int(t), int(P), float(beta), float(eta_full), float(eta_block), wp,
                                    cf, int(iters), hp, _ptr(host_group_sumsq), _ptr(group_sumsq), _ptr(ws),
                                    _nbytes(ws) if ws_bytes is None else int(ws_bytes), _stream(stream),
                                    _stream(copy_stream))
    _check(st, "qmuon_step_from_host")


def qmuon_update_normalize_noalloc(q8, absmax, grad, rows: int, cols: int, q8_kind, grad_dtype, beta: float,
                                   sumsq=None, inv_norm=None, stream=None):
    """The single-tensor update whose scratch is a static array in the
    library (no plan, no workspace, no device allocation)."""
    t = tensor_desc(q8, absmax, grad, rows, cols)
    st = lib().qmuon_update_normalize_noalloc(C.byref(t), Q8_KINDS.get(q8_kind, q8_kind),
                                              DTYPES.get(grad_dtype, grad_dtype), float(beta), _ptr(sumsq),
                                              _ptr(inv_norm), _stream(stream))
    _check(st, "qmuon_update_normalize_noalloc")


def qmuon_noalloc_sync_status(stream=None):
    """Waits for the stream and raises if a kernel of the allocation-free
    update recorded a failure since the last read (the record is cleared)."""
    _check(lib().qmuon_noalloc_sync_status(_stream(stream)), "qmuon_noalloc_sync_status")


def qmuon_noalloc_inject_status(status: int, site: int = 0):
    """Records ``status`` as if a kernel of the allocation-free update had
    failed at ``site`` (for testing a caller's failure handling)."""
    _check(lib().qmuon_noalloc_inject_status(int(status), int(site)), "qmuon_noalloc_inject_status")


def qmuon_get_counters() -> dict:
    """The library's path and dtype tallies (calls that returned OK, and the
    tensors they read or wrote), field name -> count."""
    c = qmuon_counters()
    _check(lib().qmuon_get_counters(C.byref(c), C.sizeof(c)), "qmuon_get_counters")
    return {f: int(getattr(c, f)) for f in COUNTER_FIELDS}


def qmuon_reset_counters():
    lib().qmuon_reset_counters()


def qmuon_step_prepare(plan: Plan, weights, ws, ws_bytes: Optional[int] = None):
    wp = (C.c_void_p * max(1, len(weights)))(*[_ptr(w) for w in weights])
    _check(lib().qmuon_step_prepare(plan.handle, wp, _ptr(ws), _nbytes(ws) if ws_bytes is None else int(ws_bytes)),
           "qmuon_step_prepare")


def qmuon_sync_status(ws, stream=None):
    _check(lib().qmuon_sync_status(_ptr(ws), _stream(stream)), "qmuon_sync_status")


# --------------------------------------------------------------------------
# 4-bit GRASP momentum state
# --------------------------------------------------------------------------

def grasp_matrix(rows: int, cols: int, res, res_rmax, res_cmax, p, p_rmax, p_cmax, r, r_rmax, r_cmax,
                 grad) -> qmuon_grasp_matrix:
    return qmuon_grasp_matrix(int(rows), int(cols), _ptr(res), _ptr(res_rmax), _ptr(res_cmax), _ptr(p), _ptr(p_rmax),
                              _ptr(p_cmax), _ptr(r), _ptr(r_rmax), _ptr(r_cmax), _ptr(grad))


def _grasp_array(matrices: Sequence):
    arr = (qmuon_grasp_matrix * max(1, len(matrices)))(*matrices)
    return arr, len(matrices)


def qmuon_grasp_workspace_size(matrices: Sequence) -> int:
    arr, n = _grasp_array(matrices)
    return int(lib().qmuon_grasp_workspace_size(arr, n))


def qmuon_grasp_step(matrices: Sequence, mu: float, ws, ws_bytes: Optional[int] = None, stream=None):
    arr, n = _grasp_array(matrices)
    _check(lib().qmuon_grasp_step(arr, n, float(mu), _ptr(ws), _nbytes(ws) if ws_bytes is None else int(ws_bytes),
                                  _stream(stream)), "qmuon_grasp_step")


# --------------------------------------------------------------------------
# beside the Muon step: gradient clipping, AdamW, RMS norm
# --------------------------------------------------------------------------
# These entries take a model's own tensors.  Torch tensors are checked: their type,
# that they are on the GPU, and that they hold what the call reads and writes there;
# a mismatch is QMUON_ERR_INVALID_ARGUMENT.  Raw addresses are taken as they are.

_types: dict = {}   # torch dtype of a qmuon_dtype


def _type_of(code):
    """The torch dtype of a qmuon_dtype; None for a code that the library refuses."""
    if not _types:
        import torch
        _types.update({QMUON_BF16: torch.bfloat16, QMUON_FP16: torch.float16, QMUON_FP32: torch.float32})
    return _types.get(code)


def _refuse(x, where: str, what: str, need: str):
    raise QmuonError(QMUON_ERR_INVALID_ARGUMENT, where,
                     f"{what} has to be {need}; it is {tuple(x.shape)}, strides {x.stride()}, of {x.dtype} on {x.device}")


def _rows_apart(x, rows: int, cols: int, ld: int) -> bool:
    """Whether a tensor that is not contiguous is rows `ld` apart in all of its leading dimensions together."""
    *lead, width = zip(x.shape, x.stride())
    if width[0] < cols or (width[1] != 1 and cols != 1):
        return False
    n = 1
    for size, stride in reversed(lead):
        if size != 1 and stride != ld * n:
            return False
        n *= size
    return bool(lead) and n >= rows


def _dense(x) -> bool:
    """Whether a tensor's elements lie side by side in some order."""
    n = 1
    for stride, size in sorted(zip(x.stride(), x.shape)):
        if size != 1:
            if stride != n:
                return False
            n *= size
    return True


def _array(x, dtype, n: int, where: str, what: str, beside=None) -> int:
    """The address of n elements side by side (of a torch dtype; None: any), a tensor or an address.  `beside`: the
    arrays that are gone through together with this one: it may then be in any order that is theirs too."""
    try:
        if (x.dtype is dtype or dtype is None) and x.is_cuda and x.numel() >= n:
            if x.is_contiguous():
                return x.data_ptr()
            if beside is not None and _dense(x) and all(
                    b is None or isinstance(b, int) or b.shape != x.shape or b.stride() == x.stride() for b in beside):
                return x.data_ptr()
    except AttributeError:
        if x is None or isinstance(x, int):
            return x or 0
        raise
    _refuse(x, where, what, f"a contiguous GPU tensor of {n} or more elements" + (f" of {dtype}" if dtype else "") +
            ("" if beside is None else ", or one in the same order as the others"))


def _bytes(x, n: int, where: str, what: str) -> int:
    """The address of n elements of any type of one byte."""
    if x is not None and not isinstance(x, int) and x.element_size() != 1:
        _refuse(x, where, what, "of one byte per element")
    return _array(x, None, n, where, what)


def _matrix(x, dtype, rows: int, cols: int, ld: int, where: str, what: str) -> int:
    """The address of `rows` rows of `cols` elements, `ld` apart (a tensor or an address)."""
    try:
        if (x.dtype is dtype or dtype is None) and x.is_cuda:
            if x.is_contiguous():
                n = x.numel()
                if n >= rows * ld or n >= (rows - 1) * ld + cols:
                    return x.data_ptr()
            elif _rows_apart(x, rows, cols, ld):
                return x.data_ptr()
    except AttributeError:
        if x is None or isinstance(x, int):
            return x or 0
        raise
    _refuse(x, where, what, f"a GPU tensor of {rows} x {cols} elements of {dtype}, rows {ld} elements apart")


def _on_gpu(x, where: str, what: str) -> Optional[int]:
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        _refuse(x, where, what, "on the GPU")
    return x.data_ptr()


class ClipPlan:
    """An owned ``qmuon_clip_plan*`` (destroyed with the object)."""

    def __init__(self, handle: int, keepalive):
        self.handle = handle
        self._keep = keepalive

    def __del__(self):
        qmuon_clip_plan_destroy(self)


def qmuon_clip_plan_create(grads: Sequence) -> ClipPlan:
    """``grads``: ``qmuon_grad`` or ``(gradient tensor, dtype name)`` tuples.

    The plan holds the gradients' addresses: zero them in place, do not let them go (``set_to_none=False``).
    """
    def desc(g):
        if isinstance(g, qmuon_grad):
            return g
        n, dtype = int(g[0].numel()), DTYPES.get(g[1], g[1])
        return qmuon_grad(_array(g[0], _type_of(dtype), n, "qmuon_clip_plan_create", "a gradient", ()), n, dtype, 0)
    descs = [desc(g) for g in grads]
    arr = (qmuon_grad * max(1, len(descs)))(*descs)
    out = C.c_void_p()
    _check(lib().qmuon_clip_plan_create(arr, len(descs), C.byref(out)), "qmuon_clip_plan_create")
    return ClipPlan(out.value, grads)


def qmuon_clip_plan_destroy(plan: ClipPlan):
    h, plan.handle = getattr(plan, "handle", None), None
    if h and _lib_handle is not None:
        _lib_handle.qmuon_clip_plan_destroy(h)


def qmuon_clip_workspace_size(plan: ClipPlan) -> int:
    return int(lib().qmuon_clip_workspace_size(plan.handle))


def qmuon_grad_clip(plan: ClipPlan, max_norm: float, apply: bool, norm, ws, ws_bytes: Optional[int] = None, stream=None):
    """``norm``: a device fp32 tensor of two: the norm and the coefficient."""
    where = "qmuon_grad_clip"
    st = (_lib_handle or lib()).qmuon_grad_clip(
        plan.handle, float(max_norm), int(apply), _array(norm, _types.get(QMUON_FP32) or _type_of(QMUON_FP32), 2, where, "norm"),
        _on_gpu(ws, where, "ws"), _nbytes(ws) if ws_bytes is None else int(ws_bytes),
        _raw_stream() if stream is None and _raw_stream else _stream(stream))
    if st != QMUON_OK:
        raise QmuonError(st, where)


class AdamwPlan:
    """An owned ``qmuon_adamw_plan*`` (destroyed with the object)."""

    def __init__(self, handle: int, keepalive):
        self.handle = handle
        self._keep = keepalive

    def __del__(self):
        qmuon_adamw_plan_destroy(self)


def adamw_tensor(param, grad, m, v, numel: int, grad_dtype="bf16", m_absmax=None, v_absmax=None, copy=None,
                 copy_dtype="bf16", weight_decay: float = 0.0, lr_scale: float = 1.0) -> qmuon_adamw_tensor:
    """The plan made of it holds these addresses, and is where the types of m and v are checked."""
    n, where = int(numel), "adamw_tensor"
    grad_dtype, copy_dtype = DTYPES.get(grad_dtype, grad_dtype), DTYPES.get(copy_dtype, copy_dtype)
    f32 = _type_of(QMUON_FP32)
    these = (param, grad, copy, m, v)
    t = qmuon_adamw_tensor(_array(param, f32, n, where, "param", these),
                           _array(grad, _types.get(grad_dtype), n, where, "grad", these),
                           None if copy is None else _array(copy, _types.get(copy_dtype), n, where, "copy", these),
                           _array(m, None, n, where, "m", these), _array(v, None, n, where, "v", these),
                           None if m_absmax is None else _array(m_absmax, f32, -(-n // 256), where, "m_absmax"),
                           None if v_absmax is None else _array(v_absmax, f32, -(-n // 256), where, "v_absmax"), n, float(lr_scale),
                           float(weight_decay), grad_dtype, copy_dtype)
    t._keep = (param, grad, copy, m, v, m_absmax, v_absmax)
    return t


def qmuon_adamw_plan_create(tensors: Sequence, state="f32") -> AdamwPlan:
    """``tensors``: ``adamw_tensor(...)``; ``state``: "f32" or "e4m3"."""
    kind = STATE_KINDS.get(state, state)
    held = _type_of(QMUON_FP32) if kind == QMUON_STATE_F32 else None    # None: one byte
    for t in tensors:
        for x in getattr(t, "_keep", ())[3:5]:
            if x is not None and not isinstance(x, int) and (x.dtype is not held if held else x.element_size() != 1):
                _refuse(x, "qmuon_adamw_plan_create", "m" if x is t._keep[3] else "v", f"of {held or 'one byte per element'}")
    arr = (qmuon_adamw_tensor * max(1, len(tensors)))(*tensors)
    out = C.c_void_p()
    st = lib().qmuon_adamw_plan_create(arr, len(tensors), kind, C.byref(out))
    _check(st, "qmuon_adamw_plan_create")
    return AdamwPlan(out.value, tensors)


def qmuon_adamw_plan_destroy(plan: AdamwPlan):
    h, plan.handle = getattr(plan, "handle", None), None
    if h and _lib_handle is not None:
        _lib_handle.qmuon_adamw_plan_destroy(h)


def qmuon_adamw_step(plan: AdamwPlan, t: int, lr: float, beta1: float, beta2: float, eps: float, grad_scale=None,
                     stream=None):
    """``grad_scale``: a device fp32 tensor of one (a clipping coefficient), or None."""
    where = "qmuon_adamw_step"
    scale = None if grad_scale is None else _array(grad_scale, _types.get(QMUON_FP32) or _type_of(QMUON_FP32), 1, where, "grad_scale")
    st = (_lib_handle or lib()).qmuon_adamw_step(plan.handle, int(t), lr, beta1, beta2, eps, scale,
                                                 _raw_stream() if stream is None and _raw_stream else _stream(stream))
    if st != QMUON_OK:
        raise QmuonError(st, where)


def qmuon_adamw_step_sr(plan: AdamwPlan, t: int, lr: float, beta1: float, beta2: float, eps: float, seed: int,
                        grad_scale=None, stream=None):
    where = "qmuon_adamw_step_sr"
    _check(lib().qmuon_adamw_step_sr(plan.handle, int(t), lr, beta1, beta2, eps, int(seed) & 0xFFFFFFFFFFFFFFFF,
                                     _array(grad_scale, _type_of(QMUON_FP32), 1, where, "grad_scale"), _stream(stream)), where)


# The structures as bytes, which take a sixth of a ctypes object's time, and the entries that take them so: most of what
# the checks of the tensors cost a small call comes back here.
_RMSNORM, _RMSNORM_GRAD = struct.Struct("@7Q6qfi").pack, struct.Struct("@6Q6qfi").pack
_bytes_entries: dict = {}


def _by_bytes(name: str):
    fn = lib()[name]    # a function object of its own
    fn.restype, fn.argtypes = C.c_int32, [C.c_char_p, *getattr(lib(), name).argtypes[1:]]
    _bytes_entries[name] = fn
    return fn


def qmuon_rmsnorm_forward(x, gain, rows: int, cols: int, dtype, eps: float, y=None, residual=None, sum=None,
                          payload=None, scale_inv=None, ld_x: Optional[int] = None, ld_residual: Optional[int] = None,
                          ld_sum: Optional[int] = None, ld_y: Optional[int] = None, stream=None):
    """The ``ld_*`` default to ``cols`` (rows next to one another)."""
    where = "qmuon_rmsnorm_forward"
    dtype = DTYPES.get(dtype, dtype)
    t = _types.get(dtype) or _type_of(dtype)
    if ld_x is None:
        ld_x = cols
    if ld_residual is None:
        ld_residual = cols
    if ld_sum is None:
        ld_sum = cols
    if ld_y is None:
        ld_y = cols
    try:
        n = _RMSNORM(_matrix(x, t, rows, cols, ld_x, where, "x"),
                     0 if residual is None else _matrix(residual, t, rows, cols, ld_residual, where, "residual"),
                     _array(gain, _types[QMUON_FP32], cols, where, "gain"),
                     0 if sum is None else _matrix(sum, t, rows, cols, ld_sum, where, "sum"),
                     0 if y is None else _matrix(y, t, rows, cols, ld_y, where, "y"),
                     0 if payload is None else _bytes(payload, rows * cols, where, "payload"),
                     0 if scale_inv is None else _bytes(scale_inv, rows * (cols // 32), where, "scale_inv"), rows, cols, ld_x,
                     ld_residual, ld_sum, ld_y, eps, dtype)
    except (struct.error, OverflowError) as e:
        raise QmuonError(QMUON_ERR_INVALID_ARGUMENT, where, str(e)) from None
    st = (_bytes_entries.get(where) or _by_bytes(where))(n, _raw_stream() if stream is None and _raw_stream else _stream(stream))
    if st != QMUON_OK:
        raise QmuonError(st, where)


def qmuon_rmsnorm_workspace_size(rows: int, cols: int) -> int:
    return int(lib().qmuon_rmsnorm_workspace_size(int(rows), int(cols)))


def qmuon_rmsnorm_backward(dy, h, gain, rows: int, cols: int, dtype, eps: float, dx, dgain, ws, dsum=None,
                           ld_dy: Optional[int] = None, ld_h: Optional[int] = None, ld_dsum: Optional[int] = None,
                           ld_dx: Optional[int] = None, ws_bytes: Optional[int] = None, stream=None):
    where = "qmuon_rmsnorm_backward"
    dtype = DTYPES.get(dtype, dtype)
    t = _types.get(dtype) or _type_of(dtype)
    if ld_dy is None:
        ld_dy = cols
    if ld_h is None:
        ld_h = cols
    if ld_dsum is None:
        ld_dsum = cols
    if ld_dx is None:
        ld_dx = cols
    try:
        n = _RMSNORM_GRAD(_matrix(dy, t, rows, cols, ld_dy, where, "dy"), _matrix(h, t, rows, cols, ld_h, where, "h"),
                          0 if dsum is None else _matrix(dsum, t, rows, cols, ld_dsum, where, "dsum"),
                          _array(gain, _types[QMUON_FP32], cols, where, "gain"), _matrix(dx, t, rows, cols, ld_dx, where, "dx"),
                          _array(dgain, _types[QMUON_FP32], cols, where, "dgain"), rows, cols, ld_dy, ld_h, ld_dsum, ld_dx, eps,
                          dtype)
    except (struct.error, OverflowError) as e:
        raise QmuonError(QMUON_ERR_INVALID_ARGUMENT, where, str(e)) from None
    st = (_bytes_entries.get(where) or _by_bytes(where))(
        n, _on_gpu(ws, where, "ws"), _nbytes(ws) if ws_bytes is None else int(ws_bytes),
        _raw_stream() if stream is None and _raw_stream else _stream(stream))
    if st != QMUON_OK:
        raise QmuonError(st, where)
