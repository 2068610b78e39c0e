"""Thin Python binding of the C ABI in include/saf.h (ctypes).

The functions here have the C names and only marshal arguments: torch CUDA
tensors become device pointers, the current torch stream becomes the
cudaStream_t, and a nonzero status becomes SafError. Every step of the layer
runs in the CUDA library; if libsaf.so is missing, importing this module
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsaf.so")

SAF_BF16 = 0
SAF_FP32 = 1

SAF_OK = 0
SAF_EINVAL = -1
SAF_EALIGN = -2
SAF_EUNSUPPORTED = -3
SAF_ELAUNCH = -4
SAF_EWORKSPACE = -5
SAF_ETIMEOUT = -6
SAF_ECUDA = -8
SAF_ESCRATCH = -9
SAF_EPAGE = -10

# Every symbol that include/saf.h declares.
EXPORTED = ("saf_attn_workspace_bytes", "saf_attn_fwd", "saf_attn_bwd", "saf_device_status",
            "saf_error_string", "saf_version", "saf_set_trace_events", "saf_launch_count",
            "saf_attn_fwd_noalloc", "saf_fit_workspace_bytes", "saf_fit_compact",
            "saf_pattern_grad", "saf_attn_fwd_gqa", "saf_attn_bwd_gqa", "saf_fit_stats_workspace_bytes",
            "saf_fit_target_stats", "saf_fit_from_target_workspace_bytes", "saf_fit_from_target",
            "saf_attn_fwd_diag", "saf_frozen_state_bytes", "saf_frozen_prepare", "saf_attn_fwd_prepared",
            "saf_attn_bwd_prepared", "saf_pattern_grad_tc_workspace_bytes", "saf_pattern_grad_tc",
            "saf_attn_fwd_window", "saf_attn_bwd_window", "saf_kv_append", "saf_attn_paged_workspace_bytes",
            "saf_attn_paged", "saf_attn_paged_shared", "saf_kv_append_quant", "saf_kv_read_quant",
            "saf_attn_paged_quant_workspace_bytes", "saf_attn_paged_quant", "saf_attn_paged_shared_quant")

SAF_KERNEL_NONE = 0
SAF_KERNEL_LOGNORM = 1
SAF_KERNEL_FWD = 2
SAF_KERNEL_BWD_DELTA = 3
SAF_KERNEL_BWD_KV = 4
SAF_KERNEL_BWD_Q = 5
SAF_KERNEL_BWD = 6
SAF_KERNEL_DQ_FINISH = 7
SAF_KERNEL_PATTERN_PREP = 8
SAF_KERNEL_PATTERN_GRAD = 9
SAF_KERNEL_KV_APPEND = 10
SAF_KERNEL_PAGED = 11
SAF_KERNEL_KV_READ = 12


class SafError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status} ({_lib.saf_error_string(status).decode()})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m softmax_attention_hybrid_gb300.build_lib`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.saf_attn_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.saf_attn_workspace_bytes.restype = sz
    lib.saf_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_fwd.restype = i
    lib.saf_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp, vp, vp]
    lib.saf_attn_fwd_noalloc.restype = i
    lib.saf_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.saf_fit_stats_workspace_bytes.restype = sz
    lib.saf_fit_stats_workspace_bytes.argtypes = [i, i]
    lib.saf_fit_target_stats.restype = i
    lib.saf_fit_target_stats.argtypes = [vp, i, i, vp, vp, vp, vp, sz, vp]
    lib.saf_fit_from_target_workspace_bytes.restype = sz
    lib.saf_fit_from_target_workspace_bytes.argtypes = [i, i]
    lib.saf_fit_from_target.restype = i
    lib.saf_fit_from_target.argtypes = [vp, i, i, i, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp]
    lib.saf_frozen_state_bytes.restype = sz
    lib.saf_frozen_state_bytes.argtypes = [i, i, i]
    lib.saf_frozen_prepare.restype = i
    lib.saf_frozen_prepare.argtypes = [vp, vp, i, vp, i, i, i, vp, sz, vp]
    lib.saf_attn_fwd_prepared.restype = i
    lib.saf_attn_fwd_prepared.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_bwd_prepared.restype = i
    lib.saf_attn_bwd_prepared.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, vp, vp, vp,
                                          vp, sz, vp]
    lib.saf_attn_fwd_diag.restype = i
    lib.saf_attn_fwd_diag.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp, vp, vp, sz, vp, i,
                                      ctypes.c_uint]
    lib.saf_attn_fwd_gqa.restype = i
    lib.saf_attn_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_bwd_gqa.restype = i
    lib.saf_attn_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.saf_attn_bwd.restype = i
    lib.saf_device_status.argtypes = [vp, vp]
    lib.saf_device_status.restype = i
    lib.saf_error_string.argtypes = [i]
    lib.saf_error_string.restype = ctypes.c_char_p
    lib.saf_version.argtypes = []
    lib.saf_version.restype = i
    lib.saf_set_trace_events.argtypes = [i, vp, vp]
    lib.saf_set_trace_events.restype = i
    lib.saf_launch_count.argtypes = []
    lib.saf_launch_count.restype = ctypes.c_ulonglong
    lib.saf_fit_workspace_bytes.argtypes = [i, i]
    lib.saf_fit_workspace_bytes.restype = sz
    lib.saf_fit_compact.argtypes = [vp, vp, i, i, i, ctypes.c_float, vp, vp, vp, vp, sz, vp]
    lib.saf_fit_compact.restype = i
    lib.saf_pattern_grad.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, vp, vp, vp]
    lib.saf_pattern_grad.restype = i
    lib.saf_pattern_grad_tc_workspace_bytes.argtypes = [i, i, i, i]
    lib.saf_pattern_grad_tc_workspace_bytes.restype = sz
    lib.saf_pattern_grad_tc.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_pattern_grad_tc.restype = i
    lib.saf_attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_fwd_window.restype = i
    lib.saf_attn_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i, vp, vp, vp,
                                        vp, sz, vp]
    lib.saf_attn_bwd_window.restype = i
    lib.saf_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, vp, i, i, ctypes.c_int64, vp, i, i, i, i, i, i, i, i,
                                  vp, vp, vp, vp, vp]
    lib.saf_kv_append.restype = i
    lib.saf_attn_paged_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.saf_attn_paged_workspace_bytes.restype = sz
    lib.saf_attn_paged.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, i, i, i, i, vp, vp,
                                   vp, sz, vp]
    lib.saf_attn_paged.restype = i
    lib.saf_attn_paged_shared.argtypes = [vp, vp, vp, vp, i, vp, i, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, i, i,
                                          i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_paged_shared.restype = i
    lib.saf_kv_append_quant.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, vp, i, i, ctypes.c_int64, vp, i, i, i, i, i, i,
                                       i, i, vp, vp, vp, vp, vp, vp, vp]
    lib.saf_kv_append_quant.restype = i
    lib.saf_kv_read_quant.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, vp, vp, vp, vp]
    lib.saf_kv_read_quant.restype = i
    lib.saf_attn_paged_quant_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.saf_attn_paged_quant_workspace_bytes.restype = sz
    lib.saf_attn_paged_quant.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, i, i,
                                        i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_paged_quant.restype = i
    lib.saf_attn_paged_shared_quant.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, i, vp, vp, vp, vp, i, vp, i, i, i, i, i,
                                               i, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.saf_attn_paged_shared_quant.restype = i
    return lib


_lib = _load()


def library():
    """The loaded ctypes handle of libsaf.so."""
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SAF_BF16
    if t.dtype == torch.float32:
        return SAF_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _frozen_bytes(frozen, H):
    if frozen is None:
        return None
    vals = [1 if int(x) else 0 for x in (frozen.tolist() if torch.is_tensor(frozen) else frozen)]
    if len(vals) != H:
        raise ValueError("frozen mask must have H entries")
    return (ctypes.c_uint8 * H)(*vals)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def saf_error_string(status: int) -> str:
    return _lib.saf_error_string(int(status)).decode()


def saf_version() -> int:
    return _lib.saf_version()


def saf_attn_workspace_bytes(B, H, T, d, dtype, backward) -> int:
    dt = SAF_BF16 if dtype in (torch.bfloat16, SAF_BF16, "bf16") else SAF_FP32
    return int(_lib.saf_attn_workspace_bytes(int(B), int(H), int(T), int(d), dt, 1 if backward else 0))


def alloc_workspace(B, H, T, d, dtype, backward, device="cuda"):
    """A workspace buffer for saf_attn_fwd / saf_attn_bwd (256-byte aligned by torch)."""
    n = saf_attn_workspace_bytes(B, H, T, d, dtype, backward)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def saf_attn_fwd(q, k, v, a, r, frozen, o=None, lse=None, workspace=None, stream=None):
    """Forward pass; returns (o, lse). q, k, v: [B, H, T, d] CUDA tensors;
    a, r: [H, ld_prior] fp32 CUDA tensors (or None when nothing is frozen);
    frozen: H flags (list or tensor, read on the host)."""
    B, H, T, d = v.shape
    if o is None:
        o = torch.empty_like(v)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, False, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), int(ld), _frozen_bytes(frozen, H),
                           B, H, T, d, _dt(v), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                           _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_fwd")
    return o, lse


def saf_attn_fwd_diag(q, k, v, a, r, frozen, withhold, wait_limit_us, o=None, lse=None, workspace=None,
                      stream=None):
    """Diagnostic forward for testing failure detection: with withhold=1 the
    kernel's producer publishes no work item and every bounded wait expires
    after wait_limit_us; returns (o, lse, workspace). Read the result with
    saf_device_status(workspace)."""
    B, H, T, d = v.shape
    if o is None:
        o = torch.empty_like(v)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, False, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_fwd_diag(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), int(ld), _frozen_bytes(frozen, H),
                                B, H, T, d, _dt(v), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                _stream(stream), int(withhold), int(wait_limit_us))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_fwd_diag")
    return o, lse, workspace


def saf_attn_fwd_noalloc(q, k, v, a, r, frozen, o=None, lse=None, stream=None):
    """Forward pass without a workspace, for callers that cannot allocate
    device memory: the library uses its fixed 8 MiB device scratch instead.
    Same outputs as saf_attn_fwd; raises SafError (SAF_ESCRATCH) when the
    problem does not fit. Calls on one device share that scratch, so they
    must be ordered on one stream."""
    B, H, T, d = v.shape
    if o is None:
        o = torch.empty_like(v)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), int(ld), _frozen_bytes(frozen, H),
                                   B, H, T, d, _dt(v), _ptr(o), _ptr(lse), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_fwd_noalloc")
    return o, lse


def saf_attn_bwd(q, k, v, o, do, lse, a, r, frozen, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward pass; returns (dq, dk, dv)."""
    B, H, T, d = v.shape
    dq = torch.empty_like(v) if dq is None else dq
    dk = torch.empty_like(v) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, True, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(a), _ptr(r), int(ld),
                           _frozen_bytes(frozen, H), B, H, T, d, _dt(v), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_bwd")
    return dq, dk, dv


def _gqa_shape(q, v, frozen):
    B, Hkv, T, d = v.shape
    if q is not None:
        H = q.shape[1]
    elif frozen is not None:
        H = len(frozen)
    else:
        raise ValueError("q is needed unless the frozen mask gives H")
    return B, H, Hkv, T, d


def saf_attn_fwd_gqa(q, k, v, a, r, frozen, o=None, lse=None, workspace=None, stream=None):
    """Grouped-query forward; returns (o, lse). q: [B, H, T, d]; k, v:
    [B, Hkv, T, d] with H a multiple of Hkv (query head h reads key/value head
    h // (H // Hkv)); a, r, frozen per query head, as for saf_attn_fwd."""
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    if o is None:
        o = torch.empty((B, H, T, d), dtype=v.dtype, device=v.device)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, False, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), int(ld), _frozen_bytes(frozen, H),
                               B, H, Hkv, T, d, _dt(v), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                               _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_fwd_gqa")
    return o, lse


def saf_attn_bwd_gqa(q, k, v, o, do, lse, a, r, frozen, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Grouped-query backward; returns dq [B, H, T, d] and dk, dv [B, Hkv, T, d]
    (a shared head's gradient is the sum over its query heads)."""
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    dq = torch.empty((B, H, T, d), dtype=v.dtype, device=v.device) if dq is None else dq
    dk = torch.empty_like(v) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, True, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(a), _ptr(r), int(ld),
                               _frozen_bytes(frozen, H), B, H, Hkv, T, d, _dt(v), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_bwd_gqa")
    return dq, dk, dv


def saf_frozen_prepare(a, r, frozen, T, dtype, state=None, stream=None):
    """Fill (and return) the prepared frozen-pattern state of a, r ([H, ld_prior]
    fp32 CUDA tensors) for sequences of length T in `dtype`."""
    H = a.shape[0]
    dt = SAF_BF16 if dtype in (torch.bfloat16, SAF_BF16, "bf16") else SAF_FP32
    n = int(_lib.saf_frozen_state_bytes(H, int(T), dt))
    if state is None:
        state = torch.empty(max(n, 256), dtype=torch.uint8, device=a.device)
    st = _lib.saf_frozen_prepare(_ptr(a), _ptr(r), int(a.shape[1]), _frozen_bytes(frozen, H), H, int(T), dt,
                                 _ptr(state), state.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_frozen_prepare")
    return state


def _state(state, H, T, dt):
    """The prepared state, which the kernels read by the sizes of the call."""
    if state is not None and state.numel() * state.element_size() < _lib.saf_frozen_state_bytes(H, T, dt):
        raise ValueError(f"the prepared state is shorter than one of {H} heads and {T} tokens")
    return state


def saf_attn_fwd_prepared(q, k, v, a, r, frozen, state, o=None, lse=None, workspace=None, stream=None):
    """Forward with the frozen-pattern data from a prepared state (grouped-query
    shapes allowed: k, v [B, Hkv, T, d]); returns (o, lse)."""
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    if o is None:
        o = torch.empty((B, H, T, d), dtype=v.dtype, device=v.device)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, False, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_fwd_prepared(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), int(ld), _frozen_bytes(frozen, H),
                                    _ptr(_state(state, H, T, _dt(v))), B, H, Hkv, T, d, _dt(v), _ptr(o), _ptr(lse),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_fwd_prepared")
    return o, lse


def saf_attn_bwd_prepared(q, k, v, o, do, lse, a, r, frozen, state, dq=None, dk=None, dv=None, workspace=None,
                          stream=None):
    """Backward with the frozen-pattern data from a prepared state; returns (dq, dk, dv)."""
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    dq = torch.empty((B, H, T, d), dtype=v.dtype, device=v.device) if dq is None else dq
    dk = torch.empty_like(v) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, v.dtype, True, v.device)
    ld = a.shape[1] if a is not None else T
    st = _lib.saf_attn_bwd_prepared(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(a), _ptr(r),
                                    int(ld), _frozen_bytes(frozen, H), _ptr(_state(state, H, T, _dt(v))), B, H, Hkv,
                                    T, d, _dt(v), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
                                    _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_attn_bwd_prepared")
    return dq, dk, dv


# The calls below are short enough on the GPU that their checks in Python count: what every call
# has is checked in one expression, and what is wrong is named on a second look (_at).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_F32, _I32, _U8, _E4M3 = torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_I64x9 = ctypes.c_int64 * 9
_2G, _8E = 2 ** 31, 2 ** 63   # ctypes would cut a larger int to its low 32 (64) bits


def _fits(top=_2G, **given):
    """Raise for the first of the given numbers that a C integer of [-top, top) does not hold."""
    for name, x in given.items():
        if not -top <= x < top:
            raise ValueError(f"{name} = {x} is out of range")


def _at(t, idx, dtype):
    """Address of an optional contiguous tensor of `dtype` on device `idx`."""
    if t is None:
        return None
    if t.get_device() != idx or t.dtype is not dtype or not t.is_contiguous():
        _refuse(t, idx, dtype)
    return t.data_ptr()


def _refuse(t, idx, dtype):
    if t.get_device() != idx:
        raise ValueError(f"a tensor of shape {tuple(t.shape)} must live on cuda:{idx}")
    if t.dtype is not dtype:
        raise TypeError(f"a tensor of shape {tuple(t.shape)} must be {dtype}, got {t.dtype}")
    raise ValueError(f"a tensor of shape {tuple(t.shape)} must be contiguous")


def _device(t):
    idx = t.get_device()
    if idx < 0:
        raise ValueError("tensor must live on a CUDA device")
    return idx


def _shapes(*given):
    """Raise for the first (name, tensor or None, shape) whose shape is another."""
    for name, t, shape in given:
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _flags(frozen, H):
    """The frozen flags as H bytes; a bytes object is passed on as it is."""
    if frozen is None:
        return None
    if type(frozen) is bytes:
        if len(frozen) != H:
            raise ValueError("frozen mask must have H entries")
        return frozen
    return bytes(_frozen_bytes(frozen, H))


def _run(where, fn, idx, *args):
    """fn(*args, stream) with device `idx` current, on its current stream."""
    if _get_device() != idx:
        with torch.cuda.device(idx):
            return _run(where, fn, idx, *args)
    raw = _raw_stream(idx) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    st = fn(*args, raw)
    if st != SAF_OK:
        raise SafError(st, where)


def _on(stream, t, call):
    """call() on `stream`, of t's device: what the call allocates and clears belongs to that stream."""
    if stream.device != t.device:
        raise ValueError("stream and tensors must be of one device")
    with torch.cuda.stream(stream):
        return call()


def _prior(a, r, H, idx, none):
    """Addresses and row length of a, r ([H, ld_prior] fp32, or None when nothing is frozen)."""
    if a is None or r is None:
        return None, None, none
    shape = a.shape
    if len(shape) != 2 or shape[0] != H or r.shape != shape:
        raise ValueError("a and r must both be [H, ld_prior]")
    return _at(a, idx, torch.float32), _at(r, idx, torch.float32), shape[1]


def saf_attn_fwd_window(q, k, v, a, r, frozen, window, sinks=0, state=None, o=None, lse=None, workspace=None,
                        stream=None):
    """Forward of the layer whose ordinary heads see the last `window` keys and the first
    `sinks` (query i: keys j <= i with i - j < window or j < sinks; window 0: every key);
    returns (o, lse). q: [B, H, T, d]; k, v: [B, Hkv, T, d]; a, r, frozen as for
    saf_attn_fwd_gqa; state: a prepared frozen-pattern state (saf_frozen_prepare) or None."""
    if stream is not None:
        return _on(stream, v, lambda: saf_attn_fwd_window(q, k, v, a, r, frozen, window, sinks, state, o,
                   lse, workspace))
    if not (-_2G <= window < _2G and -_2G <= sinks < _2G):
        _fits(window=window, sinks=sinks)
    idx, dt = _device(v), v.dtype
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    full, rows = (B, H, T, d), (B, H, T)
    if ((q is not None and q.shape != full) or (k is not None and k.shape != v.shape)
            or (o is not None and o.shape != full) or (lse is not None and lse.shape != rows)):
        _shapes(("q", q, full), ("k", k, v.shape), ("o", o, full), ("lse", lse, rows))
    if o is None:
        o = torch.empty(full, dtype=dt, device=v.device)
    if lse is None:
        lse = torch.empty(rows, dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, dt, False, v.device)
    ap, rp, ld = _prior(a, r, H, idx, T)
    _run("saf_attn_fwd_window", _lib.saf_attn_fwd_window, idx, _at(q, idx, dt), _at(k, idx, dt),
         _at(v, idx, dt), ap, rp, ld, _flags(frozen, H), _at(_state(state, H, T, _dt(v)), idx, torch.uint8),
         int(window), int(sinks), B, H, Hkv, T, d, _dt(v), _at(o, idx, dt), _at(lse, idx, torch.float32),
         _at(workspace, idx, torch.uint8), workspace.numel())
    return o, lse


def saf_attn_bwd_window(q, k, v, o, do, lse, a, r, frozen, window, sinks=0, state=None, dq=None, dk=None, dv=None,
                        workspace=None, stream=None):
    """Backward of saf_attn_fwd_window (o, lse: its outputs for the same inputs); returns
    dq [B, H, T, d] and dk, dv [B, Hkv, T, d]."""
    if stream is not None:
        return _on(stream, v, lambda: saf_attn_bwd_window(q, k, v, o, do, lse, a, r, frozen, window, sinks,
                   state, dq, dk, dv, workspace))
    if not (-_2G <= window < _2G and -_2G <= sinks < _2G):
        _fits(window=window, sinks=sinks)
    idx, dt = _device(v), v.dtype
    B, H, Hkv, T, d = _gqa_shape(q, v, frozen)
    full, kv = (B, H, T, d), v.shape
    _shapes(("q", q, full), ("k", k, kv), ("o", o, full), ("do", do, full), ("lse", lse, (B, H, T)),
            ("dq", dq, full), ("dk", dk, kv), ("dv", dv, kv))
    dq = torch.empty(full, dtype=dt, device=v.device) if dq is None else dq
    dk = torch.empty(kv, dtype=dt, device=v.device) if dk is None else dk
    dv = torch.empty(kv, dtype=dt, device=v.device) if dv is None else dv
    if workspace is None:
        workspace = alloc_workspace(B, H, T, d, dt, True, v.device)
    ap, rp, ld = _prior(a, r, H, idx, T)
    _run("saf_attn_bwd_window", _lib.saf_attn_bwd_window, idx, _at(q, idx, dt), _at(k, idx, dt),
         _at(v, idx, dt), _at(o, idx, dt), _at(do, idx, dt), _at(lse, idx, torch.float32), ap, rp, ld,
         _flags(frozen, H), _at(_state(state, H, T, _dt(v)), idx, torch.uint8), int(window), int(sinks), B, H, Hkv,
         T, d, _dt(v), _at(dq, idx, dt),
         _at(dk, idx, dt), _at(dv, idx, dt), _at(workspace, idx, torch.uint8), workspace.numel())
    return dq, dk, dv


def _strided(t, idx, dt):
    """Address and (sequence, head, token) strides of a [B, heads, T, d] tensor with contiguous rows."""
    s = t.stride()
    if t.get_device() != idx or t.dtype is not dt:
        _refuse(t, idx, dt)
    if s[3] != 1:
        raise ValueError(f"a tensor of shape {tuple(t.shape)} must have contiguous rows")
    return t.data_ptr(), s[:3]


def _table(ctx, n_new, page_table, B):
    """max_pages, after the shapes of the counts and the page table of B sequences."""
    shape = page_table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    if ctx.shape != (B,) or (n_new is not None and n_new.shape != (B,)):
        raise ValueError("ctx and n_new must be [B]")
    return shape[1]


def saf_kv_append(k, v, k_cache, v_cache, page_table, ctx, n_new=None, q=None, q_out=None, inv_freq=None,
                  interleaved=False, pos_base=0, frozen=None, status=None, stream=None):
    """Write the new tokens' k, v [B, Hkv, T, d] (any strides with contiguous rows) into the
    paged caches [num_pages, Hkv, page_size, d] at slots ctx[b] + t of page_table [B, max_pages],
    with the rotary rotation of k, and of q [B, H, T, d] into q_out; returns q_out (None
    without q). ctx, n_new: int32 [B] on the device (n_new None: T tokens each).
    inv_freq: rope_dim / 2 angles per position (CPU float64 tensor or a sequence; None: no
    rotation). frozen: flags of the H query heads (their q, and keys that no ordinary head
    reads, are left alone); without q it also gives H (default Hkv). status: a CUDA tensor
    whose first 8 bytes, zeroed once by the caller, collect errors for saf_device_status
    (None: errors are not recorded)."""
    if stream is not None:
        return _on(stream, v, lambda: saf_kv_append(k, v, k_cache, v_cache, page_table, ctx, n_new, q,
                   q_out, inv_freq, interleaved, pos_base, frozen, status))
    if not -_8E <= pos_base < _8E:
        _fits(_8E, pos_base=pos_base)
    idx, dt, i32 = _device(v), v.dtype, torch.int32
    shape, caches = v.shape, v_cache.shape
    B, Hkv, T, d = shape
    num_pages, heads, page_size, width = caches
    max_pages = _table(ctx, n_new, page_table, B)
    if heads != Hkv or width != d or (k_cache is not None and k_cache.shape != caches):
        raise ValueError("the caches must be [num_pages, Hkv, page_size, d]")
    if k is not None and k.shape != shape:
        raise ValueError("k must have v's shape")
    if q is not None:
        full = q.shape
        H = full[1]
        if full[0] != B or full[2] != T or full[3] != d:
            raise ValueError("q must be [B, H, T, d]")
        if q_out is None:
            # rows that are not written (frozen heads, rows without a token) come back as zeros
            q_out = torch.zeros(full, dtype=dt, device=v.device)
        elif q_out.shape != full:
            raise ValueError("q_out must have q's shape")
        qp, (qb, qh, qt) = _strided(q, idx, dt)
        qo = _at(q_out, idx, dt)
    else:
        H = len(frozen) if frozen is not None else Hkv
        qp = qo = None
        qb = qh = qt = 0
    if k is not None:
        kp, (kb, kh, kt) = _strided(k, idx, dt)
    else:
        kp, kb, kh, kt = None, 0, 0, 0
    vp, (vb, vh, vt) = _strided(v, idx, dt)
    freq, rope = None, 0
    if inv_freq is not None:
        if not (torch.is_tensor(inv_freq) and inv_freq.dtype is torch.float64 and inv_freq.get_device() < 0
                and inv_freq.is_contiguous()):
            inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
        rope = 2 * inv_freq.numel()
        freq = inv_freq.data_ptr() if rope else None
    if status is not None and status.numel() * status.element_size() < 8:
        raise ValueError("status needs 8 bytes")
    _run("saf_kv_append", _lib.saf_kv_append, idx, qp, kp, vp, _I64x9(qb, qh, qt, kb, kh, kt, vb, vh, vt),
         _at(ctx, idx, i32), _at(n_new, idx, i32), _at(page_table, idx, i32), max_pages, freq, rope,
         1 if interleaved else 0, pos_base, _flags(frozen, H), B, H, Hkv, T, d, num_pages, page_size, _dt(v), qo,
         _at(k_cache, idx, dt), _at(v_cache, idx, dt), None if status is None else _at(status, idx, status.dtype))
    return q_out


def saf_attn_paged_workspace_bytes(B, H, Hkv, T, d, max_len, dtype, prefix_len=0) -> int:
    dt = SAF_BF16 if dtype in (torch.bfloat16, SAF_BF16, "bf16") else SAF_FP32
    if not all(-_2G <= n < _2G for n in (B, H, Hkv, T, d, max_len, prefix_len)):
        return 0
    return int(_lib.saf_attn_paged_workspace_bytes(B, H, Hkv, T, d, int(max_len), int(prefix_len), dt))


def alloc_paged_workspace(B, H, Hkv, T, d, max_len, dtype, prefix_len=0, device="cuda"):
    """A workspace for saf_attn_paged / saf_attn_paged_shared with cleared status words (for these
    sizes: a smaller batch may need a larger one)."""
    n = saf_attn_paged_workspace_bytes(B, H, Hkv, T, d, max_len, dtype, prefix_len)
    w = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    w[:256].zero_()
    return w


def saf_attn_paged_quant_workspace_bytes(B, H, Hkv, T, d, max_len, dtype, prefix_len=0) -> int:
    dt = SAF_BF16 if dtype in (torch.bfloat16, SAF_BF16, "bf16") else SAF_FP32
    if not all(-_2G <= n < _2G for n in (B, H, Hkv, T, d, max_len, prefix_len)):
        return 0
    return int(_lib.saf_attn_paged_quant_workspace_bytes(B, H, Hkv, T, d, int(max_len), int(prefix_len), dt))


def alloc_paged_quant_workspace(B, H, Hkv, T, d, max_len, dtype, prefix_len=0, device="cuda"):
    """alloc_paged_workspace for saf_attn_paged_quant / saf_attn_paged_shared_quant (dtype: q's)."""
    n = saf_attn_paged_quant_workspace_bytes(B, H, Hkv, T, d, max_len, dtype, prefix_len)
    w = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    w[:256].zero_()
    return w


def _scales(k_scale, v_scale, caches, idx):
    """Addresses of the scales of 8-bit caches of shape `caches`."""
    if v_scale.shape != caches[:3] or (k_scale is not None and k_scale.shape != caches[:3]):
        raise ValueError("the scales must be [num_pages, Hkv, page_size]")
    return _at(k_scale, idx, _F32), _at(v_scale, idx, _F32)


def _paged(where, fn, q, k_cache, v_cache, prefix, P, page_table, ctx, max_len, n_new, a, r, frozen, window, sinks, o,
           lse, workspace, scales=None):
    # scales: those of 8-bit caches, (k_scale, v_scale)
    if not (-_2G <= window < _2G and -_2G <= sinks < _2G and -_2G <= max_len < _2G):
        _fits(window=window, sinks=sinks, max_len=max_len)
    idx, dt = _device(q), q.dtype
    full, caches, table = q.shape, v_cache.shape, page_table.shape
    B, H, T, d = full
    num_pages, Hkv, page_size, width = caches
    if width != d or (k_cache is not None and k_cache.shape != caches):
        raise ValueError("the caches must both be [num_pages, Hkv, page_size, d]")
    if len(table) != 2 or table[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    if ctx.shape != (B,) or (n_new is not None and n_new.shape != (B,)):
        raise ValueError("ctx and n_new must be [B]")
    if o is None:
        o = torch.empty(full, dtype=dt, device=q.device)
    if lse is None:
        lse = torch.empty(full[:3], dtype=_F32, device=q.device)
    if o.shape != full or lse.shape != full[:3]:
        raise ValueError(f"o and lse must have shapes {tuple(full)} and {tuple(full[:3])}")
    cdt, at_scales = dt, ()
    if scales is not None:
        cdt, at_scales = _E4M3, _scales(*scales, caches, idx)
    if workspace is None:
        alloc = alloc_paged_workspace if scales is None else alloc_paged_quant_workspace
        workspace = alloc(B, H, Hkv, T, d, max_len, dt, P, q.device)
    if not (idx == v_cache.get_device() == page_table.get_device() == ctx.get_device() == o.get_device()
            == lse.get_device() == workspace.get_device()
            and cdt is v_cache.dtype and dt is o.dtype and lse.dtype is _F32 and page_table.dtype is _I32
            and ctx.dtype is _I32 and workspace.dtype is _U8
            and q.is_contiguous() and v_cache.is_contiguous() and page_table.is_contiguous() and ctx.is_contiguous()
            and o.is_contiguous() and lse.is_contiguous() and workspace.is_contiguous()):
        for t, want in ((q, dt), (v_cache, cdt), (page_table, _I32), (ctx, _I32), (o, dt), (lse, _F32), (workspace, _U8)):
            _at(t, idx, want)
    ap, rp, ld = _prior(a, r, H, idx, P + max_len)
    _run(where, fn, idx, q.data_ptr(), _at(k_cache, idx, cdt), v_cache.data_ptr(), *at_scales, *prefix,
         page_table.data_ptr(), table[1], ctx.data_ptr(), _at(n_new, idx, _I32), ap, rp, ld,
         _flags(frozen, H), int(window), int(sinks), B, H, Hkv, T, d, max_len, num_pages, page_size, _dt(q),
         o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return o, lse


def saf_attn_paged(q, k_cache, v_cache, page_table, ctx, max_len, n_new=None, a=None, r=None, frozen=None, window=0,
                   sinks=0, o=None, lse=None, workspace=None, stream=None):
    """Attention of the newest tokens q [B, H, T, d] over the paged caches
    [num_pages, Hkv, page_size, d]; returns (o, lse). Token t of sequence b stands at position
    ctx[b] + t; rows t >= n_new[b] come back as o = 0, lse = -inf. max_len: an upper bound of
    ctx[b] + n_new[b]. a, r [H, ld_prior >= max_len] and frozen as for saf_attn_fwd; window and
    sinks as for saf_attn_fwd_window. workspace: alloc_paged_workspace."""
    if stream is not None:
        return _on(stream, q, lambda: saf_attn_paged(q, k_cache, v_cache, page_table, ctx, max_len, n_new,
                   a, r, frozen, window, sinks, o, lse, workspace))
    return _paged("saf_attn_paged", _lib.saf_attn_paged, q, k_cache, v_cache, (), 0, page_table, ctx, max_len, n_new, a,
                  r, frozen, window, sinks, o, lse, workspace)


def saf_attn_paged_shared(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, ctx, max_len, n_new=None, a=None,
                          r=None, frozen=None, window=0, sinks=0, o=None, lse=None, workspace=None, stream=None):
    """saf_attn_paged for sequences that share a prefix of prefix_len tokens, held once in the
    pages prefix_pages (int32, on the device): token t of sequence b stands at position
    prefix_len + ctx[b] + t, and ctx, n_new, max_len and page_table count own tokens."""
    if stream is not None:
        return _on(stream, q, lambda: saf_attn_paged_shared(q, k_cache, v_cache, prefix_pages, prefix_len,
                   page_table, ctx, max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace))
    if not -_2G <= prefix_len < _2G:
        _fits(prefix_len=prefix_len)
    if prefix_pages is not None and prefix_pages.numel() * v_cache.shape[2] < prefix_len:
        raise ValueError("prefix_pages holds fewer pages than prefix_len tokens take")
    prefix = (_at(prefix_pages, _device(q), torch.int32), prefix_len)
    return _paged("saf_attn_paged_shared", _lib.saf_attn_paged_shared, q, k_cache, v_cache, prefix, prefix_len,
                  page_table, ctx, max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace)


def saf_kv_append_quant(k, v, k_cache, v_cache, k_scale, v_scale, page_table, ctx, n_new=None, q=None, q_out=None,
                       inv_freq=None, interleaved=False, pos_base=0, frozen=None, status=None, stream=None):
    """saf_kv_append into 8-bit caches: k_cache, v_cache [num_pages, Hkv, page_size, d] of
    torch.float8_e4m3fn with fp32 scales k_scale, v_scale [num_pages, Hkv, page_size]. A row y is
    held as scale = max(max |y| / 448, 2^-126) and codes y / scale. k, v and q are bf16 or fp32;
    everything else is as for saf_kv_append."""
    if stream is not None:
        return _on(stream, v, lambda: saf_kv_append_quant(k, v, k_cache, v_cache, k_scale, v_scale, page_table, ctx,
                   n_new, q, q_out, inv_freq, interleaved, pos_base, frozen, status))
    if not -_8E <= pos_base < _8E:
        _fits(_8E, pos_base=pos_base)
    idx, dt = _device(v), v.dtype
    shape, caches = v.shape, v_cache.shape
    B, Hkv, T, d = shape
    num_pages, heads, page_size, width = caches
    max_pages = _table(ctx, n_new, page_table, B)
    if heads != Hkv or width != d or (k_cache is not None and k_cache.shape != caches):
        raise ValueError("the caches must be [num_pages, Hkv, page_size, d]")
    ks, vs = _scales(k_scale, v_scale, caches, idx)
    if k is not None and k.shape != shape:
        raise ValueError("k must have v's shape")
    qp = qo = kp = None
    q_strides = k_strides = (0, 0, 0)
    if q is not None:
        full = q.shape
        H = full[1]
        if full[0] != B or full[2] != T or full[3] != d:
            raise ValueError("q must be [B, H, T, d]")
        if q_out is None:
            # rows that are not written (frozen heads, rows without a token) come back as zeros
            q_out = torch.zeros(full, dtype=dt, device=v.device)
        elif q_out.shape != full:
            raise ValueError("q_out must have q's shape")
        qp, q_strides = _strided(q, idx, dt)
        qo = _at(q_out, idx, dt)
    else:
        H = len(frozen) if frozen is not None else Hkv
    if k is not None:
        kp, k_strides = _strided(k, idx, dt)
    vp, v_strides = _strided(v, idx, dt)
    freq, rope = None, 0
    if inv_freq is not None:
        if not (torch.is_tensor(inv_freq) and inv_freq.dtype is torch.float64 and inv_freq.get_device() < 0
                and inv_freq.is_contiguous()):
            inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
        rope = 2 * inv_freq.numel()
        freq = inv_freq.data_ptr() if rope else None
    if status is not None and status.numel() * status.element_size() < 8:
        raise ValueError("status needs 8 bytes")
    _run("saf_kv_append_quant", _lib.saf_kv_append_quant, idx, qp, kp, vp, _I64x9(*q_strides, *k_strides, *v_strides),
         _at(ctx, idx, _I32), _at(n_new, idx, _I32), _at(page_table, idx, _I32), max_pages, freq, rope,
         1 if interleaved else 0, pos_base, _flags(frozen, H), B, H, Hkv, T, d, num_pages, page_size, _dt(v), qo,
         _at(k_cache, idx, _E4M3), _at(v_cache, idx, _E4M3), ks, vs,
         None if status is None else _at(status, idx, status.dtype))
    return q_out


def saf_kv_read_quant(k_cache, v_cache, k_scale, v_scale, page_table, first=None, count=None, T=None, dtype=None,
                     k_out=None, v_out=None, status=None, stream=None):
    """Rows of 8-bit caches read back: slots first[b] .. first[b] + count[b] - 1 of each sequence of
    page_table [B, max_pages] as k_out, v_out [B, Hkv, T, d] (bf16 or fp32; rows behind them are
    zeros); returns (k_out, v_out). first, count: int32 [B] on the device (None: 0, and T each).
    T and dtype size the outputs where v_out is not given. k_cache and k_scale may be None
    (values only: k_out is None). status as for saf_kv_append."""
    if stream is not None:
        return _on(stream, v_cache, lambda: saf_kv_read_quant(k_cache, v_cache, k_scale, v_scale, page_table, first,
                   count, T, dtype, k_out, v_out, status))
    idx, caches = _device(v_cache), v_cache.shape
    num_pages, Hkv, page_size, d = caches
    if len(page_table.shape) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    _shapes(("k_cache", k_cache, caches), ("first", first, (B,)), ("count", count, (B,)))
    if k_cache is None and (k_scale is not None or k_out is not None):
        raise ValueError("k_scale and k_out need k_cache")
    if k_cache is not None and k_scale is None:
        raise ValueError("k_cache needs k_scale")
    ks, vs = _scales(k_scale, v_scale, caches, idx)
    if v_out is None:
        if T is None or dtype is None:
            raise ValueError("T and dtype are needed without v_out")
        _fits(T=T)
        v_out = torch.empty((B, Hkv, T, d), dtype=dtype, device=v_cache.device)
    dt, full = v_out.dtype, v_out.shape
    if len(full) != 4 or full[0] != B or full[1] != Hkv or full[3] != d:
        raise ValueError("v_out must be [B, Hkv, T, d]")
    if (T is not None and T != full[2]) or (dtype is not None and dtype != dt):
        raise ValueError("v_out is of another T or dtype")
    if k_cache is not None and k_out is None:
        k_out = torch.empty(full, dtype=dt, device=v_cache.device)
    _shapes(("k_out", k_out, full))
    if status is not None and status.numel() * status.element_size() < 8:
        raise ValueError("status needs 8 bytes")
    _run("saf_kv_read_quant", _lib.saf_kv_read_quant, idx, _at(k_cache, idx, _E4M3), _at(v_cache, idx, _E4M3), ks, vs,
         _at(page_table, idx, _I32), max_pages, _at(first, idx, _I32), _at(count, idx, _I32), B, Hkv, full[2], d,
         num_pages, page_size, _dt(v_out), _at(k_out, idx, dt), _at(v_out, idx, dt),
         None if status is None else _at(status, idx, status.dtype))
    return k_out, v_out


def saf_attn_paged_quant(q, k_cache, v_cache, k_scale, v_scale, page_table, ctx, max_len, n_new=None, a=None, r=None,
                        frozen=None, window=0, sinks=0, o=None, lse=None, workspace=None, stream=None):
    """saf_attn_paged over 8-bit caches (torch.float8_e4m3fn [num_pages, Hkv, page_size, d]) with fp32
    scales [num_pages, Hkv, page_size]; q, o bf16 or fp32. workspace: alloc_paged_quant_workspace."""
    if stream is not None:
        return _on(stream, q, lambda: saf_attn_paged_quant(q, k_cache, v_cache, k_scale, v_scale, page_table, ctx,
                   max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace))
    return _paged("saf_attn_paged_quant", _lib.saf_attn_paged_quant, q, k_cache, v_cache, (), 0, page_table, ctx,
                  max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace, (k_scale, v_scale))


def saf_attn_paged_shared_quant(q, k_cache, v_cache, k_scale, v_scale, prefix_pages, prefix_len, page_table, ctx,
                               max_len, n_new=None, a=None, r=None, frozen=None, window=0, sinks=0, o=None, lse=None,
                               workspace=None, stream=None):
    """saf_attn_paged_shared over 8-bit caches, as saf_attn_paged_quant."""
    if stream is not None:
        return _on(stream, q, lambda: saf_attn_paged_shared_quant(q, k_cache, v_cache, k_scale, v_scale, prefix_pages,
                   prefix_len, page_table, ctx, max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace))
    if not -_2G <= prefix_len < _2G:
        _fits(prefix_len=prefix_len)
    if prefix_pages is not None and prefix_pages.numel() * v_cache.shape[2] < prefix_len:
        raise ValueError("prefix_pages holds fewer pages than prefix_len tokens take")
    prefix = (_at(prefix_pages, _device(q), torch.int32), prefix_len)
    return _paged("saf_attn_paged_shared_quant", _lib.saf_attn_paged_shared_quant, q, k_cache, v_cache, prefix,
                  prefix_len, page_table, ctx, max_len, n_new, a, r, frozen, window, sinks, o, lse, workspace,
                  (k_scale, v_scale))


def saf_set_trace_events(kernel: int, start=None, stop=None) -> None:
    """Record torch.cuda.Event `start`/`stop` around every launch of `kernel`
    (a SAF_KERNEL_* id) from now on; kernel 0 or None events switch it off."""
    sp = ctypes.c_void_p(start.cuda_event) if start is not None else None
    ep = ctypes.c_void_p(stop.cuda_event) if stop is not None else None
    st = _lib.saf_set_trace_events(int(kernel), sp, ep)
    if st != SAF_OK:
        raise SafError(st, "saf_set_trace_events")


def saf_launch_count() -> int:
    return int(_lib.saf_launch_count())


def saf_device_status(workspace, stream=None) -> int:
    return int(_lib.saf_device_status(_ptr(workspace), _stream(stream)))


def saf_fit_workspace_bytes(H, T) -> int:
    return int(_lib.saf_fit_workspace_bytes(int(H), int(T)))


def saf_fit_compact(eta_abs, eta_rel, steps=400, lr=0.05, a=None, r=None, loss=None, workspace=None, stream=None):
    """Fit a, r of Eq. 3 to target marginals eta_abs, eta_rel (fp32 CUDA tensors
    [H, T]); returns (a, r, loss) as fp32 CUDA tensors [H, T], [H, T], [H]."""
    H, T = eta_abs.shape
    dev = eta_abs.device
    a = torch.empty((H, T), dtype=torch.float32, device=dev) if a is None else a
    r = torch.empty((H, T), dtype=torch.float32, device=dev) if r is None else r
    loss = torch.empty((H,), dtype=torch.float32, device=dev) if loss is None else loss
    if workspace is None:
        workspace = torch.empty(max(saf_fit_workspace_bytes(H, T), 256), dtype=torch.uint8, device=dev)
    st = _lib.saf_fit_compact(_ptr(eta_abs), _ptr(eta_rel), H, T, int(steps), float(lr), _ptr(a), _ptr(r),
                              _ptr(loss), _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_fit_compact")
    return a, r, loss


def saf_fit_target_stats(A, stream=None):
    """eta_abs, eta_rel [H, T] and negent [H] of the floored, row-normalised
    targets of A (fp32 CUDA tensor [H, T, T])."""
    H, T, _ = A.shape
    dev = A.device
    ea = torch.empty((H, T), dtype=torch.float32, device=dev)
    er = torch.empty((H, T), dtype=torch.float32, device=dev)
    ng = torch.empty((H,), dtype=torch.float32, device=dev)
    ws = torch.empty(max(int(_lib.saf_fit_stats_workspace_bytes(H, T)), 256), dtype=torch.uint8, device=dev)
    st = _lib.saf_fit_target_stats(_ptr(A), H, T, _ptr(ea), _ptr(er), _ptr(ng), _ptr(ws), ws.numel(),
                                   _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_fit_target_stats")
    return ea, er, ng


def saf_fit_from_target(A, steps=400, lr=0.05, tol=0.2, stream=None):
    """Fit every head of A (fp32 CUDA tensor [H, T, T]) from its measured
    pattern to accept / reject on the device; returns a, r [H, T], kappa [H]
    and accept [H] (uint8)."""
    H, T, _ = A.shape
    dev = A.device
    a = torch.empty((H, T), dtype=torch.float32, device=dev)
    r = torch.empty((H, T), dtype=torch.float32, device=dev)
    kappa = torch.empty((H,), dtype=torch.float32, device=dev)
    accept = torch.empty((H,), dtype=torch.uint8, device=dev)
    ws = torch.empty(max(int(_lib.saf_fit_from_target_workspace_bytes(H, T)), 256), dtype=torch.uint8, device=dev)
    st = _lib.saf_fit_from_target(_ptr(A), H, T, int(steps), float(lr), float(tol), _ptr(a), _ptr(r), _ptr(kappa),
                                  _ptr(accept), _ptr(ws), ws.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_fit_from_target")
    return a, r, kappa, accept


def saf_pattern_grad(v, do, o, lse, a, r, frozen, da=None, dr=None, stream=None):
    """Gradients of a and r of the frozen heads (fp32 CUDA tensors [H, T])."""
    B, H, T, d = v.shape
    da = torch.empty((H, T), dtype=torch.float32, device=v.device) if da is None else da
    dr = torch.empty((H, T), dtype=torch.float32, device=v.device) if dr is None else dr
    st = _lib.saf_pattern_grad(_ptr(v), _ptr(do), _ptr(o), _ptr(lse), _ptr(a), _ptr(r), a.shape[-1],
                               _frozen_bytes(frozen, H), B, H, T, d, _dt(v), _ptr(da), _ptr(dr), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_pattern_grad")
    return da, dr


def saf_pattern_grad_tc_workspace_bytes(B, H, T, n_frozen):
    return int(_lib.saf_pattern_grad_tc_workspace_bytes(B, H, T, n_frozen))


def saf_pattern_grad_tc(v, do, o, lse, a, r, frozen, da=None, dr=None, workspace=None, stream=None):
    """Gradients of a and r of the frozen heads on the tensor cores (bf16 v, do, o
    [B, H, T, d], d = 64, 96 or 128); fp32 CUDA tensors [H, T], the same bits on
    every run.
    `workspace` (uint8 CUDA tensor) is allocated when not given."""
    B, H, T, d = v.shape
    fz = _frozen_bytes(frozen, H)
    nf = sum(fz) if fz is not None else 0
    da = torch.empty((H, T), dtype=torch.float32, device=v.device) if da is None else da
    dr = torch.empty((H, T), dtype=torch.float32, device=v.device) if dr is None else dr
    if workspace is None:
        n = max(saf_pattern_grad_tc_workspace_bytes(B, H, T, nf), 256)
        workspace = torch.empty(n, dtype=torch.uint8, device=v.device)
    st = _lib.saf_pattern_grad_tc(_ptr(v), _ptr(do), _ptr(o), _ptr(lse), _ptr(a), _ptr(r), a.shape[-1], fz, B, H,
                                  T, d, _ptr(da), _ptr(dr), _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SAF_OK:
        raise SafError(st, "saf_pattern_grad_tc")
    return da, dr
