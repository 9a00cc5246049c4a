"""ctypes binding of libla2.so -- argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and sizes, passes the caller's
current CUDA stream, and raises on a non-OK status.  There is no fallback: if
the library is missing or a shape is unsupported, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libla2.so")

LA2_OK = 0
LA2_ERR_INVALID_ARG = 1
LA2_ERR_UNSUPPORTED = 2
LA2_ERR_WORKSPACE = 3
LA2_ERR_CUDA = 4
LA2_ERR_TIMEOUT = 5

LA2_DTYPE_F32 = 0
LA2_DTYPE_BF16 = 1

# Every entry point include/la2.h declares.
EXPORTS = ("la2_workspace_bytes", "la2_fwd", "la2_fwd_state", "la2_fwd_ex", "la2_bwd", "la2_bwd_ex",
           "la2_decode", "la2_status_str", "la2_device_status", "la2_last_launch_count",
           "la2_fwd_noalloc", "la2_set_schedule", "la2_plan_info", "la2_selftest_timeout",
           "la2_bwd_state", "la2_dlambda", "la2_dlambda_workspace_bytes",
           "la2_norm_workspace_bytes", "la2_fwd_norm", "la2_bwd_norm",
           "la2_gdr_workspace_bytes", "la2_gdr_fwd", "la2_gdr_bwd", "la2_gdr_decode",
           "la2_gdr_selftest_timeout", "la2_state_copy")

LA2_LAYOUT_BHTD = 0
LA2_LAYOUT_BTHD = 1
_LAYOUTS = {"bhtd": LA2_LAYOUT_BHTD, "bthd": LA2_LAYOUT_BTHD}

LA2_SCHEDULE_AUTO = 0
LA2_SCHEDULE_UNIFORM = 1
LA2_SCHEDULE_BALANCED = 2
_SCHEDULES = {"auto": LA2_SCHEDULE_AUTO, "uniform": LA2_SCHEDULE_UNIFORM, "balanced": LA2_SCHEDULE_BALANCED}


class LA2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {la2_status_str(status)} ({status})")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libla2.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libla2.so not found at {path}; build it with "
                           "`python -m causal_linear_attention_la2_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.la2_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.la2_workspace_bytes.restype = sz
    lib.la2_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_fwd.restype = i
    lib.la2_fwd_state.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_fwd_state.restype = i
    lib.la2_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_bwd.restype = i
    lib.la2_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_fwd_ex.restype = i
    lib.la2_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, vp, sz,
                               vp]
    lib.la2_bwd_ex.restype = i
    lib.la2_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.la2_decode.restype = i
    lib.la2_status_str.argtypes = [i]
    lib.la2_status_str.restype = ctypes.c_char_p
    lib.la2_device_status.argtypes = [ctypes.POINTER(ctypes.c_int), i]
    lib.la2_device_status.restype = i
    lib.la2_last_launch_count.argtypes = []
    lib.la2_last_launch_count.restype = i
    lib.la2_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
    lib.la2_fwd_noalloc.restype = i
    lib.la2_set_schedule.argtypes = [i]
    lib.la2_set_schedule.restype = i
    lib.la2_plan_info.argtypes = [i, i, i, i, i, i, i, i, ctypes.POINTER(LA2Plan), i]
    lib.la2_plan_info.restype = i
    lib.la2_selftest_timeout.argtypes = [vp, vp, vp, vp, vp, i, i, i, ctypes.c_uint, vp]
    lib.la2_selftest_timeout.restype = i
    lib.la2_bwd_state.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                  i, i, vp, sz, vp]
    lib.la2_bwd_state.restype = i
    lib.la2_dlambda_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.la2_dlambda_workspace_bytes.restype = sz
    lib.la2_dlambda.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_dlambda.restype = i
    lib.la2_norm_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.la2_norm_workspace_bytes.restype = sz
    lib.la2_fwd_norm.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]
    lib.la2_fwd_norm.restype = i
    lib.la2_bwd_norm.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                 vp, sz, vp]
    lib.la2_bwd_norm.restype = i
    lib.la2_gdr_workspace_bytes.argtypes = [i] * 8
    lib.la2_gdr_workspace_bytes.restype = sz
    lib.la2_gdr_fwd.argtypes = [vp] * 9 + [i] * 9 + [vp, sz, vp]
    lib.la2_gdr_fwd.restype = i
    lib.la2_gdr_bwd.argtypes = [vp] * 15 + [i] * 9 + [vp, sz, vp]
    lib.la2_gdr_bwd.restype = i
    lib.la2_gdr_decode.argtypes = [vp] * 7 + [i, vp] + [i] * 6 + [vp]
    lib.la2_gdr_decode.restype = i
    lib.la2_gdr_selftest_timeout.argtypes = [i, vp, sz, vp]
    lib.la2_gdr_selftest_timeout.restype = i
    lib.la2_state_copy.argtypes = [vp, vp, vp, i, i, ctypes.c_longlong, vp]
    lib.la2_state_copy.restype = i
    _lib = lib
    return lib


def la2_status_str(status: int) -> str:
    return load().la2_status_str(int(status)).decode()


def la2_workspace_bytes(B, H, T, d, e, block, dtype, is_bwd) -> int:
    return int(load().la2_workspace_bytes(B, H, T, d, e, block, dtype, int(is_bwd)))


def la2_device_status(reset: bool = True) -> int:
    code = ctypes.c_int(0)
    st = load().la2_device_status(ctypes.byref(code), int(reset))
    if st != LA2_OK:
        raise LA2Error(st, "la2_device_status")
    return code.value


def la2_last_launch_count() -> int:
    return int(load().la2_last_launch_count())


class LA2Plan(ctypes.Structure):
    """la2_plan of include/la2.h."""
    _fields_ = [("d", ctypes.c_int), ("e", ctypes.c_int), ("schedule", ctypes.c_int),
                ("units", ctypes.c_longlong), ("segments", ctypes.c_int), ("tiles_per_cta", ctypes.c_int),
                ("ctas", ctypes.c_longlong), ("prepass_ctas", ctypes.c_longlong)]


def la2_plan_info(B, H, T, d, e, block=128, dtype=LA2_DTYPE_BF16, is_bwd=False) -> list:
    """The launch plan(s) of a bf16 call of these sizes, as dicts (one per
    launch group); [] for an empty problem or fp32 inputs."""
    plans = (LA2Plan * 2)()
    n = int(load().la2_plan_info(B, H, T, d, e, block, dtype, int(is_bwd), plans, 2))
    if n < 0:
        raise LA2Error(LA2_ERR_INVALID_ARG, "la2_plan_info")
    names = {LA2_SCHEDULE_UNIFORM: "uniform", LA2_SCHEDULE_BALANCED: "balanced"}
    return [{"d": p.d, "e": p.e, "schedule": names[p.schedule], "units": p.units, "segments": p.segments,
             "tiles_per_cta": p.tiles_per_cta, "ctas": p.ctas, "prepass_ctas": p.prepass_ctas}
            for p in plans[:n]]


def la2_set_schedule(schedule: str) -> str:
    """Sets how the bf16 kernels spread their work over CTAs ("auto",
    "uniform" or "balanced"); returns the previous setting."""
    prev = int(load().la2_set_schedule(_SCHEDULES[schedule]))
    return {v: k for k, v in _SCHEDULES.items()}[prev]


# ---------------------------------------------------------------- raw C calls

def la2_selftest_timeout_raw(q, k, v, decay, out, T, d, e, limit_us, stream=0) -> int:
    """Failure-path self-test: the bf16 forward kernel waits, bounded by
    limit_us, on a flag nothing sets and records LA2_ERR_TIMEOUT; returns the
    launch status (read the recorded code with la2_device_status)."""
    return int(load().la2_selftest_timeout(q, k, v, decay, out, T, d, e, limit_us, stream))


def la2_fwd_raw(q, k, v, decay, out, B, H, T, d, e, block, dtype, workspace=0, ws_bytes=0,
                stream=0) -> int:
    """The C call with integer pointers; returns the status code."""
    return int(load().la2_fwd(q, k, v, decay, out, B, H, T, d, e, block, dtype, workspace,
                              ws_bytes, stream))


def la2_fwd_noalloc_raw(q, k, v, decay, out, B, H, T, d, e, block, dtype, stream=0) -> int:
    """The allocation-free forward (scratch built into the library); returns the status."""
    return int(load().la2_fwd_noalloc(q, k, v, decay, out, B, H, T, d, e, block, dtype, stream))


def la2_bwd_raw(q, k, v, decay, dout, dq, dk, dv, B, H, T, d, e, block, dtype, workspace=0,
                ws_bytes=0, stream=0) -> int:
    return int(load().la2_bwd(q, k, v, decay, dout, dq, dk, dv, B, H, T, d, e, block, dtype,
                              workspace, ws_bytes, stream))


# ------------------------------------------------------------- torch wrappers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LA2_DTYPE_BF16
    if t.dtype == torch.float32:
        return LA2_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float32")


def _out_dtype(out_dtype) -> tuple:
    """(torch dtype, la2_dtype code) of the outputs: fp32 (None) or bf16."""
    if out_dtype is None or out_dtype == torch.float32:
        return torch.float32, LA2_DTYPE_F32
    if out_dtype == torch.bfloat16:
        return torch.bfloat16, LA2_DTYPE_BF16
    raise TypeError(f"unsupported out_dtype {out_dtype}; expected torch.float32 or torch.bfloat16")


def _check(t: torch.Tensor, name: str, shape, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_ptr(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


_ws_cache: dict = {}


def _workspace(nbytes: int, device, workspace=None):
    """(pointer, size) of a device workspace of at least nbytes (256-byte aligned).

    A caller-provided uint8 tensor is used as is; otherwise one buffer per
    device is kept and grown on demand (torch's allocator, plumbing only).
    """
    if nbytes <= 0:
        return 0, 0
    if workspace is not None:
        if not workspace.is_cuda or workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must be a CUDA buffer of at least {nbytes} bytes")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    key = torch.device(device).index
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf.data_ptr(), buf.numel()


def la2_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
            out: torch.Tensor | None = None, block: int = 128, stream=None,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """o[b,h,t] = sum_{s<=t} decay[h]^(t-s) (q[b,h,t] . k[b,h,s]) v[b,h,s], on q's device.

    q, k, v: bf16 or fp32; the output is fp32 (la2_fwd_ex also writes bf16)."""
    B, H, T, d = q.shape
    e = v.shape[-1]
    dt = _dtype_code(q)
    _check(q, "q", (B, H, T, d), q.dtype)
    _check(k, "k", (B, H, T, d), q.dtype)
    _check(v, "v", (B, H, T, e), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    if out is None:
        out = torch.empty((B, H, T, e), dtype=torch.float32, device=q.device)
    _check(out, "out", (B, H, T, e), torch.float32)
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 0), q.device, workspace)
    st = la2_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), out.data_ptr(),
                     B, H, T, d, e, block, dt, wp, wn, _stream_ptr(stream))
    if st != LA2_OK:
        raise LA2Error(st, "la2_fwd")
    return out


def la2_fwd_state_raw(q, k, v, decay, out, init_state, final_state, B, H, T, d, e, block, dtype,
                      workspace=0, ws_bytes=0, stream=0) -> int:
    """The C call with integer pointers (0 = NULL for the states); returns the status."""
    return int(load().la2_fwd_state(q, k, v, decay, out, init_state, final_state, B, H, T, d, e,
                                    block, dtype, workspace, ws_bytes, stream))


def la2_fwd_state(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
                  init_state: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  final_state: torch.Tensor | None = None, block: int = 128, stream=None,
                  workspace: torch.Tensor | None = None):
    """(out, final_state): la2_fwd started from init_state ([B, H, d, e] fp32, None = 0),
    returning the state after the last position as well."""
    B, H, T, d = q.shape
    e = v.shape[-1]
    dt = _dtype_code(q)
    _check(q, "q", (B, H, T, d), q.dtype)
    _check(k, "k", (B, H, T, d), q.dtype)
    _check(v, "v", (B, H, T, e), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    out = torch.empty((B, H, T, e), **f32) if out is None else out
    final_state = torch.empty((B, H, d, e), **f32) if final_state is None else final_state
    _check(out, "out", (B, H, T, e), torch.float32)
    _check(final_state, "final_state", (B, H, d, e), torch.float32)
    ip = 0
    if init_state is not None:
        _check(init_state, "init_state", (B, H, d, e), torch.float32)
        ip = init_state.data_ptr()
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 0), q.device, workspace)
    st = la2_fwd_state_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                           out.data_ptr(), ip, final_state.data_ptr(), B, H, T, d, e, block, dt,
                           wp, wn, _stream_ptr(stream))
    if st != LA2_OK:
        raise LA2Error(st, "la2_fwd_state")
    return out, final_state


def _dims(q, v, layout):
    """(B, H, T, d, e) from q's and v's shapes in the given layout."""
    if layout == "bhtd":
        B, H, T, d = q.shape
    elif layout == "bthd":
        B, T, H, d = q.shape
    else:
        raise ValueError(f"unknown layout {layout!r}; expected 'bhtd' or 'bthd'")
    return B, H, T, d, v.shape[-1]


def _shape(layout, B, H, T, D):
    return (B, H, T, D) if layout == "bhtd" else (B, T, H, D)


def la2_fwd_ex(q, k, v, decay, layout: str = "bhtd", init_state=None, out=None, final_state=None,
               want_final: bool = False, block: int = 128, stream=None, workspace=None,
               out_dtype=None):
    """la2_fwd_state for q, k, v (and out) laid out [B, H, T, D] ('bhtd') or
    [B, T, H, D] ('bthd'), out of type out_dtype (torch.float32, the default, or
    torch.bfloat16).  Returns out, or (out, final_state) with want_final or a
    final_state buffer given."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    odt, oc = _out_dtype(out_dtype)
    _check(q, "q", _shape(layout, B, H, T, d), q.dtype)
    _check(k, "k", _shape(layout, B, H, T, d), q.dtype)
    _check(v, "v", _shape(layout, B, H, T, e), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    out = torch.empty(_shape(layout, B, H, T, e), dtype=odt, device=q.device) if out is None else out
    _check(out, "out", _shape(layout, B, H, T, e), odt)
    if final_state is None and want_final:
        final_state = torch.empty((B, H, d, e), **f32)
    fp = 0
    if final_state is not None:
        _check(final_state, "final_state", (B, H, d, e), torch.float32)
        fp = final_state.data_ptr()
    ip = 0
    if init_state is not None:
        _check(init_state, "init_state", (B, H, d, e), torch.float32)
        ip = init_state.data_ptr()
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 0), q.device, workspace)
    st = int(load().la2_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                               out.data_ptr(), ip, fp, B, H, T, d, e, block, dt, oc,
                               _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_fwd_ex")
    return (out, final_state) if final_state is not None else out


def la2_bwd_ex(q, k, v, decay, dout, layout: str = "bhtd", dq=None, dk=None, dv=None,
               block: int = 128, stream=None, workspace=None, out_dtype=None):
    """la2_bwd for tensors laid out [B, H, T, D] ('bhtd') or [B, T, H, D] ('bthd'),
    dq, dk, dv of type out_dtype (torch.float32, the default, or torch.bfloat16)."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    odt, oc = _out_dtype(out_dtype)
    for t, n, D in ((q, "q", d), (k, "k", d), (v, "v", e), (dout, "dout", e)):
        _check(t, n, _shape(layout, B, H, T, D), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    o = dict(dtype=odt, device=q.device)
    dq = torch.empty(_shape(layout, B, H, T, d), **o) if dq is None else dq
    dk = torch.empty(_shape(layout, B, H, T, d), **o) if dk is None else dk
    dv = torch.empty(_shape(layout, B, H, T, e), **o) if dv is None else dv
    for t, n, D in ((dq, "dq", d), (dk, "dk", d), (dv, "dv", e)):
        _check(t, n, _shape(layout, B, H, T, D), odt)
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 1), q.device, workspace)
    st = int(load().la2_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                               dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, T,
                               d, e, block, dt, oc, _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_bwd_ex")
    return dq, dk, dv


def la2_bwd_state(q, k, v, decay, dout, init_state=None, d_final_state=None, layout: str = "bhtd",
                  dq=None, dk=None, dv=None, d_init_state=None, want_d_init: bool = True,
                  block: int = 128, stream=None, workspace=None, out_dtype=None):
    """(dq, dk, dv, d_init_state) of sum(dout * out) + sum(d_final_state * final_state) for
    the forward la2_fwd_ex(q, k, v, decay, layout, init_state); states [B, H, d, e] fp32
    (None = zero), dq, dk, dv of type out_dtype (torch.float32 or torch.bfloat16).
    d_init_state is None unless want_d_init or a buffer is given."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    odt, oc = _out_dtype(out_dtype)
    for t, n, D in ((q, "q", d), (k, "k", d), (v, "v", e), (dout, "dout", e)):
        _check(t, n, _shape(layout, B, H, T, D), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    o = dict(dtype=odt, device=q.device)
    dq = torch.empty(_shape(layout, B, H, T, d), **o) if dq is None else dq
    dk = torch.empty(_shape(layout, B, H, T, d), **o) if dk is None else dk
    dv = torch.empty(_shape(layout, B, H, T, e), **o) if dv is None else dv
    for t, n, D in ((dq, "dq", d), (dk, "dk", d), (dv, "dv", e)):
        _check(t, n, _shape(layout, B, H, T, D), odt)
    if d_init_state is None and want_d_init:
        d_init_state = torch.empty((B, H, d, e), **f32)
    ptrs = []
    for t, n in ((init_state, "init_state"), (d_final_state, "d_final_state"),
                 (d_init_state, "d_init_state")):
        if t is not None:
            _check(t, n, (B, H, d, e), torch.float32)
        ptrs.append(0 if t is None else t.data_ptr())
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 1), q.device, workspace)
    st = int(load().la2_bwd_state(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                                  dout.data_ptr(), ptrs[0], ptrs[1], dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), ptrs[2], B, H, T, d, e, block, dt, oc,
                                  _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_bwd_state")
    return dq, dk, dv, d_init_state


def la2_dlambda_workspace_bytes(B, H, T, d, e, dtype) -> int:
    return int(load().la2_dlambda_workspace_bytes(B, H, T, d, e, dtype))


def la2_dlambda(q, k, v, decay, dout, init_state=None, d_final_state=None, layout: str = "bhtd",
                d_decay=None, stream=None, workspace=None):
    """dL/d(decay) [H] (summed over the batch) for L = sum(dout * out) + sum(d_final_state *
    final_state), the forward la2_fwd_ex(q, k, v, decay, layout, init_state)."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    for t, n, D in ((q, "q", d), (k, "k", d), (v, "v", e), (dout, "dout", e)):
        _check(t, n, _shape(layout, B, H, T, D), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    d_decay = torch.empty((H,), dtype=torch.float32, device=q.device) if d_decay is None else d_decay
    _check(d_decay, "d_decay", (H,), torch.float32)
    ptrs = []
    for t, n in ((init_state, "init_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _check(t, n, (B, H, d, e), torch.float32)
        ptrs.append(0 if t is None else t.data_ptr())
    wp, wn = _workspace(la2_dlambda_workspace_bytes(B, H, T, d, e, dt), q.device, workspace)
    st = int(load().la2_dlambda(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                                dout.data_ptr(), ptrs[0], ptrs[1], d_decay.data_ptr(), B, H, T, d, e,
                                dt, _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_dlambda")
    return d_decay


def la2_norm_workspace_bytes(B, H, T, d, e, block, dtype, is_bwd) -> int:
    return int(load().la2_norm_workspace_bytes(B, H, T, d, e, block, dtype, int(is_bwd)))


def la2_fwd_norm(q, k, v, decay, layout: str = "bhtd", y=None, den=None, block: int = 128,
                 stream=None, workspace=None):
    """(y, den): the normalised form y_t = num_t / (q_t . z_t), z_t = decay z_{t-1} + k_t."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    for t, n, D in ((q, "q", d), (k, "k", d), (v, "v", e)):
        _check(t, n, _shape(layout, B, H, T, D), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    y = torch.empty(_shape(layout, B, H, T, e), **f32) if y is None else y
    den = torch.empty((B, H, T), **f32) if den is None else den
    _check(y, "y", _shape(layout, B, H, T, e), torch.float32)
    _check(den, "den", (B, H, T), torch.float32)
    wp, wn = _workspace(la2_norm_workspace_bytes(B, H, T, d, e, block, dt, 0), q.device, workspace)
    st = int(load().la2_fwd_norm(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                                 y.data_ptr(), den.data_ptr(), B, H, T, d, e, block, dt,
                                 _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_fwd_norm")
    return y, den


def la2_bwd_norm(q, k, v, decay, y, den, dy, layout: str = "bhtd", dq=None, dk=None, dv=None,
                 block: int = 128, stream=None, workspace=None):
    """(dq, dk, dv) of sum(dy * y) for (y, den) = la2_fwd_norm(q, k, v, decay)."""
    B, H, T, d, e = _dims(q, v, layout)
    dt = _dtype_code(q)
    for t, n, D in ((q, "q", d), (k, "k", d), (v, "v", e), (dy, "dy", e)):
        _check(t, n, _shape(layout, B, H, T, D), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    _check(y, "y", _shape(layout, B, H, T, e), torch.float32)
    _check(den, "den", (B, H, T), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty(_shape(layout, B, H, T, d), **f32) if dq is None else dq
    dk = torch.empty(_shape(layout, B, H, T, d), **f32) if dk is None else dk
    dv = torch.empty(_shape(layout, B, H, T, e), **f32) if dv is None else dv
    wp, wn = _workspace(la2_norm_workspace_bytes(B, H, T, d, e, block, dt, 1), q.device, workspace)
    st = int(load().la2_bwd_norm(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                                 y.data_ptr(), den.data_ptr(), dy.data_ptr(), dq.data_ptr(),
                                 dk.data_ptr(), dv.data_ptr(), B, H, T, d, e, block, dt,
                                 _LAYOUTS[layout], wp, wn, _stream_ptr(stream)))
    if st != LA2_OK:
        raise LA2Error(st, "la2_bwd_norm")
    return dq, dk, dv


def la2_decode_raw(q, k, v, decay, state, out, B, H, d, e, dtype, stream=0) -> int:
    return int(load().la2_decode(q, k, v, decay, state, out, B, H, d, e, dtype, stream))


def la2_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
               state: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token per sequence: state <- decay state + k v^T (in place), returns state^T q.

    q, k: [B, H, d], v: [B, H, e] (bf16 or fp32); state: [B, H, d, e] fp32."""
    B, H, d = q.shape
    e = v.shape[-1]
    dt = _dtype_code(q)
    _check(q, "q", (B, H, d), q.dtype)
    _check(k, "k", (B, H, d), q.dtype)
    _check(v, "v", (B, H, e), q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    _check(state, "state", (B, H, d, e), torch.float32)
    out = torch.empty((B, H, e), dtype=torch.float32, device=q.device) if out is None else out
    _check(out, "out", (B, H, e), torch.float32)
    st = la2_decode_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(),
                        state.data_ptr(), out.data_ptr(), B, H, d, e, dt, _stream_ptr(stream))
    if st != LA2_OK:
        raise LA2Error(st, "la2_decode")
    return out


def la2_bwd(q, k, v, decay, dout, dq=None, dk=None, dv=None, block: int = 128, stream=None,
            workspace: torch.Tensor | None = None):
    """(dq, dk, dv) of sum(dout * la2_fwd(q, k, v, decay)); decay is not differentiated."""
    B, H, T, d = q.shape
    e = v.shape[-1]
    dt = _dtype_code(q)
    for t, n, shp in ((q, "q", (B, H, T, d)), (k, "k", (B, H, T, d)), (v, "v", (B, H, T, e)),
                      (dout, "dout", (B, H, T, e))):
        _check(t, n, shp, q.dtype)
    _check(decay, "decay", (H,), torch.float32)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((B, H, T, d), **f32) if dq is None else dq
    dk = torch.empty((B, H, T, d), **f32) if dk is None else dk
    dv = torch.empty((B, H, T, e), **f32) if dv is None else dv
    for t, n, shp in ((dq, "dq", (B, H, T, d)), (dk, "dk", (B, H, T, d)), (dv, "dv", (B, H, T, e))):
        _check(t, n, shp, torch.float32)
    wp, wn = _workspace(la2_workspace_bytes(B, H, T, d, e, block, dt, 1), q.device, workspace)
    st = la2_bwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), dout.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, T, d, e, block, dt, wp, wn,
                     _stream_ptr(stream))
    if st != LA2_OK:
        raise LA2Error(st, "la2_bwd")
    return dq, dk, dv


# ------------------------------------------------------- the gated delta rule

def la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dtype, is_bwd) -> int:
    return int(load().la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dtype, int(is_bwd)))


def la2_gdr_fwd_raw(q, k, v, g, beta, out, init_state, final_state, seq_lens, B, Hk, H, T, d, e,
                    dtype, out_dtype, layout, workspace=0, ws_bytes=0, stream=0) -> int:
    """The C call with integer pointers (0 = NULL); returns the status."""
    return int(load().la2_gdr_fwd(q, k, v, g, beta, out, init_state, final_state, seq_lens, B, Hk,
                                  H, T, d, e, dtype, out_dtype, layout, workspace, ws_bytes, stream))


def la2_gdr_bwd_raw(q, k, v, g, beta, dout, init_state, d_final_state, dq, dk, dv, dg, dbeta,
                    d_init_state, seq_lens, B, Hk, H, T, d, e, dtype, out_dtype, layout,
                    workspace=0, ws_bytes=0, stream=0) -> int:
    """The C call with integer pointers (0 = NULL); returns the status."""
    return int(load().la2_gdr_bwd(q, k, v, g, beta, dout, init_state, d_final_state, dq, dk, dv,
                                  dg, dbeta, d_init_state, seq_lens, B, Hk, H, T, d, e, dtype,
                                  out_dtype, layout, workspace, ws_bytes, stream))


def la2_gdr_decode_raw(q, k, v, g, beta, states, slots, n_slots, out, B, Hk, H, d, e, dtype,
                       stream=0) -> int:
    """The C call with integer pointers (0 = NULL); returns the status."""
    return int(load().la2_gdr_decode(q, k, v, g, beta, states, slots, n_slots, out, B, Hk, H, d, e,
                                     dtype, stream))


LA2_GDR_SELFTEST_BYTES = 16 << 20
LA2_GDR_KERNEL_DECODE = 0
LA2_GDR_KERNEL_GRAD = 1
LA2_GDR_KERNEL_WALK = 2
LA2_GDR_KERNEL_WALKS = 3


def la2_gdr_selftest_timeout_raw(kernel, workspace, ws_bytes, stream=0) -> int:
    """Failure-path self-test: one of the gated delta rule's kernels waits, bounded by 20 ms, for a
    copy that is never issued and records LA2_ERR_TIMEOUT; returns the launch status (read the
    recorded code with la2_device_status)."""
    return int(load().la2_gdr_selftest_timeout(kernel, workspace, ws_bytes, stream))


def la2_state_copy_raw(states, src, dst, n, n_slots, slot_elems, stream=0) -> int:
    """The C call with integer pointers; returns the status."""
    return int(load().la2_state_copy(states, src, dst, n, n_slots, slot_elems, stream))


def _same_device(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _need(t, name, shape, dtype, device) -> None:
    """_check and the device, with the usual case decided in one expression."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous() and t.is_cuda:
        return
    _check(t, name, shape, dtype)
    _same_device(device, **{name: t})


class _On:
    """The tensors' device, and the caller's stream if one is given, made current for a call: what
    the call allocates (and sets to zero) belongs to the stream that its kernels run on."""

    def __init__(self, device, stream=None):
        if device.type != "cuda":
            raise ValueError("the tensors must be CUDA tensors")
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self._guard = torch.cuda.stream(stream)
        else:
            self._guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


def _stream_on(device) -> int:
    """The current stream of the tensors' device (inside _On: the caller's stream)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _own_workspace(nbytes: int, device, workspace):
    """(pointer, size, tensor): the caller's workspace, or one of this call's own.

    A call allocates its workspace from torch's caching allocator on the stream
    that it runs on, so two calls on two streams, or two captured graphs, never
    share one; the allocator hands the memory on in stream order."""
    if workspace is not None:
        _same_device(device, workspace=workspace)
        p, n = _workspace(nbytes, device, workspace)
        return p, n, workspace
    if nbytes <= 0:
        return 0, 0, None
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf.data_ptr(), nbytes, buf


def _gdr_dims(q, v, layout):
    """(B, Hk, H, T, d, e) from q's and v's shapes in the given layout."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must have 4 dimensions")
    B, Hk, T, d, e = _dims(q, v, layout)
    H = v.shape[1] if layout == "bhtd" else v.shape[2]
    if Hk == 0 or H % Hk != 0:
        if not (H == 0 and Hk == 0):
            raise ValueError(f"{H} value heads are not a multiple of {Hk} key heads")
    return B, Hk, H, T, d, e


def _gdr_inputs(q, k, v, g, beta, layout, seq_lens, states):
    """Checks what both directions take; returns the sizes and the dtype code."""
    B, Hk, H, T, d, e = _gdr_dims(q, v, layout)
    dt, dev = _dtype_code(q), q.device
    qk = q.shape
    _need(q, "q", qk, q.dtype, dev)
    _need(k, "k", qk, q.dtype, dev)
    _need(v, "v", _shape(layout, B, H, T, e), q.dtype, dev)
    gate = (B, H, T) if layout == "bhtd" else (B, T, H)
    _need(beta, "beta", gate, torch.float32, dev)
    if g is not None:
        _need(g, "g", gate, torch.float32, dev)
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", (B,), torch.int32, dev)
    for name, s in states.items():
        if s is not None:
            _need(s, name, (B, H, d, e), torch.float32, dev)
    return B, Hk, H, T, d, e, dt


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def la2_gdr_fwd(q, k, v, g, beta, layout: str = "bhtd", init_state=None, seq_lens=None, out=None,
                final_state=None, want_final: bool = False, stream=None, workspace=None,
                out_dtype=None):
    """The gated delta rule over whole sequences:

        S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t

    q, k [B, Hk, T, d], v [B, H, T, e] (bf16 or fp32; 'bthd': [B, T, heads, .]), g (log-gate, or
    None) and beta fp32 [B, H, T] ('bthd': [B, T, H]); value head h reads key head h // (H // Hk).
    seq_lens (int32 [B]): rows of each sequence; the rows behind them are left as they were in
    `out` (zero in an out allocated here).  Returns out, or (out, final_state) with want_final or
    a final_state buffer given."""
    B, Hk, H, T, d, e, dt = _gdr_inputs(q, k, v, g, beta, layout, seq_lens,
                                        {"init_state": init_state, "final_state": final_state})
    odt, oc = _out_dtype(out_dtype)
    shape = _shape(layout, B, H, T, e)
    with _On(q.device, stream):
        sp = _stream_on(q.device)
        if out is None:
            out = (torch.empty if seq_lens is None else torch.zeros)(shape, dtype=odt, device=q.device)
        else:
            _need(out, "out", shape, odt, q.device)
        if final_state is None and want_final:
            final_state = torch.empty((B, H, d, e), dtype=torch.float32, device=q.device)
        wp, wn, keep = _own_workspace(la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dt, 0), q.device, workspace)
        st = la2_gdr_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), beta.data_ptr(),
                             out.data_ptr(), _ptr(init_state), _ptr(final_state), _ptr(seq_lens),
                             B, Hk, H, T, d, e, dt, oc, _LAYOUTS[layout], wp, wn, sp)
    if st != LA2_OK:
        raise LA2Error(st, "la2_gdr_fwd")
    return out if final_state is None else (out, final_state)


def la2_gdr_bwd(q, k, v, g, beta, dout, layout: str = "bhtd", init_state=None, d_final_state=None,
                seq_lens=None, dq=None, dk=None, dv=None, dg=None, dbeta=None, d_init_state=None,
                want_d_init: bool = False, stream=None, workspace=None, out_dtype=None):
    """(dq, dk, dv, dg, dbeta[, d_init_state]) of sum(dout * out) + sum(d_final_state * final_state)
    for la2_gdr_fwd; dg is None without a gate.  d_init_state is returned with want_d_init or a
    buffer given.  Rows behind seq_lens are left as they were (zero in tensors allocated here)."""
    B, Hk, H, T, d, e, dt = _gdr_inputs(q, k, v, g, beta, layout, seq_lens,
                                        {"init_state": init_state, "d_final_state": d_final_state,
                                         "d_init_state": d_init_state})
    odt, oc = _out_dtype(out_dtype)
    _need(dout, "dout", v.shape, q.dtype, q.device)
    if dg is not None and g is None:
        raise ValueError("dg needs a gate g")
    gate = tuple(beta.shape)
    new = torch.empty if seq_lens is None else torch.zeros
    with _On(q.device, stream):
        sp = _stream_on(q.device)
        o = dict(dtype=odt, device=q.device)
        f = dict(dtype=torch.float32, device=q.device)
        dq = new(_shape(layout, B, Hk, T, d), **o) if dq is None else dq
        dk = new(_shape(layout, B, Hk, T, d), **o) if dk is None else dk
        dv = new(_shape(layout, B, H, T, e), **o) if dv is None else dv
        dbeta = new(gate, **f) if dbeta is None else dbeta
        if g is not None and dg is None:
            dg = new(gate, **f)
        if d_init_state is None and want_d_init:
            d_init_state = torch.empty((B, H, d, e), **f)
        for name, t, shape, dtype in (("dq", dq, q.shape, odt), ("dk", dk, q.shape, odt), ("dv", dv, v.shape, odt),
                                      ("dbeta", dbeta, gate, torch.float32), ("dg", dg, gate, torch.float32)):
            if t is not None:
                _need(t, name, shape, dtype, q.device)
        wp, wn, keep = _own_workspace(la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dt, 1), q.device, workspace)
        st = la2_gdr_bwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), beta.data_ptr(),
                             dout.data_ptr(), _ptr(init_state), _ptr(d_final_state), dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), _ptr(dg), dbeta.data_ptr(),
                             _ptr(d_init_state), _ptr(seq_lens), B, Hk, H, T, d, e, dt, oc,
                             _LAYOUTS[layout], wp, wn, sp)
    if st != LA2_OK:
        raise LA2Error(st, "la2_gdr_bwd")
    r = (dq, dk, dv, dg, dbeta)
    return r if d_init_state is None else r + (d_init_state,)


def la2_gdr_decode(q, k, v, g, beta, states, slots=None, out=None, stream=None) -> torch.Tensor:
    """One token of the gated delta rule for each sequence, on its slot of the pool `states`
    ([slots, H, d, e] fp32, updated in place); returns out [B, H, e] fp32.

    q, k [B, Hk, d], v [B, H, e] (bf16 or fp32), g (or None) and beta fp32 [B, H]; slots int32 [B]
    (None: sequence b has slot b).  A slot outside the pool, or named by an earlier row already,
    gives zeros and changes no state."""
    if q.dim() != 3 or v.dim() != 3 or states.dim() != 4:
        raise ValueError("q and v must have 3 dimensions, states 4")
    B, Hk, d = q.shape
    H, e = v.shape[1:]
    dt, dev, n_slots = _dtype_code(q), q.device, states.shape[0]
    if (Hk == 0 or H % Hk != 0) and H + Hk:
        raise ValueError(f"{H} value heads are not a multiple of {Hk} key heads")
    _need(q, "q", q.shape, q.dtype, dev)
    _need(k, "k", q.shape, q.dtype, dev)
    _need(v, "v", (B, H, e), q.dtype, dev)
    _need(beta, "beta", (B, H), torch.float32, dev)
    if g is not None:
        _need(g, "g", (B, H), torch.float32, dev)
    _need(states, "states", (n_slots, H, d, e), torch.float32, dev)
    if slots is not None:
        _need(slots, "slots", (B,), torch.int32, dev)
    elif n_slots < B:
        raise ValueError(f"{B} sequences but {n_slots} slots")
    with _On(dev, stream):
        sp = _stream_on(dev)
        if out is None:
            out = torch.empty((B, H, e), dtype=torch.float32, device=dev)
        else:
            _need(out, "out", (B, H, e), torch.float32, dev)
        st = la2_gdr_decode_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), beta.data_ptr(),
                                states.data_ptr(), _ptr(slots), n_slots, out.data_ptr(), B, Hk, H,
                                d, e, dt, sp)
    if st != LA2_OK:
        raise LA2Error(st, "la2_gdr_decode")
    return out


def la2_state_copy(states, src, dst, stream=None) -> torch.Tensor:
    """Slot copies inside the pool `states` ([slots, ...] fp32, in place): slot dst[i] takes what
    slot src[i] held before the call, src[i] < 0 clears it (src, dst int32 [n]).  Pairs outside
    the pool do nothing; of several pairs with one destination the last counts.  Returns states."""
    if states.dim() < 1 or src.dim() != 1:
        raise ValueError("states must have a slot dimension, src and dst one dimension")
    n, n_slots, dev = src.shape[0], states.shape[0], states.device
    _need(states, "states", states.shape, torch.float32, dev)
    _need(src, "src", (n,), torch.int32, dev)
    _need(dst, "dst", (n,), torch.int32, dev)
    with _On(dev, stream):
        st = la2_state_copy_raw(states.data_ptr(), src.data_ptr(), dst.data_ptr(), n, n_slots,
                                states.numel() // n_slots if n_slots else 0,
                                _stream_on(dev))
    if st != LA2_OK:
        raise LA2Error(st, "la2_state_copy")
    return states
