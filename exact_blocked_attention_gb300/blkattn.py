"""Thin Python binding of libblkattn's C ABI (include/blkattn.h).

Argument marshalling only: torch tensors are turned into strided descriptors
(data pointer, sizes, strides) and the current torch stream is passed through,
here with ctypes, for the operators of a serving step (rope, paged_append,
attention_paged) in the small extension csrc/torch_bind.cpp.
Every step of the attention runs in the library's CUDA kernels; there is no
CPU or eager fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libblkattn.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_CUDA = -3
ERR_DEVICE_TIMEOUT = -4
ERR_NO_WORKSPACE = -5
ERR_SCRATCH_LIMIT = -6
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024

BF16, F32, I32, I64 = 1, 2, 3, 4
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.int32: I32, torch.int64: I64}

EXPORTED = ("blkattn_fwd", "blkattn_merge", "blkattn_status_string",
            "blkattn_check_device_error", "blkattn_debug_plan", "blkattn_debug_set_split_event",
            "blkattn_fwd_static_scratch", "blkattn_last_cuda_error", "blkattn_fwd_tree",
            "blkattn_spec_sample", "blkattn_fwd_window", "blkattn_bwd", "blkattn_bwd_window",
            "blkattn_debug_stall_next_decode", "blkattn_rope_angles", "blkattn_rope_phases", "blkattn_rope",
            "blkattn_rope_bwd", "blkattn_paged_append", "blkattn_fwd_paged")

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3}


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("sizes", ctypes.c_int64 * 4), ("strides", ctypes.c_int64 * 4), ("device", ctypes.c_int32)]


class States(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("l", ctypes.c_void_p), ("u", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("d_v", ctypes.c_int32), ("u_row_stride", ctypes.c_int64)]


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32),
                ("row_groups", ctypes.c_int32), ("chunk_keys", ctypes.c_int32),
                ("n_splits", ctypes.c_int32), ("tile_keys", ctypes.c_int32),
                ("ctas", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class RopeSpec(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("trained", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


class BlkattnError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"blkattn status {status}: {text}")
        self.status = status


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load libblkattn.so (built by exact_blocked_attention_gb300.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libblkattn.so is not built ({path}); run the package build first")
            lib = ctypes.CDLL(path)
            P = ctypes.c_void_p
            lib.blkattn_fwd.restype = ctypes.c_int
            lib.blkattn_fwd.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P]
            lib.blkattn_fwd_tree.restype = ctypes.c_int
            lib.blkattn_fwd_tree.argtypes = [P, P, P, P, P, P, P, ctypes.c_float, P, P, P]
            lib.blkattn_bwd.restype = ctypes.c_int
            lib.blkattn_bwd.argtypes = [P] * 6 + [ctypes.c_float] + [P] * 7
            lib.blkattn_bwd_window.restype = ctypes.c_int
            lib.blkattn_bwd_window.argtypes = [P] * 5 + [ctypes.c_int64, P, ctypes.c_float] + [P] * 7
            lib.blkattn_fwd_window.restype = ctypes.c_int
            lib.blkattn_fwd_window.argtypes = [P, P, P, P, P, ctypes.c_int64, P, ctypes.c_float, P, P, P]
            lib.blkattn_spec_sample.restype = ctypes.c_int
            lib.blkattn_spec_sample.argtypes = [P] * 8
            lib.blkattn_fwd_static_scratch.restype = ctypes.c_int
            lib.blkattn_fwd_static_scratch.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P]
            lib.blkattn_rope_angles.restype = ctypes.c_int
            lib.blkattn_rope_angles.argtypes = [P, P, P]
            lib.blkattn_rope_phases.restype = ctypes.c_int
            lib.blkattn_rope_phases.argtypes = [P, ctypes.c_int64, P]
            for f in (lib.blkattn_rope, lib.blkattn_rope_bwd):
                f.restype = ctypes.c_int
                f.argtypes = [P, P, P, ctypes.c_int32, ctypes.c_float, P, P]
            lib.blkattn_paged_append.restype = ctypes.c_int
            lib.blkattn_paged_append.argtypes = [P] * 7 + [ctypes.c_int32, ctypes.c_float, P, P, P]
            lib.blkattn_fwd_paged.restype = ctypes.c_int
            lib.blkattn_fwd_paged.argtypes = [P] * 7 + [ctypes.c_int64, ctypes.c_float, P, P, P]
            lib.blkattn_merge.restype = ctypes.c_int
            lib.blkattn_merge.argtypes = [P, P, P, P]
            lib.blkattn_status_string.restype = ctypes.c_char_p
            lib.blkattn_status_string.argtypes = [ctypes.c_int]
            lib.blkattn_check_device_error.restype = ctypes.c_int
            lib.blkattn_check_device_error.argtypes = [P]
            lib.blkattn_debug_plan.restype = ctypes.c_int
            lib.blkattn_debug_plan.argtypes = [ctypes.c_int64] * 6 + [ctypes.c_int32, ctypes.c_int32, P]
            lib.blkattn_debug_stall_next_decode.restype = None
            lib.blkattn_debug_stall_next_decode.argtypes = [ctypes.c_int32]
            lib.blkattn_debug_set_split_event.restype = None
            lib.blkattn_debug_set_split_event.argtypes = [P]
            lib.blkattn_last_cuda_error.restype = ctypes.c_char_p
            lib.blkattn_last_cuda_error.argtypes = []
            _lib = lib
    return _lib


_bind = None


def _load_bind():
    """The torch marshalling module (csrc/torch_bind.cpp), bound to the loaded library."""
    global _bind
    lib = load()
    with _lock:
        if _bind is None:
            try:
                from . import _torch_bind as bind
            except ImportError as e:
                raise RuntimeError(f"_torch_bind is not built or not loadable ({e}); run the package build first") from e
            bind.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (lib.blkattn_rope, lib.blkattn_rope_bwd,
                                                                        lib.blkattn_paged_append,
                                                                        lib.blkattn_fwd_paged)))
            _bind = bind
    return _bind


def status_string(status: int) -> str:
    return load().blkattn_status_string(int(status)).decode()


def _check(status: int):
    if status == OK:
        return
    text = status_string(status)
    if status == ERR_INVALID_ARG:
        raise ValueError(f"blkattn: {text}")
    if status == ERR_CUDA:
        text += f" ({load().blkattn_last_cuda_error().decode()})"
    raise BlkattnError(status, text)


def describe(t: torch.Tensor | None) -> Tensor | None:
    """Strided descriptor of a tensor (no copy, no dtype conversion)."""
    if t is None:
        return None
    if t.dtype not in _DTYPES:
        raise ValueError(f"blkattn: unsupported dtype {t.dtype}")
    if t.dim() > 4:
        raise ValueError("blkattn: at most 4 dimensions")
    d = Tensor()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _DTYPES[t.dtype]
    d.ndim = t.dim()
    d.device = t.device.index if t.is_cuda else -1  # host memory: refused by the library
    for i, (s, st) in enumerate(zip(t.shape, t.stride())):
        d.sizes[i] = s
        d.strides[i] = st
    return d


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _outputs(stream, *specs):
    """Outputs of a call, one for each (shape, dtype, device), on the call's
    stream: where that is not the current one, they are allocated on it (the
    current stream's memory may still be in use there) and the current stream
    is recorded as a reader."""
    device = specs[0][2]
    if stream is None or device.type != "cuda":
        return [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype, dev in specs]
    current = torch.cuda.current_stream(device)
    handle = _stream_handle(stream)
    handle = 0 if handle == 1 else handle  # (the legacy stream is the default one)
    if handle == current.cuda_stream:
        return [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype, dev in specs]
    if handle == 2:
        raise ValueError("blkattn: torch cannot allocate on the per-thread stream: pass the outputs")
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
        outs = [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype, dev in specs]
    for t in outs:
        t.record_stream(current)
    return outs


def _ref(x):
    return None if x is None else ctypes.byref(x)


def fwd(q, k, v, seqlens_k, q_logical_pos, mask_bias, scale: float, out, lse, stream=None, tree=None,
        window: int = 0):
    """blkattn_fwd on torch CUDA tensors; out and lse are written in place.
    tree: None, or int64 [B, T_q] token-tree node masks (blkattn_fwd_tree).
    window: 0, or a sliding window of that many keys (blkattn_fwd_window)."""
    lib = load()
    if window:
        if tree is not None:
            raise ValueError("blkattn: a call takes a tree or a window, not both")
        descs = [describe(t) for t in (q, k, v, seqlens_k, q_logical_pos, mask_bias, out, lse)]
        st = lib.blkattn_fwd_window(*[_ref(x) for x in descs[:5]], ctypes.c_int64(int(window)), _ref(descs[5]),
                                    ctypes.c_float(scale), _ref(descs[6]), _ref(descs[7]),
                                    _stream_handle(stream) if q.is_cuda else None)
        _check(st)
        return out, lse
    if tree is not None:
        descs = [describe(t) for t in (q, k, v, seqlens_k, q_logical_pos, tree, mask_bias, out, lse)]
        st = lib.blkattn_fwd_tree(*[_ref(x) for x in descs[:7]], ctypes.c_float(scale),
                                  _ref(descs[7]), _ref(descs[8]), _stream_handle(stream) if q.is_cuda else None)
        _check(st)
        return out, lse
    descs = [describe(t) for t in (q, k, v, seqlens_k, q_logical_pos, mask_bias, out, lse)]
    st = lib.blkattn_fwd(_ref(descs[0]), _ref(descs[1]), _ref(descs[2]), _ref(descs[3]),
                         _ref(descs[4]), _ref(descs[5]), ctypes.c_float(scale),
                         _ref(descs[6]), _ref(descs[7]), _stream_handle(stream) if q.is_cuda else None)
    _check(st)
    return out, lse


def bwd(q, k, v, seqlens_k, q_logical_pos, mask_bias, scale: float, out, lse, dout, dq, dk, dv, stream=None,
        window: int = 0):
    """blkattn_bwd (blkattn_bwd_window when window > 0) on torch CUDA tensors;
    dq, dk, dv are written in place."""
    lib = load()
    descs = [describe(t) for t in (q, k, v, seqlens_k, q_logical_pos, mask_bias, out, lse, dout, dq, dk, dv)]
    sh = _stream_handle(stream) if q.is_cuda else None
    if window:
        st = lib.blkattn_bwd_window(*[_ref(x) for x in descs[:5]], ctypes.c_int64(int(window)), _ref(descs[5]),
                                    ctypes.c_float(scale), *[_ref(x) for x in descs[6:]], sh)
    else:
        st = lib.blkattn_bwd(*[_ref(x) for x in descs[:6]], ctypes.c_float(scale),
                             *[_ref(x) for x in descs[6:]], sh)
    _check(st)
    return dq, dk, dv


def attention_backward(q, k, v, seqlens_k, q_logical_pos, out, lse, dout, mask_bias=None, scale=None,
                       stream=None, window: int = 0):
    """Allocate fp32 dq, dk, dv and call bwd (scale defaults to 1/sqrt(d))."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    dq, dk, dv = _outputs(stream, *((t.shape, torch.float32, t.device) for t in (q, k, v)))
    return bwd(q, k, v, seqlens_k, q_logical_pos, mask_bias, scale, out, lse, dout, dq, dk, dv, stream, window=window)


def fwd_static_scratch(q, k, v, seqlens_k, q_logical_pos, mask_bias, scale: float, out, lse,
                       stream=None):
    """blkattn_fwd_static_scratch: the same call as fwd, for callers that must
    not allocate device memory at call time; the per-split scratch is a fixed
    16 MiB array inside the library (shared by all calls on a device, so calls
    must not overlap on the GPU).  Raises BlkattnError with ERR_SCRATCH_LIMIT
    when the problem needs more scratch than that."""
    lib = load()
    descs = [describe(t) for t in (q, k, v, seqlens_k, q_logical_pos, mask_bias, out, lse)]
    st = lib.blkattn_fwd_static_scratch(_ref(descs[0]), _ref(descs[1]), _ref(descs[2]), _ref(descs[3]),
                                        _ref(descs[4]), _ref(descs[5]), ctypes.c_float(scale),
                                        _ref(descs[6]), _ref(descs[7]),
                                        _stream_handle(stream) if q.is_cuda else None)
    _check(st)
    return out, lse


def attention(q, k, v, seqlens_k, q_logical_pos, mask_bias=None, scale=None,
              out_dtype=torch.float32, stream=None, tree=None, window: int = 0):
    """Allocate out/lse with torch and run blkattn_fwd (blkattn_fwd_tree with
    a token tree)."""
    B, Hq, Tq, d = q.shape
    if scale is None:
        scale = d ** -0.5
    out, lse = _outputs(stream, ((B, Hq, Tq, v.shape[3]), out_dtype, q.device), ((B, Hq, Tq), torch.float32, q.device))
    return fwd(q, k, v, seqlens_k, q_logical_pos, mask_bias, scale, out, lse, stream, tree=tree, window=window)


def spec_sample(p, q, draft, u_accept, u_sample, n_accepted=None, token=None, stream=None):
    """blkattn_spec_sample: one speculative verification step per sequence.
    p f32 [B,k+1,V], q f32 [B,k,V], draft int32 [B,k], u_accept f32 [B,k],
    u_sample int32 [B] (32 random bits).  Returns (n_accepted, token), int32 [B]."""
    lib = load()
    B = p.shape[0]
    if n_accepted is None:
        n_accepted, = _outputs(stream, ((B,), torch.int32, p.device))
    if token is None:
        token, = _outputs(stream, ((B,), torch.int32, p.device))
    descs = [describe(t) for t in (p, q, draft, u_accept, u_sample, n_accepted, token)]
    _check(lib.blkattn_spec_sample(*[_ref(d) for d in descs], _stream_handle(stream) if p.is_cuda else None))
    return n_accepted, token


def _layout(layout) -> int:
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"blkattn: layout {layout!r} is none of {sorted(ROPE_LAYOUTS)}")
    return code


def _handle(stream):
    """A stream argument as a handle; None (the current stream of the tensors' device) stays None."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def rope_angles(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, trained: float = 0.0,
                low: float = 1.0, high: float = 32.0):
    """(angles, mscale) of blkattn_rope_angles: the angle of one position for
    each of the rot / 2 pairs (list of floats) and the factor that goes with it."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"blkattn: scaling {scaling!r} is none of {sorted(ROPE_SCALINGS)}")
    spec = RopeSpec(int(rot), ROPE_SCALINGS[scaling], base, factor, trained, low, high)
    w = (ctypes.c_double * max(1, min(int(rot), 1024) // 2))()
    m = ctypes.c_float()
    _check(load().blkattn_rope_angles(ctypes.byref(spec), w, ctypes.byref(m)))
    return list(w), m.value


def rope_phases(angles, device="cuda"):
    """The phase table of angles (blkattn_rope_phases) on the device, made once and kept by the caller."""
    angles = [float(a) for a in angles]
    w = (ctypes.c_double * max(1, len(angles)))(*angles)
    f = (ctypes.c_int64 * max(1, len(angles)))()
    _check(load().blkattn_rope_phases(w, len(angles), f))
    return torch.tensor(list(f)[:len(angles)], dtype=torch.int64, device=device)


def rope(x, pos, phases, out=None, layout="half", mscale: float = 1.0, out_dtype=None, stream=None):
    """blkattn_rope: rows x [B,H,T,d] turned by their positions pos int32
    [B,T]; out (default: a new contiguous tensor) may be x itself."""
    st, out = (_bind or _load_bind()).rope(x, pos, phases, out, _layout(layout), mscale, out_dtype, _handle(stream),
                                           False)
    _check(st)
    return out


def rope_backward(dy, pos, phases, out=None, layout="half", mscale: float = 1.0, out_dtype=None, stream=None):
    """blkattn_rope_bwd: the gradient of rope's x from that of its result."""
    st, out = (_bind or _load_bind()).rope(dy, pos, phases, out, _layout(layout), mscale, out_dtype, _handle(stream),
                                           True)
    _check(st)
    return out


def paged_append(k, v, pos, page_table, k_pages, v_pages, phases=None, layout="half", mscale: float = 1.0, q=None,
                 q_out=None, stream=None):
    """blkattn_paged_append: rows k, v [B,H_kv,T,d] into the pools [N,H_kv,P,d]
    at the cache rows pos int32 [B,T] (negative: padding, not written) through
    page_table int32 [B,entries]; with phases, k and q turn on the way.
    Returns q_out (allocated as zeros, on the call's stream, when q is given
    without it: rows of padding stay unwritten), or None."""
    st, q_out = (_bind or _load_bind()).append(k, v, pos, page_table, k_pages, v_pages, phases, _layout(layout), mscale,
                                               q, q_out, _handle(stream))
    _check(st)
    return q_out


def fwd_paged(q, k_pages, v_pages, page_table, seqlens_k, q_logical_pos, scale: float, out, lse, stream=None,
              tree=None, window: int = 0):
    """blkattn_fwd_paged: attention over the pools k_pages, v_pages
    [N,H_kv,P,d] through page_table int32 [B,entries]; out and lse are written
    in place.  tree and window as for fwd."""
    st, out, lse = (_bind or _load_bind()).fwd(q, k_pages, v_pages, page_table, seqlens_k, q_logical_pos, tree, window,
                                               scale, out, lse, None, _handle(stream))
    _check(st)
    return out, lse


def attention_paged(q, k_pages, v_pages, page_table, seqlens_k, q_logical_pos, scale=None, out_dtype=torch.float32,
                    stream=None, tree=None, window: int = 0):
    """Allocate out/lse with torch and run blkattn_fwd_paged (scale defaults to 1/sqrt(d))."""
    st, out, lse = (_bind or _load_bind()).fwd(q, k_pages, v_pages, page_table, seqlens_k, q_logical_pos, tree, window,
                                               scale, None, None, out_dtype, _handle(stream))
    _check(st)
    return out, lse


def _states(m, l, u) -> States:
    s = States()
    s.m = m.data_ptr() if m.numel() else None
    s.l = None if l is None else (l.data_ptr() if l.numel() else None)
    s.u = u.data_ptr() if u.numel() else None
    s.rows = m.shape[0]
    s.d_v = u.shape[1]
    s.u_row_stride = u.stride(0)
    for t in (m, u) + (() if l is None else (l,)):
        if t.dtype != torch.float32:
            raise ValueError("blkattn: states are float32")
    if u.stride(1) != 1:
        raise ValueError("blkattn: state u must have unit column stride")
    return s


def merge(a, b, out, stream=None):
    """blkattn_merge on (m, l, u) triples of torch tensors (l may be None)."""
    lib = load()
    sa, sb, so = _states(*a), _states(*b), _states(*out)
    _check(lib.blkattn_merge(ctypes.byref(sa), ctypes.byref(sb), ctypes.byref(so), _stream_handle(stream)))
    return out


def check_device_error(stream=None) -> int:
    """Synchronise and read/clear the device error word (test hook)."""
    return int(load().blkattn_check_device_error(_stream_handle(stream)))


def stall_next_decode(cta: int) -> None:
    """Test hook: the next tcgen05 decode launch stops CTA ``cta`` (mod the
    CTA count) at a wait nothing completes; its bounded waits run out and
    check_device_error() then reports ERR_DEVICE_TIMEOUT."""
    load().blkattn_debug_stall_next_decode(int(cta))


def set_split_event(event) -> None:
    """Record ``event`` (a torch.cuda.Event) after the main kernel of every
    later fwd call, for timing the kernels apart; None switches it off."""
    if event is None:
        load().blkattn_debug_set_split_event(None)
        return
    event.record()  # make sure the underlying CUDA event exists
    load().blkattn_debug_set_split_event(event.cuda_event)


def debug_plan(B, Hq, Hkv, Tq, Tmax, d, dtype=torch.bfloat16, num_sms=152) -> dict:
    lib = load()
    p = Plan()
    _check(lib.blkattn_debug_plan(B, Hq, Hkv, Tq, Tmax, d, _DTYPES[dtype], num_sms, ctypes.byref(p)))
    return p.as_dict()
