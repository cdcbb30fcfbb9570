"""Thin ctypes binding of libfalcon (include/falcon.h), same entry-point names.

Argument marshalling only: every step of the forward pass runs in the CUDA
library. PyTorch supplies device memory and the current stream. The library
must have been built in-tree (``python -m delta_rule_linear_falcon_b200.build``);
there is no fallback, so a missing library raises at the first call.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfalcon.so")

FALCON_OK, FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED = 0, 1, 2
FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA, FALCON_ERR_TIMEOUT = 3, 4, 5
FALCON_RULE_1, FALCON_RULE_1A, FALCON_RULE_3, FALCON_RULE_3A = 1, 2, 3, 4
FALCON_RULE_2, FALCON_RULE_2A = 5, 6
FALCON_F32, FALCON_BF16 = 0, 1
FALCON_SAME_STEP = 0x100  # OR into a rule code: pair (k_t, v_t) at step t (same-step association)
FALCON_ACT_NONE, FALCON_ACT_SILU = 0, 1
FALCON_SCAN_SOFTPLUS = 1
FALCON_NORM_NONE, FALCON_NORM_RMS, FALCON_NORM_L2 = 0, 1, 2
FALCON_ROT_HALF, FALCON_ROT_PAIRS = 0, 1
ACTS = {"none": FALCON_ACT_NONE, "silu": FALCON_ACT_SILU}
NORMS = {"none": FALCON_NORM_NONE, "rms": FALCON_NORM_RMS, "l2": FALCON_NORM_L2}
ROTS = {"half": FALCON_ROT_HALF, "pairs": FALCON_ROT_PAIRS}
RULES = {"falcon1": FALCON_RULE_1, "falcon1a": FALCON_RULE_1A, "falcon3": FALCON_RULE_3,
         "falcon3a": FALCON_RULE_3A, "falcon2": FALCON_RULE_2, "falcon2a": FALCON_RULE_2A}


class FalconError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {falcon_status_string(status)} (status {status})")
        self.status = status


class FalconArgs(ctypes.Structure):
    """Mirror of falcon_args_t."""
    _fields_ = [
        ("rule", ctypes.c_int), ("io_dtype", ctypes.c_int),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p), ("eta", ctypes.c_void_p),
        ("eps", ctypes.c_float), ("window", ctypes.c_int), ("chunk", ctypes.c_int),
        ("S0", ctypes.c_void_p), ("k_prev", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("S_out", ctypes.c_void_p), ("k_last", ctypes.c_void_p),
        ("n0", ctypes.c_void_p), ("n_out", ctypes.c_void_p),
    ]


class FalconGrads(ctypes.Structure):
    """Mirror of falcon_grads_t."""
    _fields_ = [
        ("dO", ctypes.c_void_p), ("dS_T", ctypes.c_void_p),
        ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
        ("dalpha", ctypes.c_void_p), ("deta", ctypes.c_void_p),
        ("dS0", ctypes.c_void_p), ("dk_prev", ctypes.c_void_p),
    ]


_I, _P, _F32, _LL = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong


class FalconView(ctypes.Structure):
    """Mirror of falcon_view_t."""
    _fields_ = [("p", _P), ("sb", _LL), ("sh", _LL), ("st", _LL)]


class FalconConvArgs(ctypes.Structure):
    """Mirror of falcon_conv_args_t."""
    _fields_ = [("io_dtype", _I), ("B", _I), ("H", _I), ("T", _I), ("d", _I), ("K", _I), ("act", _I),
                ("x", FalconView), ("y", FalconView), ("w", _P), ("bias", _P), ("lengths", _P),
                ("state", _P), ("state_out", _P)]


class FalconConvGrads(ctypes.Structure):
    """Mirror of falcon_conv_grads_t."""
    _fields_ = [("dy", FalconView), ("dstate_out", _P), ("dx", FalconView), ("dw", _P), ("dbias", _P),
                ("dstate", _P)]


class FalconScanArgs(ctypes.Structure):
    """Mirror of falcon_scan_args_t."""
    _fields_ = [("io_dtype", _I), ("B", _I), ("H", _I), ("T", _I), ("dk", _I), ("dv", _I), ("flags", _I),
                ("q", FalconView), ("k", FalconView), ("v", FalconView), ("delta", FalconView),
                ("z", FalconView), ("o", FalconView), ("A", _P), ("D", _P), ("delta_bias", _P),
                ("lengths", _P), ("S0", _P), ("S_out", _P)]


class FalconScanGrads(ctypes.Structure):
    """Mirror of falcon_scan_grads_t."""
    _fields_ = [("dO", FalconView), ("dS_T", _P), ("dq", FalconView), ("dk", FalconView), ("dv", FalconView),
                ("ddelta", FalconView), ("dz", FalconView), ("dA", _P), ("dD", _P), ("ddelta_bias", _P),
                ("dS0", _P)]


class FalconQknormArgs(ctypes.Structure):
    """Mirror of falcon_qknorm_args_t."""
    _fields_ = [("io_dtype", _I), ("B", _I), ("Hq", _I), ("Hk", _I), ("T", _I), ("d", _I), ("norm", _I),
                ("rot", _I), ("rot_layout", _I), ("q", FalconView), ("k", FalconView), ("q_out", FalconView),
                ("k_out", FalconView), ("wq", _P), ("wk", _P), ("eps", _F32), ("freq", _P),
                ("positions", _P), ("lengths", _P)]


class FalconQknormGrads(ctypes.Structure):
    """Mirror of falcon_qknorm_grads_t."""
    _fields_ = [("dq_out", FalconView), ("dk_out", FalconView), ("dq", FalconView), ("dk", FalconView),
                ("dwq", _P), ("dwk", _P)]

# The same structs as bytes, for the calls below: packing takes a quarter of the time of filling a ctypes.Structure.
_VIEW = "Pqqq"
_CONV_ARGS, _CONV_GRADS = struct.Struct("@7i" + 2 * _VIEW + "5P"), struct.Struct("@" + _VIEW + "P" + _VIEW + "3P")
_SCAN_ARGS, _SCAN_GRADS = struct.Struct("@7i" + 6 * _VIEW + "6P"), struct.Struct("@" + _VIEW + "P" + 5 * _VIEW + "4P")
_QKNORM_ARGS, _QKNORM_GRADS = struct.Struct("@9i" + 4 * _VIEW + "2Pf3P"), struct.Struct("@" + 4 * _VIEW + "2P")

_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libfalcon.so from the package directory (raises if it is missing)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m delta_rule_linear_falcon_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            P = ctypes.POINTER(FalconArgs)
            vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            L.falcon_workspace_size.argtypes = [P]
            L.falcon_workspace_size.restype = ctypes.c_size_t
            L.falcon_fwd_chunk.argtypes = [P, vp, ctypes.c_size_t, vp]
            L.falcon_fwd_chunk.restype = i
            L.falcon_fwd_recurrent.argtypes = [P, vp]
            L.falcon_fwd_recurrent.restype = i
            L.falcon_bwd_workspace_size.argtypes = [P]
            L.falcon_bwd_workspace_size.restype = ctypes.c_size_t
            L.falcon_bwd_recurrent.argtypes = [P, ctypes.POINTER(FalconGrads), vp, ctypes.c_size_t, vp]
            L.falcon_bwd_recurrent.restype = i
            L.falcon_decode_step.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp, vp]
            L.falcon_decode_step.restype = i
            for name in ("conv", "scan", "qknorm"):
                A = G = vp   # the address of a struct, or its packed bytes
                fwd, bwd = getattr(L, f"falcon_{name}_fwd"), getattr(L, f"falcon_{name}_bwd")
                fwd.argtypes = [A, vp, ctypes.c_size_t, vp] if name == "scan" else [A, vp]
                bwd.argtypes = [A, G, vp, ctypes.c_size_t, vp]
                fwd.restype = bwd.restype = i
                size = getattr(L, f"falcon_{name}_bwd_workspace_size")
                size.argtypes, size.restype = [A], ctypes.c_size_t
                if name != "qknorm":
                    step = getattr(L, f"falcon_{name}_step")
                    step.argtypes, step.restype = [A, vp], i
            L.falcon_scan_workspace_size.argtypes = [vp]
            L.falcon_scan_workspace_size.restype = ctypes.c_size_t
            L.falcon_status_string.argtypes = [i]
            L.falcon_status_string.restype = ctypes.c_char_p
            L.falcon_check_device_errors.argtypes = [vp]
            L.falcon_check_device_errors.restype = i
            L.falcon_version.argtypes = []
            L.falcon_version.restype = i
            L.falcon_debug_stall_next_call.argtypes = [i, ctypes.c_longlong]
            L.falcon_debug_stall_next_call.restype = i
            _lib = L
    return _lib


def falcon_status_string(status: int) -> str:
    return lib().falcon_status_string(int(status)).decode()


def falcon_version() -> int:
    return int(lib().falcon_version())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FALCON_BF16
    if t.dtype == torch.float32:
        return FALCON_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _rule_code(rule) -> int:
    """A rule name or code; FALCON_SAME_STEP may be OR-ed into a code, or a name may end in
    '+same_step'."""
    if isinstance(rule, str):
        name, _, flag = rule.partition("+")
        return RULES[name] | (FALCON_SAME_STEP if flag == "same_step" else 0)
    return int(rule)


def make_args(q, k, v, alpha, eta, *, rule, eps=1e-6, window=1, chunk=64, S0=None, k_prev=None,
              o=None, S_out=None, k_last=None, n0=None, n_out=None) -> FalconArgs:
    """Fill falcon_args_t from tensors (shapes taken from k and v)."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    io = _dtype_code(k)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (k_prev, "k_prev"), (k_last, "k_last")):
        _need(t, n, k.dtype)
    for t, n in ((alpha, "alpha"), (eta, "eta"), (S0, "S0"), (S_out, "S_out"), (n0, "n0"), (n_out, "n_out")):
        _need(t, n, torch.float32)
    return FalconArgs(_rule_code(rule), io, B, H, T, dk, dv, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                      alpha.data_ptr(), eta.data_ptr(), float(eps), int(window), int(chunk),
                      _ptr(S0), _ptr(k_prev), o.data_ptr() if o is not None else None,
                      _ptr(S_out), _ptr(k_last), _ptr(n0), _ptr(n_out))


def _outputs(k, v, o, S_out, k_last, want_state: bool):
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=k.dtype, device=k.device)
    if S_out is None and want_state:
        S_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=k.device)
    if k_last is None and want_state:
        k_last = torch.empty((B, H, dk), dtype=k.dtype, device=k.device)
    return o, S_out, k_last


def falcon_workspace_size(args: FalconArgs) -> int:
    return int(lib().falcon_workspace_size(ctypes.byref(args)))


def falcon_fwd_chunk(q, k, v, alpha, eta, *, rule, eps=1e-6, window=1, chunk=64, S0=None,
                     k_prev=None, o=None, S_out=None, k_last=None, want_state=True,
                     workspace=None, stream=None):
    """Chunk-parallel forward pass. Returns (o, S_out, k_last).

    ``workspace`` is an optional contiguous CUDA tensor of at least
    ``falcon_workspace_size(args)`` bytes (nonzero where the library splits the sequence of
    an inner-product problem with few heads, and for the two-pass path of the regression
    rules, whose blocks' solved tiles it holds); when the size is nonzero and no tensor is
    given, one is allocated here with torch for the call (on the current stream, recorded
    on ``stream`` when that is another torch stream; pass your own when ``stream`` is a raw
    handle of a different stream). A smaller tensor runs the regression rules in one
    kernel."""
    o, S_out, k_last = _outputs(k, v, o, S_out, k_last, want_state)
    args = make_args(q, k, v, alpha, eta, rule=rule, eps=eps, window=window, chunk=chunk, S0=S0,
                     k_prev=k_prev, o=o, S_out=S_out, k_last=k_last)
    need = falcon_workspace_size(args)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
        ws_ptr, ws_bytes = workspace.data_ptr(), need
        if isinstance(stream, torch.cuda.Stream):
            # the caching allocator may hand the block out again once this call returns; tie its
            # reuse to the kernels queued on the caller's stream
            workspace.record_stream(stream)
    st = lib().falcon_fwd_chunk(ctypes.byref(args), ws_ptr, ws_bytes, _stream(stream))
    if st != FALCON_OK:
        raise FalconError(st, "falcon_fwd_chunk")
    return o, S_out, k_last


def falcon_fwd_recurrent(q, k, v, alpha, eta, *, rule, eps=1e-6, window=1, S0=None, k_prev=None,
                         o=None, S_out=None, k_last=None, want_state=True, n0=None, n_out=None,
                         stream=None):
    """Recurrent forward pass (fp32 arithmetic). Returns (o, S_out, k_last); for Falcon-2/2A
    pass n_out (B, H, dk) fp32 to receive the running column energies (n0 to start from them)."""
    o, S_out, k_last = _outputs(k, v, o, S_out, k_last, want_state)
    args = make_args(q, k, v, alpha, eta, rule=rule, eps=eps, window=window, chunk=64, S0=S0,
                     k_prev=k_prev, o=o, S_out=S_out, k_last=k_last, n0=n0, n_out=n_out)
    st = lib().falcon_fwd_recurrent(ctypes.byref(args), _stream(stream))
    if st != FALCON_OK:
        raise FalconError(st, "falcon_fwd_recurrent")
    return o, S_out, k_last


def falcon_bwd_workspace_size(args: FalconArgs) -> int:
    return int(lib().falcon_bwd_workspace_size(ctypes.byref(args)))


def falcon_bwd_recurrent(q, k, v, alpha, eta, dO, *, rule, eps=1e-6, window=1, S0=None, k_prev=None,
                         dS_T=None, want_dS0=True, workspace=None, stream=None):
    """Gradients of the recurrent form for upstream gradients dO (B, H, T, dv) fp32 of the
    outputs and dS_T (B, H, dv, dk) fp32 (or None) of the final state. Returns a dict of fp32
    tensors dq, dk, dv, dalpha, deta, dS0 (None unless want_dS0) and dk_prev (None without
    k_prev). ``workspace``: a CUDA tensor of at least falcon_bwd_workspace_size(args) bytes, or
    None to allocate one here for the call."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dev = k.device
    f32 = torch.float32
    _need(dO, "dO", f32)
    _need(dS_T, "dS_T", f32)
    out = {"dq": torch.empty((B, H, T, dk), dtype=f32, device=dev),
           "dk": torch.empty((B, H, T, dk), dtype=f32, device=dev),
           "dv": torch.empty((B, H, T, dv), dtype=f32, device=dev),
           "dalpha": torch.empty((B, H, T), dtype=f32, device=dev),
           "deta": torch.empty((B, H, T), dtype=f32, device=dev),
           "dS0": torch.empty((B, H, dv, dk), dtype=f32, device=dev) if want_dS0 else None,
           "dk_prev": torch.empty((B, H, dk), dtype=f32, device=dev) if k_prev is not None else None}
    args = make_args(q, k, v, alpha, eta, rule=rule, eps=eps, window=window, chunk=64, S0=S0, k_prev=k_prev)
    grads = FalconGrads(dO.data_ptr(), _ptr(dS_T), out["dq"].data_ptr(), out["dk"].data_ptr(),
                        out["dv"].data_ptr(), out["dalpha"].data_ptr(), out["deta"].data_ptr(),
                        _ptr(out["dS0"]), _ptr(out["dk_prev"]))
    need = falcon_bwd_workspace_size(args)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().falcon_bwd_recurrent(ctypes.byref(args), ctypes.byref(grads), ws_ptr, ws_bytes, _stream(stream))
    if st != FALCON_OK:
        raise FalconError(st, "falcon_bwd_recurrent")
    return out


def falcon_decode_step(S, k_prev, q, k, v, alpha, eta, *, rule="falcon1", eps=1e-6, o=None,
                       stream=None):
    """One decode token for (N, H) heads; S and k_prev are updated in place. Returns o."""
    N, H, dv, dk = S.shape
    _need(S, "S", torch.float32)
    for t, n in ((k_prev, "k_prev"), (q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(alpha, "alpha", torch.float32)
    _need(eta, "eta", torch.float32)
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    _need(o, "o", q.dtype)
    st = lib().falcon_decode_step(_rule_code(rule), _dtype_code(q), N, H, dk, dv, S.data_ptr(),
                                  k_prev.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                  alpha.data_ptr(), eta.data_ptr(), float(eps), o.data_ptr(),
                                  _stream(stream))
    if st != FALCON_OK:
        raise FalconError(st, "falcon_decode_step")
    return o


# ---- operators around the memory: convolution, selective scan, q/k norm ------------------------------
#
# Sequence tensors are (B, H, T, d) torch views of any batch, head and token strides whose last axis is
# contiguous (a transposed slice of a fused projection goes in as it is). Every tensor of a call is on one
# device, which need not be the current one. Outputs and workspaces that a call makes are allocated on
# `stream` (default: the device's current stream), where its kernels run.

_NO_VIEW = (0, 0, 0, 0)
_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """The context in which a call allocates, and the raw stream on which it launches."""
    if stream is None:
        ctx = _HERE if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)
        return ctx, torch._C._cuda_getCurrentRawStream(dev.index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _rank(t, name, rank):
    """The tensor that a call takes its device and type from."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != rank:
        raise ValueError(f"{name} must have {rank} axes, got the shape {tuple(t.shape)}")


def _refuse(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _seq(t, name, shape, dtype, dev):
    """falcon_view_t of a (B, H, T, d) tensor, or of a (B, H, d) one as a single token."""
    if t is None:
        return _NO_VIEW
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
        _refuse(t, name, shape, dtype, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return (t.data_ptr(), s[0], s[1], s[2] if len(s) == 4 else 0)


def _arr(t, name, shape, dtype, dev):
    """Address of a contiguous parameter, state or gradient, or 0."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
        _refuse(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def _code(table, key, what) -> int:
    if key not in table:
        raise ValueError(f"{what} must be one of {sorted(table)}, got {key!r}")
    return table[key]


def _call(name, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != FALCON_OK:
        raise FalconError(st, name)


def _dense(shape, dtype, dev):
    """An uninitialised contiguous tensor."""
    strides = (1,)
    for n in shape[:0:-1]:
        strides = (n * strides[0],) + strides
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


def _token_major(B, H, T, d, dev):
    """An uninitialised fp32 (B, H, T, d) view of token-major rows."""
    return torch.empty_strided((B, H, T, d), (T * H * d, d, H * d, 1), dtype=torch.float32, device=dev)


def _rows(t, T, H, d):
    """falcon_view_t of what _token_major made (all zeros for None)."""
    return _NO_VIEW if t is None else (t.data_ptr(), T * H * d, d, H * d)


def _token_majors(n, B, H, T, d, dev):
    """n of them, made together."""
    return torch.empty_strided((n, B, H, T, d), (B * T * H * d, T * H * d, d, H * d, 1), dtype=torch.float32, device=dev).unbind()


def _workspace(workspace, need, dev):
    """(tensor, address, bytes) of the caller's workspace or of one made here."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    _need(workspace, "workspace")
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, other tensors on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _conv_args(x, w, bias, act, state, lengths, shape, state_shape, y, state_out):
    dev, io, f32 = x.device, x.dtype, torch.float32
    B, H, d = shape[0], shape[1], shape[-1]
    K = w.shape[2]
    return _CONV_ARGS.pack(
        _dtype_code(x), B, H, shape[2] if len(shape) == 4 else 1, d, K, _code(ACTS, act, "act"),
        *_seq(x, "x", shape, io, dev), *_seq(y, "y", shape, io, dev), _arr(w, "w", (H, d, K), f32, dev),
        _arr(bias, "bias", (H, d), f32, dev), _arr(lengths, "lengths", (B,), torch.int32, dev),
        _arr(state, "state", state_shape, io, dev), _arr(state_out, "state_out", state_shape, io, dev))


def make_conv_args(x, w, *, bias=None, act="silu", state=None, lengths=None, y=None, state_out=None) -> FalconConvArgs:
    """The argument struct of falcon_conv_fwd / _bwd for these tensors, for falcon_conv_bwd_workspace_size."""
    _rank(x, "x", 4)
    _rank(w, "w", 3)
    B, H, T, d = shape = tuple(x.shape)
    return FalconConvArgs.from_buffer_copy(_conv_args(x, w, bias, act, state, lengths, shape, (B, H, max(w.shape[2] - 1, 0), d), y, state_out))


def falcon_conv_bwd_workspace_size(args: FalconConvArgs) -> int:
    return int((_lib or lib()).falcon_conv_bwd_workspace_size(ctypes.byref(args)))


def falcon_conv_fwd(x, w, *, bias=None, act="silu", state=None, lengths=None, y=None, state_out=None,
                    want_state=False, stream=None):
    """Causal depthwise convolution over the last K tokens: x (B, H, T, d), w (H, d, K) fp32. Returns
    (y, state_out); y is head-major (B, H, T, d) unless given, state_out (B, H, K - 1, d) is the last
    K - 1 inputs, made where want_state asks for it (it may be `state` itself). With ``lengths`` (B,)
    int32, rows of y behind a sequence's end are left as they were (uninitialised in a y made here)."""
    _rank(x, "x", 4)
    _rank(w, "w", 3)
    shape = B, H, T, d = tuple(x.shape)
    tail = (B, H, max(w.shape[2] - 1, 0), d)
    ctx, raw = _on(x.device, stream)
    with ctx:
        if y is None:
            y = _dense(shape, x.dtype, x.device)
        if state_out is None and want_state:
            state_out = _dense(tail, x.dtype, x.device)
        a = _conv_args(x, w, bias, act, state, lengths, shape, tail, y, state_out)
        _call("falcon_conv_fwd", a, raw)
    return y, state_out


def falcon_conv_step(x, w, state, *, bias=None, act="silu", state_out=None, y=None, stream=None):
    """One token of the convolution for N sequences: x (N, H, d), state (N, H, K - 1, d), which is updated
    in place unless state_out is given. Returns y (N, H, d)."""
    _rank(x, "x", 3)
    _rank(w, "w", 3)
    shape = N, H, d = tuple(x.shape)
    ctx, raw = _on(x.device, stream)
    with ctx:
        if y is None:
            y = _dense(shape, x.dtype, x.device)
        a = _conv_args(x, w, bias, act, state, None, shape, (N, H, max(w.shape[2] - 1, 0), d), y,
                       state if state_out is None else state_out)
        _call("falcon_conv_step", a, raw)
    return y


def falcon_conv_bwd(x, w, dy, *, bias=None, act="silu", state=None, lengths=None, dstate_out=None, dx=None,
                    workspace=None, stream=None):
    """Gradients of falcon_conv_fwd for dy (B, H, T, d) fp32 and dstate_out (B, H, K - 1, d) fp32 or None.
    Returns a dict of fp32 tensors dx (token-major rows like a projection's, seen as (B, H, T, d), unless
    given), dw, dbias (None without bias) and dstate (None without state). ``workspace``: a CUDA tensor of at least
    falcon_conv_bwd_workspace_size(make_conv_args(x, w)) bytes, or None to allocate one here for the call."""
    _rank(x, "x", 4)
    _rank(w, "w", 3)
    f32, dev = torch.float32, x.device
    shape = B, H, T, d = tuple(x.shape)
    K = w.shape[2]
    tail = (B, H, max(K - 1, 0), d)
    ctx, raw = _on(dev, stream)
    with ctx:
        if dx is None:
            dx = _token_major(B, H, T, d, dev)
            to = _rows(dx, T, H, d)
        else:
            to = _seq(dx, "dx", shape, f32, dev)
        out = {"dx": dx, "dw": _dense((H, d, K), f32, dev),
               "dbias": _dense((H, d), f32, dev) if bias is not None else None,
               "dstate": _dense(tail, f32, dev) if state is not None else None}
        a = _conv_args(x, w, bias, act, state, lengths, shape, tail, None, None)
        g = _CONV_GRADS.pack(*_seq(dy, "dy", shape, f32, dev), _arr(dstate_out, "dstate_out", tail, f32, dev),
                             *to, _at(out["dw"]), _at(out["dbias"]), _at(out["dstate"]))
        need = int((_lib or lib()).falcon_conv_bwd_workspace_size(a))
        workspace, p, n = _workspace(workspace, need, dev)
        _call("falcon_conv_bwd", a, g, p, n, raw)
    return out


def _scan_shapes(k, v, rank):
    """(B, H, T, dk, dv), the shape of v and that of k."""
    _rank(v, "v", rank)
    _rank(k, "k", rank)
    vs = tuple(v.shape)
    dk = k.shape[-1]
    return (vs[0], vs[1], vs[2] if rank == 4 else 1, dk, vs[-1]), vs, vs[:-1] + (dk,)


def _scan_args(sizes, vs, ks, q, k, v, delta, A, D, z, delta_bias, softplus, lengths, S0, o, S_out):
    B, H, T, dk, dv = sizes
    dev, io, f32 = v.device, v.dtype, torch.float32
    state = (B, H, dv, dk)
    return _SCAN_ARGS.pack(
        _dtype_code(v), B, H, T, dk, dv, FALCON_SCAN_SOFTPLUS if softplus else 0, *_seq(q, "q", ks, io, dev),
        *_seq(k, "k", ks, io, dev), *_seq(v, "v", vs, io, dev), *_seq(delta, "delta", vs, io, dev),
        *_seq(z, "z", vs, io, dev), *_seq(o, "o", vs, io, dev), _arr(A, "A", (H, dv, dk), f32, dev), _arr(D, "D", (H, dv), f32, dev),
        _arr(delta_bias, "delta_bias", (H, dv), f32, dev), _arr(lengths, "lengths", (B,), torch.int32, dev),
        _arr(S0, "S0", state, f32, dev), _arr(S_out, "S_out", state, f32, dev))


def make_scan_args(q, k, v, delta, A, *, D=None, z=None, delta_bias=None, softplus=True, S0=None, lengths=None, o=None,
                   S_out=None) -> FalconScanArgs:
    """The argument struct of falcon_scan_fwd / _bwd for these tensors, for falcon_scan_workspace_size and
    falcon_scan_bwd_workspace_size."""
    sizes, vs, ks = _scan_shapes(k, v, 4)
    return FalconScanArgs.from_buffer_copy(_scan_args(sizes, vs, ks, q, k, v, delta, A, D, z, delta_bias, softplus, lengths, S0, o, S_out))


def falcon_scan_workspace_size(args: FalconScanArgs) -> int:
    return int((_lib or lib()).falcon_scan_workspace_size(ctypes.byref(args)))


def falcon_scan_bwd_workspace_size(args: FalconScanArgs) -> int:
    return int((_lib or lib()).falcon_scan_bwd_workspace_size(ctypes.byref(args)))


def falcon_scan_fwd(q, k, v, delta, A, *, D=None, z=None, delta_bias=None, softplus=True, S0=None, lengths=None,
                    o=None, S_out=None, want_state=True, workspace=None, stream=None):
    """Selective scan: q, k (B, H, T, dk), v, delta and z (B, H, T, dv), A (H, dv, dk), D and delta_bias
    (H, dv), S0 (B, H, dv, dk); parameters and states fp32. Returns (o, S_out). With few channels the
    sequence is split, for which a workspace of falcon_scan_workspace_size(make_scan_args(q, k, v, delta, A)) bytes is
    made here unless one is given (a smaller one runs it whole)."""
    sizes, vs, ks = _scan_shapes(k, v, 4)
    B, H, T, dk, dv = sizes
    dev = v.device
    ctx, raw = _on(dev, stream)
    with ctx:
        if o is None:
            o = _dense(vs, v.dtype, dev)
        if S_out is None and want_state:
            S_out = _dense((B, H, dv, dk), torch.float32, dev)
        a = _scan_args(sizes, vs, ks, q, k, v, delta, A, D, z, delta_bias, softplus, lengths, S0, o, S_out)
        need = int((_lib or lib()).falcon_scan_workspace_size(a)) if workspace is None else 0
        workspace, p, n = _workspace(workspace, need, dev)
        _call("falcon_scan_fwd", a, p, n, raw)
    return o, S_out


def falcon_scan_step(q, k, v, delta, A, S, *, D=None, z=None, delta_bias=None, softplus=True, S_out=None, o=None,
                     stream=None):
    """One token of the scan for N sequences: q, k (N, H, dk), v, delta, z (N, H, dv); S (N, H, dv, dk) fp32 is
    updated in place unless S_out is given. Returns o (N, H, dv)."""
    sizes, vs, ks = _scan_shapes(k, v, 3)
    ctx, raw = _on(v.device, stream)
    with ctx:
        if o is None:
            o = _dense(vs, v.dtype, v.device)
        a = _scan_args(sizes, vs, ks, q, k, v, delta, A, D, z, delta_bias, softplus, None, S, o, S if S_out is None else S_out)
        _call("falcon_scan_step", a, raw)
    return o


def falcon_scan_bwd(q, k, v, delta, A, dO, *, D=None, z=None, delta_bias=None, softplus=True, S0=None, lengths=None,
                    dS_T=None, workspace=None, stream=None):
    """Gradients of falcon_scan_fwd for dO (B, H, T, dv) fp32 and dS_T (B, H, dv, dk) fp32 or None. Returns a
    dict of fp32 tensors dq, dk, dv, ddelta, dA and, for the inputs that were given, dD, ddelta_bias, dz, dS0
    (None otherwise). Sequence gradients are token-major rows seen as (B, H, T, d). ``workspace``: a CUDA tensor of at
    least falcon_scan_bwd_workspace_size(make_scan_args(q, k, v, delta, A)) bytes, or None to allocate one here."""
    sizes, vs, ks = _scan_shapes(k, v, 4)
    B, H, T, dk, dv = sizes
    dev, f32 = v.device, torch.float32
    ctx, raw = _on(dev, stream)
    with ctx:
        dq, dk_ = _token_majors(2, B, H, T, dk, dev)
        wide = _token_majors(2 if z is None else 3, B, H, T, dv, dev)
        out = {"dq": dq, "dk": dk_, "dv": wide[0], "ddelta": wide[1], "dz": None if z is None else wide[2],
               "dA": _dense((H, dv, dk), f32, dev),
               "dD": _dense((H, dv), f32, dev) if D is not None else None,
               "ddelta_bias": _dense((H, dv), f32, dev) if delta_bias is not None else None,
               "dS0": _dense((B, H, dv, dk), f32, dev) if S0 is not None else None}
        a = _scan_args(sizes, vs, ks, q, k, v, delta, A, D, z, delta_bias, softplus, lengths, S0, None, None)
        g = _SCAN_GRADS.pack(*_seq(dO, "dO", vs, f32, dev), _arr(dS_T, "dS_T", (B, H, dv, dk), f32, dev),
                             *_rows(dq, T, H, dk), *_rows(dk_, T, H, dk), *_rows(wide[0], T, H, dv),
                             *_rows(wide[1], T, H, dv), *_rows(out["dz"], T, H, dv), _at(out["dA"]), _at(out["dD"]), _at(out["ddelta_bias"]), _at(out["dS0"]))
        need = int((_lib or lib()).falcon_scan_bwd_workspace_size(a))
        workspace, p, n = _workspace(workspace, need, dev)
        _call("falcon_scan_bwd", a, g, p, n, raw)
    return out


def _qknorm_shapes(q, k):
    """The tensor that is there (q or k may be None: no heads of it), and the shapes of q and k."""
    x = q if q is not None else k
    if x is None:
        raise TypeError("q or k must be given")
    for t, n in ((q, "q"), (k, "k")):
        if t is not None:
            _rank(t, n, 4)
    B, _, T, d = x.shape
    return x, (B, q.shape[1] if q is not None else 0, T, d), (B, k.shape[1] if k is not None else 0, T, d)


def _qknorm_args(x, qs, ks, q, k, q_out, k_out, wq, wk, norm, eps, rot, layout, freq, positions, lengths):
    dev, io, f32 = x.device, x.dtype, torch.float32
    B, Hq, T, d = qs
    rot = int(rot)
    return _QKNORM_ARGS.pack(
        _dtype_code(x), B, Hq, ks[1], T, d, _code(NORMS, norm, "norm"), rot, _code(ROTS, layout, "layout"),
        *_seq(q, "q", qs, io, dev), *_seq(k, "k", ks, io, dev), *_seq(q_out, "q_out", qs, io, dev),
        *_seq(k_out, "k_out", ks, io, dev),
        _arr(wq, "wq", (d,), f32, dev), _arr(wk, "wk", (d,), f32, dev), float(eps), _arr(freq, "freq", (rot // 2,), f32, dev),
        _arr(positions, "positions", (B, T), torch.int32, dev), _arr(lengths, "lengths", (B,), torch.int32, dev))


def make_qknorm_args(q, k, *, wq=None, wk=None, norm="rms", eps=1e-6, rot=0, layout="half", freq=None, positions=None,
                     lengths=None, q_out=None, k_out=None) -> FalconQknormArgs:
    """The argument struct of falcon_qknorm_fwd / _bwd for these tensors, for falcon_qknorm_bwd_workspace_size (which
    needs freq where rot > 0)."""
    x, qs, ks = _qknorm_shapes(q, k)
    return FalconQknormArgs.from_buffer_copy(_qknorm_args(x, qs, ks, q, k, q_out, k_out, wq, wk, norm, eps, rot, layout, freq, positions, lengths))


def falcon_qknorm_bwd_workspace_size(args: FalconQknormArgs) -> int:
    return int((_lib or lib()).falcon_qknorm_bwd_workspace_size(ctypes.byref(args)))


def falcon_qknorm_fwd(q, k, *, wq=None, wk=None, norm="rms", eps=1e-6, rot=0, layout="half", freq=None, positions=None,
                      lengths=None, q_out=None, k_out=None, stream=None):
    """Norm of each head's rows of q (B, Hq, T, d) and k (B, Hk, T, d) with the rotation of their first ``rot``
    channels by positions (B, T) int32 (default: 0, 1, ..) times freq (rot / 2) fp32. Either of q and k may be
    None. Returns (q_out, k_out), head-major unless given; q_out may be q itself, k_out k."""
    x, qs, ks = _qknorm_shapes(q, k)
    ctx, raw = _on(x.device, stream)
    with ctx:
        if q_out is None and q is not None:
            q_out = _dense(qs, x.dtype, x.device)
        if k_out is None and k is not None:
            k_out = _dense(ks, x.dtype, x.device)
        a = _qknorm_args(x, qs, ks, q, k, q_out, k_out, wq, wk, norm, eps, rot, layout, freq, positions, lengths)
        _call("falcon_qknorm_fwd", a, raw)
    return q_out, k_out


def falcon_qknorm_bwd(q, k, dq_out, dk_out, *, wq=None, wk=None, norm="rms", eps=1e-6, rot=0, layout="half", freq=None,
                      positions=None, lengths=None, workspace=None, stream=None):
    """Gradients of falcon_qknorm_fwd for dq_out, dk_out (fp32, the shapes of q and k). Returns a dict of fp32
    tensors dq, dk (token-major rows seen as (B, H, T, d); None where q or k is), dwq and dwk (None without
    the weight). ``workspace`` (used where a weight is given): a CUDA tensor of at least
    falcon_qknorm_bwd_workspace_size(make_qknorm_args(q, k)) bytes, or None to allocate one here for the call."""
    x, qs, ks = _qknorm_shapes(q, k)
    dev, f32 = x.device, torch.float32
    ctx, raw = _on(dev, stream)
    with ctx:
        rows = lambda s: _token_major(*s, dev)
        out = {"dq": rows(qs) if q is not None else None, "dk": rows(ks) if k is not None else None,
               "dwq": _dense(qs[3:], f32, dev) if wq is not None else None,
               "dwk": _dense(qs[3:], f32, dev) if wk is not None else None}
        a = _qknorm_args(x, qs, ks, q, k, None, None, wq, wk, norm, eps, rot, layout, freq, positions, lengths)
        g = _QKNORM_GRADS.pack(*_seq(dq_out, "dq_out", qs, f32, dev), *_seq(dk_out, "dk_out", ks, f32, dev),
                               *_rows(out["dq"], qs[2], qs[1], qs[3]), *_rows(out["dk"], ks[2], ks[1], ks[3]),
                               _at(out["dwq"]), _at(out["dwk"]))
        need = int((_lib or lib()).falcon_qknorm_bwd_workspace_size(a)) if wq is not None or wk is not None else 0
        workspace, p, n = _workspace(workspace, need, dev)
        _call("falcon_qknorm_bwd", a, g, p, n, raw)
    return out


def falcon_debug_stall_next_call(block: int, wait_budget_cycles: int) -> int:
    """Test hook: the next chunk call of this thread stalls its TMA producers at ``block`` and
    gives up its waits after ``wait_budget_cycles`` SM clocks (see include/falcon.h)."""
    return int(lib().falcon_debug_stall_next_call(int(block), int(wait_budget_cycles)))


def falcon_check_device_errors(stream=None) -> int:
    return int(lib().falcon_check_device_errors(_stream(stream)))
