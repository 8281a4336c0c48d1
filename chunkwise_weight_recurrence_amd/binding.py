"""ctypes binding of libttt.so: same entry points as ``include/ttt.h``.

Argument marshalling only.  Tensors (torch, on the GPU) are passed as raw
device pointers; ``None`` becomes NULL; a plain int is taken as a pointer.
Every computation happens in the library's HIP kernels.  A missing library
raises at load time: there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from enum import IntEnum

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libttt.so")

EXPORTS = ("ttt_workspace_size", "ttt_saved_size", "ttt_chunk_fwd", "ttt_chunk_bwd", "inplace_ttt_workspace_size",
           "inplace_ttt_fwd", "inplace_ttt_guarded_workspace_size", "inplace_ttt_fwd_guarded",
           "inplace_ttt_bwd_workspace_size", "inplace_ttt_bwd", "inplace_ttt_bwd_guarded_workspace_size",
           "inplace_ttt_bwd_guarded", "ttt_mlp_workspace_size", "ttt_mlp_chunk_fwd",
           "ttt_mlp_bwd_workspace_size", "ttt_mlp_chunk_bwd", "ttt_mlp_saved_size",
           "ttt_last_error", "ttt_version", "ttt_timing_enable", "ttt_timing_read", "ttt_chunk_bwd_noalloc",
           "ttt_noalloc_scratch_bytes", "ttt_recurrence_workspace_size", "ttt_recurrence_saved_size",
           "ttt_recurrence_fwd", "ttt_recurrence_bwd", "ttt_recurrence_step", "ttt_layernorm_fwd",
           "ttt_layernorm_workspace_size", "ttt_layernorm_bwd")


class Status(IntEnum):
    OK = 0
    INVALID_ARG = -1
    UNSUPPORTED = -2
    WORKSPACE = -3
    HIP = -4


class DType(IntEnum):
    F32 = 0
    BF16 = 1


class Loss(IntEnum):
    MSE = 0
    IP = 1
    L1 = 2
    RMSE = 3


class Act(IntEnum):
    NONE = 0
    SILU = 1
    GELU = 2
    NORM = 3


class Decay(IntEnum):
    NONE = 0
    SCALAR = 1
    VECTOR = 2


class Gate(IntEnum):
    SIGMOID = 0
    LOG = 1


class RecInput(IntEnum):
    PLAIN = 0
    CONVEX = 1


class Kernel(IntEnum):
    """Mirror of ``ttt_kernel`` (per-kernel timing ids)."""
    FWD = 0
    BWD_SEQ = 1
    BWD_CROSS = 2
    DGAMMA = 3
    GENERIC_FWD = 4
    GENERIC_BWD = 5
    DECAY_CUMSUM = 6
    INPLACE_APPLY = 7
    INPLACE_UPDATE = 8
    DECAY_PREP = 9
    INPLACE_NORM = 10
    LIN_STATE = 11
    LIN_SCAN = 12
    LIN_OUT = 13
    INPLACE_BWD_W = 14
    INPLACE_BWD_DZ = 15
    INPLACE_BWD_DV = 16
    INPLACE_BWD_DW = 17
    MLP_FWD = 18
    MLP_BWD = 19
    NORM_FWD = 20
    NORM_BWD = 21
    NORM_QUERY = 22
    NORM_BWD_PRE = 23
    MLP_QUERY = 24
    MLP_BWD_PRE = 25
    REC_FWD = 26
    REC_BWD = 27
    REC_STEP = 28
    LN_FWD = 29
    LN_BWD = 30
    LN_REDUCE = 31
    REC_CLEAR = 32


ENTRY_FWD = 0
ENTRY_BWD = 1


class TTTDesc(ctypes.Structure):
    """Mirror of ``ttt_desc``."""
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("C", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("loss", ctypes.c_int32), ("act", ctypes.c_int32),
                ("decay", ctypes.c_int32), ("lr_bias", ctypes.c_float)]


class TTTMlpDesc(ctypes.Structure):
    """Mirror of ``ttt_mlp_desc``."""
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dh", ctypes.c_int32), ("dv", ctypes.c_int32), ("C", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("loss", ctypes.c_int32), ("act", ctypes.c_int32),
                ("decay", ctypes.c_int32), ("lr_bias", ctypes.c_float)]


class TTTRecDesc(ctypes.Structure):
    """Mirror of ``ttt_rec_desc``."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("packed", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32), ("input", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldg", ctypes.c_int64)]


class TTTLnDesc(ctypes.Structure):
    """Mirror of ``ttt_ln_desc``."""
    _fields_ = [("rows", ctypes.c_int64), ("ldx", ctypes.c_int64), ("D", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("period", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class TTTError(RuntimeError):
    def __init__(self, status, message):
        self.status = Status(status) if status in Status._value2member_map_ else status
        super().__init__(f"{self.status!r}: {message}")


_lib = None


def lib():
    """Load libttt.so (once).  Raises OSError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise OSError(f"{LIB_PATH} is missing: build it with "
                      "`python -m chunkwise_weight_recurrence_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    dptr = ctypes.POINTER(TTTDesc)
    L.ttt_workspace_size.argtypes = [dptr, i32, ctypes.POINTER(sz)]
    L.ttt_workspace_size.restype = i32
    L.ttt_saved_size.argtypes = [dptr, ctypes.POINTER(sz)]
    L.ttt_saved_size.restype = i32
    L.ttt_chunk_fwd.argtypes = [dptr] + [vp] * 11 + [vp, sz, vp]
    L.ttt_chunk_fwd.restype = i32
    L.ttt_chunk_bwd.argtypes = [dptr] + [vp] * 18 + [vp, sz, vp]
    L.ttt_chunk_bwd.restype = i32
    L.ttt_chunk_bwd_noalloc.argtypes = [dptr] + [vp] * 18 + [vp]
    L.ttt_chunk_bwd_noalloc.restype = i32
    L.ttt_noalloc_scratch_bytes.argtypes = []
    L.ttt_noalloc_scratch_bytes.restype = sz
    L.inplace_ttt_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.inplace_ttt_workspace_size.restype = i32
    L.inplace_ttt_fwd.argtypes = [i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    L.inplace_ttt_fwd.restype = i32
    L.inplace_ttt_guarded_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.inplace_ttt_guarded_workspace_size.restype = i32
    L.inplace_ttt_fwd_guarded.argtypes = [i32, i32, i32, i32, i32, f32, f32, ctypes.POINTER(ctypes.c_int64), i32,
                                          vp, vp, vp, vp, vp, vp, sz, vp]
    L.inplace_ttt_fwd_guarded.restype = i32
    L.inplace_ttt_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.inplace_ttt_bwd_workspace_size.restype = i32
    L.inplace_ttt_bwd.argtypes = [i32, i32, i32, i32, i32, f32] + [vp] * 9 + [sz, vp]
    L.inplace_ttt_bwd.restype = i32
    L.inplace_ttt_bwd_guarded_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.inplace_ttt_bwd_guarded_workspace_size.restype = i32
    L.inplace_ttt_bwd_guarded.argtypes = [i32, i32, i32, i32, i32, f32, f32, ctypes.POINTER(ctypes.c_int64), i32] + \
        [vp] * 12 + [sz, vp]
    L.inplace_ttt_bwd_guarded.restype = i32
    mptr = ctypes.POINTER(TTTMlpDesc)
    L.ttt_mlp_workspace_size.argtypes = [mptr, ctypes.POINTER(sz)]
    L.ttt_mlp_workspace_size.restype = i32
    L.ttt_mlp_chunk_fwd.argtypes = [mptr] + [vp] * 13 + [vp, sz, vp]
    L.ttt_mlp_saved_size.argtypes = [mptr, ctypes.POINTER(sz)]
    L.ttt_mlp_saved_size.restype = i32
    L.ttt_mlp_chunk_fwd.restype = i32
    L.ttt_mlp_bwd_workspace_size.argtypes = [mptr, ctypes.POINTER(sz)]
    L.ttt_mlp_bwd_workspace_size.restype = i32
    L.ttt_mlp_chunk_bwd.argtypes = [mptr] + [vp] * 18 + [vp, sz, vp]
    L.ttt_mlp_chunk_bwd.restype = i32
    rptr, nptr = ctypes.POINTER(TTTRecDesc), ctypes.POINTER(TTTLnDesc)
    L.ttt_recurrence_workspace_size.argtypes = [rptr, i32, ctypes.POINTER(sz)]
    L.ttt_recurrence_saved_size.argtypes = [rptr, ctypes.POINTER(sz)]
    L.ttt_recurrence_fwd.argtypes = [rptr] + [vp] * 8 + [sz, vp]
    L.ttt_recurrence_bwd.argtypes = [rptr] + [vp] * 11 + [sz, vp]
    L.ttt_recurrence_step.argtypes = [rptr] + [vp] * 3 + [i32] + [vp] * 3
    L.ttt_layernorm_fwd.argtypes = [nptr] + [vp] * 9
    L.ttt_layernorm_workspace_size.argtypes = [nptr, ctypes.POINTER(sz)]
    L.ttt_layernorm_bwd.argtypes = [nptr] + [vp] * 10 + [sz, vp]
    for name in EXPORTS[-8:]:
        getattr(L, name).restype = i32
    L.ttt_last_error.argtypes = []
    L.ttt_last_error.restype = ctypes.c_char_p
    L.ttt_version.argtypes = []
    L.ttt_version.restype = ctypes.c_char_p
    L.ttt_timing_enable.argtypes = [i32]
    L.ttt_timing_enable.restype = i32
    L.ttt_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    L.ttt_timing_read.restype = i32
    _lib = L
    return L


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError("tensors passed to libttt must be contiguous")
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)!r} as a device pointer")


def _stream(stream):
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available() and torch.cuda.is_initialized():
                return torch.cuda.current_stream().cuda_stream
        except Exception:  # pragma: no cover - torch is optional for this module
            pass
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status):
    if status != 0:
        raise TTTError(status, ttt_last_error())


def make_desc(B, H, T, dk, dv, C, dtype="bf16", loss="mse", act="none", decay="none", lr_bias=-4.0):
    """Build a TTTDesc from names ("bf16"/"f32", "mse"/"ip"/"l1", "none"/"silu"/"gelu"/"norm",
    "none"/"scalar"/"vector")."""
    def enum(cls, x):
        return int(cls[x.upper()]) if isinstance(x, str) else int(x)
    return TTTDesc(B, H, T, dk, dv, C, enum(DType, dtype), enum(Loss, loss), enum(Act, act),
                   enum(Decay, decay), float(lr_bias))


def make_mlp_desc(B, H, T, dk, dh, dv, C, dtype="bf16", loss="mse", act="gelu", decay="none", lr_bias=-4.0):
    """Build a TTTMlpDesc from names, as make_desc (decay "none" or "scalar")."""
    def enum(cls, x):
        return int(cls[x.upper()]) if isinstance(x, str) else int(x)
    return TTTMlpDesc(B, H, T, dk, dh, dv, C, enum(DType, dtype), enum(Loss, loss), enum(Act, act),
                      enum(Decay, decay), float(lr_bias))


def _fit32(**sizes):
    """Raises where ctypes would keep the low 32 bits of a size in silence."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} must fit in 32 bits (got {v})")


def make_rec_desc(B, T, D, dtype="bf16", gate="sigmoid", input="convex", packed=False, ldx=0, ldg=0):
    """Build a TTTRecDesc from names ("bf16"/"f32", "sigmoid"/"log", "plain"/"convex")."""
    def enum(cls, x):
        return int(cls[x.upper()]) if isinstance(x, str) else int(x)
    _fit32(B=B, T=T, D=D)
    return TTTRecDesc(B, T, D, int(packed), enum(DType, dtype), enum(Gate, gate), enum(RecInput, input), 0, ldx, ldg)


def make_ln_desc(rows, D, dtype="bf16", groups=1, period=1, eps=1e-5, ldx=0):
    """Build a TTTLnDesc; ``dtype`` by name ("bf16"/"f32")."""
    _fit32(D=D, groups=groups, period=period)
    return TTTLnDesc(rows, ldx, D, groups, period, int(DType[dtype.upper()]) if isinstance(dtype, str) else int(dtype),
                     float(eps), 0)


def ttt_last_error() -> str:
    return lib().ttt_last_error().decode()


def ttt_version() -> str:
    return lib().ttt_version().decode()


def ttt_workspace_size(desc: TTTDesc, entry: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_workspace_size(ctypes.byref(desc), int(entry), ctypes.byref(n)))
    return n.value


def ttt_saved_size(desc: TTTDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_saved_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_chunk_fwd(desc, q, k, v, beta, gamma, log_decay, w0, o, w_final, w_ckpt, saved, ws, ws_bytes=None,
                  stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ttt_chunk_fwd(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(beta), _p(gamma),
                               _p(log_decay), _p(w0), _p(o), _p(w_final), _p(w_ckpt), _p(saved), _p(ws),
                               int(ws_bytes), _stream(stream)))


def ttt_chunk_bwd(desc, q, k, v, beta, gamma, log_decay, w0, w_ckpt, saved, d_o, d_wfinal, dq, dk, dv,
                  dbeta, dgamma, dlog_decay, dw0, ws, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ttt_chunk_bwd(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(beta), _p(gamma),
                               _p(log_decay), _p(w0), _p(w_ckpt), _p(saved), _p(d_o), _p(d_wfinal), _p(dq),
                               _p(dk), _p(dv), _p(dbeta), _p(dgamma), _p(dlog_decay), _p(dw0),
                               _p(ws), int(ws_bytes), _stream(stream)))


def ttt_chunk_bwd_noalloc(desc, q, k, v, beta, gamma, log_decay, w0, w_ckpt, saved, d_o, d_wfinal, dq, dk, dv,
                          dbeta, dgamma, dlog_decay, dw0, stream=None):
    _check(lib().ttt_chunk_bwd_noalloc(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(beta), _p(gamma),
                                       _p(log_decay), _p(w0), _p(w_ckpt), _p(saved), _p(d_o), _p(d_wfinal), _p(dq),
                                       _p(dk), _p(dv), _p(dbeta), _p(dgamma), _p(dlog_decay), _p(dw0),
                                       _stream(stream)))


def ttt_noalloc_scratch_bytes() -> int:
    return int(lib().ttt_noalloc_scratch_bytes())


def ttt_mlp_workspace_size(desc: TTTMlpDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_mlp_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_mlp_chunk_fwd(desc, q, k, v, beta, gamma, w1_0, w2_0, o, w1_final, w2_final, w1_ckpt, w2_ckpt, saved,
                      ws, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ttt_mlp_chunk_fwd(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(beta), _p(gamma), _p(w1_0),
                                   _p(w2_0), _p(o), _p(w1_final), _p(w2_final), _p(w1_ckpt), _p(w2_ckpt),
                                   _p(saved), _p(ws), int(ws_bytes), _stream(stream)))


def ttt_mlp_saved_size(desc: TTTMlpDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_mlp_saved_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_mlp_bwd_workspace_size(desc: TTTMlpDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_mlp_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_mlp_chunk_bwd(desc, q, k, v, beta, gamma, w1_ckpt, w2_ckpt, saved, d_o, d_w1final, d_w2final, dq, dk, dv,
                      dbeta, dgamma, dw1_0, dw2_0, ws, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ttt_mlp_chunk_bwd(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(beta), _p(gamma), _p(w1_ckpt),
                                   _p(w2_ckpt), _p(saved), _p(d_o), _p(d_w1final), _p(d_w2final), _p(dq), _p(dk), _p(dv),
                                   _p(dbeta), _p(dgamma), _p(dw1_0), _p(dw2_0), _p(ws), int(ws_bytes),
                                   _stream(stream)))


def inplace_ttt_workspace_size(B, T, d_model, d_ff, C) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().inplace_ttt_workspace_size(int(B), int(T), int(d_model), int(d_ff), int(C), ctypes.byref(n)))
    return n.value


def inplace_ttt_fwd(B, T, d_model, d_ff, C, eta, z, vhat, w_down, o, ws=None, ws_bytes=0, stream=None):
    _check(lib().inplace_ttt_fwd(int(B), int(T), int(d_model), int(d_ff), int(C), float(eta),
                                 _p(z), _p(vhat), _p(w_down), _p(o), _p(ws), int(ws_bytes), _stream(stream)))


def inplace_ttt_guarded_workspace_size(B, T, d_model, d_ff, C) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().inplace_ttt_guarded_workspace_size(int(B), int(T), int(d_model), int(d_ff), int(C),
                                                    ctypes.byref(n)))
    return n.value


def inplace_ttt_fwd_guarded(B, T, d_model, d_ff, C, eta, clip_tau, doc_starts, z, vhat, w_init, w_down, o,
                            ws=None, ws_bytes=0, stream=None):
    """``doc_starts``: host sequence of flat positions b * T + t (0 < t < T), increasing."""
    starts = [int(p) for p in (doc_starts or [])]
    arr = (ctypes.c_int64 * len(starts))(*starts) if starts else None
    _check(lib().inplace_ttt_fwd_guarded(int(B), int(T), int(d_model), int(d_ff), int(C), float(eta),
                                         float(clip_tau), arr, len(starts), _p(z), _p(vhat), _p(w_init),
                                         _p(w_down), _p(o), _p(ws), int(ws_bytes), _stream(stream)))


def inplace_ttt_bwd_workspace_size(B, T, d_model, d_ff, C) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().inplace_ttt_bwd_workspace_size(int(B), int(T), int(d_model), int(d_ff), int(C), ctypes.byref(n)))
    return n.value


def inplace_ttt_bwd(B, T, d_model, d_ff, C, eta, z, vhat, w_final, d_o, d_wfinal, dz, dvhat, dw0, ws, ws_bytes,
                    stream=None):
    _check(lib().inplace_ttt_bwd(int(B), int(T), int(d_model), int(d_ff), int(C), float(eta), _p(z), _p(vhat),
                                 _p(w_final), _p(d_o), _p(d_wfinal), _p(dz), _p(dvhat), _p(dw0), _p(ws), int(ws_bytes),
                                 _stream(stream)))


def inplace_ttt_bwd_guarded_workspace_size(B, T, d_model, d_ff, C) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().inplace_ttt_bwd_guarded_workspace_size(int(B), int(T), int(d_model), int(d_ff), int(C),
                                                        ctypes.byref(n)))
    return n.value


def inplace_ttt_bwd_guarded(B, T, d_model, d_ff, C, eta, clip_tau, doc_starts, z, vhat, w0, w_init, w_final, d_o,
                            d_wfinal, dz, dvhat, dw0, dw_init, ws, ws_bytes, stream=None):
    """``doc_starts``: host sequence of flat positions b * T + t (0 < t < T), increasing."""
    starts = [int(p) for p in (doc_starts or [])]
    arr = (ctypes.c_int64 * len(starts))(*starts) if starts else None
    _check(lib().inplace_ttt_bwd_guarded(int(B), int(T), int(d_model), int(d_ff), int(C), float(eta),
                                         float(clip_tau), arr, len(starts), _p(z), _p(vhat), _p(w0), _p(w_init),
                                         _p(w_final), _p(d_o), _p(d_wfinal), _p(dz), _p(dvhat), _p(dw0),
                                         _p(dw_init), _p(ws), int(ws_bytes), _stream(stream)))


_torch_types = None
_raw_stream = None


def _types():
    """torch's types by DType, then int32 and uint8; torch is imported with the first tensor call."""
    global _torch_types, _raw_stream
    if _torch_types is None:
        import torch
        # the current stream's handle without the Stream object around it, where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _torch_types = (torch.float32, torch.bfloat16, torch.int32, torch.uint8)
    return _torch_types


def _io_type(desc):
    """The torch type of a desc's tensors (None for an invalid dtype, which the library rejects)."""
    return _types()[desc.dtype] if desc.dtype in (0, 1) else None


def _device(x):
    """The device index of a call's first tensor (-1 on the host), None for a raw pointer."""
    return x.get_device() if hasattr(x, "get_device") else None


def _arg(name, x, dev, dtype, rows, cols, ld=0):
    """The pointer of one tensor of a call: ``rows`` rows of ``cols`` elements, ``ld`` elements apart (0: dense).

    A tensor on the host, on another device than the call's first, of another
    type or with fewer elements than the kernels touch would fault the GPU; it
    raises ValueError here.  Integers are device pointers and are taken as they are."""
    if x is None or type(x) is int:
        return x
    try:
        if x.dtype is dtype and x.get_device() == dev and dev >= 0 and (not ld or ld == cols) and x.is_contiguous() \
                and x.numel() >= rows * cols:
            return x.data_ptr()
    except AttributeError:
        raise TypeError(f"cannot pass {type(x)!r} as a device pointer") from None
    if x.get_device() < 0:
        raise ValueError(f"{name} must be on the GPU, not on {x.device}")
    if dev is not None and x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, the tensors before it on cuda:{dev}")
    if dtype is not None and x.dtype is not dtype:
        raise ValueError(f"{name} must be {str(dtype)[6:]}, not {str(x.dtype)[6:]}")
    if ld and ld != cols:
        st = x.stride()
        if x.dim() < 2 or st[-1] != 1 or x.shape[-1] != cols or (x.shape[-2] > 1 and st[-2] != ld) or \
                any(x.shape[i] > 1 and st[i] != ld * math.prod(x.shape[i + 1:-1]) for i in range(x.dim() - 2)):
            raise ValueError(f"{name} must have rows of {cols} elements, {ld} apart (got shape {tuple(x.shape)}, "
                             f"strides {st})")
    elif not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if x.numel() < rows * cols:
        raise ValueError(f"{name} has {x.numel()} elements, {rows * cols} are needed")
    return x.data_ptr()


def _ws(ws, ws_bytes, dev):
    """(pointer, bytes) of a workspace."""
    if hasattr(ws, "data_ptr"):
        size = ws.numel() * ws.element_size()
        return _arg("ws", ws, dev, ws.dtype, 0, 0), size if ws_bytes is None else min(size, int(ws_bytes))
    return ws, int(ws_bytes or 0)


def _call(f, dev, stream, *args):
    """Call ``f`` with device ``dev`` current, on ``stream`` (None: that device's current stream)."""
    if dev is None:
        _check(f(*args, _stream(stream)))
        return
    import torch
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _check(f(*args, _raw_stream(dev) if stream is None else _stream(stream)))
        return
    status = f(*args, _raw_stream(dev) if stream is None else _stream(stream))
    if status != 0:
        raise TTTError(status, ttt_last_error())


def ttt_recurrence_workspace_size(desc: TTTRecDesc, entry: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_recurrence_workspace_size(ctypes.byref(desc), int(entry), ctypes.byref(n)))
    return n.value


def ttt_recurrence_saved_size(desc: TTTRecDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_recurrence_saved_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_recurrence_fwd(desc, x, gate, h0, seq_starts, o, h_final, saved, ws, ws_bytes=None, stream=None):
    """``seq_starts``: int32 device tensor of B + 1 positions for a packed desc, else None."""
    f32, _, i32, u8 = _types()
    dt, dev, B, D = _io_type(desc), _device(x), desc.B, desc.D
    n = desc.T if desc.packed else B * desc.T
    _call(lib().ttt_recurrence_fwd, dev, stream, ctypes.byref(desc), _arg("x", x, dev, dt, n, D, desc.ldx),
          _arg("gate", gate, dev, dt, n, D, desc.ldg), _arg("h0", h0, dev, f32, B, D),
          _arg("seq_starts", seq_starts, dev, i32, 1, B + 1), _arg("o", o, dev, dt, n, D),
          _arg("h_final", h_final, dev, f32, B, D),
          _arg("saved", saved, dev, u8, 1, 0 if saved is None else ttt_recurrence_saved_size(desc)),
          *_ws(ws, ws_bytes, dev))


def ttt_recurrence_bwd(desc, x, gate, h0, seq_starts, saved, d_o, d_hfinal, dx, dgate, dh0, ws, ws_bytes=None,
                       stream=None):
    f32, _, i32, u8 = _types()
    dt, dev, B, D = _io_type(desc), _device(x), desc.B, desc.D
    n = desc.T if desc.packed else B * desc.T
    _call(lib().ttt_recurrence_bwd, dev, stream, ctypes.byref(desc), _arg("x", x, dev, dt, n, D, desc.ldx),
          _arg("gate", gate, dev, dt, n, D, desc.ldg), _arg("h0", h0, dev, f32, B, D),
          _arg("seq_starts", seq_starts, dev, i32, 1, B + 1),
          _arg("saved", saved, dev, u8, 1, 0 if saved is None else ttt_recurrence_saved_size(desc)),
          _arg("d_o", d_o, dev, dt, n, D), _arg("d_hfinal", d_hfinal, dev, f32, B, D),
          _arg("dx", dx, dev, dt, n, D, desc.ldx), _arg("dgate", dgate, dev, dt, n, D, desc.ldg),
          _arg("dh0", dh0, dev, f32, B, D), *_ws(ws, ws_bytes, dev))


def ttt_recurrence_step(desc, x, gate, slots, h, o, n_states=None, stream=None):
    """``h``: [n_states, D] float32, updated in place; ``n_states`` is only needed where h is a raw pointer."""
    f32, _, i32, _ = _types()
    dt, dev, n, D = _io_type(desc), _device(x), desc.B, desc.D
    if n_states is None:
        n_states = h.numel() // D if hasattr(h, "numel") and D > 0 else 0
    if not -2 ** 31 <= n_states < 2 ** 31:
        _fit32(n_states=n_states)
    _call(lib().ttt_recurrence_step, dev, stream, ctypes.byref(desc), _arg("x", x, dev, dt, n, D, desc.ldx),
          _arg("gate", gate, dev, dt, n, D, desc.ldg), _arg("slots", slots, dev, i32, 1, n), n_states,
          _arg("h", h, dev, f32, n_states, D), _arg("o", o, dev, dt, n, D))


def ttt_layernorm_workspace_size(desc: TTTLnDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ttt_layernorm_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_layernorm_fwd(desc, x, res, w, b, y, r, mean, rstd, stream=None):
    f32 = _types()[0]
    dt, dev, n, D, G = _io_type(desc), _device(x), desc.rows, desc.D, desc.groups
    _call(lib().ttt_layernorm_fwd, dev, stream, ctypes.byref(desc), _arg("x", x, dev, dt, n, D, desc.ldx),
          _arg("res", res, dev, dt, n, D), _arg("w", w, dev, f32, G, D), _arg("b", b, dev, f32, G, D),
          _arg("y", y, dev, dt, n, D), _arg("r", r, dev, dt, n, D), _arg("mean", mean, dev, f32, n, 1),
          _arg("rstd", rstd, dev, f32, n, 1))


def ttt_layernorm_bwd(desc, x, w, mean, rstd, dy, dr, dx, dw, db, ws, ws_bytes=None, stream=None):
    f32 = _types()[0]
    dt, dev, n, D, G = _io_type(desc), _device(x), desc.rows, desc.D, desc.groups
    _call(lib().ttt_layernorm_bwd, dev, stream, ctypes.byref(desc), _arg("x", x, dev, dt, n, D, desc.ldx),
          _arg("w", w, dev, f32, G, D), _arg("mean", mean, dev, f32, n, 1), _arg("rstd", rstd, dev, f32, n, 1),
          _arg("dy", dy, dev, dt, n, D), _arg("dr", dr, dev, dt, n, D), _arg("dx", dx, dev, dt, n, D, desc.ldx),
          _arg("dw", dw, dev, f32, G, D), _arg("db", db, dev, f32, G, D), *_ws(ws, ws_bytes, dev))


def ttt_timing_enable(on: bool) -> None:
    _check(lib().ttt_timing_enable(1 if on else 0))


def ttt_timing_read(kernel) -> tuple[float, int]:
    """(summed device milliseconds, launch count) of one kernel since the last enable."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    status = lib().ttt_timing_read(int(kernel), ctypes.byref(ms), ctypes.byref(n))
    if status != 0:
        raise TTTError(status, "ttt_timing_read failed")
    return ms.value, n.value
