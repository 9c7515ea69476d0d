"""Python binding of ``libgdr.so`` (the C ABI in include/gdr.h).

Argument marshalling only: torch tensors are checked for device, dtype, shape and
contiguity, their device pointers and the current HIP stream are handed to the C entry
points, and a non-zero status is raised as ``GdrError``. Every step of the computation
runs in the library's HIP kernels. There is no fallback: if the library is missing the
import fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_F32, GDR_BF16 = 0, 1
GDR_READ_PRE, GDR_REVERSE, GDR_ACCUMULATE, GDR_QK_L2NORM, GDR_HEAD_DECAY = 1, 2, 4, 8, 16

STATUS = {0: "GDR_OK", 1: "GDR_ERR_NULL", 2: "GDR_ERR_DIMS", 3: "GDR_ERR_DTYPE", 4: "GDR_ERR_CHUNK",
          5: "GDR_ERR_ALIGN", 6: "GDR_ERR_ALIAS", 7: "GDR_ERR_UNSUPPORTED", 8: "GDR_ERR_FLAGS",
          9: "GDR_ERR_HIP"}

# every symbol include/gdr.h declares
EXPORTS = ("gdr_chunk_fwd", "gdr_chunk_fwd_bidir", "gdr_chunk_fwd_gated", "gdr_decode_step", "gdr_decode_step_gated",
           "gdr_gdn2_chunk_fwd", "gdr_gdn2_chunk_fwd_bidir", "gdr_gdn2_chunk_fwd_noalloc", "gdr_gdn2_chunk_fwd_workspace_bytes",
           "gdr_gdn2_decode_step",
           "gdr_delta_product_fwd",
           "gdr_chunk_bwd", "gdr_chunk_bwd_workspace_bytes",
           "gdr_channel_scan_fwd", "gdr_channel_scan_fwd_workspace_bytes", "gdr_channel_scan_states_elems",
           "gdr_channel_scan_bwd", "gdr_channel_scan_bwd_workspace_bytes", "gdr_channel_scan_step",
           "gdr_gated_ffn_fwd", "gdr_gated_ffn_bwd", "gdr_gated_ffn_bwd_workspace_bytes",
           "gdr_linear_ce_fwd", "gdr_linear_ce_fwd_workspace_bytes", "gdr_linear_ce_bwd",
           "gdr_linear_ce_bwd_workspace_bytes",
           "gdr_linear_attn_fwd", "gdr_linear_attn_fwd_workspace_bytes", "gdr_linear_attn_bwd",
           "gdr_linear_attn_bwd_workspace_bytes", "gdr_linear_attn_step",
           "gdr_qk_norm_rope_fwd", "gdr_qk_norm_rope_bwd", "gdr_qk_norm_rope_bwd_workspace_bytes",
           "gdr_status_string", "gdr_last_error", "gdr_abi_version", "gdr_selftest_mfma")


class GdrError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__("%s: %s" % (self.name, detail))


class ChunkDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("Hv", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("num_seqs", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class ScanDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int64),
                ("num_seqs", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class FfnDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("D", ctypes.c_int64), ("F", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32)]


class CeDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("D", ctypes.c_int64), ("V", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class QkDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "Hq", "Hk", "d", "rot", "q_stride", "k_stride", "dq_stride", "dk_stride")] + \
        [("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class DecodeDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("Hk", ctypes.c_int64), ("Hv", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError("%s is missing: build it with `python -m gated_delta_rule_70_amd.build` "
                          "(there is no fallback path)" % path)
    lib = ctypes.CDLL(path)
    p, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.gdr_chunk_fwd.argtypes = [p, p, p, p, p, p, p, i32, p, p, ctypes.POINTER(ChunkDims), p]
    lib.gdr_chunk_fwd.restype = ctypes.c_int
    lib.gdr_chunk_fwd_gated.argtypes = [p, p, p, p, p, p, p, p, p, i32, p, p, ctypes.POINTER(ChunkDims), p]
    lib.gdr_chunk_fwd_gated.restype = ctypes.c_int
    lib.gdr_chunk_fwd_bidir.argtypes = [p] * 10 + [i32, p, p, p, ctypes.POINTER(ChunkDims), p]
    lib.gdr_chunk_fwd_bidir.restype = ctypes.c_int
    lib.gdr_decode_step.argtypes = [p, p, p, p, p, p, p, p, ctypes.POINTER(DecodeDims), p]
    lib.gdr_decode_step.restype = ctypes.c_int
    lib.gdr_decode_step_gated.argtypes = [p, p, p, p, p, p, p, p, p, p, ctypes.POINTER(DecodeDims), p]
    lib.gdr_decode_step_gated.restype = ctypes.c_int
    lib.gdr_chunk_bwd.argtypes = [p] * 15 + [p, ctypes.c_int64, ctypes.POINTER(ChunkDims), p]
    lib.gdr_chunk_bwd.restype = ctypes.c_int
    lib.gdr_chunk_bwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDims), i32]
    lib.gdr_chunk_bwd_workspace_bytes.restype = ctypes.c_int64
    lib.gdr_delta_product_fwd.argtypes = [p, p, p, p, p, p, p, i32, i32, p, p, ctypes.POINTER(ChunkDims), p]
    lib.gdr_delta_product_fwd.restype = ctypes.c_int
    lib.gdr_gdn2_chunk_fwd.argtypes = [p, p, p, p, p, p, p, p, i32, p, p, p, ctypes.c_int64,
                                       ctypes.POINTER(ChunkDims), p]
    lib.gdr_gdn2_chunk_fwd.restype = ctypes.c_int
    lib.gdr_gdn2_chunk_fwd_bidir.argtypes = [p] * 11 + [p, i32, p, p, p, p, ctypes.c_int64, ctypes.POINTER(ChunkDims), p]
    lib.gdr_gdn2_chunk_fwd_bidir.restype = ctypes.c_int
    lib.gdr_gdn2_chunk_fwd_noalloc.argtypes = [p, p, p, p, p, p, p, p, i32, p, p, ctypes.POINTER(ChunkDims), p]
    lib.gdr_gdn2_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.gdr_gdn2_chunk_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDims), i32, i32]
    lib.gdr_gdn2_chunk_fwd_workspace_bytes.restype = ctypes.c_int64
    lib.gdr_gdn2_decode_step.argtypes = [p, p, p, p, p, p, p, p, p, ctypes.POINTER(DecodeDims), p]
    lib.gdr_gdn2_decode_step.restype = ctypes.c_int
    i64 = ctypes.c_int64
    for name, args in (("gdr_channel_scan_fwd", [p] * 11 + [i64, ctypes.POINTER(ScanDims), p]),
                       ("gdr_channel_scan_bwd", [p] * 16 + [i64, ctypes.POINTER(ScanDims), p]),
                       ("gdr_channel_scan_step", [p] * 8 + [ctypes.POINTER(ScanDims), p]),
                       ("gdr_gated_ffn_fwd", [p] * 6 + [ctypes.POINTER(FfnDims), p]),
                       ("gdr_gated_ffn_bwd", [p] * 10 + [i64, ctypes.POINTER(FfnDims), p]),
                       ("gdr_linear_ce_fwd", [p] * 6 + [i64, ctypes.POINTER(CeDims), p]),
                       ("gdr_linear_ce_bwd", [p] * 8 + [i64, ctypes.POINTER(CeDims), p]),
                       ("gdr_linear_attn_fwd", [p] * 9 + [i64, ctypes.POINTER(ChunkDims), p]),
                       ("gdr_linear_attn_bwd", [p] * 14 + [i64, ctypes.POINTER(ChunkDims), p]),
                       ("gdr_linear_attn_step", [p] * 7 + [ctypes.POINTER(DecodeDims), p]),
                       ("gdr_qk_norm_rope_fwd", [p] * 8 + [ctypes.POINTER(QkDims), p]),
                       ("gdr_qk_norm_rope_bwd", [p] * 13 + [i64, ctypes.POINTER(QkDims), p])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    for name, args in (("gdr_channel_scan_states_elems", [ctypes.POINTER(ScanDims), i32]),
                       ("gdr_channel_scan_fwd_workspace_bytes", [ctypes.POINTER(ScanDims), i32]),
                       ("gdr_channel_scan_bwd_workspace_bytes", [ctypes.POINTER(ScanDims), i32]),
                       ("gdr_gated_ffn_bwd_workspace_bytes", [ctypes.POINTER(FfnDims)]),
                       ("gdr_linear_ce_fwd_workspace_bytes", [ctypes.POINTER(CeDims)]),
                       ("gdr_linear_ce_bwd_workspace_bytes", [ctypes.POINTER(CeDims)]),
                       ("gdr_linear_attn_fwd_workspace_bytes", [ctypes.POINTER(ChunkDims), i32]),
                       ("gdr_linear_attn_bwd_workspace_bytes", [ctypes.POINTER(ChunkDims), i32]),
                       ("gdr_qk_norm_rope_bwd_workspace_bytes", [ctypes.POINTER(QkDims)])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i64
    lib.gdr_status_string.argtypes = [ctypes.c_int]
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_last_error.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    lib.gdr_abi_version.argtypes = []
    lib.gdr_abi_version.restype = ctypes.c_int32
    lib.gdr_selftest_mfma.argtypes = [p, p, p, p]
    lib.gdr_selftest_mfma.restype = ctypes.c_int
    return lib


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _check(status: int):
    if status != 0:
        raise GdrError(status, lib().gdr_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    return torch._C._cuda_getCurrentRawStream(t.device.index)  # current_stream(...).cuda_stream, without the object


def _run(t, fn, *args):
    """fn on t's device, which need not be the current one, and on the stream that is current there."""
    if t.device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(t.device):
            return _run(t, fn, *args)
    status = fn(*args, _stream(t))
    if status:
        _check(status)


def _need(t, name, dtype=None, shape=None, device=None):
    # what nearly every call brings, checked in one expression: a step's checks cost it more than its kernel
    if (device is not None and type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _dtype_code(dt, what="q, k, v"):
    if dt == torch.bfloat16:
        return GDR_BF16
    if dt == torch.float32:
        return GDR_F32
    raise ValueError("%s must be bfloat16 or float32 (got %s)" % (what, dt))


def chunk_fwd(q, k, v, log_alpha, beta, h0=None, cu_seqlens=None, *, chunk: int = 64,
              read: str = "post", reverse: bool = False, out=None, accumulate: bool = False,
              hT=None, want_state: bool = True, l2norm: bool = False):
    """Chunked forward (``gdr_chunk_fwd``).

    q, k [B, Hk, T, dk]; v [B, Hv, T, dv] (bf16 or fp32, same dtype); log_alpha, beta
    [B, Hv, T] fp32; h0 [S, Hv, dk, dv] fp32 or None; cu_seqlens int32 [S+1] (device) or
    None. Returns (out [B, Hv, T, dv], hT [S, Hv, dk, dv] or None). ``out`` may be given
    (required for ``accumulate``); ``hT`` may be given (it may be ``h0`` itself).
    ``l2norm`` normalises each row of q and k in the kernel (``GDR_QK_L2NORM``).
    """
    return _chunk(q, k, v, log_alpha, beta, None, None, h0, cu_seqlens, chunk, read, reverse, out,
                  accumulate, hT, want_state, l2norm)


def chunk_fwd_gated(q, k, v, a, b, A_log, dt_bias, h0=None, cu_seqlens=None, *, chunk: int = 64,
                    read: str = "post", reverse: bool = False, out=None, accumulate: bool = False,
                    hT=None, want_state: bool = True, l2norm: bool = True):
    """Chunked forward with the gates formed in the kernel (``gdr_chunk_fwd_gated``): a, b
    [B, Hv, T] fp32 raw inputs, A_log, dt_bias [Hv] fp32; the rest as ``chunk_fwd``."""
    return _chunk(q, k, v, a, b, A_log, dt_bias, h0, cu_seqlens, chunk, read, reverse, out,
                  accumulate, hT, want_state, l2norm)


def chunk_fwd_bidir(q, k, v, log_alpha_fwd, beta_fwd, log_alpha_rev, beta_rev, h0_fwd=None, h0_rev=None,
                    cu_seqlens=None, *, chunk: int = 64, read: str = "pre", out=None, accumulate: bool = False,
                    want_state: bool = True, l2norm: bool = False):
    """Both scans of a bidirectional layer, summed per token (``gdr_chunk_fwd_bidir``): the
    forward scan and the in-segment reversed scan, each with its own gates [B, Hv, T] fp32 (indexed
    by token) and initial state [S, Hv, dk, dv] fp32 or None, the same ``read`` for both. Returns
    (out [B, Hv, T, dv], hT_fwd, hT_rev), the final states None without ``want_state``."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    for t, n in ((log_alpha_fwd, "log_alpha_fwd"), (beta_fwd, "beta_fwd"), (log_alpha_rev, "log_alpha_rev"),
                 (beta_rev, "beta_rev")):
        _need(t, n, torch.float32, (B, Hv, T), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    for t, n in ((h0_fwd, "h0_fwd"), (h0_rev, "h0_rev")):
        if t is not None:
            _need(t, n, torch.float32, (S, Hv, dk, dv), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((B, Hv, T, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (B, Hv, T, dv), dev)
    hT_f = hT_r = None
    if want_state:
        hT_f = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
        hT_r = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_ACCUMULATE if accumulate else 0) | \
        (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    _run(q, lib().gdr_chunk_fwd_bidir, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha_fwd), _ptr(beta_fwd),
         _ptr(log_alpha_rev), _ptr(beta_rev), _ptr(h0_fwd), _ptr(h0_rev),
         _ptr(cu_seqlens), int(chunk), _ptr(out), _ptr(hT_f), _ptr(hT_r),
         ctypes.byref(dims))
    return out, hT_f, hT_r


def _chunk(q, k, v, ga, gb, A_log, dt_bias, h0, cu_seqlens, chunk, read, reverse, out, accumulate,
           hT, want_state, l2norm):
    gated = A_log is not None or dt_bias is not None
    na, nb = ("a", "b") if gated else ("log_alpha", "beta")
    _need(q, "q")
    dev = q.device
    dt = q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    _need(ga, na, torch.float32, (B, Hv, T), dev)
    _need(gb, nb, torch.float32, (B, Hv, T), dev)
    if gated:
        _need(A_log, "A_log", torch.float32, (Hv,), dev)
        _need(dt_bias, "dt_bias", torch.float32, (Hv,), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (S, Hv, dk, dv), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((B, Hv, T, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (B, Hv, T, dv), dev)
    if hT is None and want_state:
        hT = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _need(hT, "hT", torch.float32, (S, Hv, dk, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_REVERSE if reverse else 0) | \
        (GDR_ACCUMULATE if accumulate else 0) | (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    if gated:
        _run(q, lib().gdr_chunk_fwd_gated, _ptr(q), _ptr(k), _ptr(v), _ptr(ga), _ptr(gb), _ptr(A_log),
             _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), int(chunk), _ptr(out),
             _ptr(hT), ctypes.byref(dims))
    else:
        _run(q, lib().gdr_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(ga), _ptr(gb), _ptr(h0),
             _ptr(cu_seqlens), int(chunk), _ptr(out), _ptr(hT),
             ctypes.byref(dims))
    return out, hT


def decode_step(q, k, v, log_alpha, beta, state_in, state_out=None, out=None, *, read: str = "post",
                l2norm: bool = False):
    """One decode step (``gdr_decode_step``). q, k [N, Hk, dk]; v [N, Hv, dv]; log_alpha,
    beta [N, Hv] fp32; state_in [N, Hv, dk, dv] fp32. ``state_out`` defaults to a new
    tensor; pass ``state_in`` itself to update in place. Returns (out, state_out).
    ``l2norm`` normalises q and k in the kernel (``GDR_QK_L2NORM``)."""
    return _decode(q, k, v, log_alpha, beta, None, None, state_in, state_out, out, read, l2norm)


def decode_step_gated(q, k, v, a, b, A_log, dt_bias, state_in, state_out=None, out=None, *,
                      read: str = "post", l2norm: bool = True):
    """One decode step with the gates formed in the kernel (``gdr_decode_step_gated``): a, b
    [N, Hv] fp32 raw inputs, A_log, dt_bias [Hv] fp32; the rest as ``decode_step``."""
    return _decode(q, k, v, a, b, A_log, dt_bias, state_in, state_out, out, read, l2norm)


def _decode(q, k, v, ga, gb, A_log, dt_bias, state_in, state_out, out, read, l2norm):
    gated = A_log is not None or dt_bias is not None
    na, nb = ("a", "b") if gated else ("log_alpha", "beta")
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    _need(k, "k", dt, (N, Hk, dk), dev)
    _need(v, "v", dt, (N, Hv, dv), dev)
    _need(ga, na, torch.float32, (N, Hv), dev)
    _need(gb, nb, torch.float32, (N, Hv), dev)
    if gated:
        _need(A_log, "A_log", torch.float32, (Hv,), dev)
        _need(dt_bias, "dt_bias", torch.float32, (Hv,), dev)
    _need(state_in, "state_in", torch.float32, (N, Hv, dk, dv), dev)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    else:
        _need(state_out, "state_out", torch.float32, (N, Hv, dk, dv), dev)
    if out is None:
        out = torch.empty((N, Hv, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (N, Hv, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_QK_L2NORM if l2norm else 0)
    dims = DecodeDims(N, Hk, Hv, dk, dv, code, flags)
    if gated:
        _run(q, lib().gdr_decode_step_gated, _ptr(q), _ptr(k), _ptr(v), _ptr(ga), _ptr(gb), _ptr(A_log),
             _ptr(dt_bias), _ptr(state_in), _ptr(state_out), _ptr(out),
             ctypes.byref(dims))
    else:
        _run(q, lib().gdr_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(ga), _ptr(gb), _ptr(state_in),
             _ptr(state_out), _ptr(out), ctypes.byref(dims))
    return out, state_out


def chunk_bwd(q, k, v, log_alpha, beta, dout, h0=None, cu_seqlens=None, dhT=None, *, read: str = "post",
              reverse: bool = False, want_dh0: bool = True, workspace=None):
    """Gradients of ``chunk_fwd`` (``gdr_chunk_bwd``): the inputs as given to the forward, dout
    [B, Hv, T, dv] in their dtype, dhT [S, Hv, dk, dv] fp32 or None. Returns fp32 tensors
    (dq, dk, dv, dlog_alpha, dbeta, dh0 or None). ``workspace`` (a uint8 GPU tensor of at least
    ``chunk_bwd_workspace_bytes`` bytes) is allocated here when not given."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    _need(dout, "dout", dt, (B, Hv, T, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (B, Hv, T), dev)
    _need(beta, "beta", torch.float32, (B, Hv, T), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _need(t, name, torch.float32, (S, Hv, dk, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_REVERSE if reverse else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    need = lib().gdr_chunk_bwd_workspace_bytes(ctypes.byref(dims), int(cu_seqlens is not None))
    if need < 0:
        raise ValueError("invalid sizes for the backward workspace")
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif workspace.numel() < need:
        raise ValueError("workspace holds %d bytes, %d needed" % (workspace.numel(), need))
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk_ = torch.empty((B, Hk, T, dk), **f32), torch.empty((B, Hk, T, dk), **f32)
    dv_ = torch.empty((B, Hv, T, dv), **f32)
    dla, dbe = torch.empty((B, Hv, T), **f32), torch.empty((B, Hv, T), **f32)
    dh0 = torch.empty((S, Hv, dk, dv), **f32) if want_dh0 else None
    _run(q, lib().gdr_chunk_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
         _ptr(dout), _ptr(dhT), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dla), _ptr(dbe), _ptr(dh0),
         _ptr(workspace), ctypes.c_int64(workspace.numel()), ctypes.byref(dims))
    return dq, dk_, dv_, dla, dbe, dh0


def chunk_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, num_seqs=0, dtype=torch.bfloat16) -> int:
    """Bytes of workspace ``gdr_chunk_bwd`` needs (num_seqs > 0: packed sequences)."""
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, num_seqs, _dtype_code(dtype), 0)
    return int(lib().gdr_chunk_bwd_workspace_bytes(ctypes.byref(dims), int(num_seqs > 0)))


def delta_product_fwd(q, k, v, log_alpha, beta, h0=None, cu_seqlens=None, *, chunk: int = 64,
                      read: str = "pre", out=None, accumulate: bool = False, hT=None, want_state: bool = True,
                      l2norm: bool = False):
    """DeltaProduct forward (``gdr_delta_product_fwd``): q [B, Hk, T, dk]; k [B, Hk, T, n, dk];
    v [B, Hv, T, n, dv]; log_alpha [B, Hv, T] fp32; beta [B, Hv, T, n] fp32. ``read`` defaults
    to the pre-write read of the page this variant comes from. Returns (out, hT)."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    n = k.shape[3]
    Hv, dv = v.shape[1], v.shape[4]
    _need(k, "k", dt, (B, Hk, T, n, dk), dev)
    _need(v, "v", dt, (B, Hv, T, n, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (B, Hv, T), dev)
    _need(beta, "beta", torch.float32, (B, Hv, T, n), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (S, Hv, dk, dv), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((B, Hv, T, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (B, Hv, T, dv), dev)
    if hT is None and want_state:
        hT = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _need(hT, "hT", torch.float32, (S, Hv, dk, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_ACCUMULATE if accumulate else 0) | \
        (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    _run(q, lib().gdr_delta_product_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(h0),
         _ptr(cu_seqlens), int(n), int(chunk), _ptr(out), _ptr(hT),
         ctypes.byref(dims))
    return out, hT


def gdn2_chunk_fwd(q, k, v, g, b, w, h0=None, cu_seqlens=None, *, chunk: int = 64, read: str = "post",
                   reverse: bool = False, out=None, accumulate: bool = False, hT=None, want_state: bool = True,
                   l2norm: bool = False, workspace=None, fused: bool = False):
    """GDN-2 chunked forward (``gdr_gdn2_chunk_fwd``).

    q, k [B, Hk, T, dk] and v [B, Hv, T, dv] (bf16 or fp32, one dtype); g [B, Hk, T, dk] fp32 log
    decay per key channel; b [B, Hk, T, dk] erase gate and w [B, Hv, T, dv] write gate in the
    dtype of q. The rest as ``chunk_fwd``. The two-pass form runs with ``workspace`` (a uint8 GPU
    tensor of at least ``gdn2_chunk_fwd_workspace_bytes`` bytes, allocated here when not given);
    ``fused=True`` passes no workspace and runs the one-pass kernel.
    """
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    _need(g, "g", torch.float32, (B, Hk, T, dk), dev)
    _need(b, "b", dt, (B, Hk, T, dk), dev)
    _need(w, "w", dt, (B, Hv, T, dv), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (S, Hv, dk, dv), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((B, Hv, T, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (B, Hv, T, dv), dev)
    if hT is None and want_state:
        hT = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _need(hT, "hT", torch.float32, (S, Hv, dk, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_REVERSE if reverse else 0) | \
        (GDR_ACCUMULATE if accumulate else 0) | (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    ws_ptr, ws_bytes = None, 0
    if not fused:
        need = lib().gdr_gdn2_chunk_fwd_workspace_bytes(ctypes.byref(dims), int(chunk), int(cu_seqlens is not None))
        if need < 0:
            raise ValueError("invalid sizes for the GDN-2 workspace")
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        _need(workspace, "workspace", torch.uint8, None, dev)
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()
    _run(q, lib().gdr_gdn2_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(h0),
         _ptr(cu_seqlens), int(chunk), _ptr(out), _ptr(hT), ws_ptr, ws_bytes,
         ctypes.byref(dims))
    return out, hT


def gdn2_chunk_fwd_bidir(q, k, v, fwd_gates, rev_gates, h0_fwd=None, h0_rev=None, cu_seqlens=None, *,
                         chunk: int = 64, read: str = "pre", out=None, accumulate: bool = False,
                         want_state: bool = True, l2norm: bool = False, workspace=None, fused: bool = False):
    """Both GDN-2 scans of a bidirectional layer, summed per token (``gdr_gdn2_chunk_fwd_bidir``):
    ``fwd_gates`` and ``rev_gates`` are (g, b, w) triples in ``gdn2_chunk_fwd``'s layouts; the rest
    as ``chunk_fwd_bidir`` and ``gdn2_chunk_fwd`` (one workspace serves both passes). Returns
    (out, hT_fwd, hT_rev)."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    for name, (g, b, w) in (("fwd", fwd_gates), ("rev", rev_gates)):
        _need(g, "g_" + name, torch.float32, (B, Hk, T, dk), dev)
        _need(b, "b_" + name, dt, (B, Hk, T, dk), dev)
        _need(w, "w_" + name, dt, (B, Hv, T, dv), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    for t, n in ((h0_fwd, "h0_fwd"), (h0_rev, "h0_rev")):
        if t is not None:
            _need(t, n, torch.float32, (S, Hv, dk, dv), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((B, Hv, T, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (B, Hv, T, dv), dev)
    hT_f = hT_r = None
    if want_state:
        hT_f = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
        hT_r = torch.empty((S, Hv, dk, dv), dtype=torch.float32, device=dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_ACCUMULATE if accumulate else 0) | \
        (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, flags)
    ws_ptr, ws_bytes = None, 0
    if not fused:
        need = lib().gdr_gdn2_chunk_fwd_workspace_bytes(ctypes.byref(dims), int(chunk), int(cu_seqlens is not None))
        if need < 0:
            raise ValueError("invalid sizes for the GDN-2 workspace")
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        _need(workspace, "workspace", torch.uint8, None, dev)
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()
    (gf, bf, wf), (gr, br, wr) = fwd_gates, rev_gates
    _run(q, lib().gdr_gdn2_chunk_fwd_bidir, _ptr(q), _ptr(k), _ptr(v), _ptr(gf), _ptr(bf), _ptr(wf), _ptr(gr),
         _ptr(br), _ptr(wr), _ptr(h0_fwd), _ptr(h0_rev), _ptr(cu_seqlens), int(chunk),
         _ptr(out), _ptr(hT_f), _ptr(hT_r), ws_ptr, ws_bytes, ctypes.byref(dims))
    return out, hT_f, hT_r


def gdn2_chunk_fwd_noalloc(q, k, v, g, b, w, h0, cu_seqlens, out, hT, *, chunk: int = 64, read: str = "post",
                           reverse: bool = False, accumulate: bool = False, l2norm: bool = False):
    """``gdr_gdn2_chunk_fwd_noalloc``: the two-pass GDN-2 forward on the library's fixed device
    scratch (no workspace, nothing allocated by the call). Arguments as ``gdn2_chunk_fwd``; ``out``
    and ``hT`` (or None for no final state) must be given, so that nothing is allocated here either."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    for name, t, tdt, shape in (("k", k, dt, (B, Hk, T, dk)), ("v", v, dt, (B, Hv, T, dv)),
                                ("g", g, torch.float32, (B, Hk, T, dk)), ("b", b, dt, (B, Hk, T, dk)),
                                ("w", w, dt, (B, Hv, T, dv)), ("out", out, dt, (B, Hv, T, dv))):
        _need(t, name, tdt, shape, dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        S = cu_seqlens.shape[0] - 1
    for name, t in (("h0", h0), ("hT", hT)):
        if t is not None:
            _need(t, name, torch.float32, (S, Hv, dk, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_REVERSE if reverse else 0) | \
        (GDR_ACCUMULATE if accumulate else 0) | (GDR_QK_L2NORM if l2norm else 0)
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, _dtype_code(dt), flags)
    _run(q, lib().gdr_gdn2_chunk_fwd_noalloc, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(h0),
         _ptr(cu_seqlens), int(chunk), _ptr(out), _ptr(hT), ctypes.byref(dims))
    return out, hT


def gdn2_chunk_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, num_seqs=0, dtype=torch.bfloat16) -> int:
    """Bytes of workspace the two-pass ``gdr_gdn2_chunk_fwd`` needs (num_seqs > 0: packed)."""
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, num_seqs, _dtype_code(dtype), 0)
    return int(lib().gdr_gdn2_chunk_fwd_workspace_bytes(ctypes.byref(dims), int(chunk), int(num_seqs > 0)))


def gdn2_decode_step(q, k, v, g, b, w, state_in, state_out=None, out=None, *, read: str = "post",
                     l2norm: bool = False):
    """One GDN-2 decode step (``gdr_gdn2_decode_step``). q, k, b [N, Hk, dk] and v, w [N, Hv, dv]
    in one dtype; g [N, Hk, dk] fp32; state_in [N, Hv, dk, dv] fp32. Returns (out, state_out)."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    _need(k, "k", dt, (N, Hk, dk), dev)
    _need(b, "b", dt, (N, Hk, dk), dev)
    _need(g, "g", torch.float32, (N, Hk, dk), dev)
    _need(v, "v", dt, (N, Hv, dv), dev)
    _need(w, "w", dt, (N, Hv, dv), dev)
    _need(state_in, "state_in", torch.float32, (N, Hv, dk, dv), dev)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    else:
        _need(state_out, "state_out", torch.float32, (N, Hv, dk, dv), dev)
    if out is None:
        out = torch.empty((N, Hv, dv), dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (N, Hv, dv), dev)
    if read not in ("pre", "post"):
        raise ValueError("read must be 'pre' or 'post'")
    flags = (GDR_READ_PRE if read == "pre" else 0) | (GDR_QK_L2NORM if l2norm else 0)
    dims = DecodeDims(N, Hk, Hv, dk, dv, code, flags)
    _run(q, lib().gdr_gdn2_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(state_in),
         _ptr(state_out), _ptr(out), ctypes.byref(dims))
    return out, state_out


def _workspace(t, need, dev):
    """The caller's workspace, or a new one of ``need`` bytes (None where none is needed)."""
    if need < 0:
        raise GdrError(2, lib().gdr_last_error().decode())
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _need(t, "workspace", torch.uint8, None, dev)
    return t


def _scan_args(x, a, b, A_log, dt_bias, cu_seqlens, reverse):
    _need(x, "x")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt, "x, a, b")
    if x.dim() != 3:
        raise ValueError("x must have shape (B, T, D) (got %s)" % (tuple(x.shape),))
    B, T, D = x.shape
    _need(a, "a", dt, (B, T, D), dev)
    _need(b, "b", dt, (B, T, D), dev)
    _need(A_log, "A_log", torch.float32, (D,), dev)
    _need(dt_bias, "dt_bias", torch.float32, (D,), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must have shape (S + 1,), S >= 1 (got %s)" % (tuple(cu_seqlens.shape),))
        S = cu_seqlens.shape[0] - 1
    return ScanDims(B, T, D, S if cu_seqlens is not None else 0, code, GDR_REVERSE if reverse else 0), S, dev


def channel_scan_fwd(x, a, b, A_log, dt_bias, h0=None, cu_seqlens=None, *, reverse: bool = False, out=None,
                     hT=None, want_state: bool = True, want_states: bool = False, workspace=None):
    """The gated linear recurrence per channel over whole sequences (``gdr_channel_scan_fwd``).

    x, a, b [B, T, D] (bf16 or fp32, one dtype); A_log, dt_bias [D] fp32; h0 [S, D] fp32 or None;
    cu_seqlens int32 [S+1] (device) or None. Returns (out [B, T, D], hT [S, D] or None, states or
    None); ``want_states`` keeps the block states ``channel_scan_bwd`` needs. ``hT`` may be ``h0``."""
    dims, S, dev = _scan_args(x, a, b, A_log, dt_bias, cu_seqlens, reverse)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (S, dims.D), dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", x.dtype, x.shape, dev)
    if hT is not None:
        _need(hT, "hT", torch.float32, (S, dims.D), dev)
    elif want_state:
        hT = torch.empty((S, dims.D), dtype=torch.float32, device=dev)
    packed = int(cu_seqlens is not None)
    d = ctypes.byref(dims)
    states = None
    if want_states:
        n = lib().gdr_channel_scan_states_elems(d, packed)
        if n < 0:
            raise GdrError(2, lib().gdr_last_error().decode())
        states = torch.empty(n, dtype=torch.float32, device=dev)
    ws = _workspace(workspace, lib().gdr_channel_scan_fwd_workspace_bytes(d, packed), dev)
    _run(x, lib().gdr_channel_scan_fwd, _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(h0),
         _ptr(cu_seqlens), _ptr(out), _ptr(hT), _ptr(states), _ptr(ws),
         0 if ws is None else ws.numel(), d)
    return out, hT, states


def channel_scan_bwd(x, a, b, A_log, dt_bias, states, dout, cu_seqlens=None, dhT=None, *, reverse: bool = False,
                     want_dh0: bool = True, workspace=None):
    """Gradients of ``channel_scan_fwd`` (``gdr_channel_scan_bwd``): its inputs, the ``states`` it
    kept, dout [B, T, D] and dhT [S, D] fp32 or None. Returns (dx, da, db [B, T, D] in x's dtype,
    dA_log, ddt_bias [D] fp32, dh0 [S, D] fp32 or None)."""
    dims, S, dev = _scan_args(x, a, b, A_log, dt_bias, cu_seqlens, reverse)
    packed = int(cu_seqlens is not None)
    d = ctypes.byref(dims)
    _need(dout, "dout", x.dtype, x.shape, dev)
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (S, dims.D), dev)
    _need(states, "states", torch.float32, (lib().gdr_channel_scan_states_elems(d, packed),), dev)
    dx, da, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dA_log, ddt_bias = torch.empty_like(A_log), torch.empty_like(A_log)
    dh0 = torch.empty((S, dims.D), dtype=torch.float32, device=dev) if want_dh0 else None
    ws = _workspace(workspace, lib().gdr_channel_scan_bwd_workspace_bytes(d, packed), dev)
    _run(x, lib().gdr_channel_scan_bwd, _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(states),
         _ptr(cu_seqlens), _ptr(dout), _ptr(dhT), _ptr(dx), _ptr(da), _ptr(db),
         _ptr(dA_log), _ptr(ddt_bias), _ptr(dh0), _ptr(ws),
         0 if ws is None else ws.numel(), d)
    return dx, da, db, dA_log, ddt_bias, dh0


def channel_scan_step(x, a, b, A_log, dt_bias, state_in, state_out=None, out=None):
    """One token of the channel scan (``gdr_channel_scan_step``): x, a, b [N, D]; state_in [N, D] fp32.
    ``state_out`` defaults to a new tensor; pass ``state_in`` itself to update in place. Returns
    (out [N, D], state_out)."""
    _need(x, "x")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt, "x, a, b")
    if x.dim() != 2:
        raise ValueError("x must have shape (N, D) (got %s)" % (tuple(x.shape),))
    N, D = x.shape
    _need(a, "a", dt, (N, D), dev)
    _need(b, "b", dt, (N, D), dev)
    _need(A_log, "A_log", torch.float32, (D,), dev)
    _need(dt_bias, "dt_bias", torch.float32, (D,), dev)
    _need(state_in, "state_in", torch.float32, (N, D), dev)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    else:
        _need(state_out, "state_out", torch.float32, (N, D), dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", dt, (N, D), dev)
    dims = ScanDims(N, 1, D, 0, code, 0)
    _run(x, lib().gdr_channel_scan_step, _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(state_in),
         _ptr(state_out), _ptr(out), ctypes.byref(dims))
    return out, state_out


ACTS = {"silu": 0, "gelu_tanh": 1}
GDR_FFN_KEEP_F32 = 256


def _ffn_args(x, w_gate, w_up, act):
    _need(x, "x")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt, "x, w_gate, w_up")
    if type(w_gate) is not torch.Tensor:
        _need(w_gate, "w_gate")
    if x.dim() < 1 or w_gate.dim() != 2:
        raise ValueError("x must have shape (..., D) and w_gate (F, D) (got %s, %s)" % (tuple(x.shape), tuple(w_gate.shape)))
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTS)))
    D, F = x.shape[-1], w_gate.shape[0]
    _need(w_gate, "w_gate", dt, (F, D), dev)
    _need(w_up, "w_up", dt, (F, D), dev)
    M = 1
    for n in x.shape[:-1]:
        M *= n
    return FfnDims(M, D, F, code, ACTS[act]), dev


def _keep(dims, dt, xdt, name):
    """Marks in which dtype gate and up are kept."""
    if dt == torch.float32:
        dims.act |= GDR_FFN_KEEP_F32
    elif dt != xdt:
        raise ValueError("%s must be torch.float32 or %s (got %s)" % (name, xdt, dt))


def gated_ffn_fwd(x, w_gate, w_up, *, act: str = "silu", out=None, want_saved: bool = False, saved_dtype=torch.float32):
    """Both projections of a gated feed-forward block, the activation and the product
    (``gdr_gated_ffn_fwd``): h = act(x w_gate^T) * (x w_up^T). x [..., D]; w_gate, w_up [F, D] (bf16
    or fp32, one dtype). Returns (h [..., F], gate, up); the projections gate and up [..., F] are kept
    for ``gated_ffn_bwd`` with ``want_saved``, else None. They are kept in ``saved_dtype``: fp32
    (``GDR_FFN_KEEP_F32``), or x's dtype, which for bf16 takes half the memory and leaves a third more
    error in the gradients."""
    dims, dev = _ffn_args(x, w_gate, w_up, act)
    if want_saved:
        _keep(dims, saved_dtype, x.dtype, "saved_dtype")
    shape = tuple(x.shape[:-1]) + (dims.F,)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
    else:
        _need(out, "out", x.dtype, shape, dev)
    gate = torch.empty(shape, dtype=saved_dtype, device=dev) if want_saved else None
    up = torch.empty_like(gate) if want_saved else None
    _run(x, lib().gdr_gated_ffn_fwd, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(out), _ptr(gate), _ptr(up),
         ctypes.byref(dims))
    return out, gate, up


def gated_ffn_bwd(x, w_gate, w_up, gate, up, dh, *, act: str = "silu", workspace=None):
    """Gradients of ``gated_ffn_fwd`` (``gdr_gated_ffn_bwd``): its inputs, the gate and up it kept (fp32 or
    x's dtype, both the same) and dh [..., F]. Returns (dx [..., D], dw_gate, dw_up [F, D]) in x's dtype."""
    dims, dev = _ffn_args(x, w_gate, w_up, act)
    shape = tuple(x.shape[:-1]) + (dims.F,)
    _need(gate, "gate", None, shape, dev)
    _keep(dims, gate.dtype, x.dtype, "gate")
    _need(up, "up", gate.dtype, shape, dev)
    _need(dh, "dh", x.dtype, shape, dev)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w_gate), torch.empty_like(w_up)
    ws = _workspace(workspace, lib().gdr_gated_ffn_bwd_workspace_bytes(ctypes.byref(dims)), dev)
    _run(x, lib().gdr_gated_ffn_bwd, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(gate), _ptr(up), _ptr(dh), _ptr(dx),
         _ptr(dwg), _ptr(dwu), _ptr(ws), 0 if ws is None else ws.numel(),
         ctypes.byref(dims))
    return dx, dwg, dwu


def _ce_args(x, weight, targets):
    _need(x, "x")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt, "x, weight")
    if type(weight) is not torch.Tensor:
        _need(weight, "weight")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must have shape (N, D) and weight (V, D) (got %s, %s)" % (tuple(x.shape), tuple(weight.shape)))
    N, D = x.shape
    V = weight.shape[0]
    _need(weight, "weight", dt, (V, D), dev)
    _need(targets, "targets", torch.int64, (N,), dev)
    return CeDims(N, D, V, code, 0), dev


def linear_ce_fwd(x, weight, targets, *, workspace=None):
    """Softmax cross entropy of x weight^T per token, the logits never kept (``gdr_linear_ce_fwd``).
    x [N, D], weight [V, D] (bf16 or fp32, one dtype); targets [N] int64, a value outside 0 .. V-1 (as
    -100) for a token that bears no loss. Returns (loss [N], lse [N]) fp32."""
    dims, dev = _ce_args(x, weight, targets)
    loss = torch.empty(dims.N, dtype=torch.float32, device=dev)
    lse = torch.empty_like(loss)
    ws = _workspace(workspace, lib().gdr_linear_ce_fwd_workspace_bytes(ctypes.byref(dims)), dev)
    _run(x, lib().gdr_linear_ce_fwd, _ptr(x), _ptr(weight), _ptr(targets), _ptr(loss), _ptr(lse), _ptr(ws),
         0 if ws is None else ws.numel(), ctypes.byref(dims))
    return loss, lse


def linear_ce_bwd(x, weight, targets, lse, dloss, *, workspace=None):
    """Gradients of ``linear_ce_fwd`` (``gdr_linear_ce_bwd``): its inputs, the lse it returned and
    dloss [N] fp32, the gradient of each token's loss. Returns (dx [N, D], dweight [V, D]) in x's dtype."""
    dims, dev = _ce_args(x, weight, targets)
    _need(lse, "lse", torch.float32, (dims.N,), dev)
    _need(dloss, "dloss", torch.float32, (dims.N,), dev)
    dx, dw = torch.empty_like(x), torch.empty_like(weight)
    ws = _workspace(workspace, lib().gdr_linear_ce_bwd_workspace_bytes(ctypes.byref(dims)), dev)
    _run(x, lib().gdr_linear_ce_bwd, _ptr(x), _ptr(weight), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(dx), _ptr(dw),
         _ptr(ws), 0 if ws is None else ws.numel(), ctypes.byref(dims))
    return dx, dw


def _attn_args(q, k, v, log_alpha, cu_seqlens):
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    if type(v) is not torch.Tensor:
        _need(v, "v")
    if type(log_alpha) is not torch.Tensor:
        _need(log_alpha, "log_alpha")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must have shape (B, Hk, T, dk) and v (B, Hv, T, dv) (got %s, %s)" % (tuple(q.shape), tuple(v.shape)))
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    _need(k, "k", dt, (B, Hk, T, dk), dev)
    _need(v, "v", dt, (B, Hv, T, dv), dev)
    head = log_alpha.dim() == 1
    _need(log_alpha, "log_alpha", torch.float32, (Hv,) if head else (B, Hv, T), dev)
    S = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must have shape (S + 1,), S >= 1 (got %s)" % (tuple(cu_seqlens.shape),))
        S = cu_seqlens.shape[0] - 1
    dims = ChunkDims(B, T, Hk, Hv, dk, dv, S if cu_seqlens is not None else 0, code, GDR_HEAD_DECAY if head else 0)
    return dims, (S, Hv, dk, dv), dev


def linear_attn_fwd(q, k, v, log_alpha, h0=None, cu_seqlens=None, *, out=None, hT=None, want_state: bool = True,
                    workspace=None):
    """Linear attention with a decay for each head over whole sequences (``gdr_linear_attn_fwd``):
    H_t = exp(log_alpha_t) H_{t-1} + k_t v_t^T, o_t = H_t^T q_t.

    q, k [B, Hk, T, dk]; v [B, Hv, T, dv] (bf16 or fp32, one dtype); log_alpha fp32, [B, Hv, T] or, one
    decay for each head, [Hv]; h0 [S, Hv, dk, dv] fp32 or None; cu_seqlens int32 [S+1] (device) or None.
    Returns (out [B, Hv, T, dv], hT [S, Hv, dk, dv] or None). ``hT`` may be ``h0`` itself."""
    dims, state, dev = _attn_args(q, k, v, log_alpha, cu_seqlens)
    if h0 is not None:
        _need(h0, "h0", torch.float32, state, dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need(out, "out", v.dtype, v.shape, dev)
    if hT is not None:
        _need(hT, "hT", torch.float32, state, dev)
    elif want_state:
        hT = torch.empty(state, dtype=torch.float32, device=dev)
    d = ctypes.byref(dims)
    ws = _workspace(workspace, lib().gdr_linear_attn_fwd_workspace_bytes(d, int(cu_seqlens is not None)), dev)
    _run(q, lib().gdr_linear_attn_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(cu_seqlens), _ptr(out),
         _ptr(hT), _ptr(ws), 0 if ws is None else ws.numel(), d)
    return out, hT


def linear_attn_bwd(q, k, v, log_alpha, dout, h0=None, cu_seqlens=None, dhT=None, *, want_dh0: bool = True,
                    workspace=None):
    """Gradients of ``linear_attn_fwd`` (``gdr_linear_attn_bwd``): its inputs, dout [B, Hv, T, dv] and dhT
    [S, Hv, dk, dv] fp32 or None. Returns (dq, dk [B, Hk, T, dk] and dv [B, Hv, T, dv] in q's dtype,
    dlog_alpha fp32 like log_alpha, dh0 [S, Hv, dk, dv] fp32 or None)."""
    dims, state, dev = _attn_args(q, k, v, log_alpha, cu_seqlens)
    _need(dout, "dout", v.dtype, v.shape, dev)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _need(t, name, torch.float32, state, dev)
    dq, dk, dv, dla = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(log_alpha)
    dh0 = torch.empty(state, dtype=torch.float32, device=dev) if want_dh0 else None
    d = ctypes.byref(dims)
    ws = _workspace(workspace, lib().gdr_linear_attn_bwd_workspace_bytes(d, int(cu_seqlens is not None)), dev)
    _run(q, lib().gdr_linear_attn_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(cu_seqlens), _ptr(dout),
         _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dla), _ptr(dh0), _ptr(ws),
         0 if ws is None else ws.numel(), d)
    return dq, dk, dv, dla, dh0


def linear_attn_step(q, k, v, log_alpha, state_in, state_out=None, out=None):
    """One token of linear attention (``gdr_linear_attn_step``): q, k [N, Hk, dk]; v [N, Hv, dv]; log_alpha
    fp32 [N, Hv] or [Hv]; state_in [N, Hv, dk, dv] fp32. ``state_out`` defaults to a new tensor; pass
    ``state_in`` itself to update in place. Returns (out [N, Hv, dv], state_out)."""
    _need(q, "q")
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    if type(v) is not torch.Tensor:
        _need(v, "v")
    if type(log_alpha) is not torch.Tensor:
        _need(log_alpha, "log_alpha")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q must have shape (N, Hk, dk) and v (N, Hv, dv) (got %s, %s)" % (tuple(q.shape), tuple(v.shape)))
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    head = log_alpha.dim() == 1
    _need(k, "k", dt, (N, Hk, dk), dev)
    _need(v, "v", dt, (N, Hv, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (Hv,) if head else (N, Hv), dev)
    _need(state_in, "state_in", torch.float32, (N, Hv, dk, dv), dev)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    else:
        _need(state_out, "state_out", torch.float32, (N, Hv, dk, dv), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need(out, "out", dt, (N, Hv, dv), dev)
    dims = DecodeDims(N, Hk, Hv, dk, dv, code, GDR_HEAD_DECAY if head else 0)
    _run(q, lib().gdr_linear_attn_step, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(state_in), _ptr(state_out),
         _ptr(out), ctypes.byref(dims))
    return out, state_out


GDR_ROPE_NEIGHBOURS = 1


def _head_rows(t, name, dtype=None, lead=None, d=None, device=None):
    """The stride between the rows of t [..., H, d]: each token's heads are one piece, tokens are evenly apart (as a
    part of a projection's rows is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    shape, st = t.shape, t.stride()
    if len(shape) not in (3, 4) or (lead is not None and (shape[:-2] != lead or shape[-1] != d)):
        want = "(B, T, H, d) or (N, H, d)" if lead is None else tuple(lead) + ("H", d)
        raise ValueError("%s must have shape %s (got %s)" % (name, want, tuple(shape)))
    H, d = shape[-2], shape[-1]
    if t.is_contiguous():
        return H * d
    # a part of a projection's rows, as nearly every call brings it
    if len(shape) == 4 and st[3] == 1 and st[2] == d and st[1] >= H * d and st[0] == shape[1] * st[1]:
        return st[1]
    if (d > 1 and st[-1] != 1) or (H > 1 and st[-2] != d):
        raise ValueError("%s must have each token's heads in one piece (strides %s)" % (name, tuple(st)))
    outer = [(n, s) for n, s in zip(shape[:-2], st[:-2]) if n > 1]
    if not outer:
        return H * d
    row = outer[-1][1]
    if len(outer) == 2 and outer[0][1] != outer[1][0] * row:
        raise ValueError("%s must have its tokens evenly apart (strides %s)" % (name, tuple(st)))
    return row


def _qk_args(q, k, w_q, w_k, inv_freq, positions, eps, interleaved):
    """The call's sizes, the device, and the shapes of the results."""
    qs = _head_rows(q, "q")
    dev, dt, shape = q.device, q.dtype, q.shape
    lead, Hq, d = shape[:-2], shape[-2], shape[-1]
    code = _dtype_code(dt, "q, k")
    ks = _head_rows(k, "k", dt, lead, d, dev)
    Hk = k.shape[-2]
    if w_q is not None:
        _need(w_q, "w_q", torch.float32, (d,), dev)
    if w_k is not None:
        _need(w_k, "w_k", torch.float32, (d,), dev)
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, None, dev)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must have shape (rot / 2,) (got %s)" % (tuple(inv_freq.shape),))
        rot = 2 * inv_freq.shape[0]
    if positions is not None:
        _need(positions, "positions", torch.int64, lead, dev)
    if len(lead) == 2:
        B, T = lead
        like_q, like_k = (B, Hq, T, d), (B, Hk, T, d)
    else:
        B, T = lead[0], 1
        like_q, like_k = (B, Hq, d), (B, Hk, d)
    return QkDims(B, T, Hq, Hk, d, rot, qs, ks, 0, 0, eps, code, GDR_ROPE_NEIGHBOURS if interleaved else 0), dev, like_q, like_k


def qk_norm_rope_fwd(q, k, w_q, w_k, inv_freq, positions=None, *, eps: float = 1e-6, interleaved: bool = False,
                     out_q=None, out_k=None):
    """The norm of each query and key head and the rotation by its position, in one pass
    (``gdr_qk_norm_rope_fwd``): y = R(p) (x rsqrt(mean(x^2) + eps) w).

    q [B, T, Hq, d], k [B, T, Hk, d] (bf16 or fp32, one dtype), each token's heads in one piece: parts of a
    projection's rows are taken as they are; w_q, w_k [d] fp32 or None for ones; inv_freq [rot / 2] fp32, the
    first rot channels' angles by position, or None for no rotation; positions [B, T] int64 or None for
    0 .. T-1. Channels i and rot / 2 + i are a pair, 2i and 2i + 1 with ``interleaved``. Returns (oq
    [B, Hq, T, d], ok [B, Hk, T, d]). One token of N sequences: q [N, Hq, d], k [N, Hk, d], positions [N];
    returns [N, Hq, d], [N, Hk, d]."""
    dims, dev, like_q, like_k = _qk_args(q, k, w_q, w_k, inv_freq, positions, eps, interleaved)
    if out_q is None:
        out_q = q.new_empty(like_q)
    else:
        _need(out_q, "out_q", q.dtype, like_q, dev)
    if out_k is None:
        out_k = k.new_empty(like_k)
    else:
        _need(out_k, "out_k", q.dtype, like_k, dev)
    _run(q, lib().gdr_qk_norm_rope_fwd, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k), _ptr(inv_freq), _ptr(positions), _ptr(out_q),
         _ptr(out_k), ctypes.byref(dims))
    return out_q, out_k


def qk_norm_rope_bwd(q, k, w_q, w_k, inv_freq, doq, dok, positions=None, *, eps: float = 1e-6, interleaved: bool = False,
                     dq=None, dk=None, workspace=None):
    """Gradients of ``qk_norm_rope_fwd`` (``gdr_qk_norm_rope_bwd``): its inputs, doq and dok like its results.
    Returns (dq like q, dk like k in q's dtype, dw_q, dw_k [d] fp32 or None where there is no weight). dq and dk
    may be given, as parts of one buffer of rows too."""
    dims, dev, like_q, like_k = _qk_args(q, k, w_q, w_k, inv_freq, positions, eps, interleaved)
    _need(doq, "doq", q.dtype, like_q, dev)
    _need(dok, "dok", q.dtype, like_k, dev)
    if dq is None:
        dq = q.new_empty(q.shape)
        dims.dq_stride = dims.Hq * dims.d
    elif tuple(dq.shape) != tuple(q.shape):
        raise ValueError("dq must have shape %s (got %s)" % (tuple(q.shape), tuple(dq.shape)))
    else:
        dims.dq_stride = _head_rows(dq, "dq", q.dtype, q.shape[:-2], q.shape[-1], dev)
    if dk is None:
        dk = k.new_empty(k.shape)
        dims.dk_stride = dims.Hk * dims.d
    elif tuple(dk.shape) != tuple(k.shape):
        raise ValueError("dk must have shape %s (got %s)" % (tuple(k.shape), tuple(dk.shape)))
    else:
        dims.dk_stride = _head_rows(dk, "dk", q.dtype, q.shape[:-2], q.shape[-1], dev)
    dw_q = None if w_q is None else torch.empty_like(w_q)
    dw_k = None if w_k is None else torch.empty_like(w_k)
    need = lib().gdr_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(dims)) if dw_q is not None or dw_k is not None else 0
    ws = _workspace(workspace, need, dev)
    _run(q, lib().gdr_qk_norm_rope_bwd, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k), _ptr(inv_freq), _ptr(positions), _ptr(doq), _ptr(dok),
         _ptr(dq), _ptr(dk), _ptr(dw_q), _ptr(dw_k), _ptr(ws), 0 if ws is None else ws.numel(),
         ctypes.byref(dims))
    return dq, dk, dw_q, dw_k


def selftest_mfma(a, b):
    """Diagnostic: the 16x16 product of a [16, 32] and b [32, 16] (fp32 GPU tensors) through
    the library's matrix-core operand layouts. Returns d [3, 16, 16] (see include/gdr.h)."""
    _need(a, "a", torch.float32, (16, 32))
    _need(b, "b", torch.float32, (32, 16), a.device)
    d = torch.empty((3, 16, 16), dtype=torch.float32, device=a.device)
    _run(a, lib().gdr_selftest_mfma, _ptr(a), _ptr(b), _ptr(d))
    return d
