"""Packed (block-diagonal causal) attention on GB300: Python binding of libpa.

Thin ctypes marshalling over the C ABI in include/pa.h: every function here
has the same name as its C entry point, checks that the torch tensors it is
given have the layout the ABI expects, and passes their device pointers and
the current CUDA stream through. All computation happens in the CUDA kernels
of libpa.so; there is no other code path. If the library has not been built
(``python -m segment_masked_causal_gb300.build``), importing works but every
call raises ``LibraryMissing``.

Semantics (mlx-train-perf changelog, PACKED kernels; 0.5.1 README,
"Sequence packing"): token i attends token j iff j <= i and seg[i] == seg[j].
q/out/dout/dq are (B, Hq, N, D) bf16; k/v/dk/dv are (B, Hkv, N, D) bf16; lse
is (B, Hq, N) fp32; seg is (B, N) int32; D in {64, 96, 128}. The *_strided
calls take (B, H, N, D) views with any strides (last dim contiguous); N need
not be a multiple of 128 except in the single-step calls.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpa.so")

PA_OK = 0
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_NULL", 2: "PA_ERR_HEAD_DIM", 3: "PA_ERR_GQA", 4: "PA_ERR_SHAPE",
                5: "PA_ERR_ALIGN", 6: "PA_ERR_WORKSPACE", 7: "PA_ERR_ARCH", 8: "PA_ERR_CUDA", 9: "PA_ERR_DTYPE",
                10: "PA_ERR_HOST_MEMORY"}
PA_IO_BF16, PA_IO_F32 = 0, 1
PA_CKPT_INT8, PA_CKPT_E4M3 = 0, 1
PA_CKPT_MAX_TENSORS = 8
EXPORTS = ["pa_workspace_bytes", "pa_fwd", "pa_bwd", "pa_fwd_causal", "pa_bwd_causal", "pa_build_tile_table",
           "pa_fwd_tiles", "pa_bwd_delta", "pa_bwd_dq", "pa_bwd_dkv", "pa_bwd_noalloc", "pa_device_status",
           "pa_selftest_wait_timeout", "pa_selftest_exp2_fma", "pa_pack_first_fit", "pa_workspace_bytes_strided", "pa_fwd_strided",
           "pa_bwd_strided", "pa_lce_workspace_bytes", "pa_lce_fwd", "pa_lce_bwd_workspace_bytes", "pa_lce_bwd",
           "pa_bwd_fused_workspace_bytes", "pa_bwd_fused", "pa_logp_workspace_bytes", "pa_logp_plan", "pa_logp_fwd",
           "pa_logp_bwd_workspace_bytes", "pa_logp_bwd", "pa_ckpt_save", "pa_ckpt_load", "pa_bwd_ckpt_workspace_bytes",
           "pa_bwd_ckpt", "pa_status_string"]


class LibraryMissing(RuntimeError):
    pass


class PAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class pa_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("D", ctypes.c_int32), ("scale", ctypes.c_float)]


class pa_strides(ctypes.Structure):
    _fields_ = [("q_b", ctypes.c_int64), ("q_h", ctypes.c_int64), ("q_n", ctypes.c_int64),
                ("k_b", ctypes.c_int64), ("k_h", ctypes.c_int64), ("k_n", ctypes.c_int64)]


class pa_ckpt_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("C", ctypes.c_int32),
                ("s_b", ctypes.c_int64), ("s_h", ctypes.c_int64), ("s_n", ctypes.c_int64)]


class pa_ckpt(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded libpa.so (ctypes), with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise LibraryMissing(f"{LIB_PATH} not built; run python -m segment_masked_causal_gb300.build")
            L = ctypes.CDLL(LIB_PATH)
            P, S = ctypes.c_void_p, ctypes.c_size_t
            D = ctypes.POINTER(pa_dims)
            L.pa_workspace_bytes.argtypes = [D]
            L.pa_workspace_bytes.restype = S
            L.pa_fwd.argtypes = [D, P, P, P, P, P, P, P, S, P]
            L.pa_fwd_causal.argtypes = [D, P, P, P, P, P, P, S, P]
            L.pa_bwd.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_causal.argtypes = [D, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_build_tile_table.argtypes = [D, P, P, S, P]
            L.pa_fwd_tiles.argtypes = [D, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_delta.argtypes = [D, P, P, P, P, S, P]
            L.pa_bwd_dq.argtypes = [D, P, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_dkv.argtypes = [D, P, P, P, P, P, P, P, P, P, S, P]
            for f in ("pa_fwd", "pa_fwd_causal", "pa_bwd", "pa_bwd_causal", "pa_build_tile_table", "pa_fwd_tiles",
                      "pa_bwd_delta", "pa_bwd_dq", "pa_bwd_dkv"):
                getattr(L, f).restype = ctypes.c_int
            L.pa_bwd_fused_workspace_bytes.argtypes = [D]
            L.pa_bwd_fused_workspace_bytes.restype = S
            L.pa_bwd_fused.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_fused.restype = ctypes.c_int
            L.pa_bwd_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(ctypes.c_uint32), P]
            L.pa_bwd_noalloc.restype = ctypes.c_int
            L.pa_selftest_wait_timeout.argtypes = [P, S, P]
            L.pa_selftest_wait_timeout.restype = ctypes.c_int
            L.pa_selftest_exp2_fma.argtypes = [P, P, ctypes.c_int64, P]
            L.pa_selftest_exp2_fma.restype = ctypes.c_int
            L.pa_device_status.argtypes = [P, P]
            L.pa_device_status.restype = ctypes.c_uint32
            ST = ctypes.POINTER(pa_strides)
            L.pa_workspace_bytes_strided.argtypes = [D]
            L.pa_workspace_bytes_strided.restype = S
            L.pa_fwd_strided.argtypes = [D, ST, ctypes.c_int32, P, P, P, P, P, P, P, S, P]
            L.pa_fwd_strided.restype = ctypes.c_int
            L.pa_bwd_strided.argtypes = [D, ST, ctypes.c_int32, P, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_strided.restype = ctypes.c_int
            I32, U64 = ctypes.c_int32, ctypes.c_uint64
            L.pa_lce_workspace_bytes.argtypes = [I32, I32, I32]
            L.pa_lce_workspace_bytes.restype = S
            L.pa_lce_fwd.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, S, P]
            L.pa_lce_fwd.restype = ctypes.c_int
            L.pa_lce_bwd_workspace_bytes.argtypes = [I32, I32, I32]
            L.pa_lce_bwd_workspace_bytes.restype = S
            L.pa_lce_bwd.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, S, P]
            L.pa_lce_bwd.restype = ctypes.c_int
            F = ctypes.c_float
            L.pa_logp_workspace_bytes.argtypes = [I32, I32, I32, I32]
            L.pa_logp_workspace_bytes.restype = S
            L.pa_logp_fwd.argtypes = [I32, I32, I32, F, I32, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_logp_fwd.restype = ctypes.c_int
            L.pa_logp_plan.argtypes = [I32, I32, I32, I32, P]
            L.pa_logp_plan.restype = ctypes.c_int
            L.pa_logp_bwd_workspace_bytes.argtypes = [I32, I32, I32]
            L.pa_logp_bwd_workspace_bytes.restype = S
            L.pa_logp_bwd.argtypes = [I32, I32, I32, F, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_logp_bwd.restype = ctypes.c_int
            CK = ctypes.POINTER(pa_ckpt)
            L.pa_ckpt_save.argtypes = [I32, P, I32, I32, I32, P]  # an array of pa_ckpt_tensor, or its bytes
            L.pa_ckpt_save.restype = ctypes.c_int
            L.pa_ckpt_load.argtypes = [I32, P, I32, I32, I32, P]
            L.pa_ckpt_load.restype = ctypes.c_int
            L.pa_bwd_ckpt_workspace_bytes.argtypes = [D]
            L.pa_bwd_ckpt_workspace_bytes.restype = S
            L.pa_bwd_ckpt.argtypes = [D, ST, I32, I32, CK, CK, CK, CK, P, P, P, P, P, P, P, S, P]
            L.pa_bwd_ckpt.restype = ctypes.c_int
            L.pa_pack_first_fit.argtypes = [P, P, I32, P, I32, I32, I32, U64, U64, P, P, P, P, P, P, P]
            L.pa_pack_first_fit.restype = ctypes.c_int
            L.pa_status_string.argtypes = [ctypes.c_int]
            L.pa_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def make_dims(B, Hq, Hkv, N, D, scale=0.0) -> pa_dims:
    return pa_dims(int(B), int(Hq), int(Hkv), int(N), int(D), float(scale))


def _check(code: int):
    if code != PA_OK:
        raise PAError(code, lib().pa_status_string(code).decode())


def _ptr(t, dtype=None, name=""):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        # the same stream without building a Stream object (3 us of a launch-bound call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dims_of(q, k, scale):
    B, Hq, N, D = q.shape
    return make_dims(B, Hq, k.shape[1], N, D, scale)


def pa_workspace_bytes(B, Hq, Hkv, N, D) -> int:
    d = make_dims(B, Hq, Hkv, N, D)
    return int(lib().pa_workspace_bytes(ctypes.byref(d)))


def pa_workspace_bytes_strided(B, Hq, Hkv, N, D) -> int:
    d = make_dims(B, Hq, Hkv, N, D)
    return int(lib().pa_workspace_bytes_strided(ctypes.byref(d)))


def workspace(q, k, device=None, strided=False):
    """A device workspace sized for q/k (caller-owned torch uint8 tensor);
    strided=True sizes it for pa_fwd_strided / pa_bwd_strided."""
    import torch
    B, Hq, N, D = q.shape
    f = pa_workspace_bytes_strided if strided else pa_workspace_bytes
    n = f(B, Hq, k.shape[1], N, D)
    if n == 0:
        raise PAError(4, "invalid dims")
    return torch.empty(n, dtype=torch.uint8, device=device or q.device)


def _ptr_rows(t, dtype, name, like=None):
    """Device pointer of a (B, H, N, D) CUDA tensor whose last dim is
    contiguous; `like` (if given) must have the same strides."""
    if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a 4-d CUDA tensor with a contiguous last dim")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if like is not None and tuple(t.stride()) != tuple(like.stride()):
        raise ValueError(f"{name} must have the strides of its group's first tensor")
    return t.data_ptr()


def _strides_of(q, k):
    return pa_strides(q.stride(0), q.stride(1), q.stride(2), k.stride(0), k.stride(1), k.stride(2))


def _io_dtype(q):
    import torch
    if q.dtype == torch.bfloat16:
        return q.dtype, PA_IO_BF16
    if q.dtype == torch.float32:
        return q.dtype, PA_IO_F32
    raise ValueError(f"q must be bfloat16 or float32, got {q.dtype}")


def pa_fwd_strided(q, k, v, seg, out, lse, ws, scale=0.0, stream=None):
    """pa_fwd on (B, H, N, D) views with any strides (e.g. (B, N, H, D) memory
    transposed), bf16 or fp32 (all tensors alike; fp32 is rounded to bf16 on
    the way in); seg None = plain causal. out must share q's strides."""
    import torch
    bf, io = _io_dtype(q)
    d = _dims_of(q, k, scale)
    st = _strides_of(q, k)
    _check(lib().pa_fwd_strided(ctypes.byref(d), ctypes.byref(st), io, _ptr_rows(q, bf, "q"), _ptr_rows(k, bf, "k"),
                                _ptr_rows(v, bf, "v", k), _ptr(seg, torch.int32, "seg"),
                                _ptr_rows(out, bf, "out", q), _ptr(lse, torch.float32, "lse"),
                                _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_bwd_strided(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale=0.0, stream=None):
    """pa_bwd on strided (B, H, N, D) views, bf16 or fp32 (all alike): out,
    dout and dq share q's strides; v, dk and dv share k's. seg None = plain
    causal."""
    import torch
    bf, io = _io_dtype(q)
    d = _dims_of(q, k, scale)
    st = _strides_of(q, k)
    _check(lib().pa_bwd_strided(ctypes.byref(d), ctypes.byref(st), io, _ptr_rows(q, bf, "q"), _ptr_rows(k, bf, "k"),
                                _ptr_rows(v, bf, "v", k), _ptr_rows(out, bf, "out", q),
                                _ptr_rows(dout, bf, "dout", q), _ptr(lse, torch.float32, "lse"),
                                _ptr(seg, torch.int32, "seg"), _ptr_rows(dq, bf, "dq", q), _ptr_rows(dk, bf, "dk", k),
                                _ptr_rows(dv, bf, "dv", k), _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_fwd(q, k, v, seg, out, lse, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_fwd(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                        _ptr(seg, torch.int32, "seg"), _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"),
                        _ptr(ws, None, "ws"), ws.numel() if hasattr(ws, "numel") else 0, _stream(stream)))


def pa_fwd_causal(q, k, v, out, lse, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_fwd_causal(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                               _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"), _ptr(ws, None, "ws"),
                               ws.numel(), _stream(stream)))


def pa_bwd(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                        _ptr(out, bf, "out"), _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"),
                        _ptr(seg, torch.int32, "seg"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"), _ptr(dv, bf, "dv"),
                        _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_bwd_fused_workspace_bytes(B, Hq, Hkv, N, D) -> int:
    d = make_dims(B, Hq, Hkv, N, D)
    return int(lib().pa_bwd_fused_workspace_bytes(ctypes.byref(d)))


def pa_bwd_fused(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale=0.0, stream=None):
    """The single-pass backward (seg None = plain causal); ws sized by
    pa_bwd_fused_workspace_bytes."""
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd_fused(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                              _ptr(out, bf, "out"), _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"),
                              _ptr(seg, torch.int32, "seg"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"),
                              _ptr(dv, bf, "dv"), _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def backward_fused(q, k, v, out, dout, lse, seg=None, scale=0.0, ws=None):
    """Allocate dq/dk/dv and run the single-pass backward (contiguous bf16,
    N % 128 == 0); dq is not bitwise reproducible from run to run."""
    import torch
    B, Hq, N, D = q.shape
    if ws is None:
        n = pa_bwd_fused_workspace_bytes(B, Hq, k.shape[1], N, D)
        if n == 0:
            raise PAError(4, "invalid dims for the single-pass backward")
        ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    pa_bwd_fused(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale)
    return dq, dk, dv


def pa_bwd_causal(q, k, v, out, dout, lse, dq, dk, dv, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd_causal(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                               _ptr(out, bf, "out"), _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"),
                               _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"), _ptr(dv, bf, "dv"), _ptr(ws, None, "ws"),
                               ws.numel(), _stream(stream)))


def pa_build_tile_table(q, k, seg, ws, scale=0.0, stream=None):
    import torch
    d = _dims_of(q, k, scale)
    _check(lib().pa_build_tile_table(ctypes.byref(d), _ptr(seg, torch.int32, "seg"), _ptr(ws, None, "ws"),
                                     ws.numel(), _stream(stream)))


def pa_fwd_tiles(q, k, v, seg, out, lse, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_fwd_tiles(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                              _ptr(seg, torch.int32, "seg"), _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"),
                              _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_bwd_delta(q, k, out, dout, lse, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd_delta(ctypes.byref(d), _ptr(out, bf, "out"), _ptr(dout, bf, "dout"),
                              _ptr(lse, torch.float32, "lse"), _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_bwd_dq(q, k, v, dout, lse, seg, dq, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd_dq(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                           _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"), _ptr(seg, torch.int32, "seg"),
                           _ptr(dq, bf, "dq"), _ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_bwd_dkv(q, k, v, dout, lse, seg, dk, dv, ws, scale=0.0, stream=None):
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    _check(lib().pa_bwd_dkv(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                            _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"), _ptr(seg, torch.int32, "seg"),
                            _ptr(dk, bf, "dk"), _ptr(dv, bf, "dv"), _ptr(ws, None, "ws"), ws.numel(),
                            _stream(stream)))


def pa_bwd_noalloc(q, k, v, out, dout, lse, seg, dq, dk, dv, scale=0.0, stream=None, wait_status=False):
    """pa_bwd without a workspace, for callers that cannot allocate device
    memory (the scratch is a fixed 8 MiB array inside the library). Returns the
    device status word when wait_status is true (the call then synchronises),
    else None. Calls that overlap on the GPU share that array and race."""
    import torch
    bf = torch.bfloat16
    d = _dims_of(q, k, scale)
    st = ctypes.c_uint32(0xFFFFFFFF)
    _check(lib().pa_bwd_noalloc(ctypes.byref(d), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                                _ptr(out, bf, "out"), _ptr(dout, bf, "dout"), _ptr(lse, torch.float32, "lse"),
                                _ptr(seg, torch.int32, "seg"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"),
                                _ptr(dv, bf, "dv"), ctypes.byref(st) if wait_status else None, _stream(stream)))
    return int(st.value) if wait_status else None


def pa_selftest_wait_timeout(ws, stream=None):
    """Launch the bounded-wait self-test into the workspace status word (see
    include/pa.h); read the result with pa_device_status."""
    _check(lib().pa_selftest_wait_timeout(_ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


def pa_selftest_exp2_fma(x, y, stream=None):
    """y = 2^x through the FMA-pipe exponential (see include/pa.h);
    x and y are fp32 CUDA tensors of the same number of elements."""
    import torch
    if x.numel() != y.numel():
        raise ValueError("x and y differ in size")
    _check(lib().pa_selftest_exp2_fma(_ptr(x, torch.float32, "x"), _ptr(y, torch.float32, "y"), x.numel(),
                                      _stream(stream)))


def pa_device_status(ws, stream=None) -> int:
    return int(lib().pa_device_status(_ptr(ws, None, "ws"), _stream(stream)))


def pa_pack_first_fit(lengths, rows, N, seed=0, epoch=0, offsets=None, tokens=None, pad_token=0):
    """Pack sequences into `rows` rows of N tokens (host call; see include/pa.h).

    lengths/offsets: per-sequence token counts and prompt lengths (offsets
    None = all 0); tokens: the sequences' tokens concatenated in input order,
    or None to skip the token rows. Returns a dict of numpy arrays: seg and
    loss_mask (rows, N), row_tokens and row_targets (rows, N) or None,
    placement (count,) int64 flat start index or -1, and the ints rows_used
    and placed_tokens. row_targets holds, where loss_mask is 1, the next token
    of the same sequence, and -1 elsewhere (an ignored target for
    pa_lce_fwd)."""
    import numpy as np
    lengths = np.ascontiguousarray(lengths, dtype=np.int32).reshape(-1)
    count = lengths.size
    off = None if offsets is None else np.ascontiguousarray(offsets, dtype=np.int32).reshape(-1)
    if off is not None and off.size != count:
        raise ValueError("offsets must have one entry per sequence")
    tok = None if tokens is None else np.ascontiguousarray(tokens, dtype=np.int32).reshape(-1)
    if tok is not None and tok.size != int(lengths.astype(np.int64).sum()):
        raise ValueError("tokens must hold sum(lengths) values")
    rows, N = int(rows), int(N)
    cells = max(rows, 0) * max(N, 0)
    seg = np.empty(cells, np.int32)
    mask = np.empty(cells, np.uint8)
    row_tokens = np.empty(cells, np.int32) if tok is not None else None
    row_targets = np.empty(cells, np.int32) if tok is not None else None
    placement = np.empty(count, np.int64)
    used, placed = ctypes.c_int32(0), ctypes.c_int64(0)

    def p(a):
        return None if a is None or a.size == 0 else a.ctypes.data

    _check(lib().pa_pack_first_fit(p(lengths), p(off), count, p(tok), int(pad_token), rows, N,
                                   int(seed) & 0xFFFFFFFFFFFFFFFF, int(epoch) & 0xFFFFFFFFFFFFFFFF,
                                   seg.ctypes.data if cells else None, p(mask), p(row_tokens), p(row_targets),
                                   p(placement),
                                   ctypes.byref(used), ctypes.byref(placed)))
    return {"seg": seg.reshape(rows, N), "loss_mask": mask.reshape(rows, N),
            "row_tokens": None if row_tokens is None else row_tokens.reshape(rows, N),
            "row_targets": None if row_targets is None else row_targets.reshape(rows, N),
            "placement": placement, "rows_used": int(used.value), "placed_tokens": int(placed.value)}


def packed_batches(lengths, B, N, seed, epoch, offsets=None, tokens=None, pad_token=0, rank=0, world=1):
    """One epoch of fixed-shape packed batches: pack every sequence with
    pa_pack_first_fit into as many rows as it needs, then yield consecutive
    groups of B rows as dicts of seg, loss_mask, row_tokens and row_targets,
    each (B, N).
    Rows of the last batch that hold no sequence are one padding segment with
    no supervised token. Sequences longer than N are left out.

    Data parallel: with world > 1, every rank packs the same epoch (same seed
    and epoch give the same rows) and takes batches rank, rank + world, ...;
    every rank gets the same number of batches, the missing ones being all
    padding (no supervised token), so ranks that step together never wait on
    one that ran out."""
    import numpy as np
    B, world, rank = int(B), int(world), int(rank)
    if not 0 <= rank < world:
        raise ValueError("need 0 <= rank < world")
    count = len(lengths)
    rows = max(-(-count // B), 1) * B
    r = pa_pack_first_fit(lengths, rows, N, seed, epoch, offsets, tokens, pad_token)
    keys = ("seg", "loss_mask", "row_tokens", "row_targets")
    fill = {"seg": 0, "loss_mask": 0, "row_tokens": pad_token, "row_targets": -1}
    n_batches = -(-r["rows_used"] // B)
    per_rank = -(-n_batches // world)
    for i in range(per_rank):
        b = rank + i * world
        if b < n_batches:
            sl = slice(b * B, (b + 1) * B)
            yield {k: (None if r[k] is None else r[k][sl]) for k in keys}
        else:
            yield {k: (None if r[k] is None else np.full((B, N), fill[k], dtype=r[k].dtype)) for k in keys}


def pa_lce_workspace_bytes(N, V, D) -> int:
    return int(lib().pa_lce_workspace_bytes(int(N), int(V), int(D)))


def pa_lce_fwd(hidden, head, targets, nll, lse, target_logit, ws, stream=None):
    """Fused linear cross-entropy forward (see include/pa.h): hidden (N, D)
    and head (V, D) bf16, targets (N) int32; writes nll, lse and
    target_logit, (N) fp32 each."""
    import torch
    N, D = hidden.shape
    V = head.shape[0]
    if head.shape[1] != D:
        raise ValueError("head must be (V, D) with the hidden states' D")
    f = torch.float32
    _check(lib().pa_lce_fwd(N, V, D, _ptr(hidden, torch.bfloat16, "hidden"), _ptr(head, torch.bfloat16, "head"),
                            _ptr(targets, torch.int32, "targets"), _ptr(nll, f, "nll"), _ptr(lse, f, "lse"),
                            _ptr(target_logit, f, "target_logit"), _ptr(ws, None, "ws"), ws.numel(),
                            _stream(stream)))


def linear_cross_entropy_forward(hidden, head, targets, ws=None):
    """Allocate the outputs (and a workspace) and run pa_lce_fwd; returns
    (nll, lse, target_logit)."""
    import torch
    N, D = hidden.shape
    out = [torch.empty(N, dtype=torch.float32, device=hidden.device) for _ in range(3)]
    if ws is None:
        n = pa_lce_workspace_bytes(N, head.shape[0], D)
        if n == 0:
            raise PAError(4, "invalid linear cross-entropy dims")
        ws = torch.empty(n, dtype=torch.uint8, device=hidden.device)
    pa_lce_fwd(hidden, head, targets, *out, ws)
    return tuple(out)


def pa_lce_bwd_workspace_bytes(N, V, D) -> int:
    return int(lib().pa_lce_bwd_workspace_bytes(int(N), int(V), int(D)))


def pa_lce_bwd(hidden, head, targets, lse, g, dhidden, dhead, ws, stream=None):
    """Fused linear cross-entropy backward (see include/pa.h): writes dhidden
    (N, D) bf16 and, unless dhead is None, dhead (V, D) bf16, for the loss
    sum_i g[i] nll[i] with the forward's lse."""
    import torch
    N, D = hidden.shape
    V = head.shape[0]
    if head.shape[1] != D or tuple(dhidden.shape) != (N, D) or (dhead is not None and tuple(dhead.shape) != (V, D)):
        raise ValueError("hidden/dhidden must be (N, D) and head/dhead (V, D)")
    f, bf = torch.float32, torch.bfloat16
    _check(lib().pa_lce_bwd(N, V, D, _ptr(hidden, bf, "hidden"), _ptr(head, bf, "head"),
                            _ptr(targets, torch.int32, "targets"), _ptr(lse, f, "lse"), _ptr(g, f, "g"),
                            _ptr(dhidden, bf, "dhidden"), _ptr(dhead, bf, "dhead"), _ptr(ws, None, "ws"),
                            ws.numel(), _stream(stream)))


def linear_cross_entropy_backward(hidden, head, targets, lse, g, train_head=True, ws=None):
    """Allocate the outputs (and a workspace) and run pa_lce_bwd; returns
    (dhidden, dhead), dhead None when the head does not train."""
    import torch
    N, D = hidden.shape
    dh = torch.empty_like(hidden)
    dw = torch.empty_like(head) if train_head else None
    if ws is None:
        n = pa_lce_bwd_workspace_bytes(N, head.shape[0], D)
        if n == 0:
            raise PAError(4, "invalid linear cross-entropy dims")
        ws = torch.empty(n, dtype=torch.uint8, device=hidden.device)
    pa_lce_bwd(hidden, head, targets, lse, g, dh, dw, ws)
    return dh, dw


# ------------------------------------------------- token log probabilities
def _on_current_device(*ts):
    """The tensors share one CUDA device and it is the current one (whose
    stream the call takes)."""
    import torch
    at = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != at:  # -1 for a CPU tensor
            raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at}), got one on {t.device}")


def _logp_dims(hidden, head, targets):
    hs, ws = hidden.shape, head.shape
    if len(hs) != 2 or len(ws) != 2 or hs[1] != ws[1]:
        raise ValueError("hidden must be (N, D) and head (V, D)")
    if targets.shape != hs[:1]:
        raise ValueError("targets must be (N,)")
    return hs[0], ws[0], hs[1]


def _logp_inputs(hidden, head, targets):
    """The three inputs' types, layout and device."""
    import torch
    if hidden.dtype != torch.bfloat16 or head.dtype != torch.bfloat16 or targets.dtype != torch.int32:
        raise ValueError(f"hidden and head must be bfloat16 and targets int32, got {hidden.dtype}, {head.dtype} and {targets.dtype}")
    at = torch.cuda.current_device()
    if not hidden.get_device() == head.get_device() == targets.get_device() == at:
        raise ValueError(f"hidden, head and targets must be on the current CUDA device (cuda:{at})")
    if not (hidden.is_contiguous() and head.is_contiguous() and targets.is_contiguous()):
        raise ValueError("hidden, head and targets must be contiguous")


def _want(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


@functools.lru_cache(maxsize=256)  # a function of the numbers alone
def pa_logp_workspace_bytes(N, V, D, top=0) -> int:
    return int(lib().pa_logp_workspace_bytes(int(N), int(V), int(D), int(top)))


def pa_logp_plan(N, V, D, sms=None):
    """How the forward cuts its work: (pairs of CTAs, splits, units of 32 rows
    per split, units per logit tile); sms defaults to the current device's."""
    import torch
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    plan = (ctypes.c_int32 * 4)()
    _check(lib().pa_logp_plan(int(N), int(V), int(D), int(sms), plan))
    return bool(plan[0]), plan[1], plan[2], plan[3]


def pa_logp_fwd(hidden, head, targets, logp, lse, entropy, top_ids, top_logp, ws, temperature=1.0, top=0, stream=None):
    """logp, lse and entropy (N,) fp32 and, with top > 0, top_ids (N, top)
    int32 and top_logp (N, top) fp32, all outputs (see include/pa.h)."""
    import torch
    N, V, D = _logp_dims(hidden, head, targets)
    f, i32 = torch.float32, torch.int32
    for t, n in ((logp, "logp"), (lse, "lse"), (entropy, "entropy")):
        _want(t, (N,), n)
    for t, n in ((top_ids, "top_ids"), (top_logp, "top_logp")):
        _want(t, (N, top), n)
    _logp_inputs(hidden, head, targets)
    _on_current_device(logp, lse, entropy, top_ids, top_logp, ws)
    _check(lib().pa_logp_fwd(N, V, D, float(temperature), int(top), hidden.data_ptr(), head.data_ptr(), targets.data_ptr(),
                             _ptr(logp, f, "logp"), _ptr(lse, f, "lse"), _ptr(entropy, f, "entropy"),
                             _ptr(top_ids, i32, "top_ids"), _ptr(top_logp, f, "top_logp"), _ptr(ws, torch.uint8, "ws"),
                             ws.numel(), _stream(stream)))


def token_logprobs_forward(hidden, head, targets, temperature=1.0, top=0, ws=None):
    """Log probabilities of `targets` under softmax(hidden head^T / temperature)
    with the entropy and the `top` most likely alternatives, without the
    logits. hidden (N, D) and head (V, D) bf16; targets (N,) int32, outside
    [0, V) = not scored (logp 0). Returns (logp, lse, entropy, top_ids,
    top_logp), the last two None when top is 0."""
    import torch
    N, V, D = _logp_dims(hidden, head, targets)
    dev, f, empty = hidden.device, torch.float32, torch.empty
    if ws is None:
        n = pa_logp_workspace_bytes(N, V, D, top)
        if n == 0:
            raise PAError(4, "invalid token log probability dims")
        ws = empty(n, dtype=torch.uint8, device=dev)
    logp, lse, entropy = empty(N, dtype=f, device=dev), empty(N, dtype=f, device=dev), empty(N, dtype=f, device=dev)
    ids, alt = (empty((N, top), dtype=torch.int32, device=dev), empty((N, top), dtype=f, device=dev)) if top else (None, None)
    _logp_inputs(hidden, head, targets)
    _on_current_device(ws)
    _check(lib().pa_logp_fwd(N, V, D, float(temperature), top, hidden.data_ptr(), head.data_ptr(), targets.data_ptr(),
                             logp.data_ptr(), lse.data_ptr(), entropy.data_ptr(), ids.data_ptr() if top else None,
                             alt.data_ptr() if top else None, _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(None)))
    return logp, lse, entropy, ids, alt


@functools.lru_cache(maxsize=256)  # a function of the numbers alone
def pa_logp_bwd_workspace_bytes(N, V, D) -> int:
    return int(lib().pa_logp_bwd_workspace_bytes(int(N), int(V), int(D)))


def pa_logp_bwd(hidden, head, targets, lse, entropy, g_logp, g_entropy, dhidden, dhead, ws, temperature=1.0, stream=None):
    """dhidden (N, D) and dhead (V, D) bf16 are outputs (dhead None when the
    head does not train); g_logp and g_entropy (N,) fp32 = dL/dlogp and
    dL/dentropy per token, g_entropy None for no entropy term."""
    import torch
    N, V, D = _logp_dims(hidden, head, targets)
    f, bf = torch.float32, torch.bfloat16
    for t, n in ((lse, "lse"), (entropy, "entropy"), (g_logp, "g_logp"), (g_entropy, "g_entropy")):
        _want(t, (N,), n)
    _want(dhidden, (N, D), "dhidden")
    _want(dhead, (V, D), "dhead")
    _logp_inputs(hidden, head, targets)
    _on_current_device(lse, entropy, g_logp, g_entropy, dhidden, dhead, ws)
    _check(lib().pa_logp_bwd(N, V, D, float(temperature), hidden.data_ptr(), head.data_ptr(), targets.data_ptr(),
                             _ptr(lse, f, "lse"), _ptr(entropy, f, "entropy"),
                             _ptr(g_logp, f, "g_logp"), _ptr(g_entropy, f, "g_entropy"), _ptr(dhidden, bf, "dhidden"),
                             _ptr(dhead, bf, "dhead"), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def token_logprobs_backward(hidden, head, targets, lse, entropy, g_logp, g_entropy=None, temperature=1.0,
                            train_head=True, ws=None):
    """Gradients of sum(g_logp * logp + g_entropy * entropy) into hidden and
    head: (dhidden, dhead), dhead None when the head does not train. hidden
    may be a Checkpoint (of a (N, D) tensor): its values are brought back for
    the call. The gradients are bf16, about 1.7e-3 of their norm off for up to
    128 tokens and 2.4e-3 for more (see include/pa.h)."""
    import torch
    if isinstance(hidden, Checkpoint):
        hidden = checkpoint_load([hidden])[0]
    if ws is None:
        n = pa_logp_bwd_workspace_bytes(*_logp_dims(hidden, head, targets))
        if n == 0:
            raise PAError(4, "invalid token log probability dims")
        ws = torch.empty(n, dtype=torch.uint8, device=hidden.device)
    dh = torch.empty_like(hidden)
    dw = torch.empty_like(head) if train_head else None
    pa_logp_bwd(hidden, head, targets, lse, entropy, g_logp, g_entropy, dh, dw, ws, temperature)
    return dh, dw


# ------------------------------------------------------- 8-bit checkpoints
class Checkpoint:
    """A tensor kept in 8 bits: codes (int8 or float8_e4m3fn, the tensor's
    shape, contiguous) and fp32 scales, one per block of the last dim; dtype
    is what loading gives back."""
    __slots__ = ("codes", "scales", "block", "dtype")

    def __init__(self, codes, scales, block=64, dtype=None):
        import torch
        if block not in (32, 64, 128):
            raise ValueError(f"block must be 32, 64 or 128, got {block}")
        if codes.dtype != torch.int8:
            _ckpt_format(codes.dtype)
        shape, blocks = codes.shape, scales.shape
        if len(shape) != len(blocks) or shape[:-1] != blocks[:-1] or blocks[-1] != -(-shape[-1] // block):
            raise ValueError(f"scales must be {(*shape[:-1], -(-shape[-1] // block))}, got {tuple(blocks)}")
        self.codes, self.scales, self.block, self.dtype = codes, scales, block, torch.bfloat16 if dtype is None else dtype

    @property
    def shape(self):
        return self.codes.shape

    @property
    def nbytes(self):
        return self.codes.numel() + 4 * self.scales.numel()


def _ckpt_format(dtype):
    import torch
    if dtype == torch.int8:
        return PA_CKPT_INT8
    if dtype == torch.float8_e4m3fn:
        return PA_CKPT_E4M3
    raise ValueError(f"codes must be int8 or float8_e4m3fn, got {dtype}")


_CKPT_FIELDS = struct.Struct("PPPiiiiqqq")  # pa_ckpt_tensor
_ONES, _ZEROS = ((), (1,), (1, 1), (1, 1, 1)), ((), (0,), (0, 0), (0, 0, 0))


def _ckpt_of(x, codes, scales, at):
    """The bytes of the C description of tensor x (1 to 4 dims, the last
    contiguous) with codes and scales (contiguous) on device `at`."""
    shape, stride = x.shape, x.stride()
    pad = 4 - len(shape)
    if not 0 <= pad <= 3 or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError("a checkpointed tensor has 1 to 4 dims, the last contiguous")
    if not x.get_device() == codes.get_device() == scales.get_device() == at:
        raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
    try:
        return _CKPT_FIELDS.pack(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), *_ONES[pad], *shape, *_ZEROS[pad],
                                 *stride[:-1])
    except struct.error:
        raise PAError(4, f"a dimension of {tuple(shape)} is past 2^31 - 1") from None


def _ckpt_call(fn, parts, io, fmt, block, stream):
    st = _stream(stream)
    for i in range(0, len(parts), PA_CKPT_MAX_TENSORS):
        some = parts[i:i + PA_CKPT_MAX_TENSORS]
        _check(fn(len(some), b"".join(some), io, fmt, block, st))


def _ckpt_lists(fn, xs, cs, stream):
    """pa_ckpt_save or pa_ckpt_load of matching lists, PA_CKPT_MAX_TENSORS a launch."""
    import torch
    if len(xs) != len(cs):
        raise ValueError("one checkpoint per tensor")
    if not xs:
        return
    dtype, kind, block, f32 = xs[0].dtype, cs[0].codes.dtype, cs[0].block, torch.float32
    io, fmt, at, parts = _io_dtype(xs[0])[1], _ckpt_format(kind), torch.cuda.current_device(), []
    for x, c in zip(xs, cs):
        codes, scales = c.codes, c.scales
        if x.dtype != dtype or codes.dtype != kind or c.block != block:
            raise ValueError("the tensors of one call share their type, format and block")
        if codes.shape != x.shape:
            raise ValueError(f"codes must be {tuple(x.shape)}, got {tuple(codes.shape)}")
        if not (codes.is_contiguous() and scales.is_contiguous()) or scales.dtype != f32:
            raise ValueError("codes and scales must be contiguous, scales float32")
        parts.append(_ckpt_of(x, codes, scales, at))
    _ckpt_call(fn, parts, io, fmt, block, stream)


def pa_ckpt_save(tensors, checkpoints, stream=None):
    """Fill the checkpoints' codes and scales (see include/pa.h)."""
    _ckpt_lists(lib().pa_ckpt_save, tensors, checkpoints, stream)


def pa_ckpt_load(tensors, checkpoints, stream=None):
    """Fill the tensors from the checkpoints (see include/pa.h)."""
    _ckpt_lists(lib().pa_ckpt_load, tensors, checkpoints, stream)


def checkpoint_save(tensors, format="int8", block=64):
    """Keep activations in 8 bits: a list of Checkpoints of the given tensors
    (bf16 or fp32, all alike; 1 to 4 dims, the last contiguous and a multiple
    of 8). format "int8" or "e4m3"; one scale per `block` elements of the
    last dim (32, 64 or 128). One launch for up to eight tensors."""
    import torch
    if format not in ("int8", "e4m3"):
        raise ValueError(f"format must be int8 or e4m3, got {format!r}")
    if block not in (32, 64, 128):
        raise ValueError(f"block must be 32, 64 or 128, got {block}")
    tensors = list(tensors)
    if not tensors:
        return []
    kept, parts, empty, f32, new = [], [], torch.empty, torch.float32, object.__new__
    kind, fmt = (torch.int8, PA_CKPT_INT8) if format == "int8" else (torch.float8_e4m3fn, PA_CKPT_E4M3)
    (dtype, io), at = _io_dtype(tensors[0]), torch.cuda.current_device()
    for x in tensors:
        if x.dtype != dtype:
            raise ValueError("the tensors of one call share their type")
        shape, dev, c = x.shape, x.device, new(Checkpoint)
        if not shape:
            raise ValueError("a checkpointed tensor has 1 to 4 dims, the last contiguous")
        c.codes = codes = empty(shape, dtype=kind, device=dev)
        c.scales = scales = empty((*shape[:-1], -(-shape[-1] // block)), dtype=f32, device=dev)
        c.block, c.dtype = block, dtype
        kept.append(c)
        parts.append(_ckpt_of(x, codes, scales, at))
    _ckpt_call(lib().pa_ckpt_save, parts, io, fmt, block, None)
    return kept


def checkpoint_load(checkpoints, out=None):
    """The checkpoints' values as contiguous tensors of their dtypes, or into
    the tensors `out` (any strides with the last dim contiguous)."""
    import torch
    checkpoints, empty = list(checkpoints), torch.empty
    out = [empty(c.codes.shape, dtype=c.dtype, device=c.codes.device) for c in checkpoints] if out is None else list(out)
    pa_ckpt_load(out, checkpoints)
    return out


@functools.lru_cache(maxsize=256)  # a function of the numbers alone
def pa_bwd_ckpt_workspace_bytes(B, Hq, Hkv, N, D) -> int:
    d = make_dims(B, Hq, Hkv, N, D)
    return int(lib().pa_bwd_ckpt_workspace_bytes(ctypes.byref(d)))


def pa_bwd_ckpt(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale=0.0, stream=None):
    """pa_bwd from Checkpoints of q, k, v and out (one format and block).
    dout and dq share their strides, dk and dv theirs; seg None = plain
    causal."""
    import torch
    bf, f, kind, block, at = torch.bfloat16, torch.float32, q.codes.dtype, q.block, torch.cuda.current_device()
    qs, ks = q.codes.shape, k.codes.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q and k must be checkpoints of (B, H, N, D) tensors")
    B, Hq, N, D = qs
    Hkv = ks[1]
    kept = []
    for c, want, n in ((q, qs, "q"), (k, (B, Hkv, N, D), "k"), (v, ks, "v"), (out, qs, "out")):
        codes, scales = c.codes, c.scales
        if codes.shape != want:
            raise ValueError(f"{n} must be {tuple(want)}, got {tuple(codes.shape)}")
        if codes.dtype != kind or c.block != block or c.dtype != bf or scales.dtype != f:
            raise ValueError("q, k, v and out must be bf16 checkpoints in one format and block")
        if not codes.get_device() == scales.get_device() == at or not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError(f"{n} must be contiguous and on the current CUDA device (cuda:{at})")
        kept.append(ctypes.byref(pa_ckpt(codes.data_ptr(), scales.data_ptr())))
    plain = True
    for t, want, n in ((dout, qs, "dout"), (dq, qs, "dq"), (dk, ks, "dk"), (dv, ks, "dv")):
        if t.shape != want or t.dtype != bf or t.get_device() != at or t.stride(3) != 1:
            raise ValueError(f"{n} must be {tuple(want)} {bf} with a contiguous last dim on the current CUDA device (cuda:{at})")
        plain = plain and t.is_contiguous()
    if lse.shape != (B, Hq, N) or (seg is not None and seg.shape != (B, N)):
        raise ValueError(f"lse must be {(B, Hq, N)} and seg {(B, N)}")
    _on_current_device(lse, seg, ws)
    st = None
    if not plain:
        if dq.stride() != dout.stride() or dk.stride() != dv.stride():
            raise ValueError("dq must have dout's strides and dv dk's")
        st = ctypes.byref(_strides_of(dout, dk))
    _check(lib().pa_bwd_ckpt(ctypes.byref(pa_dims(B, Hq, Hkv, N, D, scale)), st, _ckpt_format(kind), block, *kept,
                             dout.data_ptr(), _ptr(lse, f, "lse"), _ptr(seg, torch.int32, "seg"), dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def backward_from_checkpoint(q, k, v, out, dout, lse, seg=None, scale=0.0, ws=None):
    """The attention backward from 8-bit Checkpoints of q, k, v and out:
    (dq, dk, dv) in bf16. They take dout's memory order: contiguous, or
    (B, N, H, D) memory for a dout that is a view of such."""
    import torch
    if q.codes.dim() != 4 or k.codes.dim() != 4:
        raise ValueError("q and k must be checkpoints of (B, H, N, D) tensors")
    B, Hq, N, D = q.codes.shape
    Hkv = k.codes.shape[1]
    if ws is None:
        n = pa_bwd_ckpt_workspace_bytes(B, Hq, Hkv, N, D)
        if n == 0:
            raise PAError(4, "invalid dims")
        ws = torch.empty(n, dtype=torch.uint8, device=dout.device)
    if dout.is_contiguous():
        dq, shape, stride = torch.empty_like(dout), (B, Hkv, N, D), (Hkv * N * D, N * D, D, 1)
    else:
        dq = torch.empty_strided(dout.shape, dout.stride(), dtype=dout.dtype, device=dout.device)
        shape, stride = (B, Hkv, N, D), (N * Hkv * D, D, Hkv * D, 1)
    dk, dv = (torch.empty_strided(shape, stride, dtype=dout.dtype, device=dout.device) for _ in range(2))
    pa_bwd_ckpt(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale)
    return dq, dk, dv


def pa_status_string(code: int) -> str:
    return lib().pa_status_string(code).decode()


# ---------------------------------------------------------------- conveniences
def _all_contiguous(*ts):
    return all(t.is_contiguous() for t in ts)


def forward(q, k, v, seg=None, scale=0.0, ws=None):
    """Allocate out/lse and run pa_fwd (seg given) or pa_fwd_causal (seg None);
    strided q/k/v go through pa_fwd_strided (out then takes q's strides)."""
    import torch
    B, Hq, N, D = q.shape
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if not _all_contiguous(q, k, v) or q.dtype == torch.float32:
        out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
        ws = workspace(q, k, strided=True) if ws is None else ws
        pa_fwd_strided(q, k, v, seg, out, lse, ws, scale)
        return out, lse
    out = torch.empty_like(q)
    ws = workspace(q, k) if ws is None else ws
    if seg is None:
        pa_fwd_causal(q, k, v, out, lse, ws, scale)
    else:
        pa_fwd(q, k, v, seg, out, lse, ws, scale)
    return out, lse


def backward(q, k, v, out, dout, lse, seg=None, scale=0.0, ws=None):
    """Allocate dq/dk/dv and run pa_bwd (seg given) or pa_bwd_causal (seg None);
    strided tensors go through pa_bwd_strided (dq takes q's strides, dk/dv k's)."""
    import torch
    if not _all_contiguous(q, k, v, out, dout) or q.dtype == torch.float32:
        dq = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
        dk = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
        dv = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
        ws = workspace(q, k, strided=True) if ws is None else ws
        pa_bwd_strided(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale)
        return dq, dk, dv
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = workspace(q, k) if ws is None else ws
    if seg is None:
        pa_bwd_causal(q, k, v, out, dout, lse, dq, dk, dv, ws, scale)
    else:
        pa_bwd(q, k, v, out, dout, lse, seg, dq, dk, dv, ws, scale)
    return dq, dk, dv
