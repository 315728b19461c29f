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
PA_ROPE_HALF, PA_ROPE_INTERLEAVED = 0, 1
PA_ROPE_MAX_TENSORS, PA_ROPE_MAX_PAIRS = 4, 64
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}
EXPORTS = ["pa_workspace_bytes", "pa_fwd", "pa_bwd", "pa_fwd_causal", "pa_bwd_causal", "pa_build_tile_table",
           "pa_fwd_tiles", "pa_bwd_delta", "pa_bwd_dq", "pa_bwd_dkv", "pa_bwd_noalloc", "pa_device_status",
           "pa_selftest_wait_timeout", "pa_selftest_exp2_fma", "pa_pack_first_fit", "pa_workspace_bytes_strided", "pa_fwd_strided",
           "pa_bwd_strided", "pa_lce_workspace_bytes", "pa_lce_fwd", "pa_lce_bwd_workspace_bytes", "pa_lce_bwd",
           "pa_bwd_fused_workspace_bytes", "pa_bwd_fused", "pa_logp_workspace_bytes", "pa_logp_plan", "pa_logp_fwd",
           "pa_logp_bwd_workspace_bytes", "pa_logp_bwd", "pa_ckpt_save", "pa_ckpt_load", "pa_bwd_ckpt_workspace_bytes",
           "pa_bwd_ckpt", "pa_rotary_frequencies", "pa_rotary_init", "pa_positions", "pa_rope", "pa_paged_append",
           "pa_paged_workspace_bytes", "pa_paged_fwd", "pa_selftest_paged_units", "pa_status_string"]


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


class pa_rotary(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("ready", ctypes.c_int32), ("turns", ctypes.c_uint64 * PA_ROPE_MAX_PAIRS)]


class pa_rope_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("x_b", ctypes.c_int64), ("x_h", ctypes.c_int64), ("x_n", ctypes.c_int64),
                ("y_b", ctypes.c_int64), ("y_h", ctypes.c_int64), ("y_n", ctypes.c_int64)]


class pa_paged_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "T", "Hq", "Hkv", "D", "pages", "page", "width")] + [("scale", ctypes.c_float)]


class pa_paged_strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("q_t", "q_h", "n_t", "n_h", "o_t", "o_h", "p_p", "p_h", "p_n")]


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
            DB = ctypes.c_double
            L.pa_rotary_frequencies.argtypes = [I32, I32, DB, DB, DB, DB, DB, P]
            L.pa_rotary_frequencies.restype = ctypes.c_int
            L.pa_rotary_init.argtypes = [P, I32, I32, P, DB]
            L.pa_rotary_init.restype = ctypes.c_int
            L.pa_positions.argtypes = [I32, I32, P, P, P]
            L.pa_positions.restype = ctypes.c_int
            L.pa_rope.argtypes = [P, I32, P, I32, I32, I32, I32, P, I32, P]  # an array of pa_rope_tensor, or its bytes
            L.pa_rope.restype = ctypes.c_int
            # pa_paged_dims and pa_paged_strides, or their bytes
            L.pa_paged_append.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, P]
            L.pa_paged_append.restype = ctypes.c_int
            L.pa_paged_workspace_bytes.argtypes = [I32]
            L.pa_paged_workspace_bytes.restype = S
            L.pa_paged_fwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, S, P]
            L.pa_paged_fwd.restype = ctypes.c_int
            L.pa_selftest_paged_units.argtypes = [P, P, P, P]
            L.pa_selftest_paged_units.restype = ctypes.c_int
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


# -------------------------------------------------------- rotary positions
class Rotary:
    """Rotary positions on the first `rot` elements of a head, in pairs of
    halves or of neighbours (interleaved): frequencies theta^(-2i / rot) with
    `scaling` "plain", "linear", "base" or "bands" by `factor` (see
    include/pa.h; "bands" takes original, low and high and is linear in a pair's
    turns: a model whose ramp is linear in the pair's index gives its `frequencies`), or the given
    `frequencies` (rot / 2 radians a position). `amplitude` multiplies cosine and
    sine. Holds no device memory."""
    __slots__ = ("c", "ref", "rot", "interleaved", "amplitude", "frequencies")

    def __init__(self, rot, theta=10000.0, interleaved=False, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0,
                 amplitude=1.0, frequencies=None):
        rot = int(rot)
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        if frequencies is None:
            f = (ctypes.c_double * PA_ROPE_MAX_PAIRS)()
            _check(lib().pa_rotary_frequencies(rot, ROPE_SCALINGS[scaling], float(theta), float(factor), float(original),
                                               float(low), float(high), f))
        else:
            if scaling != "plain":
                raise ValueError("frequencies come as they are used: no scaling beside them")
            given = [float(x) for x in frequencies]
            if len(given) != rot // 2 or len(given) > PA_ROPE_MAX_PAIRS:
                raise ValueError(f"frequencies must be rot / 2 = {rot // 2} numbers (at most {PA_ROPE_MAX_PAIRS}), got {len(given)}")
            f = (ctypes.c_double * PA_ROPE_MAX_PAIRS)(*given)
        self.c = pa_rotary()
        self.ref = ctypes.byref(self.c)
        _check(lib().pa_rotary_init(self.ref, rot, int(bool(interleaved)), f, float(amplitude)))
        self.rot, self.interleaved, self.amplitude = rot, bool(interleaved), float(amplitude)
        self.frequencies = tuple(f[:rot // 2])

    def __reduce__(self):  # copies and pickles are made again from what it was made of: `ref` is an address
        return _rotary_of, (self.rot, self.interleaved, self.amplitude, self.frequencies)


def _rotary_of(rot, interleaved, amplitude, frequencies):
    return Rotary(rot, interleaved=interleaved, amplitude=amplitude, frequencies=frequencies)


def pa_positions(seg, positions, stream=None):
    """positions[b, n] = n minus the start of its run of equal ids; both (B, N) int32."""
    import torch
    shape, i32, at = seg.shape, torch.int32, torch.cuda.current_device()
    if len(shape) != 2:
        raise ValueError("seg must be (B, N)")
    if positions.shape != shape:
        raise ValueError(f"positions must be {tuple(shape)}, got {tuple(positions.shape)}")
    if seg.dtype != i32 or positions.dtype != i32:
        raise ValueError(f"seg and positions must be int32, got {seg.dtype} and {positions.dtype}")
    if not seg.get_device() == positions.get_device() == at:
        raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
    if not (seg.is_contiguous() and positions.is_contiguous()):
        raise ValueError("seg and positions must be contiguous")
    _check(lib().pa_positions(shape[0], shape[1], seg.data_ptr(), positions.data_ptr(), _stream(stream)))


def segment_positions(seg):
    """Positions of packed rows from their segment ids, counting from 0 in each
    segment: (B, N) int32."""
    import torch
    positions = torch.empty(seg.shape, dtype=torch.int32, device=seg.device)
    pa_positions(seg, positions)
    return positions


_ROPE_FIELDS = struct.Struct("PPi4xqqqqqq")  # pa_rope_tensor


def _rope_refusals(parts, B, N, D, unit):
    """What pa_rope refuses of single tensors, for all of them before the first launch
    (a list of several launches is turned whole or not at all)."""
    for p in parts:
        x, y, H, *s = _ROPE_FIELDS.unpack(p)
        used = [i for i, n in enumerate((B, H, N)) if n > 1]
        if not 0 < H <= 65535 or any(s[i] < D or s[i + 3] < D for i in used):
            raise PAError(4, pa_status_string(4))
        if any(s[i] % unit or s[i + 3] % unit for i in used) or x % 16 or y % 16:
            raise PAError(5, pa_status_string(5))
        if x == y and any(s[i] != s[i + 3] for i in used):
            raise PAError(4, pa_status_string(4))


def pa_rope(tensors, out, rotary, positions=None, backward=False, stream=None):
    """Rotate the (B, H, N, D) tensors into `out` (which may be the tensors
    themselves; None: new tensors in the same memory order), or take their
    gradients back; see include/pa.h. Returns the outputs."""
    import torch
    tensors = list(tensors)
    made = out is None
    out = [torch.empty_like(x) for x in tensors] if made else list(out)
    if len(tensors) != len(out):
        raise ValueError("one output per tensor")
    if not tensors:
        return out
    parts, at, pack = [], torch.cuda.current_device(), _ROPE_FIELDS.pack
    dtype, io = _io_dtype(tensors[0])
    first = None
    for x, y in zip(tensors, out):
        shape = x.shape
        if len(shape) != 4:
            raise ValueError("tensors must be (B, H, N, D)")
        B, H, N, D = shape
        if first is None:
            first = (B, N, D)
        elif first != (B, N, D):
            raise ValueError("the tensors of one call are (B, H, N, D) with one B, N and D")
        if x.dtype != dtype:
            raise ValueError("the tensors of one call share their type")
        if x.get_device() != at:
            raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
        x_b, x_h, x_n, x_c = x.stride()
        y_b, y_h, y_n, y_c = y.stride()
        if not made:
            if y.shape != shape or y.dtype != dtype:
                raise ValueError("out must have the tensors' shapes and type")
            if y.get_device() != at:
                raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
        if (x_c != 1 or y_c != 1) and D > 1:
            raise ValueError("the tensors' last dim must be contiguous")
        parts.append(pack(x.data_ptr(), y.data_ptr(), H, x_b, x_h, x_n, y_b, y_h, y_n))
    B, N, D = first
    pos = None
    if positions is not None:
        if positions.shape != (B, N) or positions.dtype != torch.int32:
            raise ValueError(f"positions must be {(B, N)} int32, got {tuple(positions.shape)} {positions.dtype}")
        if positions.get_device() != at:
            raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at}), got positions on {positions.device}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        pos = positions.data_ptr()
    st, fn = _stream(stream), lib().pa_rope
    if len(parts) > PA_ROPE_MAX_TENSORS:
        _rope_refusals(parts, B, N, D, 16 // tensors[0].element_size())
    for i in range(0, len(parts), PA_ROPE_MAX_TENSORS):
        some = parts[i:i + PA_ROPE_MAX_TENSORS]
        _check(fn(rotary.ref, len(some), b"".join(some), B, N, D, io, pos, 1 if backward else 0, st))
    return out


def rotary_forward(tensors, rotary, positions=None, out=None):
    """The (B, H, N, D) tensors (q and k, say; bf16 or fp32, any strides with
    the last dim contiguous) rotated to their positions ((B, N) int32, or None
    for 0, 1, ...), as new tensors in the same memory order or into `out`."""
    return pa_rope(tensors, out, rotary, positions)


def rotary_backward(grads, rotary, positions=None, out=None):
    """Gradients of rotary_forward's inputs from those of its outputs."""
    return pa_rope(grads, out, rotary, positions, backward=True)


# -------------------------------------------------------------- paged cache
class PagedCache:
    """Pages of keys and values: two (pages, Hkv, page, D) bf16 tensors on one
    device with the same strides, the last dim contiguous; (pages, page, Hkv, D)
    memory comes as its transpose(1, 2). Holds the tensors."""
    __slots__ = ("k", "v", "pages", "Hkv", "page", "D", "strides", "device_index")

    def __init__(self, k_pages, v_pages):
        import torch
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must be (pages, Hkv, page, D)")
        if k_pages.dtype != torch.bfloat16 or v_pages.dtype != torch.bfloat16:
            raise ValueError(f"k_pages and v_pages must be bfloat16, got {k_pages.dtype} and {v_pages.dtype}")
        if k_pages.stride() != v_pages.stride() or k_pages.stride(3) != 1:
            raise ValueError("k_pages and v_pages must share their strides, the last dim contiguous")
        if k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must be on one device")
        self.k, self.v, self.device_index = k_pages, v_pages, k_pages.get_device()
        self.pages, self.Hkv, self.page, self.D = k_pages.shape
        self.strides = k_pages.stride()[:3]


def _rows_of(t, H, D, at, name):
    """A (T, H, D) bf16 tensor on device `at`, its last dim contiguous (H None: any): its sizes and strides."""
    import torch
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (H is not None and shape[1] != H):
        raise ValueError(f"{name} must be (T, {'H' if H is None else H}, {D}), got {tuple(shape)}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.get_device() != at:
        raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at}), got {name} on {t.device}")
    s_t, s_h, s_c = t.stride()
    if s_c != 1:
        raise ValueError(f"{name}'s last dim must be contiguous")
    return shape[0], shape[1], s_t, s_h


def _paged_tables(cache, page_table, q_start, kv_len, at):
    """S and width, the step's three arrays checked."""
    import torch
    i32, shape = torch.int32, page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be (S, width)")
    S, width = shape
    if q_start.shape != (S + 1,) or kv_len.shape != (S,):
        raise ValueError(f"q_start must be {(S + 1,)} and kv_len {(S,)}, got {tuple(q_start.shape)} and {tuple(kv_len.shape)}")
    if not page_table.dtype == q_start.dtype == kv_len.dtype == i32:
        raise ValueError("page_table, q_start and kv_len must be int32")
    if not page_table.get_device() == q_start.get_device() == kv_len.get_device() == cache.device_index == at:
        raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
    if not (page_table.is_contiguous() and q_start.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError("page_table, q_start and kv_len must be contiguous")
    return S, width


_PAGED_DIMS, _PAGED_STRIDES = struct.Struct("8if"), struct.Struct("9q")  # pa_paged_dims, pa_paged_strides


def pa_paged_append(cache, q, k, v, page_table, q_start, kv_len, rotary=None, positions=None, q_out=None, stream=None):
    """New tokens' keys and values into the cache, their queries rotated into
    q_out (see include/pa.h); q and q_out may both be None."""
    import torch
    at, Hkv, D = torch.cuda.current_device(), cache.Hkv, cache.D
    S, width = _paged_tables(cache, page_table, q_start, kv_len, at)
    T, _, n_t, n_h = _rows_of(k, Hkv, D, at, "k")
    if _rows_of(v, Hkv, D, at, "v") != (T, Hkv, n_t, n_h):  # strides of dimensions of one are never used
        Tv, _, m_t, m_h = _rows_of(v, Hkv, D, at, "v")
        if Tv != T or (T > 1 and m_t != n_t) or (Hkv > 1 and m_h != n_h):
            raise ValueError("v must have k's shape and strides")
    Hq, q_t, q_h, o_t, o_h, q_ptr, o_ptr = Hkv, D * Hkv, D, D * Hkv, D, None, None
    if q is not None and q_out is not None:
        Tq, Hq, q_t, q_h = _rows_of(q, None, D, at, "q")
        To, _, o_t, o_h = _rows_of(q_out, Hq, D, at, "q_out")
        if Tq != T or To != T:
            raise ValueError(f"q and q_out must have k's {T} rows")
        q_ptr, o_ptr = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out come together")
    pos = None
    if positions is not None:
        _want(positions, (T,), "positions")
        _on_current_device(positions)
        pos = _ptr(positions, torch.int32, "positions")
    _check(lib().pa_paged_append(_PAGED_DIMS.pack(S, T, Hq, Hkv, D, cache.pages, cache.page, width, 0.0),
                                 _PAGED_STRIDES.pack(q_t, q_h, n_t, n_h, o_t, o_h, *cache.strides),
                                 None if rotary is None else rotary.ref, q_ptr, k.data_ptr(), v.data_ptr(),
                                 page_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), pos, o_ptr,
                                 cache.k.data_ptr(), cache.v.data_ptr(), _stream(stream)))


def paged_append(cache, q, k, v, page_table, q_start, kv_len, rotary=None, positions=None, q_out=None):
    """Write a step's new keys (T, Hkv, D), rotated, and values into their places
    in the cache and return the queries (T, Hq, D) rotated to their positions (in
    q_out, which may be q, or a new tensor whose rows behind the last sequence are
    not set; None for q None). Sequence s's new tokens are rows q_start[s] to
    q_start[s + 1] - 1, the last of its kv_len[s] tokens; page_table (S, width)
    lists its pages. All int32 on the device."""
    import torch
    if q is not None and q_out is None:
        q_out = torch.empty_like(q)
    pa_paged_append(cache, q, k, v, page_table, q_start, kv_len, rotary, positions, q_out)
    return q_out


@functools.lru_cache(maxsize=16)  # a function of the number alone
def pa_paged_workspace_bytes(D) -> int:
    return int(lib().pa_paged_workspace_bytes(int(D)))


def _paged_workspace(q, cache):
    import torch
    n = pa_paged_workspace_bytes(cache.D)
    if n == 0:
        raise PAError(2, "head dim must be 64, 96 or 128")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def paged_workspace(q, cache):
    """A device workspace for paged_forward on q and cache (uint8; any lengths), its
    status word clear: a step without rows, which launches nothing, leaves it so."""
    ws = _paged_workspace(q, cache)
    ws[:4].zero_()
    return ws


def pa_paged_fwd(q, cache, page_table, q_start, kv_len, out, lse, ws, scale=0.0, stream=None):
    """Attention of a step's queries over the cache (see include/pa.h): out (T, Hq,
    D) bf16 and lse (T, Hq) fp32 are outputs."""
    import torch
    at, D = torch.cuda.current_device(), cache.D
    S, width = _paged_tables(cache, page_table, q_start, kv_len, at)
    T, Hq, q_t, q_h = _rows_of(q, None, D, at, "q")
    To, _, o_t, o_h = _rows_of(out, Hq, D, at, "out")
    if To != T or lse.shape != (T, Hq):
        raise ValueError(f"out must have q's shape and lse be {(T, Hq)}, got {tuple(out.shape)} and {tuple(lse.shape)}")
    if lse.dtype != torch.float32 or ws.dtype != torch.uint8:
        raise ValueError(f"lse must be float32 and ws uint8, got {lse.dtype} and {ws.dtype}")
    if not (lse.is_contiguous() and ws.is_contiguous()):
        raise ValueError("lse and ws must be contiguous")
    if not lse.get_device() == ws.get_device() == at:
        raise ValueError(f"every tensor must be on the current CUDA device (cuda:{at})")
    _check(lib().pa_paged_fwd(_PAGED_DIMS.pack(S, T, Hq, cache.Hkv, D, cache.pages, cache.page, width, scale),
                              _PAGED_STRIDES.pack(q_t, q_h, 0, 0, o_t, o_h, *cache.strides), q.data_ptr(),
                              cache.k.data_ptr(), cache.v.data_ptr(), page_table.data_ptr(), q_start.data_ptr(),
                              kv_len.data_ptr(), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))


def paged_forward(q, cache, page_table, q_start, kv_len, scale=0.0, out=None, lse=None, ws=None):
    """Attention of a step's new tokens over the paged cache, their own keys and
    values among it (paged_append). q (T, Hq, D) bf16, rows as in paged_append;
    returns (out, lse), lse (T, Hq) fp32. Rows of no sequence are left as they
    are (not set, in new outputs). ws is a paged_workspace, which a program keeps: it
    spares the allocation, and pa_device_status(ws), which waits for the stream, tells
    whether the call came through (without one, its status goes with its memory)."""
    import torch
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if ws is None:
        ws = _paged_workspace(q, cache)
    pa_paged_fwd(q, cache, page_table, q_start, kv_len, out, lse, ws, scale)
    return out, lse


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
