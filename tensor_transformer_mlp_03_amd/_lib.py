"""ctypes binding of libtpmlp (include/tpmlp.h).

Argument marshalling only: every step of the MLP runs in the library's HIP
kernels.  Functions keep the C names; tensors are torch tensors on the GPU
(bf16 data as ``torch.bfloat16`` or ``torch.uint16``/``torch.int16`` bits,
float32 outputs as ``torch.float32``); sizes come from the tensors' shapes.
A status other than TPMLP_OK raises :class:`TpmlpError`.

If the shared library has not been built, loading fails loudly; there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtpmlp.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "tpmlp.h")

STATUS = {
    0: "TPMLP_OK", 1: "TPMLP_ERR_NULL", 2: "TPMLP_ERR_SHAPE", 3: "TPMLP_ERR_ALIGN",
    4: "TPMLP_ERR_WORKSPACE", 5: "TPMLP_ERR_SHARDS", 6: "TPMLP_ERR_HIP",
    7: "TPMLP_ERR_UNSUPPORTED", 8: "TPMLP_ERR_ALIAS", 9: "TPMLP_ERR_NO_FORWARD",
}
KERNEL_COUNT = 13
MAX_SHARDS = 64


class TpmlpError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__(f"{func}: {STATUS.get(status, status)} ({detail})")


_lib = None

_vp, _sz, _i64, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
_PP = ctypes.POINTER(ctypes.c_void_p)


class EdgeDesc(ctypes.Structure):
    """tpmlp_edge: the description of the edge between two blocks."""
    _fields_ = [("M", _i64), ("H", _i64), ("post", ctypes.c_int32), ("pre", ctypes.c_int32),
                ("y_type", ctypes.c_int32), ("r_type", ctypes.c_int32), ("param_type", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("eps", ctypes.c_float), ("w_post", _vp), ("b_post", _vp),
                ("w_pre", _vp), ("b_pre", _vp), ("gate", _vp), ("gate_rows", _i64), ("ld_gate", _i64)]
    gate_tokens = None  # how many tokens the gate's rows are enough for, where it is known


_EP = ctypes.POINTER(EdgeDesc)
_SIGS = {
    "tpmlp_abi_version": ([], _int),
    "tpmlp_status_str": ([_int], ctypes.c_char_p),
    "tpmlp_last_error": ([], ctypes.c_char_p),
    "tpmlp_kernel_name": ([_int], ctypes.c_char_p),
    "tpmlp_fwd_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "tpmlp_bwd_workspace_bytes": ([_i64, _i64, _i64, _int], _sz),
    "tpmlp_tp_workspace_bytes": ([_int, _i64, _i64, _i64], _sz),
    "tpmlp_saved_activation_bytes": ([_i64, _i64, _i64, _int], _sz),
    "tpmlp_recompute_policy": ([_i64, _i64, _i64, _sz], _int),
    "tpmlp_fwd": ([_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_tp_fwd": ([_vp, _PP, _PP, _PP, _PP, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_tp_bwd": ([_vp, _vp, _PP, _PP, _PP, _PP, _PP, _PP, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_tp_fwd_full": ([_vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_tp_bwd_full": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_shard_sum": ([_PP, _int, _vp, _i64, _vp], _int),
    "tpmlp_fwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp], _int),
    "tpmlp_sp_workspace_bytes": ([_int, _i64, _i64, _i64], _sz),
    "tpmlp_sp_fwd": ([_PP, _PP, _PP, _PP, _PP, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_sp_bwd": ([_PP, _PP, _PP, _PP, _PP, _PP, _PP, _PP, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_fp8_workspace_bytes": ([_int, _i64, _i64, _i64], _sz),
    "tpmlp_fp8_tp_fwd": ([_vp, _PP, _PP, _PP, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_fp8_tp_bwd": ([_vp, _vp, _PP, _PP, _PP, _PP, _PP, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_fp8_quantize": ([_vp, _i64, _i64, _int, _int, _vp, _vp, _vp], _int),
    "tpmlp_edge_fwd": ([_EP, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp], _int),
    "tpmlp_edge_bwd_workspace_bytes": ([_EP], _sz),
    "tpmlp_edge_bwd": ([_EP, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _int, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                        _vp, _vp, _vp, _sz, _vp], _int),
    "tpmlp_route_rows": ([_i64, _int, _int, _int, _int], _i64),
    "tpmlp_route_workspace_bytes": ([_i64, _int, _int], _sz),
    "tpmlp_route_sort": ([_vp, _int, _i64, _int, _int, _int, _int, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "tpmlp_route_dispatch": ([_vp, _i64, _vp, _vp, _i64, _int, _i64, _i64, _vp, _i64, _vp], _int),
    "tpmlp_route_combine": ([_vp, _int, _i64, _vp, _vp, _i64, _int, _i64, _i64, _vp, _int, _i64, _vp], _int),
    "tpmlp_route_combine_bwd": ([_vp, _int, _i64, _vp, _int, _i64, _vp, _vp, _vp, _i64, _int, _i64, _i64, _vp, _i64,
                                 _vp, _vp], _int),
    "tpmlp_grad_workspace_bytes": ([_vp, _int], _sz),
    "tpmlp_grad_sumsq": ([_vp, _vp, _vp, _int, _vp, _vp, _sz, _vp], _int),
    "tpmlp_grad_clip": ([_vp, _vp, _vp, _vp, _int, _vp, ctypes.c_float, ctypes.c_float, _vp, _vp], _int),
    "tpmlp_clip_grad_norm": ([_vp, _vp, _vp, _vp, _int, ctypes.c_float, ctypes.c_float, _vp, _vp, _sz, _vp], _int),
    "tpmlp_glu_fwd_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "tpmlp_glu_fwd": ([_vp, _vp, _vp, _vp, _int, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_glu_bwd_workspace_bytes": ([_i64, _i64, _i64, _int], _sz),
    "tpmlp_glu_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _int, _int, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    "tpmlp_dropout_fwd": ([_vp, _int, _i64, _vp, _int, _vp, _i64, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _vp,
                           ctypes.c_uint32, _i64, _vp], _int),
    "tpmlp_dropout_bwd_workspace_bytes": ([_i64, _i64], _sz),
    "tpmlp_dropout_bwd": ([_vp, _int, _i64, _vp, _int, _i64, _vp, _i64, _i64, ctypes.c_float, _vp, ctypes.c_uint32, _i64,
                           _vp, _sz, _vp], _int),
    "tpmlp_edge_fwd_fp8": ([_EP, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp], _int),
    "tpmlp_fp4_quantize": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], _int),
    "tpmlp_fp4_packed_bytes": ([_i64, _i64, _int], _sz),
    "tpmlp_fp4_pack": ([_vp, _vp, _vp, _int, _i64, _i64, _vp], _int),
    "tpmlp_fp4_fwd": ([_vp, _int, _i64, _vp, _vp, _vp, _int, _i64, _int, _int, _i64, _i64, _i64, _vp], _int),
    "tpmlp_timing_begin": ([_int], _int),
    "tpmlp_timing_begin_kinds": ([_int, ctypes.c_uint], _int),
    "tpmlp_timing_end": ([ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_int)], _int),
    "tpmlp_timing_records": ([ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_double), _int], _int),
    "tpmlp_timing_dispatches": ([ctypes.POINTER(_int), _int], _int),
}


def header_functions() -> list:
    """Names of the functions include/tpmlp.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tpmlp_\w+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """The loaded library (loads it on first use).  Raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m tensor_transformer_mlp_03_amd.build` "
                "(hipcc for gfx950). There is no fallback path.")
        try:  # share torch's HIP runtime (same soname) when torch is present
            import torch  # noqa: F401
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, func: str):
    if status != 0:
        raise TpmlpError(status, func, lib().tpmlp_last_error().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = _device = None  # torch's functions behind _current_stream


def _current_stream() -> int:
    """hipStream_t of torch's current stream.  torch.cuda.current_stream() builds a Stream
    object for it, which takes longer than a small call's launch (2.8 us against 0.1)."""
    global _raw_stream, _device
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if raw is None or device is None:
            raw, device = (lambda _: torch.cuda.current_stream().cuda_stream), (lambda: None)
        _device, _raw_stream = device, raw
    return _raw_stream(_device())


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(_device()) if _raw_stream else _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr_array(items: Optional[Sequence], n: int):
    if items is None:
        return None
    arr = (ctypes.c_void_p * n)()
    for i in range(n):
        arr[i] = _ptr(items[i]) if items[i] is not None else None
    return ctypes.cast(arr, _PP)


def _bf16(t, name):
    import torch
    if t.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError(f"{name} must hold bf16 bits (bfloat16/uint16/int16), got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32(t, name):
    import torch
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    return t


# --- queries ------------------------------------------------------------------
def tpmlp_abi_version() -> int:
    return lib().tpmlp_abi_version()


def tpmlp_status_str(status: int) -> str:
    return lib().tpmlp_status_str(status).decode()


def tpmlp_kernel_name(kind: int) -> str:
    return lib().tpmlp_kernel_name(kind).decode()


def tpmlp_fwd_workspace_bytes(M: int, H: int, F_i: int) -> int:
    return lib().tpmlp_fwd_workspace_bytes(M, H, F_i)


def tpmlp_bwd_workspace_bytes(M: int, H: int, F_i: int, recompute: bool) -> int:
    return lib().tpmlp_bwd_workspace_bytes(M, H, F_i, int(bool(recompute)))


def tpmlp_tp_workspace_bytes(t: int, M: int, H: int, F_i: int) -> int:
    return lib().tpmlp_tp_workspace_bytes(t, M, H, F_i)


# --- compute ------------------------------------------------------------------
def tpmlp_fwd(X, A_i, B_i, Z_i, P_save, ws, stream=None):
    """Rank i's forward; shapes X[M,H], A_i[H,F_i], B_i[F_i,H], Z_i[M,H] float32."""
    M, H = X.shape
    F = A_i.shape[1]
    _bf16(X, "X"), _bf16(A_i, "A_i"), _bf16(B_i, "B_i"), _f32(Z_i, "Z_i")
    _shape(B_i, (F, H), "B_i"), _shape(Z_i, (M, H), "Z_i")
    if P_save is not None:
        _bf16(P_save, "P_save"), _shape(P_save, (M, F), "P_save")
    st = lib().tpmlp_fwd(_ptr(X), _ptr(A_i), _ptr(B_i), _ptr(Z_i), _ptr(P_save), M, H, F,
                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_fwd")


NOALLOC_SCRATCH_BYTES = 64 << 20  # TPMLP_NOALLOC_SCRATCH_BYTES


def tpmlp_fwd_noalloc(X, A_i, B_i, Z_i, P_save, stream=None):
    """tpmlp_fwd with the library's own device scratch array as its workspace (no
    allocation); shapes whose forward workspace exceeds NOALLOC_SCRATCH_BYTES are
    rejected with TPMLP_ERR_WORKSPACE."""
    M, H = X.shape
    F = A_i.shape[1]
    _bf16(X, "X"), _bf16(A_i, "A_i"), _bf16(B_i, "B_i"), _f32(Z_i, "Z_i")
    _shape(B_i, (F, H), "B_i"), _shape(Z_i, (M, H), "Z_i")
    if P_save is not None:
        _bf16(P_save, "P_save"), _shape(P_save, (M, F), "P_save")
    st = lib().tpmlp_fwd_noalloc(_ptr(X), _ptr(A_i), _ptr(B_i), _ptr(Z_i), _ptr(P_save), M, H, F, _stream(stream))
    _check(st, "tpmlp_fwd_noalloc")


def tpmlp_bwd(dZ, X, A_i, B_i, P_saved, dX_i, dA_i, dB_i, ws, stream=None):
    """Rank i's backward; P_saved None recomputes the pre-activation."""
    M, H = X.shape
    F = A_i.shape[1]
    for t, n in ((dZ, "dZ"), (X, "X"), (A_i, "A_i"), (B_i, "B_i")):
        _bf16(t, n)
    for t, n in ((dX_i, "dX_i"), (dA_i, "dA_i"), (dB_i, "dB_i")):
        _f32(t, n)
    for t, n, shp in ((dZ, "dZ", (M, H)), (A_i, "A_i", (H, F)), (B_i, "B_i", (F, H)), (dX_i, "dX_i", (M, H)),
                      (dA_i, "dA_i", (H, F)), (dB_i, "dB_i", (F, H))):
        _shape(t, shp, n)
    if P_saved is not None:
        _bf16(P_saved, "P_saved"), _shape(P_saved, (M, F), "P_saved")
    st = lib().tpmlp_bwd(_ptr(dZ), _ptr(X), _ptr(A_i), _ptr(B_i), _ptr(P_saved), _ptr(dX_i), _ptr(dA_i),
                         _ptr(dB_i), M, H, F, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_bwd")


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _shards(items, t, shape, name, check, nullable=False):
    """Checks a list of t per-shard tensors (entries None allowed if nullable)."""
    if items is None:
        return
    if len(items) != t:
        raise ValueError(f"{name} has {len(items)} entries, expected t = {t}")
    for i, x in enumerate(items):
        if x is None:
            if not nullable:
                raise ValueError(f"{name}[{i}] is None")
            continue
        check(x, f"{name}[{i}]")
        _shape(x, shape, f"{name}[{i}]")


def _whole(A, B, t, H):
    """F_i of the whole weights A[H, t F_i], B[t F_i, H]."""
    if t < 1 or A.shape[1] % t:
        raise ValueError(f"A has {A.shape[1]} columns, not a multiple of t = {t}")
    _shape(A, (H, A.shape[1]), "A")
    _shape(B, (A.shape[1], H), "B")
    return A.shape[1] // t


def tpmlp_tp_fwd(X, A_sh, B_sh, P_sh, Z_sh, Z, ws, stream=None):
    """All t shards' forward, partials summed into Z[M,H] float32."""
    t = len(A_sh)
    M, H = X.shape
    F = A_sh[0].shape[1]
    _bf16(X, "X"), _f32(Z, "Z"), _shape(Z, (M, H), "Z")
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (M, F), "P_sh", _bf16, nullable=True)
    _shards(Z_sh, t, (M, H), "Z_sh", _f32, nullable=True)
    st = lib().tpmlp_tp_fwd(_ptr(X), _ptr_array(A_sh, t), _ptr_array(B_sh, t), _ptr_array(P_sh, t),
                            _ptr_array(Z_sh, t), _ptr(Z), t, M, H, F, _ptr(ws),
                            ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_tp_fwd")


def tpmlp_tp_bwd(dZ, X, A_sh, B_sh, P_sh, dA_sh, dB_sh, dX_sh, dX, ws, stream=None):
    """All t shards' backward, dX = sum of the shards' partials."""
    t = len(A_sh)
    M, H = X.shape
    F = A_sh[0].shape[1]
    _bf16(dZ, "dZ"), _shape(dZ, (M, H), "dZ"), _bf16(X, "X"), _f32(dX, "dX"), _shape(dX, (M, H), "dX")
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (M, F), "P_sh", _bf16)
    _shards(dA_sh, t, (H, F), "dA_sh", _f32)
    _shards(dB_sh, t, (F, H), "dB_sh", _f32)
    _shards(dX_sh, t, (M, H), "dX_sh", _f32, nullable=True)
    st = lib().tpmlp_tp_bwd(_ptr(dZ), _ptr(X), _ptr_array(A_sh, t), _ptr_array(B_sh, t), _ptr_array(P_sh, t),
                            _ptr_array(dA_sh, t), _ptr_array(dB_sh, t), _ptr_array(dX_sh, t), _ptr(dX), t, M,
                            H, F, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_tp_bwd")


def tpmlp_tp_fwd_full(X, A, B, P, Z, t, ws, stream=None):
    """All t shards' forward over the whole weights A[H, t F_i], B[t F_i, H] (no shard
    copies); P: None or t blocks [M, F_i] of bf16; Z[M,H] float32 the summed output."""
    M, H = X.shape
    F = _whole(A, B, t, H)
    _bf16(X, "X"), _bf16(A, "A"), _bf16(B, "B"), _f32(Z, "Z"), _shape(Z, (M, H), "Z")
    if P is not None:
        _bf16(P, "P")
        if P.numel() != t * M * F:
            raise ValueError(f"P holds {P.numel()} elements, expected t * M * F_i = {t * M * F}")
    st = lib().tpmlp_tp_fwd_full(_ptr(X), _ptr(A), _ptr(B), _ptr(P), _ptr(Z), t, M, H, F, _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_tp_fwd_full")


def tpmlp_tp_bwd_full(dZ, X, A, B, P, dA, dB, dX, t, ws, stream=None):
    """All t shards' backward over the whole weights; dA[H, t F_i] and dB[t F_i, H] are
    the whole float32 weight gradients, dX the sum of the shards' partials."""
    M, H = X.shape
    F = _whole(A, B, t, H)
    for x, n in ((dZ, "dZ"), (X, "X"), (A, "A"), (B, "B")):
        _bf16(x, n)
    _shape(dZ, (M, H), "dZ")
    for x, n, shp in ((dA, "dA", (H, t * F)), (dB, "dB", (t * F, H)), (dX, "dX", (M, H))):
        _f32(x, n), _shape(x, shp, n)
    if P is not None:
        _bf16(P, "P")
        if P.numel() != t * M * F:
            raise ValueError(f"P holds {P.numel()} elements, expected t * M * F_i = {t * M * F}")
    st = lib().tpmlp_tp_bwd_full(_ptr(dZ), _ptr(X), _ptr(A), _ptr(B), _ptr(P), _ptr(dA), _ptr(dB), _ptr(dX), t,
                                 M, H, F, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_tp_bwd_full")


def tpmlp_sp_workspace_bytes(t: int, M: int, H: int, F_i: int) -> int:
    return lib().tpmlp_sp_workspace_bytes(t, M, H, F_i)


def tpmlp_sp_fwd(X_sl, A_sh, B_sh, P_sh, Z_sl, ws, stream=None):
    """Forward at the sequence-parallel boundary: X_sl[r] and Z_sl[r] are rank r's
    token rows [M/t, H] (bf16 in, float32 out); P_sh: None or t tensors [M, F_i]."""
    t = len(A_sh)
    S, H = X_sl[0].shape
    F = A_sh[0].shape[1]
    _shards(X_sl, t, (S, H), "X_sl", _bf16)
    _shards(Z_sl, t, (S, H), "Z_sl", _f32)
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (S * t, F), "P_sh", _bf16, nullable=True)
    st = lib().tpmlp_sp_fwd(_ptr_array(X_sl, t), _ptr_array(A_sh, t), _ptr_array(B_sh, t), _ptr_array(P_sh, t),
                            _ptr_array(Z_sl, t), t, S * t, H, F, _ptr(ws), ws.numel() * ws.element_size(),
                            _stream(stream))
    _check(st, "tpmlp_sp_fwd")


def tpmlp_sp_bwd(dZ_sl, X_sl, A_sh, B_sh, P_sh, dA_sh, dB_sh, dX_sl, ws, stream=None):
    """Backward at the sequence-parallel boundary; P_sh None recomputes the
    pre-activations."""
    t = len(A_sh)
    S, H = X_sl[0].shape
    F = A_sh[0].shape[1]
    _shards(dZ_sl, t, (S, H), "dZ_sl", _bf16)
    _shards(X_sl, t, (S, H), "X_sl", _bf16)
    _shards(dX_sl, t, (S, H), "dX_sl", _f32)
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (S * t, F), "P_sh", _bf16)
    _shards(dA_sh, t, (H, F), "dA_sh", _f32)
    _shards(dB_sh, t, (F, H), "dB_sh", _f32)
    st = lib().tpmlp_sp_bwd(_ptr_array(dZ_sl, t), _ptr_array(X_sl, t), _ptr_array(A_sh, t), _ptr_array(B_sh, t),
                            _ptr_array(P_sh, t), _ptr_array(dA_sh, t), _ptr_array(dB_sh, t), _ptr_array(dX_sl, t),
                            t, S * t, H, F, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_sp_bwd")


def tpmlp_saved_activation_bytes(M: int, H: int, F: int, recompute: bool) -> int:
    return lib().tpmlp_saved_activation_bytes(M, H, F, int(recompute))


def tpmlp_recompute_policy(M: int, H: int, F: int, budget_bytes: int) -> int:
    """0: keep the pre-activation, 1: recompute it, -1: neither fits the budget."""
    return lib().tpmlp_recompute_policy(M, H, F, budget_bytes)


def tpmlp_shard_sum(parts, out, stream=None):
    """out = parts[0] + ... + parts[t-1] (float32, in order)."""
    t = len(parts)
    _f32(out, "out")
    for i, p in enumerate(parts):
        _f32(p, f"parts[{i}]")
        if p.numel() != out.numel():
            raise ValueError(f"parts[{i}] holds {p.numel()} elements, out {out.numel()}")
    st = lib().tpmlp_shard_sum(_ptr_array(parts, t), t, _ptr(out), out.numel(), _stream(stream))
    _check(st, "tpmlp_shard_sum")


def tpmlp_fp8_workspace_bytes(t: int, M: int, H: int, F_i: int) -> int:
    return lib().tpmlp_fp8_workspace_bytes(t, M, H, F_i)


def tpmlp_fp8_tp_fwd(X, A_sh, B_sh, P_sh, Z, ws, stream=None):
    """The t-shard forward with FP8 operands (per-tensor scaling), Z[M,H] float32."""
    t = len(A_sh)
    M, H = X.shape
    F = A_sh[0].shape[1]
    _bf16(X, "X"), _f32(Z, "Z"), _shape(Z, (M, H), "Z")
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (M, F), "P_sh", _bf16, nullable=True)
    st = lib().tpmlp_fp8_tp_fwd(_ptr(X), _ptr_array(A_sh, t), _ptr_array(B_sh, t), _ptr_array(P_sh, t), _ptr(Z),
                                t, M, H, F, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_fp8_tp_fwd")


def tpmlp_fp8_tp_bwd(dZ, X, A_sh, B_sh, P_sh, dA_sh, dB_sh, dX, ws, stream=None):
    """The t-shard backward with FP8 operands; P_sh None recomputes P_i."""
    t = len(A_sh)
    M, H = X.shape
    F = A_sh[0].shape[1]
    _bf16(dZ, "dZ"), _shape(dZ, (M, H), "dZ"), _bf16(X, "X"), _f32(dX, "dX"), _shape(dX, (M, H), "dX")
    _shards(A_sh, t, (H, F), "A_sh", _bf16)
    _shards(B_sh, t, (F, H), "B_sh", _bf16)
    _shards(P_sh, t, (M, F), "P_sh", _bf16)
    _shards(dA_sh, t, (H, F), "dA_sh", _f32)
    _shards(dB_sh, t, (F, H), "dB_sh", _f32)
    st = lib().tpmlp_fp8_tp_bwd(_ptr(dZ), _ptr(X), _ptr_array(A_sh, t), _ptr_array(B_sh, t), _ptr_array(P_sh, t),
                                _ptr_array(dA_sh, t), _ptr_array(dB_sh, t), _ptr(dX), t, M, H, F, _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tpmlp_fp8_tp_bwd")


def tpmlp_fp8_quantize(T, fmt: int, transpose: bool, codes, amax, stream=None):
    """FP8 codes of a bf16 tensor T[R,C] (uint8 codes [R,C], or [C,R] transposed) and
    its amax (one float32 element, overwritten)."""
    import torch
    R, C = T.shape
    _bf16(T, "T")
    if codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise TypeError("codes must be a contiguous uint8 tensor")
    _shape(codes, (C, R) if transpose else (R, C), "codes")
    _f32(amax, "amax")
    if amax.numel() != 1:
        raise ValueError("amax must hold one float32")
    st = lib().tpmlp_fp8_quantize(_ptr(T), R, C, int(fmt), 1 if transpose else 0, _ptr(codes), _ptr(amax),
                                  _stream(stream))
    _check(st, "tpmlp_fp8_quantize")


# --- block operators ----------------------------------------------------------------
F32, BF16 = 0, 1                                       # tpmlp_dtype
NORMS = {"none": 0, "rms": 1, "layer": 2}              # tpmlp_norm

_KINDS = {}  # torch dtype -> tpmlp_dtype


def _dtype(t, name) -> int:
    """tpmlp_dtype of a tensor (bf16 data may be uint16 or int16 bits)."""
    kind = _KINDS.get(t.dtype)
    if kind is None:
        import torch
        _KINDS.update({torch.float32: F32, torch.bfloat16: BF16, torch.int16: BF16, torch.uint16: BF16})
        kind = _KINDS.get(t.dtype)
        if kind is None:
            raise TypeError(f"{name} must be float32 or hold bf16 bits (bfloat16/uint16/int16), got {t.dtype}")
    return kind


def _gpu_here() -> bool:
    import torch
    return torch.cuda.device_count() > 0


def _host(t, name) -> None:
    """Refuses a tensor in host memory that kernels cannot reach (pinned memory they can).  Where there is no GPU the
    library refuses the call itself."""
    if t.numel() and _gpu_here() and not t.is_pinned():
        raise ValueError(f"{name} is not on the GPU")


def _rows(t, shape, name, kind=None):
    """(pointer, row stride) of a [rows, columns] tensor with contiguous columns, after
    checking its shape and, if given, its tpmlp_dtype."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        _host(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if kind is not None and _dtype(t, name) != kind:
        raise TypeError(f"{name} must be {'float32' if kind == F32 else 'bf16'}, got {t.dtype}")
    if t.is_contiguous():  # quicker than the strides, which makes up for the look at its device
        return t.data_ptr(), 0
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous columns")
    if shape[0] < 2:
        return t.data_ptr(), 0
    if row < shape[1]:  # 0 too, a broadcast: the library takes it as dense rows
        raise ValueError(f"the rows of {name} overlap (stride {row})")
    return t.data_ptr(), row


def _flat(t, n, dtype, name):
    """Pointer of a contiguous tensor of n elements."""
    if t is None:
        return None
    if not t.is_cuda:
        _host(t, name)
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    if t.numel() != n:
        raise ValueError(f"{name} holds {t.numel()} elements, expected {n}")
    return t.data_ptr()


def _ws(ws):
    if ws is None:
        return None, 0
    if not ws.is_cuda:
        _host(ws, "ws")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def edge_desc(H: int, post="none", pre="none", w_post=None, b_post=None, w_pre=None, b_pre=None, gate=None,
              gate_rows: int = 0, alpha: float = 1.0, eps: float = 1e-5) -> EdgeDesc:
    """A tpmlp_edge with its parameters (all float32 or all bf16; the gate [G, H], or [H] for
    one row); M, y_type and r_type are each call's own, which leaves this one as it is.  gate_rows 0: one row for all tokens.
    Holds the parameters' addresses: they have to stay alive and where they are."""
    params = [(n, t) for n, t in (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre),
                                  ("gate", gate)) if t is not None]
    kinds = {_dtype(t, n) for n, t in params}
    if len(kinds) > 1:
        raise TypeError("the edge's parameters must have one type")
    for n, t in params:
        if n != "gate":
            _flat(t, H, t.dtype, n)
    d = EdgeDesc(M=0, H=H, post=NORMS[post], pre=NORMS[pre], param_type=kinds.pop() if kinds else F32, alpha=alpha,
                 eps=eps, w_post=_ptr(w_post), b_post=_ptr(b_post), w_pre=_ptr(w_pre), b_pre=_ptr(b_pre))
    if gate_rows < 0:
        raise ValueError("gate_rows must not be negative")
    if gate is not None:
        g = gate if gate.dim() == 2 else gate.unsqueeze(0)
        d.gate, d.ld_gate = _rows(g, (g.shape[0], H), "gate")
        if gate_rows == 0 and g.shape[0] != 1:
            raise ValueError(f"a gate of {g.shape[0]} rows needs gate_rows")
        d.gate_rows = gate_rows or (1 << 31) - 1
        d.gate_tokens = g.shape[0] * d.gate_rows
    return d


def _of_call(d: EdgeDesc, M: int) -> EdgeDesc:
    """The description with one call's M, for the call's types to be added.  A copy: the library reads it without
    the interpreter's lock, while another thread may call through the same description."""
    c = EdgeDesc.from_buffer_copy(d)
    c.M = M
    return c


def _check_gate(d: EdgeDesc, M: int) -> None:
    if M > d.gate_tokens:
        raise ValueError(f"gate has {d.gate_tokens // d.gate_rows} rows for {d.gate_rows} tokens each, the call has {M} tokens")


def _gate_groups(d: EdgeDesc, M: int) -> int:
    return -(-M // d.gate_rows) if d.gate else 0


def tpmlp_edge_fwd(d: EdgeDesc, y, r, r_out, x, stream=None):
    """r_out = alpha r + gate * N_post(y), x = N_pre(r_out); y None: no block before the edge."""
    M, H = r.shape[0], d.H
    if d.gate_tokens is not None:
        _check_gate(d, M)
    c = _of_call(d, M)
    c.r_type = _dtype(r, "r")
    pr, lr = _rows(r, (M, H), "r")
    py = ly = None
    if y is not None:
        c.y_type = _dtype(y, "y")
        py, ly = _rows(y, (M, H), "y")
    po, lo = _rows(r_out, (M, H), "r_out", c.r_type)
    px, lx = _rows(x, (M, H), "x", BF16)
    st = lib().tpmlp_edge_fwd(ctypes.byref(c), py, ly or 0, pr, lr, po, lo, px, lx, _stream(stream))
    if st:
        _check(st, "tpmlp_edge_fwd")


def tpmlp_edge_bwd_workspace_bytes(d: EdgeDesc, M: int) -> int:
    return lib().tpmlp_edge_bwd_workspace_bytes(ctypes.byref(_of_call(d, M)))


def tpmlp_edge_bwd(d: EdgeDesc, y, r_out, dr_out, dx, dr, dy, dw_post=None, db_post=None, dw_pre=None, db_pre=None,
                   dgate=None, ws=None, stream=None):
    """Backward of the edge; r_out is the stream the forward wrote, dr and dy are written."""
    import torch
    M, H = dr.shape[0], d.H
    if d.gate_tokens is not None:
        _check_gate(d, M)
    c = _of_call(d, M)
    c.r_type = _dtype(dr, "dr")
    pr, lr = _rows(r_out, (M, H), "r_out", c.r_type)
    po, lo = _rows(dr_out, (M, H), "dr_out", c.r_type)
    px, lx = _rows(dx, (M, H), "dx")
    pd, ld = _rows(dr, (M, H), "dr")
    py, ly = _rows(y, (M, H), "y")
    if y is not None:
        c.y_type = _dtype(y, "y")
    pg, lg = _rows(dy, (M, H), "dy", BF16)
    f32 = torch.float32
    grads = [_flat(dw_post, H, f32, "dw_post"), _flat(db_post, H, f32, "db_post"), _flat(dw_pre, H, f32, "dw_pre"),
             _flat(db_pre, H, f32, "db_pre"),
             _flat(dgate, _gate_groups(d, M) * H, f32, "dgate") if dgate is not None else None]
    pw, nw = _ws(ws)
    st = lib().tpmlp_edge_bwd(ctypes.byref(c), py, ly, pr, lr, po, lo, px, _dtype(dx, "dx") if dx is not None else F32,
                              lx, pd, ld, pg, lg, *grads, pw, nw, _stream(stream))
    if st:
        _check(st, "tpmlp_edge_bwd")


def tpmlp_route_rows(T: int, K: int, E: int, align: int = 8, capacity: int = 0) -> int:
    return lib().tpmlp_route_rows(T, K, E, align, capacity)


def tpmlp_route_workspace_bytes(T: int, K: int, E: int) -> int:
    return lib().tpmlp_route_workspace_bytes(T, K, E)


def tpmlp_route_sort(ids, E: int, align: int, capacity: int, counts, offsets, row_of, src_of, ws=None, stream=None):
    """Pairs sorted by expert; ids [T,K] int32 or int64, the outputs int32."""
    import torch
    T, K = ids.shape
    if ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise TypeError("ids must be a contiguous int32 or int64 tensor")
    if not ids.is_cuda:
        _host(ids, "ids")
    i32, rows = torch.int32, max(0, tpmlp_route_rows(T, K, E, align, capacity))
    pw, nw = _ws(ws)
    st = lib().tpmlp_route_sort(ids.data_ptr(), 32 if ids.dtype == i32 else 64, T, K, E, align, capacity,
                                _flat(counts, E, i32, "counts"), _flat(offsets, E + 1, i32, "offsets"),
                                _flat(row_of, T * K, i32, "row_of"), _flat(src_of, rows, i32, "src_of"), pw, nw,
                                _stream(stream))
    if st:
        _check(st, "tpmlp_route_sort")


def tpmlp_route_dispatch(X, row_of, src_of, Xs, stream=None):
    """Xs[row_of[t,k]] = X[t], zeros on padding rows; bf16."""
    import torch
    (T, K), (rows, H) = row_of.shape, Xs.shape
    px, lx = _rows(X, (T, H), "X", BF16)
    ps, ls = _rows(Xs, (rows, H), "Xs", BF16)
    st = lib().tpmlp_route_dispatch(px, lx, _flat(row_of, T * K, torch.int32, "row_of"),
                                    _flat(src_of, rows, torch.int32, "src_of"), T, K, H, rows, ps, ls, _stream(stream))
    if st:
        _check(st, "tpmlp_route_dispatch")


def tpmlp_route_combine(Zs, row_of, w, Y, stream=None):
    """Y[t] = sum over k of w[t,k] Zs[row_of[t,k]]; w None: ones."""
    import torch
    (T, K), (rows, H) = row_of.shape, Zs.shape
    pz, lz = _rows(Zs, (rows, H), "Zs")
    py, ly = _rows(Y, (T, H), "Y")
    st = lib().tpmlp_route_combine(pz, _dtype(Zs, "Zs"), lz, _flat(row_of, T * K, torch.int32, "row_of"),
                                   _flat(w, T * K, torch.float32, "w"), T, K, H, rows, py, _dtype(Y, "Y"), ly,
                                   _stream(stream))
    if st:
        _check(st, "tpmlp_route_combine")


def tpmlp_route_combine_bwd(dY, Zs, row_of, src_of, w, dZs, dw, stream=None):
    """dZs[row_of[t,k]] = w[t,k] dY[t] (bf16) and dw[t,k] = <dY[t], Zs[row_of[t,k]]>; dZs (with
    src_of) or dw (with Zs) may be None."""
    import torch
    T, K = row_of.shape
    H = dY.shape[1]
    rows = (dZs if dZs is not None else Zs).shape[0]
    pd, ld = _rows(dY, (T, H), "dY")
    pz, lz = _rows(Zs, (rows, H), "Zs")
    po, lo = _rows(dZs, (rows, H), "dZs", BF16)
    st = lib().tpmlp_route_combine_bwd(pd, _dtype(dY, "dY"), ld, pz, _dtype(Zs, "Zs") if Zs is not None else F32, lz,
                                       _flat(row_of, T * K, torch.int32, "row_of"),
                                       _flat(src_of, rows, torch.int32, "src_of"), _flat(w, T * K, torch.float32, "w"),
                                       T, K, H, rows, po, lo, _flat(dw, T * K, torch.float32, "dw"), _stream(stream))
    if st:
        _check(st, "tpmlp_route_combine_bwd")


class GradTable:
    """The host arrays that the gradient calls take: addresses, sizes and types of float32 or
    bf16 tensors, and of the tensors that receive the scaled values (None: in place).  Keeps
    the tensors alive; their storage must stay where it is."""

    def __init__(self, grads, outs=None):
        self.grads, self.outs, n = list(grads), None if outs is None else list(outs), len(grads)
        if self.outs is not None and len(self.outs) != n:
            raise ValueError(f"outs has {len(self.outs)} entries, expected {n}")
        self.n = n
        self.ptrs, self.out_ptrs = (_vp * max(n, 1))(), (_vp * max(n, 1))()
        self.sizes, self.types = (_i64 * max(n, 1))(), (ctypes.c_int32 * max(n, 1))()
        for i, g in enumerate(self.grads):
            o = g if self.outs is None else self.outs[i]
            if not g.is_contiguous() or not o.is_contiguous():
                raise ValueError(f"gradient {i} and its output must be contiguous")
            if not g.is_cuda or not o.is_cuda:
                _host(g if not g.is_cuda else o, f"gradient {i} or its output")
            if o.dtype != g.dtype or o.numel() != g.numel():
                raise ValueError(f"outs[{i}] differs from its gradient in type or size")
            self.ptrs[i], self.out_ptrs[i] = g.data_ptr(), o.data_ptr()
            self.sizes[i], self.types[i] = g.numel(), _dtype(g, f"grads[{i}]")


def tpmlp_grad_workspace_bytes(table: GradTable) -> int:
    return lib().tpmlp_grad_workspace_bytes(table.sizes, table.n)


def _one(t, dtype, name):
    if t.dtype != dtype or t.numel() != 1:
        raise TypeError(f"{name} must be one {dtype}")
    if not t.is_cuda:
        _host(t, name)
    return t.data_ptr()


def tpmlp_grad_sumsq(table: GradTable, sumsq, ws, stream=None):
    """sumsq (one float64) = sum of squares of all gradients."""
    import torch
    pw, nw = _ws(ws)
    st = lib().tpmlp_grad_sumsq(table.ptrs, table.sizes, table.types, table.n, _one(sumsq, torch.float64, "sumsq"),
                                pw, nw, _stream(stream))
    if st:
        _check(st, "tpmlp_grad_sumsq")


def tpmlp_grad_clip(table: GradTable, sumsq, max_norm: float, norm=None, scale: float = 1.0, stream=None):
    """Scales the gradients by scale * min(1, max_norm / norm), norm = |scale| sqrt(sumsq)."""
    import torch
    st = lib().tpmlp_grad_clip(table.ptrs, table.out_ptrs, table.sizes, table.types, table.n,
                               _one(sumsq, torch.float64, "sumsq"), scale, max_norm,
                               None if norm is None else _one(norm, torch.float32, "norm"), _stream(stream))
    if st:
        _check(st, "tpmlp_grad_clip")


def tpmlp_clip_grad_norm(table: GradTable, max_norm: float, norm, ws, scale: float = 1.0, stream=None):
    """tpmlp_grad_sumsq and tpmlp_grad_clip in one call."""
    import torch
    pw, nw = _ws(ws)
    st = lib().tpmlp_clip_grad_norm(table.ptrs, table.out_ptrs, table.sizes, table.types, table.n, scale, max_norm,
                                    None if norm is None else _one(norm, torch.float32, "norm"), pw, nw,
                                    _stream(stream))
    if st:
        _check(st, "tpmlp_clip_grad_norm")


# --- the gated block ------------------------------------------------------------------
ACTS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3, "sigmoid": 4}  # tpmlp_act
SCALE_ROW, SCALE_MX = 0, 1                                         # tpmlp_scale
X_BF16, X_E4M3_ROW, X_E4M3_MX = 0, 1, 2                            # tpmlp_x


def _on_gpu(t, name):
    if t is not None and not t.is_cuda:
        _host(t, name)
    return t


def _dense(t, shape, name, kind=None):
    """Pointer of a contiguous tensor of this shape and, if given, tpmlp_dtype."""
    if t is None:
        return None
    _on_gpu(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if kind is not None and _dtype(t, name) != kind:
        raise TypeError(f"{name} must be {'float32' if kind == F32 else 'bf16'}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _act(act: str) -> int:
    kind = ACTS.get(act)
    if kind is None:
        raise ValueError(f"no activation {act!r}")
    return kind


def _glu_sizes(A, B):
    (F, H), (h, f2) = B.shape, A.shape
    if h != H or f2 != 2 * F:
        raise ValueError(f"A has shape {tuple(A.shape)}, expected {(H, 2 * F)} for B {tuple(B.shape)}")
    return H, F


def tpmlp_glu_fwd_workspace_bytes(M: int, H: int, F: int) -> int:
    return lib().tpmlp_glu_fwd_workspace_bytes(M, H, F)


def tpmlp_glu_bwd_workspace_bytes(M: int, H: int, F: int, recompute: bool) -> int:
    return lib().tpmlp_glu_bwd_workspace_bytes(M, H, F, int(bool(recompute)))


def tpmlp_glu_fwd(X, A, B, Z, P_save, act: str, ws, stream=None):
    """Z[M,H] = (act(P_g) * P_u) B with P = X A; A[H, 2F], B[F,H], X bf16; Z float32 or bf16."""
    H, F = _glu_sizes(A, B)
    M = X.shape[0]
    pw, nw = _ws(ws)
    st = lib().tpmlp_glu_fwd(_dense(X, (M, H), "X", BF16), _dense(A, (H, 2 * F), "A", BF16), _dense(B, (F, H), "B", BF16),
                             _dense(Z, (M, H), "Z"), _dtype(Z, "Z"), _dense(P_save, (M, 2 * F), "P_save", BF16), _act(act), M,
                             H, F, pw, nw, _stream(stream))
    if st:
        _check(st, "tpmlp_glu_fwd")


def tpmlp_glu_bwd(dZ, X, A, B, P_saved, dX, dA, dB, act: str, ws, stream=None):
    """The gated MLP's gradients; dX, and dA with dB, float32 or bf16; P_saved None recomputes P."""
    H, F = _glu_sizes(A, B)
    M = X.shape[0]
    kind = _dtype(dA, "dA")
    pw, nw = _ws(ws)
    st = lib().tpmlp_glu_bwd(_dense(dZ, (M, H), "dZ", BF16), _dense(X, (M, H), "X", BF16), _dense(A, (H, 2 * F), "A", BF16),
                             _dense(B, (F, H), "B", BF16), _dense(P_saved, (M, 2 * F), "P_saved", BF16),
                             _dense(dX, (M, H), "dX"), _dtype(dX, "dX"), _dense(dA, (H, 2 * F), "dA"),
                             _dense(dB, (F, H), "dB", kind), kind, _act(act), M, H, F, pw, nw, _stream(stream))
    if st:
        _check(st, "tpmlp_glu_bwd")


def _state(state):
    import torch
    if state.dtype not in (torch.int64, torch.uint64) or state.numel() != 2 or not state.is_contiguous():
        raise TypeError("state must be two contiguous int64 values, the seed and the step")
    return _on_gpu(state, "state").data_ptr()


def tpmlp_dropout_fwd(y, bias, r, out, p: float, state, site: int = 0, first_row: int = 0, stream=None):
    """out = r + mask * (y + bias) / (1 - p); y float32 or bf16, out and r of one type, bias and r nullable."""
    M, H = y.shape
    kind = _dtype(out, "out")
    py, ly = _rows(y, (M, H), "y")
    po, lo = _rows(out, (M, H), "out")
    pr, lr = _rows(r, (M, H), "r", kind)
    st = lib().tpmlp_dropout_fwd(py, _dtype(y, "y"), ly, _flat(bias, H, bias.dtype, "bias") if bias is not None else None,
                                 _dtype(bias, "bias") if bias is not None else F32, pr, lr, po, kind, lo, M, H, p,
                                 _state(state), _u32(site, "site"), _u32(first_row, "first_row", 1), _stream(stream))
    if st:
        _check(st, "tpmlp_dropout_fwd")


def _u32(v: int, name: str, past: int = 0) -> int:
    if not 0 <= v < (1 << 32) + past:  # ctypes would take its low bits
        raise ValueError(f"{name} must be from 0 to 2^32" + (" - 1" if not past else ""))
    return v


def tpmlp_dropout_bwd_workspace_bytes(M: int, H: int) -> int:
    return lib().tpmlp_dropout_bwd_workspace_bytes(M, H)


def tpmlp_dropout_bwd(dout, dy, db, p: float, state, site: int = 0, first_row: int = 0, ws=None, stream=None):
    """dy = mask * dout / (1 - p); db[H] (float32, nullable) = the sum of its rows."""
    import torch
    M, H = dout.shape
    pg, lg = _rows(dout, (M, H), "dout")
    py, ly = _rows(dy, (M, H), "dy")
    pw, nw = _ws(ws)
    st = lib().tpmlp_dropout_bwd(pg, _dtype(dout, "dout"), lg, py, _dtype(dy, "dy"), ly, _flat(db, H, torch.float32, "db"), M, H,
                                 p, _state(state), _u32(site, "site"), _u32(first_row, "first_row", 1), pw, nw, _stream(stream))
    if st:
        _check(st, "tpmlp_dropout_bwd")


_BYTE_TYPES = {}  # torch's types of each kind of one-byte values, beside raw bytes


def _bytes(t, shape, name, kind):
    """(pointer, row stride) of a [rows, columns] tensor with contiguous columns of one-byte values of a
    kind: "E4M3", "E8M0" or "E2M1" (two a byte), as torch's type of that format or as uint8."""
    if not _BYTE_TYPES:
        import torch
        for k, n in (("E4M3", "float8_e4m3fn"), ("E8M0", "float8_e8m0fnu"), ("E2M1", "float4_e2m1fn_x2")):
            _BYTE_TYPES[k] = (torch.uint8, getattr(torch, n, torch.uint8))
    if t.dtype not in _BYTE_TYPES[kind]:
        raise TypeError(f"{name} must hold one-byte values, {kind} or uint8, got {t.dtype}")
    return _rows(t, shape, name)


def _scales(t, M, blocks, name):
    """(pointer, row stride, tpmlp_scale) of the scales of [M, 32 blocks] codes."""
    import torch
    if t.dtype == torch.float32:
        return _flat(t, M, torch.float32, name), 0, SCALE_ROW
    p, ld = _bytes(t, (M, blocks), name, "E8M0")
    return p, ld, SCALE_MX


def tpmlp_edge_fwd_fp8(d: EdgeDesc, y, r, r_out, codes, scales, stream=None):
    """tpmlp_edge_fwd with x as E4M3 codes [M,H] (float8_e4m3fn or uint8) and scales: float32 [M], or a
    byte for every 32 values, [M, H / 32] (float8_e8m0fnu or uint8)."""
    M, H = r.shape[0], d.H
    if d.gate_tokens is not None:
        _check_gate(d, M)
    c = _of_call(d, M)
    c.r_type = _dtype(r, "r")
    pr, lr = _rows(r, (M, H), "r")
    py = ly = None
    if y is not None:
        c.y_type = _dtype(y, "y")
        py, ly = _rows(y, (M, H), "y")
    po, lo = _rows(r_out, (M, H), "r_out", c.r_type)
    pc, lc = _bytes(codes, (M, H), "codes", "E4M3")
    ps, ls, kind = _scales(scales, M, H // 32, "scales")
    st = lib().tpmlp_edge_fwd_fp8(ctypes.byref(c), py, ly or 0, pr, lr, po, lo, pc, lc, ps, ls, kind, _stream(stream))
    if st:
        _check(st, "tpmlp_edge_fwd_fp8")


def tpmlp_fp4_quantize(W, codes, scales, stream=None):
    """E2M1 codes [N, K/2] (float4_e2m1fn_x2 or uint8) and scales [N, K/32] (float8_e8m0fnu or uint8) of
    bf16 weights W[K,N]."""
    K, N = W.shape
    pw, lw = _rows(W, (K, N), "W", BF16)
    pc, lc = _bytes(codes, (N, K // 2), "codes", "E2M1")
    ps, ls = _bytes(scales, (N, K // 32), "scales", "E8M0")
    if lc or ls:
        raise ValueError("codes and scales must be contiguous")
    _check(lib().tpmlp_fp4_quantize(pw, lw, K, N, pc, ps, _stream(stream)), "tpmlp_fp4_quantize")


def tpmlp_fp4_packed_bytes(N: int, K: int, gated: bool = False) -> int:
    return lib().tpmlp_fp4_packed_bytes(N, K, int(bool(gated)))


def tpmlp_fp4_pack(codes, scales, packed, gated: bool = False, stream=None):
    """Codes [N, K/2] and scales [N, K/32] (gated: 2N rows) in the order that tpmlp_fp4_fwd reads;
    packed: tpmlp_fp4_packed_bytes one-byte values."""
    import torch
    rows, K = codes.shape[0], 2 * codes.shape[1]
    if gated and rows % 2:
        raise ValueError(f"a gated weight has an even number of rows, not {rows}")
    N = rows // 2 if gated else rows
    pc, lc = _bytes(codes, (rows, K // 2), "codes", "E2M1")
    ps, ls = _bytes(scales, (rows, K // 32), "scales", "E8M0")
    if lc or ls:
        raise ValueError("codes and scales must be contiguous")
    pp = _flat(packed, tpmlp_fp4_packed_bytes(N, K, gated), torch.uint8, "packed")
    _check(lib().tpmlp_fp4_pack(pc, ps, pp, int(bool(gated)), N, K, _stream(stream)), "tpmlp_fp4_pack")


def tpmlp_fp4_fwd(X, x_scales, packed, Y, act: str = "none", gated: bool = False, stream=None):
    """Y[M,N] = act(X W^T), or act(X W_g^T) * (X W_u^T) with W = [W_g; W_u], from a packed weight; X[M,K]
    bf16, or E4M3 codes (float8_e4m3fn or uint8) with x_scales as tpmlp_edge_fwd_fp8 writes them; Y float32 or bf16."""
    import torch
    (M, K), N = X.shape, Y.shape[1]
    ps, kind = None, X_BF16
    if X.element_size() == 1:
        if x_scales is None:
            raise ValueError("X in E4M3 needs x_scales")
        px, lx = _bytes(X, (M, K), "X", "E4M3")
        ps, ls, scale = _scales(x_scales, M, K // 32, "x_scales")
        if ls:
            raise ValueError("x_scales must be contiguous")
        kind = X_E4M3_MX if scale == SCALE_MX else X_E4M3_ROW
    else:
        px, lx = _rows(X, (M, K), "X", BF16)
        if x_scales is not None:
            raise ValueError("x_scales is given with a bf16 X")
    pp = _flat(packed, tpmlp_fp4_packed_bytes(N, K, gated), torch.uint8, "packed")
    py, ly = _rows(Y, (M, N), "Y")
    st = lib().tpmlp_fp4_fwd(px, kind, lx, ps, pp, py, _dtype(Y, "Y"), ly, _act(act), int(bool(gated)), M, N, K, _stream(stream))
    if st:
        _check(st, "tpmlp_fp4_fwd")


def tpmlp_timing_begin(capacity: int):
    _check(lib().tpmlp_timing_begin(capacity), "tpmlp_timing_begin")


def tpmlp_timing_begin_kinds(capacity: int, kinds):
    """Time only the launches of the named kernel kinds."""
    mask = 0
    for name in kinds:
        mask |= 1 << kernel_kind(name)
    _check(lib().tpmlp_timing_begin_kinds(capacity, mask), "tpmlp_timing_begin_kinds")


def kernel_kind(name: str) -> int:
    for k in range(KERNEL_COUNT):
        if tpmlp_kernel_name(k) == name:
            return k
    raise ValueError(f"no kernel kind named {name!r}")


def tpmlp_timing_end():
    """Returns ({kernel name: (launches, total ms)}, dropped)."""
    counts = (ctypes.c_int * KERNEL_COUNT)()
    total = (ctypes.c_double * KERNEL_COUNT)()
    dropped = ctypes.c_int(0)
    _check(lib().tpmlp_timing_end(counts, total, ctypes.byref(dropped)), "tpmlp_timing_end")
    return {tpmlp_kernel_name(k): (counts[k], total[k]) for k in range(KERNEL_COUNT)}, dropped.value


def tpmlp_timing_records():
    """[(kernel name, ms)] of the last timing window, in launch order."""
    n = lib().tpmlp_timing_records((ctypes.c_int * 1)(), (ctypes.c_double * 1)(), 0)
    kinds = (ctypes.c_int * max(n, 1))()
    ms = (ctypes.c_double * max(n, 1))()
    n = lib().tpmlp_timing_records(kinds, ms, n)
    return [(tpmlp_kernel_name(kinds[i]), ms[i]) for i in range(n)]


def tpmlp_timing_dispatches():
    """Kernel dispatches inside each record of the last timing window (1, or 2
    for a product run as whole-wave tiles plus a split tail)."""
    n = lib().tpmlp_timing_dispatches((ctypes.c_int * 1)(), 0)
    out = (ctypes.c_int * max(n, 1))()
    n = lib().tpmlp_timing_dispatches(out, n)
    return [out[i] for i in range(n)]
