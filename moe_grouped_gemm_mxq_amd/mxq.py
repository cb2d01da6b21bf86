"""ctypes binding of libmxq (include/mxq.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmxq.so``; PyTorch supplies device memory and streams.  Importing
this module fails loudly (RuntimeError) when the library is not built -- there
is no fallback.

Functions named like the C entry points take every buffer from the caller;
the lower-case helpers (``quantize``, ``gemm`` ...) allocate the outputs with
``torch.empty`` and call them.  A helper given a stream does both as a call within
``torch.cuda.stream(stream)`` would.

GEMM operand scale arrays are uint8 tensors of shape ``scale_shape(rows,
nblk)`` = ``(ceil128(rows) // 128, nblk, 32, 4)``: element
``[r // 128, b, r % 32, (r // 32) % 4]`` is the E8M0 scale of row ``r``,
block ``b`` (the layout of include/mxq.h: each dword holds the scales of
rows r, r+32, r+64, r+96 of a 128-row group for one block).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MXQ_LIB_PATH") or os.path.join(HERE, "libmxq.so")

MXQ_OK = 0
MXQ_ERR_INVALID_ARGUMENT = 1
MXQ_ERR_UNSUPPORTED = 2
MXQ_ERR_DEVICE = 3
MXQ_ERR_LAUNCH = 4
STATUS_NAMES = {0: "MXQ_OK", 1: "MXQ_ERR_INVALID_ARGUMENT", 2: "MXQ_ERR_UNSUPPORTED",
                3: "MXQ_ERR_DEVICE", 4: "MXQ_ERR_LAUNCH"}

MXQ_AXIS_ROW = 1
MXQ_AXIS_COLT = 2
MXQ_FMT_E4M3 = 0
MXQ_FMT_E2M1 = 1
MXQ_GG_RAGGED_M = 0
MXQ_GG_RAGGED_K = 1
MXQ_DT_F32 = 0
MXQ_DT_BF16 = 1
MXQ_SCORE_SOFTMAX = 0
MXQ_SCORE_SIGMOID = 1
MXQ_ADAMW_F32 = 0
MXQ_ADAMW_MXFP8 = 1
BLOCK = 32
BLOCK128 = 128  # elements per block of the operands with fp32 scales
MAX_GROUPS = 1024
MAX_TOPK = 32  # MXQ_MAX_TOPK
MAX_ROW_BYTES = 1 << 23  # MXQ_GEMM_MAX_ROW_BYTES: GEMM code rows (K, or K/2 for E2M1) stay below this

EXPORTED = [
    "mxq_abi_version", "mxq_last_error", "mxq_device_check", "mxq_grouped_cols_max", "mxq_operand_sizes",
    "mxq_quantize", "mxq_quantize_batched", "mxq_quantize_grouped", "mxq_qdq_fp4", "mxq_qdq_fp4_ex",
    "mxq_ste_backward_fp4", "mxq_fp4_scale_threshold", "mxq_quantize_fp4", "mxq_gemm", "mxq_grouped_gemm",
    "mxq_validate_group_end", "mxq_quantize_fp4_grouped", "mxq_expert_order_workspace", "mxq_route",
    "mxq_expert_order", "mxq_route_backward", "mxq_combine", "mxq_combine_backward", "mxq_adamw",
    "mxq_grouped128_cols_max", "mxq_quantize128", "mxq_quantize128_grouped", "mxq_gemm128", "mxq_grouped_gemm128",
    "mxq_orthogonalize_workspace", "mxq_orthogonalize", "mxq_muon",
]


class RouteConfig(ctypes.Structure):
    """mxq_route_config."""
    _fields_ = [("score", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalise", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class AdamWTensor(ctypes.Structure):
    """mxq_adamw_tensor."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("decay_scale", ctypes.c_double)]


class AdamWConfig(ctypes.Structure):
    """mxq_adamw_config."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32)]


class NewtonSchulz(ctypes.Structure):
    """mxq_newton_schulz."""
    _fields_ = [("a", ctypes.c_double), ("b", ctypes.c_double), ("c", ctypes.c_double), ("eps", ctypes.c_double),
                ("steps", ctypes.c_int32)]


class MuonConfig(ctypes.Structure):
    """mxq_muon_config."""
    _fields_ = [("ns", NewtonSchulz), ("lr", ctypes.c_double), ("momentum", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("scale", ctypes.c_double), ("grad_scale", ctypes.c_double), ("nesterov", ctypes.c_int32)]


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise RuntimeError(
            f"libmxq.so not found at {path}. Build it with "
            "`python -m moe_grouped_gemm_mxq_amd.build` (hipcc, gfx950) or point MXQ_LIB_PATH at a build.")
    lib = ctypes.CDLL(path)
    P, I64, I32, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    sig = {
        "mxq_abi_version": ([], I),
        "mxq_last_error": ([], ctypes.c_char_p),
        "mxq_device_check": ([I], I),
        "mxq_grouped_cols_max": ([I64, I32], I64),
        "mxq_operand_sizes": ([I64, I64, I, P, P], I),
        "mxq_quantize": ([P, I64, I64, I64, I, P, P, P, P, P], I),
        "mxq_quantize_batched": ([P, I64, I64, I64, I64, I64, I, P, P, P, P, P], I),
        "mxq_quantize_grouped": ([P, I64, I64, I64, P, I32, I64, I, P, P, P, P, P], I),
        "mxq_qdq_fp4": ([P, P, I64, I64, P, P, P], I),
        "mxq_qdq_fp4_ex": ([P, P, I64, I64, ctypes.c_float, P, P, P, P], I),
        "mxq_ste_backward_fp4": ([P, P, P, I64, I64, P], I),
        "mxq_fp4_scale_threshold": ([ctypes.c_float, P, P], I),
        "mxq_quantize_fp4": ([P, I64, I64, ctypes.c_float, P, P, P], I),
        "mxq_gemm": ([P, P, P, P, P, I64, I64, I64, I64, I, P], I),
        "mxq_grouped_gemm": ([I, P, P, P, P, P, I64, I64, I64, P, I32, I, P], I),
        "mxq_validate_group_end": ([P, I32, I64, P, P], I),
        "mxq_quantize_fp4_grouped": ([P, I64, I64, I64, P, I32, I64, ctypes.c_float, P, P, P], I),
        "mxq_expert_order_workspace": ([I64, I32, I32], I64),
        "mxq_route": ([P, I, I64, I32, I64, P, P, P, P, P, P, P, P, I64, P], I),
        "mxq_expert_order": ([P, I64, I32, I32, P, P, P, P, I64, P], I),
        "mxq_route_backward": ([P, I, I64, I32, I64, P, P, P, P, I64, P], I),
        "mxq_combine": ([P, I, I64, I64, P, P, I64, I32, I64, P, I, I64, P], I),
        "mxq_combine_backward": ([P, I, I64, P, I, I64, P, P, I64, I32, I64, I64, P, I, I64, P, P], I),
        "mxq_adamw": ([P, I32, I, I, I, P, P, P], I),
        "mxq_orthogonalize_workspace": ([I64, I64, I64, I], I64),
        "mxq_orthogonalize": ([P, I, I64, I64, I64, P, P, I, P, I64, P], I),
        "mxq_muon": ([P, I, P, I, P, P, I64, I64, I64, P, P, P, I64, P], I),
        "mxq_grouped128_cols_max": ([I64, I32], I64),
        "mxq_quantize128": ([P, I, I64, I64, I64, I64, I64, I, I, P, P, P, P, P], I),
        "mxq_quantize128_grouped": ([P, I, I64, I64, I64, P, I32, I64, I, P, P, P, P, P], I),
        "mxq_gemm128": ([P, P, P, P, I, P, I, I64, I64, I64, I64, P], I),
        "mxq_grouped_gemm128": ([I, P, P, P, P, P, I, I64, I64, I64, P, I32, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


ABI_VERSION = 9  # MXQ_ABI_VERSION of include/mxq.h this binding is written against

_lib = _load()
if _lib.mxq_abi_version() != ABI_VERSION:
    raise RuntimeError(f"libmxq.so at {LIB_PATH} implements ABI {_lib.mxq_abi_version()}, this binding needs "
                       f"{ABI_VERSION}: rebuild it with `python -m moe_grouped_gemm_mxq_amd.build`")


class MxqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.mxq_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")


def _check(status: int, where: str):
    if status != MXQ_OK:
        raise MxqError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it (0.1 against 2 us a call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is None:
        if _current_stream is not None and device is not None and device.index is not None:
            return _current_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t, dtype, name, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {t.dim()}")


def ceil32(v: int) -> int:
    return (v + BLOCK - 1) // BLOCK * BLOCK


def scale_shape(rows: int, nblk: int) -> tuple:
    """Shape of the GEMM-operand scale array of `rows` rows and `nblk` blocks per row."""
    return ((rows + 127) // 128, nblk, BLOCK, 4)


def _need_out(t, name, shape):
    if t is None:
        return
    _need(t, torch.uint8, name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


# ------------------------------------------------------------------ C entry points
def mxq_abi_version() -> int:
    return _lib.mxq_abi_version()


def mxq_last_error() -> str:
    return _lib.mxq_last_error().decode()


def mxq_device_check(device: int = 0) -> int:
    return _lib.mxq_device_check(device)


def mxq_grouped_cols_max(T: int, G: int) -> int:
    return _lib.mxq_grouped_cols_max(T, G)


def mxq_operand_sizes(rows: int, K: int, fmt: int = 0) -> tuple:
    """(code bytes, scale bytes) of a quantised GEMM operand of `rows` rows and reduction length K."""
    c, sc = ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.mxq_operand_sizes(rows, K, fmt, ctypes.byref(c), ctypes.byref(sc)), "mxq_operand_sizes")
    return c.value, sc.value


def mxq_quantize(x, axis_mask, q_row=None, s_row=None, q_colT=None, s_colT=None, stream=None):
    """x bf16 [R][C] (unit column stride, any row stride)."""
    _need(x, torch.bfloat16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x must have unit stride along its last dim")
    R, C = x.shape
    _need_out(q_row, "q_row", (R, ceil32(C)))
    _need_out(s_row, "s_row", scale_shape(R, ceil32(C) // BLOCK))
    _need_out(q_colT, "q_colT", (C, ceil32(R)))
    _need_out(s_colT, "s_colT", scale_shape(C, ceil32(R) // BLOCK))
    _check(_lib.mxq_quantize(_ptr(x), R, C, x.stride(0), axis_mask, _ptr(q_row), _ptr(s_row),
                             _ptr(q_colT), _ptr(s_colT), _stream(stream, x.device)), "mxq_quantize")


def mxq_quantize_batched(x, axis_mask, q_row=None, s_row=None, q_colT=None, s_colT=None, stream=None):
    """x bf16 [batch][R][C] (unit stride along C).  Outputs: q_row [batch][R][Cp],
    s_row (batch,) + scale_shape(R, Cp/32), q_colT [batch][C][Rp], s_colT (batch,) + scale_shape(C, Rp/32)."""
    _need(x, torch.bfloat16, "x", 3)
    if x.stride(2) != 1:
        raise ValueError("x must have unit stride along its last dim")
    nb, R, C = x.shape
    _need_out(q_row, "q_row", (nb, R, ceil32(C)))
    _need_out(s_row, "s_row", (nb,) + scale_shape(R, ceil32(C) // BLOCK))
    _need_out(q_colT, "q_colT", (nb, C, ceil32(R)))
    _need_out(s_colT, "s_colT", (nb,) + scale_shape(C, ceil32(R) // BLOCK))
    _check(_lib.mxq_quantize_batched(_ptr(x), nb, R, C, x.stride(1), x.stride(0), axis_mask, _ptr(q_row),
                                     _ptr(s_row), _ptr(q_colT), _ptr(s_colT), _stream(stream, x.device)),
           "mxq_quantize_batched")


def mxq_quantize_grouped(x, group_end, ldq, axis_mask, q_row=None, s_row=None, q_colT=None,
                         s_colT=None, stream=None):
    _need(x, torch.bfloat16, "x", 2)
    _need(group_end, torch.int32, "group_end", 1)
    if x.stride(1) != 1:
        raise ValueError("x must have unit stride along its last dim")
    T, C = x.shape
    _need_out(q_row, "q_row", (T, ceil32(C)))
    _need_out(s_row, "s_row", scale_shape(T, ceil32(C) // BLOCK))
    _need_out(q_colT, "q_colT", (C, ldq))
    _need_out(s_colT, "s_colT", scale_shape(C, ldq // BLOCK))
    _check(_lib.mxq_quantize_grouped(_ptr(x), T, C, x.stride(0), _ptr(group_end), group_end.numel(),
                                     ldq, axis_mask, _ptr(q_row), _ptr(s_row), _ptr(q_colT),
                                     _ptr(s_colT), _stream(stream, x.device)), "mxq_quantize_grouped")


def mxq_qdq_fp4(x, y, codes=None, scales=None, stream=None):
    """x, y fp32 contiguous, same shape; blocks along the last dim."""
    _need(x, torch.float32, "x")
    _need(y, torch.float32, "y")
    if not (x.is_contiguous() and y.is_contiguous()) or x.shape != y.shape:
        raise ValueError("x and y must be contiguous and of the same shape")
    L = x.shape[-1] if x.dim() else 1
    rows = x.numel() // L if L else 0
    _check(_lib.mxq_qdq_fp4(_ptr(x), _ptr(y), rows, L, _ptr(codes), _ptr(scales),
                            _stream(stream, x.device)), "mxq_qdq_fp4")


def _rows_L(x):
    L = x.shape[-1] if x.dim() else 1
    return (x.numel() // L if L else 0), L


def _need_u8(t, name, shape):
    if t is None:
        return
    _need(t, torch.uint8, name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")


def mxq_qdq_fp4_ex(x, y, scale_factor=6.0, codes=None, scales=None, sat_mask=None, stream=None):
    """As mxq_qdq_fp4 with a runtime scale factor and the optional saturation
    mask uint8 [rows][ceil32(L)/8] (bit j of byte k: element 8k+j clipped)."""
    _need(x, torch.float32, "x")
    _need(y, torch.float32, "y")
    if not (x.is_contiguous() and y.is_contiguous()) or x.shape != y.shape:
        raise ValueError("x and y must be contiguous and of the same shape")
    rows, L = _rows_L(x)
    _need_u8(codes, "codes", (rows, ceil32(L) // 2))
    _need_u8(scales, "scales", (rows, ceil32(L) // BLOCK))
    _need_u8(sat_mask, "sat_mask", (rows, ceil32(L) // 8))
    _check(_lib.mxq_qdq_fp4_ex(_ptr(x), _ptr(y), rows, L, float(scale_factor), _ptr(codes), _ptr(scales),
                               _ptr(sat_mask), _stream(stream, x.device)), "mxq_qdq_fp4_ex")


def mxq_ste_backward_fp4(grad_y, sat_mask, grad_x, stream=None):
    """grad_x = 0 where sat_mask marks a clipped element, grad_y elsewhere."""
    _need(grad_y, torch.float32, "grad_y")
    _need(grad_x, torch.float32, "grad_x")
    if not (grad_y.is_contiguous() and grad_x.is_contiguous()) or grad_y.shape != grad_x.shape:
        raise ValueError("grad_y and grad_x must be contiguous and of the same shape")
    rows, L = _rows_L(grad_y)
    _need_u8(sat_mask, "sat_mask", (rows, ceil32(L) // 8))
    _check(_lib.mxq_ste_backward_fp4(_ptr(grad_y), _ptr(sat_mask), _ptr(grad_x), rows, L,
                                     _stream(stream, grad_y.device)), "mxq_ste_backward_fp4")


def mxq_fp4_scale_threshold(scale_factor):
    """Host only: (F, T) of the exponent rule for this scale factor."""
    F, T = ctypes.c_int32(), ctypes.c_uint32()
    _check(_lib.mxq_fp4_scale_threshold(float(scale_factor), ctypes.byref(F), ctypes.byref(T)),
           "mxq_fp4_scale_threshold")
    return F.value, T.value


def _elems(nbytes: int, fmt: int) -> int:
    """K (elements) of an operand row of `nbytes` code bytes."""
    return nbytes * 2 if fmt == MXQ_FMT_E2M1 else nbytes


def mxq_gemm(A, sA, B, sB, C, stream=None, fmt=MXQ_FMT_E4M3):
    """A uint8 [M][K] + scales scale_shape(M, K/32), B [N][K] + scale_shape(N, K/32) -> C fp32 [M][ldc >= N].
    fmt MXQ_FMT_E2M1: A [M][K/2], B [N][K/2] (two E2M1 codes per byte)."""
    for t, n in ((A, "A"), (sA, "sA"), (B, "B"), (sB, "sB")):
        _need(t, torch.uint8, n)
    _need(C, torch.float32, "C", 2)
    M, Kb = A.shape
    K = _elems(Kb, fmt)
    N = B.shape[0]
    if (B.dim() != 2 or B.shape[1] != Kb or tuple(sA.shape) != scale_shape(M, K // BLOCK)
            or tuple(sB.shape) != scale_shape(N, K // BLOCK)):
        raise ValueError("operand shapes disagree")
    if not all(t.is_contiguous() for t in (A, sA, B, sB)):
        raise ValueError("operands must be contiguous")
    if C.shape[0] != M or C.shape[1] < N or C.stride(1) != 1:
        raise ValueError("C must be [M][>=N] with unit column stride")
    _check(_lib.mxq_gemm(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K, C.stride(0),
                         fmt, _stream(stream, A.device)), "mxq_gemm")


def mxq_grouped_gemm(mode, A, sA, B, sB, C, group_end, stream=None, fmt=MXQ_FMT_E4M3):
    """RAGGED_M: A [M][K], B [G][N][K], C [M][N].  RAGGED_K: A [M][K], B [N][K], C [G][M][N].

    Scales: sA scale_shape(M, K/32); sB (G,) + scale_shape(N, K/32) (ragged M) or scale_shape(N, K/32).
    fmt MXQ_FMT_E2M1: code rows of K/2 bytes (ragged K: from mxq_quantize_fp4_grouped)."""
    for t, n in ((A, "A"), (sA, "sA"), (B, "B"), (sB, "sB")):
        _need(t, torch.uint8, n)
    _need(C, torch.float32, "C")
    _need(group_end, torch.int32, "group_end", 1)
    G = group_end.numel()
    M, Kb = A.shape
    K = _elems(Kb, fmt)
    N = B.shape[-2]
    if mode == MXQ_GG_RAGGED_M:
        ok = (tuple(B.shape) == (G, N, Kb) and tuple(sB.shape) == (G,) + scale_shape(N, K // BLOCK)
              and tuple(C.shape) == (M, N))
    else:
        N = B.shape[0]
        ok = (tuple(B.shape) == (N, Kb) and tuple(sB.shape) == scale_shape(N, K // BLOCK)
              and tuple(C.shape) == (G, M, N))
    if not ok or tuple(sA.shape) != scale_shape(M, K // BLOCK):
        raise ValueError("grouped GEMM operand shapes disagree")
    if not all(t.is_contiguous() for t in (A, sA, B, sB, C)):
        raise ValueError("operands must be contiguous")
    _check(_lib.mxq_grouped_gemm(mode, _ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                 _ptr(group_end), G, fmt, _stream(stream, A.device)),
           "mxq_grouped_gemm")


def mxq_quantize_fp4(x, codes, scales, scale_factor=6.0, stream=None):
    """MXFP4 GEMM operand: x fp32 [rows][L] -> codes uint8 [rows][ceil32(L)/2],
    scales scale_shape(rows, ceil32(L)/32) (the GEMM operand layout)."""
    _need(x, torch.float32, "x")
    if not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D tensor")
    rows, L = x.shape
    _need_u8(codes, "codes", (rows, ceil32(L) // 2))
    _need_u8(scales, "scales", scale_shape(rows, ceil32(L) // BLOCK))
    _check(_lib.mxq_quantize_fp4(_ptr(x), rows, L, float(scale_factor), _ptr(codes), _ptr(scales),
                                 _stream(stream, x.device)), "mxq_quantize_fp4")


def mxq_quantize_fp4_grouped(x, group_end, ldq, codes, scales, scale_factor=6.0, stream=None):
    """Grouped token-axis MXFP4 operand: x fp32 [T][C] (unit column stride) ->
    codes uint8 [C][ldq/2], scales scale_shape(C, ldq/32) (the operand layout)."""
    _need(x, torch.float32, "x", 2)
    _need(group_end, torch.int32, "group_end", 1)
    if x.stride(1) != 1:
        raise ValueError("x must have unit stride along its last dim")
    T, C = x.shape
    _need_u8(codes, "codes", (C, ldq // 2))
    _need_u8(scales, "scales", scale_shape(C, ldq // BLOCK))
    _check(_lib.mxq_quantize_fp4_grouped(_ptr(x), T, C, x.stride(0), _ptr(group_end), group_end.numel(), ldq,
                                         float(scale_factor), _ptr(codes), _ptr(scales), _stream(stream, x.device)),
           "mxq_quantize_fp4_grouped")


def mxq_validate_group_end(group_end, T, flag, stream=None):
    _need(group_end, torch.int32, "group_end", 1)
    _need(flag, torch.int32, "flag")
    _check(_lib.mxq_validate_group_end(_ptr(group_end), group_end.numel(), T, _ptr(flag),
                                       _stream(stream, group_end.device)), "mxq_validate_group_end")


# ---- around the expert GEMMs: routing, combine, optimiser
_DTYPES = {torch.float32: MXQ_DT_F32, torch.bfloat16: MXQ_DT_BF16}
_SCORES = {"softmax": MXQ_SCORE_SOFTMAX, "sigmoid": MXQ_SCORE_SIGMOID, 0: MXQ_SCORE_SOFTMAX, 1: MXQ_SCORE_SIGMOID}


def _matrix(t, name):
    """(type code, rows, columns, row stride) of a float matrix on the device with unit stride along its last dim."""
    try:
        dt = _DTYPES[t.dtype]
        rows, cols = t.shape
        if t.is_cuda:
            stride, unit = t.stride()
            if unit == 1 or cols <= 1:
                # the stride of a dim of size 1 or 0 says nothing
                return dt, rows, cols, stride if rows > 1 or stride > cols else cols
    except (AttributeError, KeyError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {t.dim()}")
    raise ValueError(f"{name} must have unit stride along its last dim")


def _need_array(t, name, dtype, shape):
    """Device tensor of this type and shape, contiguous."""
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


def _type_code(dtype):
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _raw(t):
    return None if t is None else t.data_ptr()


def route_config(top_k, score="softmax", n_group=1, topk_group=1, group_top=1, renormalise=True, scale=1.0):
    """mxq_route_config; score "softmax" or "sigmoid"."""
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r}; one of 'softmax', 'sigmoid'")
    return RouteConfig(_SCORES[score], top_k, n_group, topk_group, group_top, int(bool(renormalise)), float(scale))


_kept_config = functools.lru_cache(maxsize=256)(route_config)  # the helpers' own, never handed out


@functools.lru_cache(maxsize=256)
def mxq_expert_order_workspace(T: int, top_k: int, E: int) -> int:
    return _lib.mxq_expert_order_workspace(T, top_k, E)


def mxq_route(logits, cfg, idx, weights, bias=None, group_end=None, row_token=None, slot=None, workspace=None,
              stream=None):
    """logits fp32 or bf16 [T][E] (unit column stride) -> idx int32, weights fp32 [T][top_k]; with group_end int32
    [E], row_token int32 [T * top_k], slot int32 [T][top_k] and a uint8 workspace the expert order too."""
    dt, T, E, ld = _matrix(logits, "logits")
    K = cfg.top_k
    _need_array(idx, "idx", torch.int32, (T, K))
    _need_array(weights, "weights", torch.float32, (T, K))
    if bias is not None:
        _need_array(bias, "bias", torch.float32, (E,))
    nbytes = _need_order(group_end, row_token, slot, workspace, T, K, E) if group_end is not None else 0
    _check(_lib.mxq_route(logits.data_ptr(), dt, T, E, ld, _raw(bias), ctypes.byref(cfg), idx.data_ptr(),
                          weights.data_ptr(), _raw(group_end), _raw(row_token), _raw(slot), _raw(workspace), nbytes,
                          _stream(stream, logits.device)), "mxq_route")


def _need_order(group_end, row_token, slot, workspace, T, K, E):
    _need_array(group_end, "group_end", torch.int32, (E,))
    _need_array(row_token, "row_token", torch.int32, (T * K,))
    _need_array(slot, "slot", torch.int32, (T, K))
    _need(workspace, torch.uint8, "workspace", 1)
    return workspace.numel()


def mxq_expert_order(idx, E, group_end, row_token, slot, workspace, stream=None):
    """idx int32 [T][top_k] (entries outside [0, E) dropped) -> group_end [E], row_token [T * top_k], slot [T][top_k]."""
    _need(idx, torch.int32, "idx", 2)
    T, K = idx.shape
    _need_array(idx, "idx", torch.int32, (T, K))
    nbytes = _need_order(group_end, row_token, slot, workspace, T, K, E)
    _check(_lib.mxq_expert_order(idx.data_ptr(), T, K, E, group_end.data_ptr(), row_token.data_ptr(), slot.data_ptr(),
                                 workspace.data_ptr(), nbytes, _stream(stream, idx.device)), "mxq_expert_order")


def mxq_route_backward(logits, cfg, idx, dweights, dlogits, stream=None):
    """dweights fp32 [T][top_k] -> dlogits [T][E] of the logits' type, every element written."""
    dt, T, E, ld = _matrix(logits, "logits")
    ddt, rows, cols, ldd = _matrix(dlogits, "dlogits")
    if (ddt, rows, cols) != (dt, T, E):
        raise ValueError("dlogits must have the logits' type and shape")
    _route_backward(logits, dt, T, E, ld, cfg, idx, dweights, dlogits, ldd, stream)


def _route_backward(logits, dt, T, E, ld, cfg, idx, dweights, dlogits, ldd, stream):
    pairs = (T, cfg.top_k)
    _need_array(idx, "idx", torch.int32, pairs)
    _need_array(dweights, "dweights", torch.float32, pairs)
    _check(_lib.mxq_route_backward(logits.data_ptr(), dt, T, E, ld, ctypes.byref(cfg), idx.data_ptr(), dweights.data_ptr(),
                                   dlogits.data_ptr(), ldd, _stream(stream, logits.device)), "mxq_route_backward")


def _need_pairs(slot, weights):
    shape = slot.shape if isinstance(slot, torch.Tensor) else None
    _need_array(slot, "slot", torch.int32, shape)
    if len(shape) != 2:
        raise ValueError(f"slot must have 2 dims, got {len(shape)}")
    if weights is not None:
        _need_array(weights, "weights", torch.float32, shape)
    return shape


def mxq_combine(y, slot, weights, out, stream=None):
    """out[t] = sum_k weights[t][k] * y[slot[t][k]]; y [rows][H], slot int32 [T][top_k], weights fp32 or None, out
    [T][H]; y and out fp32 or bf16 with unit column stride."""
    ydt, rows, H, ldy = _matrix(y, "y")
    odt, tokens, cols, ldo = _matrix(out, "out")
    T, K = _need_pairs(slot, weights)
    if tokens != T or cols != H:
        raise ValueError(f"out must have shape {(T, H)}, got {tuple(out.shape)}")
    _combine(y, ydt, rows, ldy, slot, weights, T, K, H, out, odt, ldo, stream)


def _combine(y, ydt, rows, ldy, slot, weights, T, K, H, out, odt, ldo, stream):
    _check(_lib.mxq_combine(y.data_ptr(), ydt, rows, ldy, slot.data_ptr(), _raw(weights), T, K, H, out.data_ptr(), odt, ldo,
                            _stream(stream, out.device)), "mxq_combine")


def mxq_combine_backward(dout, slot, rows, dy=None, dweights=None, weights=None, y=None, stream=None):
    """dy[slot[t][k]] = weights[t][k] * dout[t] ([rows][H]); dweights[t][k] = <dout[t], y[slot[t][k]]> (needs y)."""
    dt, T, K, H, ldd, ydt, ldy = _need_gradient(dout, slot, rows, weights, y)
    gdt, ldg = dt, 0
    if dy is not None:
        gdt, n, cols, ldg = _matrix(dy, "dy")
        if n != rows or cols != H:
            raise ValueError(f"dy must have shape {(rows, H)}, got {tuple(dy.shape)}")
    if dweights is not None:
        _need_array(dweights, "dweights", torch.float32, (T, K))
        if y is None:
            raise ValueError("dweights needs y")
    _combine_backward(dout, dt, ldd, y, ydt, ldy, slot, weights, T, K, H, rows, dy, gdt, ldg, dweights, stream)


def _need_gradient(dout, slot, rows, weights, y):
    dt, tokens, H, ldd = _matrix(dout, "dout")
    T, K = _need_pairs(slot, weights)
    if tokens != T:
        raise ValueError(f"dout must have {T} rows, got {tokens}")
    ydt, ldy = dt, 0
    if y is not None:
        ydt, n, cols, ldy = _matrix(y, "y")
        if n != rows or cols != H:
            raise ValueError(f"y must have shape {(rows, H)}, got {tuple(y.shape)}")
    return dt, T, K, H, ldd, ydt, ldy


def _combine_backward(dout, dt, ldd, y, ydt, ldy, slot, weights, T, K, H, rows, dy, gdt, ldg, dweights, stream):
    _check(_lib.mxq_combine_backward(dout.data_ptr(), dt, ldd, _raw(y), ydt, ldy, slot.data_ptr(), _raw(weights), T, K, H, rows,
                                     _raw(dy), gdt, ldg, _raw(dweights), _stream(stream, dout.device)),
           "mxq_combine_backward")


def mxq_adamw(tensors, n_tensors, param_dt, grad_dt, fmt, cfg, control=None, stream=None, device=None):
    """tensors: a ctypes array of AdamWTensor (see the AdamW class, which fills one from torch tensors)."""
    _check(_lib.mxq_adamw(tensors, n_tensors, param_dt, grad_dt, fmt, ctypes.byref(cfg), _raw(control),
                          _stream(stream, device)), "mxq_adamw")


# ---- FP8 with an fp32 scale for each block of 128
def ceil128(v: int) -> int:
    return (v + BLOCK128 - 1) // BLOCK128 * BLOCK128


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_device_count = functools.lru_cache(maxsize=None)(torch.cuda.device_count)
_U8, _F32 = torch.uint8, torch.float32


def _stream_here(stream, t, name, *others):
    """Handle of the stream, or of the current one of t's device, which the entry points need to be the current device; the
    others (or None) have to be there too."""
    index = 0
    if _device_count() != 1:  # (with one there is nothing to check, and small products wait for the host)
        index = t.get_device()
        if index != _current_device():
            raise ValueError(f"{name} is on {t.device}, not on the current device")
        for o in others:
            if o is not None and o.get_device() != index:
                raise ValueError(f"{name} is on {t.device}, another tensor on {o.device}")
    if stream is None and _current_stream is not None:
        return _current_stream(index)
    return _stream(stream, t.device)


def _copy128_shapes(R, C, tile, lead=(), ldq=None):
    """Shapes of the row copy's codes and scales and of the colT copy's."""
    Rp = ceil128(R) if ldq is None else ldq
    Cb = (C + BLOCK128 - 1) // BLOCK128
    return ((*lead, R, Cb * BLOCK128), (*lead, Cb, -(-R // tile)), (*lead, C, Rp), (*lead, Rp // BLOCK128, -(-C // tile)))


def _need_copies128(axis_mask, shapes, q_row, s_row, q_colT, s_colT):
    if axis_mask & MXQ_AXIS_ROW:
        _need_array(q_row, "q_row", _U8, shapes[0])
        _need_array(s_row, "s_row", _F32, shapes[1])
    if axis_mask & MXQ_AXIS_COLT:
        _need_array(q_colT, "q_colT", _U8, shapes[2])
        _need_array(s_colT, "s_colT", _F32, shapes[3])


def mxq_grouped128_cols_max(T: int, G: int) -> int:
    return _lib.mxq_grouped128_cols_max(T, G)


def mxq_quantize128(x, tile, axis_mask, q_row=None, s_row=None, q_colT=None, s_colT=None, stream=None):
    """x fp32 or bf16 [R][C] or [batch][R][C] (unit column stride) in blocks of tile x 128: q_row uint8 [R][ceil128(C)],
    s_row fp32 [C / 128][R / tile], q_colT [C][ceil128(R)], s_colT [R / 128][C / tile], each under [batch] for three dims."""
    if tile not in (1, 128):
        raise ValueError(f"tile must be 1 or 128, got {tile}")
    nb, batch_stride, lead = 1, 0, ()
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        nb, R, C = x.shape
        batch_stride, lead = x.stride(0), (nb,)
        dt, _, _, ldx = _matrix(x[0] if nb else x.new_empty((R, C)), "x")
    else:
        dt, R, C, ldx = _matrix(x, "x")
    _need_copies128(axis_mask, _copy128_shapes(R, C, tile, lead), q_row, s_row, q_colT, s_colT)
    _check(_lib.mxq_quantize128(x.data_ptr(), dt, nb, R, C, ldx, batch_stride, tile, axis_mask, _raw(q_row), _raw(s_row),
                                _raw(q_colT), _raw(s_colT), _stream_here(stream, x, "x", q_row, s_row, q_colT, s_colT)), "mxq_quantize128")


def mxq_quantize128_grouped(x, group_end, ldq, axis_mask, q_row=None, s_row=None, q_colT=None, s_colT=None, stream=None):
    """x fp32 or bf16 [T][C], rows in groups: q_colT uint8 [C][ldq], s_colT fp32 [ldq / 128][C], the blocks restarting with
    each group; q_row, s_row as mxq_quantize128's of all rows."""
    dt, T, C, ldx = _matrix(x, "x")
    G = _need_groups(group_end)
    _need_copies128(axis_mask, _copy128_shapes(T, C, 1, ldq=ldq), q_row, s_row, q_colT, s_colT)
    _check(_lib.mxq_quantize128_grouped(x.data_ptr(), dt, T, C, ldx, group_end.data_ptr(), G, ldq, axis_mask, _raw(q_row),
                                        _raw(s_row), _raw(q_colT), _raw(s_colT),
                                        _stream_here(stream, x, "x", group_end, q_row, s_row, q_colT, s_colT)), "mxq_quantize128_grouped")


def _need_groups(group_end):
    _need(group_end, torch.int32, "group_end", 1)
    _need_array(group_end, "group_end", torch.int32, group_end.shape)
    return group_end.shape[0]


def _need_operand128(codes, scales, name, lead=(), tiles=(1,)):
    """(rows, K, tile) of an operand's codes [lead.., rows, K] and scales [lead.., K / 128, rows / tile], tile one of `tiles`."""
    try:
        if codes.dtype is _U8 and scales.dtype is _F32 and codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous():
            shape, rows_of = codes.shape, scales.shape
            if len(shape) == len(rows_of) == 2 + len(lead) and (not lead or (shape[:-2] == lead and rows_of[:-2] == lead)):
                rows, K = shape[-2:]
                blocks, n = rows_of[-2:]
                if blocks * BLOCK128 == K:
                    for tile in tiles:
                        if n == (rows + tile - 1) // tile:
                            return rows, K, tile
    except (AttributeError, ValueError):
        pass
    _need(codes, _U8, name)
    if codes.dim() != 2 + len(lead) or tuple(codes.shape[:-2]) != lead or not codes.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {(*lead, 'rows', 'K')}, got {tuple(codes.shape)}")
    rows, K = codes.shape[-2:]
    _need(scales, _F32, "s" + name)
    want = " or ".join(str((*lead, K // BLOCK128, -(-rows // tile))) for tile in tiles)
    raise ValueError(f"s{name} must be a contiguous tensor of shape {want}, got {tuple(scales.shape)} (K a multiple of 128: {K})")


def _need_operands128(A, sA, B, sB):
    M, K, _ = _need_operand128(A, sA, "A")
    N, KB, tile = _need_operand128(B, sB, "B", tiles=(128, 1))
    if KB != K:
        raise ValueError(f"operand shapes disagree: A {tuple(A.shape)}, B {tuple(B.shape)}")
    return M, N, K, tile


def mxq_gemm128(A, sA, B, sB, C, stream=None):
    """A uint8 [M][K], sA fp32 [K / 128][M]; B [N][K], sB [K / 128][N] or [K / 128][ceil(N / 128)] -> C fp32 or bf16 [M][N]."""
    M, N, K, tile = _need_operands128(A, sA, B, sB)
    cdt, rows, cols, ldc = _matrix(C, "C")
    if rows != M or cols != N:
        raise ValueError(f"C must have shape {(M, N)}, got {tuple(C.shape)}")
    _gemm128(A, sA, B, sB, tile, C, cdt, M, N, K, ldc, stream)


def _gemm128(A, sA, B, sB, tile, C, cdt, M, N, K, ldc, stream):
    _check(_lib.mxq_gemm128(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), tile, C.data_ptr(), cdt, M, N, K, ldc,
                            _stream_here(stream, A, "A", sA, B, sB, C)), "mxq_gemm128")


def _need_grouped128(mode, A, sA, B, sB, group_end):
    """(M, N, K, G, shape of C)."""
    G = _need_groups(group_end)
    M, K, _ = _need_operand128(A, sA, "A")
    ragged_m = mode == MXQ_GG_RAGGED_M
    N, KB, _ = _need_operand128(B, sB, "B", (G,), (128,)) if ragged_m else _need_operand128(B, sB, "B")
    if KB != K:
        raise ValueError(f"operand shapes disagree: A {tuple(A.shape)}, B {tuple(B.shape)}")
    return M, N, K, G, (M, N) if ragged_m else (G, M, N)


def mxq_grouped_gemm128(mode, A, sA, B, sB, C, group_end, stream=None):
    """RAGGED_M: A [M][K], B [G][N][K] in 128 x 128 blocks, C [M][N].  RAGGED_K: A [M][K], B [N][K], C [G][M][N].  C fp32 or
    bf16."""
    M, N, K, G, shape = _need_grouped128(mode, A, sA, B, sB, group_end)
    _need_array(C, "C", C.dtype if isinstance(C, torch.Tensor) and C.dtype in _DTYPES else _F32, shape)
    _grouped_gemm128(mode, A, sA, B, sB, C, M, N, K, group_end, G, stream)


def _grouped_gemm128(mode, A, sA, B, sB, C, M, N, K, group_end, G, stream):
    _check(_lib.mxq_grouped_gemm128(mode, A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), C.data_ptr(), _DTYPES[C.dtype],
                                    M, N, K, group_end.data_ptr(), G, _stream_here(stream, A, "A", sA, B, sB, C, group_end)),
           "mxq_grouped_gemm128")


# ---- orthogonalised updates
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7):
    """mxq_newton_schulz."""
    return NewtonSchulz(*coefficients, eps, steps)


@functools.lru_cache(maxsize=256)
def mxq_orthogonalize_workspace(batch: int, R: int, C: int, odt: int) -> int:
    return _lib.mxq_orthogonalize_workspace(batch, R, C, odt)


def _matrices(t, name):
    """(type code, batch, R, C) of contiguous float matrices [R][C] or [batch][R][C] on the device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() not in (2, 3) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with 2 or 3 dims, got shape {tuple(t.shape)}")
    return (_DTYPES[t.dtype], 1, *t.shape) if t.dim() == 2 else (_DTYPES[t.dtype], *t.shape)


def mxq_orthogonalize(x, cfg, out, workspace, stream=None):
    """x fp32 or bf16 [R][C] or [batch][R][C], contiguous -> out of its shape, fp32 or bf16; workspace uint8."""
    dt, nb, R, C = _matrices(x, "x")
    odt = _matrices(out, "out")[0]
    if out.shape != x.shape:
        raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    _need(workspace, torch.uint8, "workspace", 1)
    _check(_lib.mxq_orthogonalize(x.data_ptr(), dt, nb, R, C, ctypes.byref(cfg), out.data_ptr(), odt, workspace.data_ptr(),
                                  workspace.numel(), _stream_here(stream, x, "x", out, workspace)), "mxq_orthogonalize")


def mxq_muon(param, grad, m, cfg, workspace, copy=None, control=None, stream=None):
    """One Muon step of param [R][C] or [batch][R][C] (see the Muon class)."""
    pdt, nb, R, C = _matrices(param, "param")
    gdt = _matrices(grad, "grad")[0]
    _need_array(m, "m", torch.float32, param.shape)
    if grad.shape != param.shape:
        raise ValueError(f"grad must have shape {tuple(param.shape)}, got {tuple(grad.shape)}")
    if copy is not None:
        _need_array(copy, "copy", torch.bfloat16, param.shape)
    if control is not None:
        _need_array(control, "control", torch.int32, (4,))
    _need(workspace, torch.uint8, "workspace", 1)
    _check(_lib.mxq_muon(param.data_ptr(), pdt, grad.data_ptr(), gdt, m.data_ptr(), _raw(copy), nb, R, C, ctypes.byref(cfg),
                         _raw(control), workspace.data_ptr(), workspace.numel(),
                         _stream_here(stream, param, "param", grad, m, copy, control, workspace)), "mxq_muon")


# ------------------------------------------------------------------ allocate-and-call helpers
def _on(stream, device):
    """Context in which `stream` is the current one, so that what is allocated belongs to it.  A helper that is given a
    stream runs as a call within it: outputs of another stream's memory could still be in use there, or be handed
    out again there before the call has ended."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), device)
    return torch.cuda.stream(stream)


def _u8(shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def quantize(x, axis_mask=MXQ_AXIS_ROW | MXQ_AXIS_COLT, stream=None):
    """Returns a dict with 'q_row', 's_row' and/or 'q_colT', 's_colT'."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize(x, axis_mask)
    R, C = x.shape
    out = {}
    if axis_mask & MXQ_AXIS_ROW:
        out["q_row"] = _u8((R, ceil32(C)), x.device)
        out["s_row"] = _u8(scale_shape(R, ceil32(C) // BLOCK), x.device)
    if axis_mask & MXQ_AXIS_COLT:
        out["q_colT"] = _u8((C, ceil32(R)), x.device)
        out["s_colT"] = _u8(scale_shape(C, ceil32(R) // BLOCK), x.device)
    mxq_quantize(x, axis_mask, out.get("q_row"), out.get("s_row"), out.get("q_colT"),
                 out.get("s_colT"))
    return out


def quantize_batched(x, axis_mask=MXQ_AXIS_ROW | MXQ_AXIS_COLT, stream=None):
    """x bf16 [batch][R][C] -> dict of batched outputs (see mxq_quantize_batched)."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize_batched(x, axis_mask)
    nb, R, C = x.shape
    out = {}
    if axis_mask & MXQ_AXIS_ROW:
        out["q_row"] = _u8((nb, R, ceil32(C)), x.device)
        out["s_row"] = _u8((nb,) + scale_shape(R, ceil32(C) // BLOCK), x.device)
    if axis_mask & MXQ_AXIS_COLT:
        out["q_colT"] = _u8((nb, C, ceil32(R)), x.device)
        out["s_colT"] = _u8((nb,) + scale_shape(C, ceil32(R) // BLOCK), x.device)
    mxq_quantize_batched(x, axis_mask, out.get("q_row"), out.get("s_row"), out.get("q_colT"), out.get("s_colT"))
    return out


def quantize_grouped(x, group_end, axis_mask=MXQ_AXIS_COLT, ldq=None, stream=None):
    if stream is not None:
        with _on(stream, x.device):
            return quantize_grouped(x, group_end, axis_mask, ldq)
    T, C = x.shape
    if ldq is None:
        ldq = mxq_grouped_cols_max(T, group_end.numel())
    out = {"ldq": ldq}
    if axis_mask & MXQ_AXIS_ROW:
        out["q_row"] = _u8((T, ceil32(C)), x.device)
        out["s_row"] = _u8(scale_shape(T, ceil32(C) // BLOCK), x.device)
    if axis_mask & MXQ_AXIS_COLT:
        out["q_colT"] = _u8((C, ldq), x.device)
        out["s_colT"] = _u8(scale_shape(C, ldq // BLOCK), x.device)
    mxq_quantize_grouped(x, group_end, ldq, axis_mask, out.get("q_row"), out.get("s_row"),
                         out.get("q_colT"), out.get("s_colT"))
    return out


def qdq_fp4(x, want_codes=False, stream=None):
    if stream is not None:
        with _on(stream, x.device):
            return qdq_fp4(x, want_codes)
    y = torch.empty_like(x)
    codes = scales = None
    if want_codes:
        L = x.shape[-1]
        rows = x.numel() // L
        codes = _u8((rows, ceil32(L) // 2), x.device)
        scales = _u8((rows, ceil32(L) // BLOCK), x.device)
    mxq_qdq_fp4(x, y, codes, scales)
    return (y, codes, scales) if want_codes else y


def quantize_fp4(x, scale_factor=6.0, stream=None):
    """MXFP4 GEMM operand of a 2-D fp32 tensor: (codes, scales in the operand layout)."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize_fp4(x, scale_factor)
    rows, L = x.shape
    codes = _u8((rows, ceil32(L) // 2), x.device)
    scales = _u8(scale_shape(rows, ceil32(L) // BLOCK), x.device)
    mxq_quantize_fp4(x, codes, scales, scale_factor)
    return codes, scales


def quantize_fp4_grouped(x, group_end, ldq=None, scale_factor=6.0, stream=None):
    """Grouped token-axis MXFP4 operand of x fp32 [T][C]: {"ldq", "codes", "scales"}."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize_fp4_grouped(x, group_end, ldq, scale_factor)
    T, C = x.shape
    if ldq is None:
        ldq = mxq_grouped_cols_max(T, group_end.numel())
    out = {"ldq": ldq, "codes": _u8((C, ldq // 2), x.device), "scales": _u8(scale_shape(C, ldq // BLOCK), x.device)}
    mxq_quantize_fp4_grouped(x, group_end, ldq, out["codes"], out["scales"], scale_factor)
    return out


def qdq_fp4_ste(x, scale_factor=6.0, want_codes=False, stream=None):
    """Forward of the clipped-STE fake quantiser: returns (y, sat_mask) or,
    with want_codes, (y, sat_mask, codes, scales)."""
    if stream is not None:
        with _on(stream, x.device):
            return qdq_fp4_ste(x, scale_factor, want_codes)
    rows, L = _rows_L(x)
    y = torch.empty_like(x)
    mask = _u8((rows, ceil32(L) // 8), x.device)
    codes = scales = None
    if want_codes:
        codes = _u8((rows, ceil32(L) // 2), x.device)
        scales = _u8((rows, ceil32(L) // BLOCK), x.device)
    mxq_qdq_fp4_ex(x, y, scale_factor, codes, scales, mask)
    return (y, mask, codes, scales) if want_codes else (y, mask)


def ste_backward_fp4(grad_y, sat_mask, stream=None):
    if stream is not None:
        with _on(stream, grad_y.device):
            return ste_backward_fp4(grad_y, sat_mask)
    grad_x = torch.empty_like(grad_y)
    mxq_ste_backward_fp4(grad_y, sat_mask, grad_x)
    return grad_x


def gemm(A, sA, B, sB, stream=None, fmt=MXQ_FMT_E4M3):
    if stream is not None:
        with _on(stream, A.device):
            return gemm(A, sA, B, sB, fmt=fmt)
    C = torch.empty((A.shape[0], B.shape[0]), dtype=torch.float32, device=A.device)
    mxq_gemm(A, sA, B, sB, C, fmt=fmt)
    return C


def grouped_gemm(mode, A, sA, B, sB, group_end, stream=None, fmt=MXQ_FMT_E4M3):
    if stream is not None:
        with _on(stream, A.device):
            return grouped_gemm(mode, A, sA, B, sB, group_end, fmt=fmt)
    if mode == MXQ_GG_RAGGED_M:
        C = torch.empty((A.shape[0], B.shape[1]), dtype=torch.float32, device=A.device)
    else:
        C = torch.empty((group_end.numel(), A.shape[0], B.shape[0]), dtype=torch.float32, device=A.device)
    mxq_grouped_gemm(mode, A, sA, B, sB, C, group_end, fmt=fmt)
    return C


def _workspace(T, top_k, E, device):
    return torch.empty(mxq_expert_order_workspace(T, top_k, E), dtype=torch.uint8, device=device)


def route(logits, top_k, *, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalise=True, scale=1.0,
          order=True, out=None, stream=None):
    """Route tokens: {"idx", "weights"} and, with order, {"group_end", "row_token", "slot"} (the expert order the grouped
    entry points and combine take).  out: a dict of such buffers to write to; with order, it may have the "workspace" too,
    which is put there for the calls after where it is missing.  stream: as a call within torch.cuda.stream(stream), whose
    memory the outputs then are."""
    if stream is not None:
        with _on(stream, logits.device):
            return route(logits, top_k, score=score, bias=bias, n_group=n_group, topk_group=topk_group, group_top=group_top,
                         renormalise=renormalise, scale=scale, order=order, out=out)
    cfg = _kept_config(top_k, score, n_group, topk_group, group_top, renormalise, scale)
    T, E = logits.shape
    if out is None:
        i32 = functools.partial(torch.empty, dtype=torch.int32, device=logits.device)
        out = {"idx": i32((T, top_k)), "weights": torch.empty((T, top_k), dtype=torch.float32, device=logits.device)}
        if order:
            out.update(group_end=i32((E,)), row_token=i32((T * top_k,)), slot=i32((T, top_k)))
    idx, weights = out["idx"], out["weights"]
    if not order:
        mxq_route(logits, cfg, idx, weights, bias)
        return {"idx": idx, "weights": weights}
    group_end, row_token, slot, ws = out["group_end"], out["row_token"], out["slot"], out.get("workspace")
    if ws is None:
        ws = out["workspace"] = _workspace(T, top_k, E, logits.device)
    mxq_route(logits, cfg, idx, weights, bias, group_end, row_token, slot, ws)
    return {"idx": idx, "weights": weights, "group_end": group_end, "row_token": row_token, "slot": slot}


def expert_order(idx, E, stream=None):
    """Expert order of chosen experts idx int32 [T][top_k]: {"group_end", "row_token", "slot"}."""
    if stream is not None:
        with _on(stream, idx.device):
            return expert_order(idx, E)
    T, K = idx.shape
    i32 = functools.partial(torch.empty, dtype=torch.int32, device=idx.device)
    out = {"group_end": i32((E,)), "row_token": i32((T * K,)), "slot": i32((T, K))}
    mxq_expert_order(idx, E, out["group_end"], out["row_token"], out["slot"], _workspace(T, K, E, idx.device))
    return out


def route_backward(logits, idx, dweights, *, score="softmax", renormalise=True, scale=1.0, stream=None):
    """Gradient of route's weights with respect to the logits."""
    if stream is not None:
        with _on(stream, logits.device):
            return route_backward(logits, idx, dweights, score=score, renormalise=renormalise, scale=scale)
    cfg = _kept_config(idx.shape[1], score, 1, 1, 1, renormalise, scale)
    dt, T, E, ld = _matrix(logits, "logits")
    dlogits = logits.new_empty((T, E))
    _route_backward(logits, dt, T, E, ld, cfg, idx, dweights, dlogits, E, None)
    return dlogits


def combine(y, slot, weights=None, dtype=torch.bfloat16, stream=None):
    """The experts' rows y [rows][H] back in token order: [T][H] of `dtype`."""
    if stream is not None:
        with _on(stream, y.device):
            return combine(y, slot, weights, dtype)
    ydt, rows, H, ldy = _matrix(y, "y")
    T, K = _need_pairs(slot, weights)
    odt = _type_code(dtype)
    out = y.new_empty((T, H), dtype=dtype)
    _combine(y, ydt, rows, ldy, slot, weights, T, K, H, out, odt, H, None)
    return out


def combine_backward(dout, slot, rows, weights=None, y=None, dtype=None, stream=None):
    """(dy [rows][H] of `dtype` (dout's), dweights [T][top_k]); dweights is None without y or weights.  Rows of dy that no
    slot names are not written (mxq_combine_backward takes a dy that the caller has filled)."""
    if stream is not None:
        with _on(stream, dout.device):
            return combine_backward(dout, slot, rows, weights, y, dtype)
    if weights is None:
        y = None
    dt, T, K, H, ldd, ydt, ldy = _need_gradient(dout, slot, rows, weights, y)
    gdt = dt if dtype is None else _type_code(dtype)
    dy = dout.new_empty((rows, H), dtype=dtype)
    dw = None if y is None else torch.empty_like(weights)
    _combine_backward(dout, dt, ldd, y, ydt, ldy, slot, weights, T, K, H, rows, dy, gdt, H, dw, None)
    return dy, dw


def dispatch(x, slot, rows, dtype=None, stream=None):
    """Tokens x [T][H] in expert order: row slot[t][k] of the result is x[t], and rows that no slot names (those past
    the last group end) are not written.  Its gradient is combine without weights."""
    return combine_backward(x, slot, rows, dtype=dtype, stream=stream)[0]


_COPY_NAMES = ((), ("q_row", "s_row"), ("q_colT", "s_colT"), ("q_row", "s_row", "q_colT", "s_colT"))


def _copies128(axis_mask, shapes, x, out):
    """The requested copies, from `out` where it is given."""
    names = _COPY_NAMES[axis_mask & 3]
    if out is not None:
        return {n: out[n] for n in names}
    of = dict(zip(("q_row", "s_row", "q_colT", "s_colT"), shapes()))
    return {n: x.new_empty(of[n], dtype=_U8 if n[0] == "q" else _F32) for n in names}


def quantize128(x, axis_mask=MXQ_AXIS_ROW, tile=1, out=None, stream=None):
    """Blocks of tile x 128 (tile 1: activations and gradients, 128: weights) of x [R][C] or [batch][R][C], fp32 or bf16: a dict
    with 'q_row', 's_row' and/or 'q_colT', 's_colT' (see mxq_quantize128).  out: a dict of such buffers to write to."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize128(x, axis_mask, tile, out)
    got = _copies128(axis_mask, lambda: _copy128_shapes(*x.shape[-2:], tile, tuple(x.shape[:-2])), x, out)
    mxq_quantize128(x, tile, axis_mask, **got)
    return got


def quantize128_grouped(x, group_end, axis_mask=MXQ_AXIS_COLT, ldq=None, out=None, stream=None):
    """Blocks of 1 x 128 of x [T][C] whose rows are in groups (see mxq_quantize128_grouped): a dict with the copies, as
    quantize128's, and "ldq"."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize128_grouped(x, group_end, axis_mask, ldq, out)
    if ldq is None:
        ldq = out["q_colT"].shape[1] if out is not None and "q_colT" in out else mxq_grouped128_cols_max(x.shape[0], group_end.numel())
    got = _copies128(axis_mask, lambda: _copy128_shapes(*x.shape, 1, ldq=ldq), x, out)
    mxq_quantize128_grouped(x, group_end, ldq, axis_mask, **got)
    got["ldq"] = ldq
    return got


def gemm128(A, sA, B, sB, dtype=torch.bfloat16, stream=None):
    """A B^T of operands with fp32 scales for blocks of 128 (see mxq_gemm128): [M][N] of `dtype`."""
    if stream is not None:
        with _on(stream, A.device):
            return gemm128(A, sA, B, sB, dtype)
    cdt = _type_code(dtype)
    M, N, K, tile = _need_operands128(A, sA, B, sB)
    C = sA.new_empty((M, N), dtype=dtype)
    _gemm128(A, sA, B, sB, tile, C, cdt, M, N, K, N, None)
    return C


def grouped_gemm128(mode, A, sA, B, sB, group_end, dtype=torch.bfloat16, stream=None):
    """Grouped products (see mxq_grouped_gemm128): [M][N] or [G][M][N] of `dtype`."""
    if stream is not None:
        with _on(stream, A.device):
            return grouped_gemm128(mode, A, sA, B, sB, group_end, dtype)
    _type_code(dtype)
    M, N, K, G, shape = _need_grouped128(mode, A, sA, B, sB, group_end)
    C = sA.new_empty(shape, dtype=dtype)
    _grouped_gemm128(mode, A, sA, B, sB, C, M, N, K, group_end, G, None)
    return C


def adamw_state(param, fmt=MXQ_ADAMW_MXFP8):
    """One moment of a parameter before the first step: fp32 zeros, or (codes, scales) of MXFP8."""
    if fmt == MXQ_ADAMW_F32:
        return torch.zeros(param.shape, dtype=torch.float32, device=param.device)
    zeros = functools.partial(torch.zeros, dtype=torch.uint8, device=param.device)
    return zeros(param.shape), zeros((ceil32(param.numel()) // BLOCK,))


def adamw_control(lr, step, seed=0, grad_scale=1.0, out=None, device="cuda"):
    """mxq_adamw_control in device memory (int32 [4]); `out`: such a tensor to overwrite, as between graph replays."""
    host = torch.tensor(struct.unpack("4i", struct.pack("2fiI", lr, grad_scale, step, seed)), dtype=torch.int32)
    return host.to(device) if out is None else out.copy_(host)


class AdamW:
    """AdamW steps of a list of tensors (mxq_adamw).

    params fp32 or bf16, grads fp32 or bf16, m and v the moments: fp32 tensors, or (codes, scales) pairs of uint8 tensors
    (MXFP8; v holds sqrt of the second moment) as adamw_state makes them.  copies: bf16 tensors that get the new
    parameters too, or None.  decay_scales: per tensor, times the weight decay.  The tensors stay the caller's: they are
    read and written where they are, so a gradient that moves to other storage needs a new AdamW."""

    def __init__(self, params, grads, m, v, copies=None, decay_scales=None):
        n = len(params)
        if not (len(grads) == len(m) == len(v) == n) or any(x is not None and len(x) != n for x in (copies, decay_scales)):
            raise ValueError("params, grads, m, v, copies and decay_scales must be of one length")
        self.device = params[0].device if n else None
        self.param_dt = self.grad_dt = MXQ_DT_F32
        self.fmt = MXQ_ADAMW_MXFP8 if n and isinstance(m[0], (tuple, list)) else MXQ_ADAMW_F32
        self.tensors = (AdamWTensor * max(n, 1))()
        self.n = n
        self.keep = (list(params), list(grads), list(m), list(v), copies and list(copies))
        for i, p in enumerate(params):
            name = f"tensor {i}: "
            pdt = self._need(p, name + "param", p, _DTYPES)
            gdt = self._need(grads[i], name + "grad", p, _DTYPES)
            if i == 0:
                self.param_dt, self.grad_dt = pdt, gdt
            elif (pdt, gdt) != (self.param_dt, self.grad_dt):
                raise TypeError(name + "all parameters must be of one type, and all gradients")
            d = self.tensors[i]
            for field, x in (("m", m[i]), ("v", v[i])):
                if isinstance(x, (tuple, list)) != (self.fmt == MXQ_ADAMW_MXFP8):
                    raise TypeError(name + "all states must be of one format")
                if self.fmt == MXQ_ADAMW_MXFP8:
                    x, scale = x
                    _need_array(scale, name + field + " scales", torch.uint8, (ceil32(p.numel()) // BLOCK,))
                    setattr(d, field + "_scale", scale.data_ptr())
                self._need(x, name + field, p, {torch.uint8 if self.fmt == MXQ_ADAMW_MXFP8 else torch.float32: 0})
                setattr(d, field, x.data_ptr())
            if copies is not None and copies[i] is not None:
                self._need(copies[i], name + "copy", p, {torch.bfloat16: 0})
                d.copy = copies[i].data_ptr()
            d.param, d.grad, d.n = p.data_ptr(), grads[i].data_ptr(), p.numel()
            d.decay_scale = 1.0 if decay_scales is None else float(decay_scales[i])

    @staticmethod
    def _need(t, name, like, types):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype not in types:
            raise TypeError(f"{name} must be {' or '.join(str(k) for k in types)}, got {t.dtype}")
        if not t.is_cuda or t.device != like.device:
            raise ValueError(f"{name} must be a device tensor, on its parameter's device")
        if t.numel() != like.numel() or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with {like.numel()} elements")
        return types[t.dtype]

    def step(self, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, step=1, grad_scale=1.0, seed=0, control=None,
             stream=None):
        """One step.  control: an adamw_control tensor whose lr, step, seed and grad_scale replace these (for graphs)."""
        if control is not None:
            _need_array(control, "control", torch.int32, (4,))
        if not self.n:
            return
        cfg = AdamWConfig(lr, betas[0], betas[1], eps, weight_decay, grad_scale, step, seed & 0xFFFFFFFF)
        mxq_adamw(self.tensors, self.n, self.param_dt, self.grad_dt, self.fmt, cfg, control, stream, self.device)


def _orthogonalize_workspace(batch, R, C, odt, device):
    return torch.empty(mxq_orthogonalize_workspace(batch, R, C, odt), dtype=torch.uint8, device=device)


def orthogonalize(x, steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7, dtype=torch.bfloat16, stream=None):
    """Newton-Schulz iterations on each matrix of x [R][C] or [batch][R][C] (see mxq_orthogonalize): a result of `dtype`, fp32
    with three times the products of bf16."""
    if stream is not None:
        with _on(stream, x.device):
            return orthogonalize(x, steps, coefficients, eps, dtype)
    odt = _type_code(dtype)
    _, nb, R, C = _matrices(x, "x")
    out = torch.empty_like(x, dtype=dtype)
    mxq_orthogonalize(x, newton_schulz(steps, coefficients, eps), out, _orthogonalize_workspace(nb, R, C, odt, x.device))
    return out


def muon_scale(shape, rule="match_rms"):
    """What an orthogonalised update of a weight [.., R][C] is multiplied by: 0.2 sqrt(max(R, C)), with which its elements are
    about the size of an AdamW update's ("match_rms"), or sqrt(max(1, R / C)) ("original")."""
    R, C = shape[-2:]
    if rule == "match_rms":
        return 0.2 * max(R, C) ** 0.5
    if rule == "original":
        return max(1.0, R / C) ** 0.5
    raise ValueError(f"unknown rule {rule!r}; one of 'match_rms', 'original'")


class Muon:
    """Muon steps of a list of weights (mxq_muon), each [R][C] or a stack [batch][R][C] of such (experts).

    params fp32 or bf16, grads fp32 or bf16, m the momenta (fp32, zeros before the first step), copies: bf16 tensors that get
    the new parameters too, or None.  The tensors stay the caller's: they are read and written where they are, so a gradient
    that moves to other storage needs a new Muon.  They are updated one after the other, in a workspace that each step
    allocates on its stream: it goes back to that stream's pool when the step has been queued, or stays the graph's where
    the step is captured (torch.cuda.graph), so a Muon need not outlive its steps."""

    def __init__(self, params, grads, m, copies=None):
        n = len(params)
        if not (len(grads) == len(m) == n) or (copies is not None and len(copies) != n):
            raise ValueError("params, grads, m and copies must be of one length")
        copies = [None] * n if copies is None else list(copies)
        need = 1
        for i, p in enumerate(params):
            name = f"tensor {i}: "
            pdt, nb, R, C = _matrices(p, name + "param")
            _matrices(grads[i], name + "grad")
            _need_array(m[i], name + "m", torch.float32, p.shape)
            if copies[i] is not None:
                _need_array(copies[i], name + "copy", torch.bfloat16, p.shape)
            if grads[i].shape != p.shape:
                raise ValueError(f"{name}grad must have shape {tuple(p.shape)}, got {tuple(grads[i].shape)}")
            if any(t is not None and t.device != params[0].device for t in (p, grads[i], m[i], copies[i])):
                raise ValueError(f"{name}all tensors must be on one device")
            room = mxq_orthogonalize_workspace(max(nb, 1), R, C, pdt)
            if room == 0:  # (what a step refuses, before it has updated the tensors before)
                raise ValueError(f"{name}matrices must have 1 to 2^20 rows and columns, in stacks of at most 65535, got {tuple(p.shape)}")
            need = max(need, room)
        self.tensors = list(zip(params, grads, m, copies))
        self.workspace_bytes = need

    def step(self, *, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.1, scale="match_rms", grad_scale=1.0, steps=5,
             coefficients=NS_COEFFICIENTS, eps=1e-7, control=None, stream=None):
        """One step.  scale: a rule of muon_scale or a number.  control: an adamw_control tensor whose lr and grad_scale replace
        these (for graphs)."""
        if not self.tensors:
            return
        device = self.tensors[0][0].device
        with contextlib.nullcontext() if stream is None else _on(stream, device):
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
            for param, grad, m, copy in self.tensors:
                factor = muon_scale(param.shape, scale) if isinstance(scale, str) else scale
                cfg = MuonConfig(newton_schulz(steps, coefficients, eps), lr, momentum, weight_decay, factor, grad_scale,
                                 int(bool(nesterov)))
                mxq_muon(param, grad, m, cfg, workspace, copy, control)
