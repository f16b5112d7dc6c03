"""Python binding of the tilegemm C ABI (``include/tilegemm.h``).

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity) and their device pointers, together with the current HIP stream,
are passed to ``libtilegemm.so``.  Every step of the computation runs in the
library's HIP kernels; there is no fallback.  If the library has not been
built, loading raises instead of computing anything another way.

PyTorch is used only for device memory and streams.
"""

from __future__ import annotations

import collections
import ctypes
import math
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
_DEFAULT_LIB = os.path.join(HERE, "libtilegemm.so")

TG_F32, TG_F16, TG_BF16 = 0, 1, 2
TG_EPI_NONE, TG_EPI_RELU = 0, 1
TG_OP_GEMM, TG_OP_DEQUANT_W4, TG_OP_MX, TG_OP_SP24, TG_OP_I8 = 0, 1, 2, 3, 4
TG_MX_E2M1, TG_MX_E4M3 = 0, 1

# exported symbols, as declared in include/tilegemm.h
EXPORTS = ("tg_gemm", "tg_gemm_ex", "tg_dequant_gemm_w4", "tg_status_str", "tg_query_config",
           "tg_query_config_ex", "tg_config_count", "tg_config_name", "tg_gemm_config",
           "tg_gemm_ex_config", "tg_dequant_gemm_w4_config", "tg_tile_map", "tg_gemm_mx",
           "tg_gemm_mx_config", "tg_gemm_sp24", "tg_gemm_sp24_config", "tg_gemm_splitk",
           "tg_gemm_splitk_workspace_size", "tg_gemm_splitk_config", "tg_gemm_splitk_noalloc",
           "tg_set_clock_stamps", "tg_set_swizzle_override", "tg_config_occupancy",
           "tg_quant_i8", "tg_gemm_i8", "tg_linear_i8", "tg_linear_i8_workspace_size",
           "tg_block_norm", "tg_block_norm_backward", "tg_block_norm_backward_workspace_size")
TG_SPLITK_SCRATCH_BYTES = 16 * 1024 * 1024

_lib = None


class BlockNormArgs(ctypes.Structure):
    """tg_block_norm_args."""

    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("xtype", ctypes.c_int),
                ("btype", ctypes.c_int), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("gate", ctypes.c_void_p),
                ("gate_rows", ctypes.c_int64), ("w_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("alpha", ctypes.c_float), ("eps", ctypes.c_float),
                ("post_norm", ctypes.c_int), ("x_out", ctypes.c_void_p),
                ("ldx_out", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("hq", ctypes.c_void_p), ("ldhq", ctypes.c_int64), ("hs", ctypes.c_void_p),
                ("r_post", ctypes.c_void_p), ("r_pre", ctypes.c_void_p)]


class BlockNormGradArgs(ctypes.Structure):
    """tg_block_norm_grad_args."""

    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("xtype", ctypes.c_int),
                ("btype", ctypes.c_int), ("x_new", ctypes.c_void_p), ("ldx_new", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("gate", ctypes.c_void_p),
                ("gate_rows", ctypes.c_int64), ("w_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("post_norm", ctypes.c_int), ("r_post", ctypes.c_void_p),
                ("r_pre", ctypes.c_void_p), ("dx_new", ctypes.c_void_p),
                ("lddx_new", ctypes.c_int64), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dy", ctypes.c_void_p),
                ("lddy", ctypes.c_int64), ("dgate", ctypes.c_void_p),
                ("dw_post", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p)]


# Result of block_norm: the new residual stream, h (block type, or int8 levels
# with their scales hs), and the norms' reciprocal roots (None unless saved).
BlockNorm = collections.namedtuple("BlockNorm", "x h hs r_post r_pre")
BlockNormGrad = collections.namedtuple("BlockNormGrad", "dx dy dgate dw_post dw_pre")


class TileGemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def library_path() -> str:
    return os.environ.get("TILEGEMM_LIB", _DEFAULT_LIB)


def load_library():
    """Load libtilegemm.so (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise FileNotFoundError(
            "libtilegemm.so not found at %s; build it with "
            "`python -m tiled_dense_gemm_07_amd.build`" % path)
    lib = ctypes.CDLL(path)
    i64, p, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.tg_gemm.argtypes = [i64, i64, i64, c_int, p, p, p, c_int, p]
    lib.tg_gemm.restype = c_int
    lib.tg_gemm_ex.argtypes = [i64, i64, i64, c_int, p, c_int, p, c_int, p, c_int, p]
    lib.tg_gemm_ex.restype = c_int
    lib.tg_gemm_ex_config.argtypes = [c_int, i64, i64, i64, c_int, p, c_int, p, c_int, p, c_int, p]
    lib.tg_gemm_ex_config.restype = c_int
    lib.tg_query_config_ex.argtypes = [c_int, i64, i64, i64, c_int, c_int, c_int, ctypes.c_char_p,
                                       ctypes.c_size_t]
    lib.tg_query_config_ex.restype = c_int
    lib.tg_dequant_gemm_w4.argtypes = [i64, i64, i64, p, p, p, p, c_int, p]
    lib.tg_dequant_gemm_w4.restype = c_int
    lib.tg_status_str.argtypes = [c_int]
    lib.tg_status_str.restype = ctypes.c_char_p
    lib.tg_query_config.argtypes = [c_int, i64, i64, i64, c_int, ctypes.c_char_p, ctypes.c_size_t]
    lib.tg_query_config.restype = c_int
    lib.tg_config_count.argtypes = [c_int, c_int]
    lib.tg_config_count.restype = c_int
    lib.tg_config_name.argtypes = [c_int, c_int, c_int, ctypes.c_char_p, ctypes.c_size_t]
    lib.tg_config_name.restype = c_int
    lib.tg_gemm_config.argtypes = [c_int, i64, i64, i64, c_int, p, p, p, c_int, p]
    lib.tg_gemm_config.restype = c_int
    lib.tg_dequant_gemm_w4_config.argtypes = [c_int, i64, i64, i64, p, p, p, p, c_int, p]
    lib.tg_dequant_gemm_w4_config.restype = c_int
    lib.tg_tile_map.argtypes = [i64, i64, c_int, p, p]
    lib.tg_tile_map.restype = c_int
    lib.tg_gemm_mx.argtypes = [i64, i64, i64, c_int, p, p, p, p, p, c_int, p]
    lib.tg_gemm_mx.restype = c_int
    lib.tg_gemm_mx_config.argtypes = [c_int, i64, i64, i64, c_int, p, p, p, p, p, c_int, p]
    lib.tg_gemm_mx_config.restype = c_int
    lib.tg_gemm_sp24.argtypes = [i64, i64, i64, c_int, p, p, p, p, c_int, p]
    lib.tg_gemm_sp24.restype = c_int
    lib.tg_gemm_sp24_config.argtypes = [c_int, i64, i64, i64, c_int, p, p, p, p, c_int, p]
    lib.tg_gemm_sp24_config.restype = c_int
    lib.tg_gemm_splitk.argtypes = [i64, i64, i64, c_int, p, p, p, c_int, c_int, p,
                                   ctypes.c_size_t, p]
    lib.tg_gemm_splitk.restype = c_int
    lib.tg_gemm_splitk_config.argtypes = [c_int, i64, i64, i64, c_int, p, p, p, c_int, c_int, p,
                                          ctypes.c_size_t, p]
    lib.tg_gemm_splitk_config.restype = c_int
    lib.tg_gemm_splitk_workspace_size.argtypes = [i64, i64, i64, c_int, c_int,
                                                  ctypes.POINTER(ctypes.c_size_t)]
    lib.tg_gemm_splitk_workspace_size.restype = c_int
    lib.tg_gemm_splitk_noalloc.argtypes = [i64, i64, i64, c_int, p, p, p, c_int, c_int, p]
    lib.tg_gemm_splitk_noalloc.restype = c_int
    lib.tg_set_clock_stamps.argtypes = [p]
    lib.tg_set_clock_stamps.restype = None
    lib.tg_set_swizzle_override.argtypes = [c_int]
    lib.tg_set_swizzle_override.restype = None
    lib.tg_config_occupancy.argtypes = [c_int, c_int, c_int, ctypes.POINTER(c_int)]
    lib.tg_config_occupancy.restype = c_int
    size_p = ctypes.POINTER(ctypes.c_size_t)
    lib.tg_quant_i8.argtypes = [i64, i64, c_int, p, i64, p, i64, p, p]
    lib.tg_gemm_i8.argtypes = [i64, i64, i64, p, i64, p, p, i64, p, p, c_int, p, i64, c_int, p]
    lib.tg_linear_i8.argtypes = [i64, i64, i64, c_int, p, i64, p, i64, p, p, p, i64, c_int, p,
                                 ctypes.c_size_t, p]
    lib.tg_linear_i8_workspace_size.argtypes = [i64, i64, i64, c_int, size_p]
    lib.tg_block_norm.argtypes = [ctypes.POINTER(BlockNormArgs), p]
    lib.tg_block_norm_backward.argtypes = [ctypes.POINTER(BlockNormGradArgs), p, ctypes.c_size_t,
                                           p]
    lib.tg_block_norm_backward_workspace_size.argtypes = [ctypes.POINTER(BlockNormGradArgs),
                                                          size_p]
    for name in ("tg_quant_i8", "tg_gemm_i8", "tg_linear_i8", "tg_linear_i8_workspace_size",
                 "tg_block_norm", "tg_block_norm_backward",
                 "tg_block_norm_backward_workspace_size"):
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().tg_status_str(status).decode()


def _check(status: int):
    if status != 0:
        raise TileGemmError(status, status_str(status))


_DTYPE_CODES = None


def _dtype_code(t) -> int:
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        import torch

        _DTYPE_CODES = {torch.float32: TG_F32, torch.float16: TG_F16, torch.bfloat16: TG_BF16}
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s (float32, float16 or bfloat16)" % t.dtype)
    return code


def _epi_code(epilogue) -> int:
    if epilogue in (None, "none", TG_EPI_NONE):
        return TG_EPI_NONE
    if epilogue in ("relu", TG_EPI_RELU):
        return TG_EPI_RELU
    raise ValueError("epilogue must be None/'none' or 'relu'")


_raw_stream = None
_torch_module = None


def _torch():
    """The torch module (a third of an import statement's time in a hot call)."""
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream_ptr(device, stream=None):
    """Handle of `stream`, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    global _raw_stream
    if _raw_stream is None:
        import torch

        # the handle without a Stream object: 0.1 us instead of 1.9 on every call
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(device.index)


def _require_gpu_tensor(name, t):
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major)" % name)


def _gemm_args(A, B, C):
    _require_gpu_tensor("A", A)
    _require_gpu_tensor("B", B)
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ: A is %s, B is %s" % (tuple(A.shape), tuple(B.shape)))
    if A.dtype != B.dtype:
        raise TypeError("A and B must share a dtype")
    if C is not None:
        _require_gpu_tensor("C", C)
        if tuple(C.shape) != (M, N) or C.dtype != A.dtype:
            raise ValueError("C must be [M, N] of the operand dtype")
    return M, N, K


def gemm(A, B, C=None, epilogue=None, stream=None):
    """C = epilogue(A @ B) on the GPU (fp32 / fp16 / bf16, row-major). Returns C."""
    M, N, K = _gemm_args(A, B, C)
    if C is None:
        import torch

        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    _check(load_library().tg_gemm(M, N, K, _dtype_code(A), A.data_ptr(), B.data_ptr(),
                                  C.data_ptr(), _epi_code(epilogue), _stream_ptr(A.device, stream)))
    return C


def gemm_with_config(index: int, A, B, C=None, epilogue=None, stream=None):
    """As :func:`gemm`, launching compiled configuration `index` (for the sweep)."""
    import torch

    M, N, K = _gemm_args(A, B, C)
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    _check(load_library().tg_gemm_config(index, M, N, K, _dtype_code(A), A.data_ptr(),
                                         B.data_ptr(), C.data_ptr(), _epi_code(epilogue),
                                         _stream_ptr(A.device, stream)))
    return C


def splitk_workspace_size(M: int, N: int, K: int, dtype: int, splits: int = 0) -> int:
    """Workspace bytes :func:`gemm_splitk` needs for this shape (0: no split)."""
    out = ctypes.c_size_t(0)
    _check(load_library().tg_gemm_splitk_workspace_size(M, N, K, dtype, splits,
                                                        ctypes.byref(out)))
    return out.value


def splitk_workspace(M: int, N: int, K: int, dtype: int, splits: int = 0, device="cuda"):
    """A zero-filled uint8 device tensor large enough for :func:`gemm_splitk`
    (None when no split would be launched).  Reusable across calls on one stream."""
    import torch

    n = splitk_workspace_size(M, N, K, dtype, splits)
    return torch.zeros((n,), dtype=torch.uint8, device=device) if n else None


def gemm_splitk(A, B, C=None, epilogue=None, splits: int = 0, workspace=None, stream=None,
                config=None):
    """As :func:`gemm`, with each output tile's K range split over `splits`
    workgroups (0: chosen by the library).  workspace: a zero-filled uint8
    device tensor of at least :func:`splitk_workspace_size` bytes (allocated
    here when None).  config: force a compiled configuration by index."""
    import torch

    M, N, K = _gemm_args(A, B, C)
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    dt = _dtype_code(A)
    if workspace is None:
        workspace = splitk_workspace(M, N, K, dt, splits, device=A.device)
    if workspace is not None:
        _require_gpu_tensor("workspace", workspace)
    wp = workspace.data_ptr() if workspace is not None else None
    wn = workspace.numel() * workspace.element_size() if workspace is not None else 0
    lib = load_library()
    args = (M, N, K, dt, A.data_ptr(), B.data_ptr(), C.data_ptr(), _epi_code(epilogue), splits,
            wp, wn, _stream_ptr(A.device, stream))
    _check(lib.tg_gemm_splitk(*args) if config is None else lib.tg_gemm_splitk_config(config, *args))
    return C


def gemm_splitk_noalloc(A, B, C, epilogue=None, splits: int = 0, stream=None):
    """As :func:`gemm_splitk`, with the partial tiles in the library's fixed
    scratch array instead of a workspace (tg_gemm_splitk_noalloc): C must be
    given, and nothing is allocated.  Calls that overlap on one GPU race."""
    M, N, K = _gemm_args(A, B, C)
    _check(load_library().tg_gemm_splitk_noalloc(
        M, N, K, _dtype_code(A), A.data_ptr(), B.data_ptr(), C.data_ptr(), _epi_code(epilogue),
        splits, _stream_ptr(A.device, stream)))
    return C


def set_clock_stamps(stamps):
    """Record the shader clock of every following launch into `stamps`, an
    int64 / uint64 device tensor of 32 elements (None: stop recording)."""
    if stamps is not None:
        _require_gpu_tensor("stamps", stamps)
        if stamps.numel() * stamps.element_size() < 32 * 8:
            raise ValueError("stamps must hold 32 64-bit values")
    load_library().tg_set_clock_stamps(stamps.data_ptr() if stamps is not None else None)


def set_swizzle_override(group_m: int):
    """Force swizzle group `group_m` on every following launch (0: none)."""
    load_library().tg_set_swizzle_override(int(group_m))


def config_occupancy(op: int, dtype: int, index: int) -> int:
    """Workgroups of configuration `index` one compute unit holds at once."""
    n = ctypes.c_int(0)
    _check(load_library().tg_config_occupancy(op, dtype, index, ctypes.byref(n)))
    return n.value


def stamp_clock_ghz(stamps) -> list:
    """Shader clock (GHz) of each workgroup 0..7 that wrote a record into the
    host copy of `stamps` (a sequence of 32 integers)."""
    out = []
    for b in range(8):
        t0, r0, t1, r1 = (int(x) for x in stamps[4 * b:4 * b + 4])
        if r1 > r0 and t1 > t0:
            out.append((t1 - t0) / ((r1 - r0) / 100e6) / 1e9)
    return out


def _gemm_ex_args(A, B, trans_a, trans_b, C):
    _require_gpu_tensor("A", A)
    _require_gpu_tensor("B", B)
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    K, M = A.shape if trans_a else (A.shape[1], A.shape[0])
    N, K2 = B.shape if trans_b else (B.shape[1], B.shape[0])
    if K != K2:
        raise ValueError("inner dimensions differ: A is %s (trans_a=%d), B is %s (trans_b=%d)"
                         % (tuple(A.shape), trans_a, tuple(B.shape), trans_b))
    if A.dtype != B.dtype:
        raise TypeError("A and B must share a dtype")
    if C is not None:
        _require_gpu_tensor("C", C)
        if tuple(C.shape) != (M, N) or C.dtype != A.dtype:
            raise ValueError("C must be [M, N] of the operand dtype")
    return M, N, K


def gemm_ex(A, B, trans_a=False, trans_b=False, C=None, epilogue=None, stream=None, config=None):
    """C = epilogue(op(A) @ op(B)): A stored [M, K] (or [K, M] with trans_a),
    B stored [K, N] (or [N, K] with trans_b).  config: force a compiled
    configuration by index (for the sweep and tests)."""
    import torch

    ta, tb = int(bool(trans_a)), int(bool(trans_b))
    M, N, K = _gemm_ex_args(A, B, ta, tb, C)
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    lib = load_library()
    args = (M, N, K, _dtype_code(A), A.data_ptr(), ta, B.data_ptr(), tb, C.data_ptr(),
            _epi_code(epilogue), _stream_ptr(A.device, stream))
    _check(lib.tg_gemm_ex(*args) if config is None else lib.tg_gemm_ex_config(config, *args))
    return C


def _w4_args(A, Wq, Ws, C):
    import torch

    for name, t in (("A", A), ("Wq", Wq), ("Ws", Ws)):
        _require_gpu_tensor(name, t)
    if A.dtype != torch.bfloat16:
        raise TypeError("activations must be bfloat16")
    if Wq.dtype != torch.uint8 or Ws.dtype != torch.uint8:
        raise TypeError("packed weights and scales must be uint8")
    M, K = A.shape
    N = Wq.shape[0]
    if tuple(Wq.shape) != (N, K // 2) or tuple(Ws.shape) != (N, K // 32) or K % 32:
        raise ValueError("expected Wq [N, K/2] and Ws [N, K/32] with K % 32 == 0")
    if C is not None:
        _require_gpu_tensor("C", C)
        if tuple(C.shape) != (M, N) or C.dtype != torch.bfloat16:
            raise ValueError("C must be bfloat16 [M, N]")
    return M, N, K


def dequant_gemm_w4(A, Wq, Ws, C=None, epilogue=None, stream=None):
    """C = epilogue(A @ W^T) with W given as packed E2M1 codes and E8M0 scales."""
    import torch

    M, N, K = _w4_args(A, Wq, Ws, C)
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(load_library().tg_dequant_gemm_w4(M, N, K, A.data_ptr(), Wq.data_ptr(), Ws.data_ptr(),
                                             C.data_ptr(), _epi_code(epilogue),
                                             _stream_ptr(A.device, stream)))
    return C


def dequant_gemm_w4_with_config(index: int, A, Wq, Ws, C=None, epilogue=None, stream=None):
    import torch

    M, N, K = _w4_args(A, Wq, Ws, C)
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(load_library().tg_dequant_gemm_w4_config(index, M, N, K, A.data_ptr(), Wq.data_ptr(),
                                                    Ws.data_ptr(), C.data_ptr(),
                                                    _epi_code(epilogue),
                                                    _stream_ptr(A.device, stream)))
    return C


def _mx_args(fmt, Aq, As, Wq, Ws, C):
    import torch

    if fmt not in (TG_MX_E2M1, TG_MX_E4M3):
        raise ValueError("activation format must be TG_MX_E2M1 or TG_MX_E4M3")
    for name, t in (("Aq", Aq), ("As", As), ("Wq", Wq), ("Ws", Ws)):
        _require_gpu_tensor(name, t)
        if t.dtype != torch.uint8:
            raise TypeError("%s must be uint8" % name)
    M = Aq.shape[0]
    K = Aq.shape[1] * (2 if fmt == TG_MX_E2M1 else 1)
    N = Wq.shape[0]
    if (tuple(As.shape) != (M, K // 32) or tuple(Wq.shape) != (N, K // 2)
            or tuple(Ws.shape) != (N, K // 32) or K % 32):
        raise ValueError("expected As [M, K/32], Wq [N, K/2], Ws [N, K/32] with K % 32 == 0")
    if C is not None:
        _require_gpu_tensor("C", C)
        if tuple(C.shape) != (M, N) or C.dtype != torch.bfloat16:
            raise ValueError("C must be bfloat16 [M, N]")
    return M, N, K


def gemm_mx(fmt: int, Aq, As, Wq, Ws, C=None, epilogue=None, stream=None, config=None):
    """C = epilogue(a @ w^T) with both operands in MX blocks: activation codes Aq
    (E2M1 [M, K/2] or E4M3 [M, K]) with E8M0 scales As [M, K/32], E2M1 weights
    Wq [N, K/2] with E8M0 scales Ws [N, K/32]; bf16 output.  `config` forces a
    compiled configuration by index."""
    import torch

    M, N, K = _mx_args(fmt, Aq, As, Wq, Ws, C)
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=Aq.device)
    args = (M, N, K, fmt, Aq.data_ptr(), As.data_ptr(), Wq.data_ptr(), Ws.data_ptr(),
            C.data_ptr(), _epi_code(epilogue), _stream_ptr(Aq.device, stream))
    lib = load_library()
    _check(lib.tg_gemm_mx(*args) if config is None else lib.tg_gemm_mx_config(config, *args))
    return C


def gemm_sp24(Ac, Ai, B, C=None, epilogue=None, stream=None, config=None):
    """C = epilogue(A @ B) with A 2:4 sparse along K, given as kept values Ac
    [M, K/2] (fp16 or bf16) and position nibbles Ai [M, K/8] (uint8); B [K, N]
    of Ac's dtype.  `config` forces a compiled configuration by index."""
    import torch

    for name, t in (("Ac", Ac), ("Ai", Ai), ("B", B)):
        _require_gpu_tensor(name, t)
    if Ac.dtype not in (torch.float16, torch.bfloat16) or B.dtype != Ac.dtype:
        raise TypeError("Ac and B must both be float16 or both bfloat16")
    if Ai.dtype != torch.uint8:
        raise TypeError("Ai must be uint8")
    M, half = Ac.shape
    K = 2 * half
    K2, N = B.shape
    if K != K2 or tuple(Ai.shape) != (M, K // 8) or K % 8:
        raise ValueError("expected Ac [M, K/2], Ai [M, K/8], B [K, N]")
    if C is None:
        C = torch.empty((M, N), dtype=Ac.dtype, device=Ac.device)
    else:
        _require_gpu_tensor("C", C)
        if tuple(C.shape) != (M, N) or C.dtype != Ac.dtype:
            raise ValueError("C must be [M, N] of Ac's dtype")
    args = (M, N, K, _dtype_code(Ac), Ac.data_ptr(), Ai.data_ptr(), B.data_ptr(),
            C.data_ptr(), _epi_code(epilogue), _stream_ptr(Ac.device, stream))
    lib = load_library()
    _check(lib.tg_gemm_sp24(*args) if config is None else lib.tg_gemm_sp24_config(config, *args))
    return C


# --------------------------------------------------------------------------
# 8-bit integer path and block norms.  These take row-strided 2-D tensors
# (unit stride along a row), for instance slices of a wider buffer.
# --------------------------------------------------------------------------
# Argument checks here cost a good part of a small call's time, so they take
# the cheapest properties of a tensor, each once.
def _rows(name, t, shape=None, dtype=None):
    """Row stride of the 2-D GPU tensor t; checks shape and dtype."""
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError("%s must be %s, got %s"
                         % (name, "2-D" if shape is None else list(shape), tuple(size)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    rows, cols = size
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError("%s must have unit stride along its rows" % name)
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError("%s must have rows that do not overlap" % name)
    return ld


def _vector(name, t, n, dtype):
    """Device pointer of the dense 1-D GPU tensor t (None: NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a dense vector of %d values" % (name, n))
    return t.data_ptr()


def _one_device(first, *others):
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("operands must be on one device: %s and %s"
                             % (first.device, t.device))


def _empty(shape, dtype, like, stream):
    """An output or workspace on like's device that belongs to the call's stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    torch = _torch()
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _empty_as(t, stream):
    """An output of t's shape and type, dense."""
    if stream is not None or not t.is_contiguous():
        return _empty(t.shape, t.dtype, t, stream)
    torch = _torch()
    return torch.empty_like(t)


def quant_i8(X, Q=None, s=None, stream=None):
    """Rows of X to 8-bit levels and one fp32 scale each (tg_quant_i8): returns
    (Q int8 [M, K], s fp32 [M]) with X about Q * s[:, None]."""
    torch = _torch()
    ldx = _rows("X", X)
    M, K = X.shape
    if Q is None:
        Q = _empty((M, K), torch.int8, X, stream)
    if s is None:
        s = _empty((M,), torch.float32, X, stream)
    ldq = _rows("Q", Q, (M, K), torch.int8)
    ps = _vector("s", s, M, torch.float32)
    _one_device(X, Q, s)
    _check(load_library().tg_quant_i8(M, K, _dtype_code(X), X.data_ptr(), ldx, Q.data_ptr(), ldq,
                                      ps, _stream_ptr(X.device, stream)))
    return Q, s


def gemm_i8(A, sa, W, sw, bias=None, out_dtype=None, C=None, epilogue=None, stream=None):
    """C = epilogue((A @ W^T) * sa[:, None] * sw + bias) with A [M, K] and W
    [N, K] in int8, fp32 scales sa [M] and sw [N], fp32 bias [N] or None; C
    [M, N] of out_dtype (bfloat16 unless C or out_dtype says otherwise)."""
    torch = _torch()
    i8, f32 = torch.int8, torch.float32
    lda = _rows("A", A, None, i8)
    ldw = _rows("W", W, None, i8)
    M, K = A.shape
    N, K2 = W.shape
    if K2 != K:
        raise ValueError("inner dimensions differ: A is %s, W is %s"
                         % (tuple(A.shape), tuple(W.shape)))
    if C is None:
        C = _empty((M, N), out_dtype or torch.bfloat16, A, stream)
    elif out_dtype is not None and C.dtype != out_dtype:
        raise TypeError("C must be %s, got %s" % (out_dtype, C.dtype))
    ldc = _rows("C", C, (M, N))
    ps, pw, pb = _vector("sa", sa, M, f32), _vector("sw", sw, N, f32), _vector("bias", bias, N, f32)
    _one_device(A, sa, W, sw, bias, C)
    _check(load_library().tg_gemm_i8(
        M, N, K, A.data_ptr(), lda, ps, W.data_ptr(), ldw, pw, pb, _dtype_code(C), C.data_ptr(),
        ldc, _epi_code(epilogue), _stream_ptr(A.device, stream)))
    return C


def linear_i8_workspace_size(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace bytes :func:`linear_i8` needs (0: none)."""
    out = ctypes.c_size_t(0)
    _check(load_library().tg_linear_i8_workspace_size(M, N, K, dtype, ctypes.byref(out)))
    return out.value


def linear_i8(X, W, sw, bias=None, C=None, epilogue=None, workspace=None, stream=None):
    """C = epilogue(X @ W^T * sw + bias) with the rows of X [M, K] (fp32, fp16
    or bf16) quantised within the call, as :func:`quant_i8` and
    :func:`gemm_i8` one after the other; C [M, N] of X's dtype.  workspace: a
    uint8 device tensor of at least :func:`linear_i8_workspace_size` bytes
    (allocated here when None and needed)."""
    torch = _torch()
    f32 = torch.float32
    ldx = _rows("X", X)
    ldw = _rows("W", W, None, torch.int8)
    M, K = X.shape
    N, K2 = W.shape
    if K2 != K:
        raise ValueError("inner dimensions differ: X is %s, W is %s"
                         % (tuple(X.shape), tuple(W.shape)))
    if C is None:
        C = _empty((M, N), X.dtype, X, stream)
    ldc = _rows("C", C, (M, N), X.dtype)
    dt = _dtype_code(X)
    wp, wn = None, 0
    if workspace is None:
        wn = linear_i8_workspace_size(M, N, K, dt)
        if wn:
            workspace = _empty((wn,), torch.uint8, X, stream)
            wp = workspace.data_ptr()
    else:
        _require_gpu_tensor("workspace", workspace)
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    pw, pb = _vector("sw", sw, N, f32), _vector("bias", bias, N, f32)
    _one_device(X, W, sw, bias, C, workspace)
    _check(load_library().tg_linear_i8(
        M, N, K, dt, X.data_ptr(), ldx, W.data_ptr(), ldw, pw, pb, C.data_ptr(), ldc,
        _epi_code(epilogue), wp, wn, _stream_ptr(X.device, stream)))
    return C


def _gate_arg(gate, gate_rows, T, D, dtype):
    """(pointer, gate_rows) of a gate [G, D] or [D]; gate_rows may be left out
    for one row (shared by every token) or one row for each token."""
    if gate is None:
        return None, 0
    size = gate.shape
    G = 1 if len(size) == 1 else size[0]
    if not gate_rows:
        if G != 1 and G != T:
            raise ValueError("gate_rows is needed: gate has %d rows for %d tokens" % (G, T))
        gate_rows = max(T, 1) if G == 1 else 1
    if not gate.is_cuda or not gate.is_contiguous():
        raise ValueError("gate must be a dense GPU tensor")
    if gate.dtype != dtype:
        raise TypeError("gate must be %s, got %s" % (dtype, gate.dtype))
    if gate_rows < 1 or size[-1] != D or len(size) > 2 or (T > 0 and G != -(-T // gate_rows)):
        raise ValueError("gate must be [ceil(T / gate_rows), D] = [%d, %d], got %s"
                         % (-(-T // max(1, gate_rows)), D, tuple(size)))
    return gate.data_ptr(), gate_rows


def block_norm(x, y=None, gate=None, gate_rows=None, w_post=None, w_pre=None, alpha=1.0, eps=1e-6,
               post_norm=True, out="h", x_out=None, h=None, hs=None, save=False, stream=None):
    """The norms, gate and residual between two blocks (tg_block_norm):

        x' = alpha x + gate * norm(y) * w_post,   h = norm(x') * w_pre

    x [T, D]: residual stream; y [T, D]: output of the block before (None: x'
    is x, whatever alpha is); gate [G, D], one row for gate_rows tokens.  out: "h" (h in y's
    type, x's without y), "i8" (h as int8 levels with scales hs) or None (x'
    only).  x_out may be x.  save: also return the norms' reciprocal roots
    for :func:`block_norm_backward`.  Returns a BlockNorm(x, h, hs, r_post,
    r_pre)."""
    torch = _torch()
    if out not in ("h", "i8", None):
        raise ValueError("out must be 'h', 'i8' or None")
    if out is None and h is not None:
        raise ValueError("h is not written with out None")
    if out != "i8" and hs is not None:
        raise ValueError("hs is not written without out 'i8'")
    ldx = _rows("x", x)
    shape = x.shape
    T, D = shape
    block = y if y is not None else (h if h is not None and out == "h" else w_pre)
    if block is None:
        block = x
    xt, bt = x.dtype, block.dtype
    a = BlockNormArgs()
    a.T, a.D, a.xtype, a.btype = T, D, _dtype_code(x), _dtype_code(block)
    a.x, a.ldx = x.data_ptr(), ldx
    a.alpha, a.eps, a.post_norm = alpha, eps, bool(post_norm)
    if y is not None:
        a.y, a.ldy = y.data_ptr(), _rows("y", y, shape)
        if x_out is None:
            x_out = _empty_as(x, stream)
            a.x_out, a.ldx_out = x_out.data_ptr(), D
    if x_out is not None and not a.x_out:
        a.x_out, a.ldx_out = x_out.data_ptr(), _rows("x_out", x_out, shape, xt)
    a.gate, a.gate_rows = _gate_arg(gate, gate_rows, T, D, bt)
    a.w_post = _vector("w_post", w_post, D, bt)
    a.w_pre = _vector("w_pre", w_pre, D, bt)
    if out == "h":
        if h is None:
            h = _empty_as(y, stream) if y is not None else _empty(shape, bt, x, stream)
            a.h, a.ldh = h.data_ptr(), D
        else:
            a.h, a.ldh = h.data_ptr(), _rows("h", h, shape, bt)
    elif out == "i8":
        if h is None:
            h = _empty(shape, torch.int8, x, stream)
        if hs is None:
            hs = _empty((T,), torch.float32, x, stream)
        a.hq, a.ldhq = h.data_ptr(), _rows("h", h, shape, torch.int8)
        a.hs = _vector("hs", hs, T, torch.float32)
    r_post = r_pre = None
    if save:
        if y is not None and post_norm:
            r_post = _empty((T,), torch.float32, x, stream)
            a.r_post = r_post.data_ptr()
        if out is not None:
            r_pre = _empty((T,), torch.float32, x, stream)
            a.r_pre = r_pre.data_ptr()
    _one_device(x, y, gate, w_post, w_pre, x_out, h, hs)
    if D == 0:  # nothing is launched: the scale of an empty row, a mean of nothing
        with torch.cuda.stream(stream):
            for t, v in ((hs, 2.0 ** -126), (r_post, math.nan), (r_pre, math.nan)):
                if t is not None:
                    t.fill_(v)
    _check(load_library().tg_block_norm(ctypes.byref(a), _stream_ptr(x.device, stream)))
    return BlockNorm(x if x_out is None else x_out, h, hs, r_post, r_pre)


def block_norm_backward(x_new, dx_new=None, dh=None, y=None, gate=None, gate_rows=None,
                        w_post=None, w_pre=None, r_post=None, r_pre=None, alpha=1.0,
                        post_norm=True, workspace=None, stream=None):
    """Gradients of :func:`block_norm` (tg_block_norm_backward) from those at
    x' (dx_new) and at h (dh), either of which may be None.  x_new, r_post and
    r_pre are the forward call's x, r_post and r_pre.  Returns a
    BlockNormGrad(dx, dy, dgate, dw_post, dw_pre), dx and dy in their inputs'
    types, the rest (None where there is no such input) in fp32."""
    torch = _torch()
    shape = x_new.shape
    ldx = _rows("x_new", x_new)
    T, D = shape
    block = y if y is not None else (dh if dh is not None else w_pre)
    if block is None:
        block = x_new
    xt, bt, f32 = x_new.dtype, block.dtype, torch.float32
    a = BlockNormGradArgs()
    a.T, a.D, a.xtype, a.btype = T, D, _dtype_code(x_new), _dtype_code(block)
    a.x_new, a.ldx_new = x_new.data_ptr(), ldx
    a.alpha, a.post_norm = alpha, bool(post_norm)
    dx = _empty_as(x_new, stream)
    a.dx, a.lddx = dx.data_ptr(), D
    dy = dgate = dw_post = dw_pre = None
    if y is not None:
        a.y, a.ldy = y.data_ptr(), _rows("y", y, shape)
        dy = _empty_as(y, stream)
        a.dy, a.lddy = dy.data_ptr(), D
        if post_norm:
            a.r_post = _vector("r_post", r_post, T, f32)
    a.gate, a.gate_rows = _gate_arg(gate, gate_rows, T, D, bt)
    if gate is not None:
        dgate = _empty(gate.shape, f32, x_new, stream)
        a.dgate = dgate.data_ptr()
    a.w_post = _vector("w_post", w_post, D, bt)
    a.w_pre = _vector("w_pre", w_pre, D, bt)
    want_pre = dh is not None and w_pre is not None
    if w_post is not None and want_pre:  # one allocation for both
        dw_post, dw_pre = _empty((2, D), f32, x_new, stream).unbind(0)
    elif w_post is not None:
        dw_post = _empty((D,), f32, x_new, stream)
    elif want_pre:
        dw_pre = _empty((D,), f32, x_new, stream)
    if dw_post is not None:
        a.dw_post = dw_post.data_ptr()
    if dw_pre is not None:
        a.dw_pre = dw_pre.data_ptr()
    if dh is not None:
        a.dh, a.lddh = dh.data_ptr(), _rows("dh", dh, shape, bt)
        a.r_pre = _vector("r_pre", r_pre, T, f32)
    if dx_new is not None:
        a.dx_new, a.lddx_new = dx_new.data_ptr(), _rows("dx_new", dx_new, shape, xt)
    if T == 0:  # sums over no tokens; nothing is launched
        with torch.cuda.stream(stream):
            for g in (dgate, dw_post, dw_pre):
                if g is not None:
                    g.zero_()
    lib = load_library()
    ref = ctypes.byref(a)
    wp, wn = None, 0
    if workspace is None:
        need = ctypes.c_size_t(0)
        _check(lib.tg_block_norm_backward_workspace_size(ref, ctypes.byref(need)))
        wn = need.value
        if wn:
            workspace = _empty((wn,), torch.uint8, x_new, stream)
            wp = workspace.data_ptr()
    else:
        _require_gpu_tensor("workspace", workspace)
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _one_device(x_new, dx_new, dh, y, gate, w_post, w_pre, r_post, r_pre, workspace)
    _check(lib.tg_block_norm_backward(ref, wp, wn, _stream_ptr(x_new.device, stream)))
    return BlockNormGrad(dx, dy, dgate, dw_post, dw_pre)


def query_config(op: int, M: int, N: int, K: int, dtype: int = TG_BF16, trans_a: bool = False,
                 trans_b: bool = False) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(load_library().tg_query_config_ex(op, M, N, K, dtype, int(trans_a), int(trans_b), buf,
                                             len(buf)))
    return buf.value.decode()


def list_configs(op: int, dtype: int = TG_BF16):
    lib = load_library()
    names = []
    for i in range(lib.tg_config_count(op, dtype)):
        buf = ctypes.create_string_buffer(128)
        _check(lib.tg_config_name(op, dtype, i, buf, len(buf)))
        names.append(buf.value.decode())
    return names


def tile_map(tiles_m: int, tiles_n: int, group_m: int):
    """The scheduler's workgroup -> (tile_m, tile_n) map, computed on the host."""
    total = tiles_m * tiles_n
    om = np.empty(total, dtype=np.int32)
    on = np.empty(total, dtype=np.int32)
    _check(load_library().tg_tile_map(tiles_m, tiles_n, group_m,
                                      om.ctypes.data_as(ctypes.c_void_p),
                                      on.ctypes.data_as(ctypes.c_void_p)))
    return om, on
