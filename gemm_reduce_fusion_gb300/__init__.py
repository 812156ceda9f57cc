"""Python binding of the tp_fused C-ABI (argument marshalling only).

Every function here has the name of the C entry point it calls
(``include/tp_fused.h``).  It reads shapes from the torch tensors it is
given and checks that every shard, output and bias has the shape, dtype,
layout and device the call implies (the C ABI sees only pointers, so a
wrong-sized buffer would otherwise be read or written out of bounds on the
device); it then passes the device pointers and the current CUDA stream to
the shared library and raises :class:`TPError` on a non-zero status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback: if the
library is missing the import fails.

Tensors are torch CUDA tensors, contiguous, row-major; inputs bfloat16,
outputs bfloat16 or float32.  Lists hold one tensor per rank/shard.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtpfused.so")

# tp_status
TP_OK = 0
TP_ERR_INVALID_ARG = 1
TP_ERR_ALIGNMENT = 2
TP_ERR_UNSUPPORTED_SHAPE = 3
TP_ERR_WORKSPACE_TOO_SMALL = 4
TP_ERR_ARCH = 5
TP_ERR_CUDA = 6
TP_ERR_DEVICE_TIMEOUT = 7
# tp_dtype
TP_BF16 = 0
TP_FP32 = 1
# tp_epilogue
TP_EPI_NONE = 0
TP_EPI_GELU = 1
TP_EPI_DGELU = 2
# tp_op
TP_OP_ROW_AR = 0
TP_OP_ROW_RS = 1
TP_OP_COL_FWD = 2
TP_OP_COL_BWD = 3
TP_OP_ROW_BWD = 4
TP_OP_AG_MM = 5
TP_OP_ROW_AR_UNFUSED = 6
TP_OP_AG_MM_BWD = 7
TP_OP_ROW_RS_BWD = 8
TP_OP_BLOCK_NORM_BWD = 9
TP_OP_COL_BWD_CKPT = 10
TP_OP_ROW_BWD_CKPT = 11
TP_OP_AG_MM_BWD_CKPT = 12
TP_OP_ROW_RS_BWD_CKPT = 13
TP_OP_COL_W4 = 14
TP_OP_ROW_W4 = 15
TP_OP_COL_FP8 = 16
TP_OP_ROW_FP8 = 17
TP_OP_COL_BWD_FP8 = 18
TP_OP_ROW_BWD_FP8 = 19
# tp_norm
TP_NORM_NONE = 0
TP_NORM_RMS = 1
TP_NORM_LAYER = 2
# largest hidden size of the block norms, and most tokens of the 4-bit forward calls
TP_BLOCK_NORM_MAX_H = 16384
TP_W4_MAX_M = 64
# tp_route_score, and the most experts of a routing call
TP_ROUTE_SOFTMAX = 0
TP_ROUTE_SIGMOID = 1
TP_ROUTE_MAX_EXPERTS = 512
# tp_debug_key
TP_DEBUG_TIMEOUT_MS = 0
TP_DEBUG_DROP_LOAD = 1
TP_DEBUG_TILE_MODE = 2
TP_DEBUG_NO_TAIL_SLICES = 3
TP_DEBUG_SPLIT_K = 4
TP_DEBUG_L2_HINTS = 5
TP_DEBUG_TMA_STORE = 6
TP_DEBUG_NO_BWD_FUSION = 7
TP_DEBUG_K_ALTERNATE = 8
# tp_row_linear_fwd_unfused flags
TP_UNFUSED_BF16_COLLECTIVE = 1


class TPError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {tp_status_string(status)} (status {status})")


class _NormDesc(ctypes.Structure):
    """tp_block_norm_desc"""
    _fields_ = [("post", ctypes.c_int), ("pre", ctypes.c_int), ("w_post", ctypes.c_void_p), ("b_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("b_pre", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_rows", ctypes.c_int64), ("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class _NormGrads(ctypes.Structure):
    """tp_block_norm_grads"""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dw_post", "db_post", "dw_pre", "db_pre", "dgate")]


class _RouteDesc(ctypes.Structure):
    """tp_route_desc"""
    _fields_ = [("score", ctypes.c_int), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_best", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class _ExpertsSaved(ctypes.Structure):
    """tp_experts_saved"""
    _fields_ = [(k, ctypes.c_void_p) for k in ("plan", "preact", "out")]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python gemm_reduce_fusion_gb300/build.py` "
            "(nvcc, sm_103a); there is no non-CUDA fallback")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    PP = ctypes.POINTER(ctypes.c_void_p)
    I = ctypes.c_int
    L = ctypes.c_int64
    S = ctypes.c_size_t
    sig = {
        "tp_workspace_size": (S, [I, I, L, L, L, L, I]),
        "tp_row_linear_fwd_allreduce": (I, [PP, PP, P, PP, I, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_fwd_reducescatter": (I, [PP, PP, P, PP, I, L, L, L, L, I, P, S, P]),
        "tp_col_linear_fwd": (I, [P, PP, PP, PP, PP, I, I, L, L, L, L, I, P, S, P]),
        "tp_col_linear_bwd": (I, [P, PP, PP, P, PP, PP, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_bwd": (I, [PP, PP, P, PP, PP, P, PP, I, L, L, L, L, I, P, S, P]),
        "tp_ag_matmul": (I, [PP, PP, PP, PP, P, I, PP, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_fwd_unfused": (I, [PP, PP, P, I, L, L, L, L, I, I, I, P, S, P]),
        "tp_ag_matmul_bwd": (I, [PP, PP, PP, PP, PP, PP, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_bwd_reducescatter": (I, [PP, PP, PP, PP, PP, P, PP, I, L, L, L, L, I, P, S, P]),
        "tp_block_norm_fwd": (I, [PP, PP, PP, PP, P, I, L, L, I, P]),
        "tp_block_norm_bwd": (I, [PP, PP, PP, PP, PP, PP, P, P, I, L, L, I, I, P, S, P]),
        "tp_ckpt_pack": (I, [PP, PP, PP, I, L, L, P]),
        "tp_ckpt_unpack": (I, [PP, PP, PP, I, I, L, L, P]),
        "tp_col_linear_bwd_ckpt": (I, [P, P, PP, PP, P, PP, PP, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_bwd_ckpt": (I, [PP, PP, PP, P, PP, PP, P, I, I, L, L, L, L, I, P, S, P]),
        "tp_ag_matmul_bwd_ckpt": (I, [PP, PP, PP, PP, PP, PP, PP, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_bwd_reducescatter_ckpt": (I, [PP, PP, PP, PP, PP, PP, P, I, I, L, L, L, L, I, P, S, P]),
        "tp_col_linear_fwd_w4": (I, [P, PP, PP, PP, PP, I, I, L, L, L, L, I, P, S, P]),
        "tp_row_linear_fwd_w4": (I, [PP, PP, PP, P, P, I, L, L, L, L, I, P, S, P]),
        "tp_w4_pack": (I, [PP, PP, PP, I, L, L, L, P]),
        "tp_w4_unpack": (I, [PP, PP, PP, I, L, L, L, P]),
        # arrays as plain pointers: half a microsecond a call less for a few of them
        "tp_fp8_pack": (I, [P, P, P, I, I, I, L, L, L, P]),
        "tp_fp8_unpack": (I, [P, P, I, L, L, L, P]),
        "tp_col_linear_fwd_fp8": (I, [P, P, P, P, P, P, I, I, L, L, L, P, S, P]),
        "tp_row_linear_fwd_fp8": (I, [P, P, P, P, I, L, L, L, P, S, P]),
        "tp_col_linear_bwd_fp8": (I, [P, P, P, P, P, P, I, L, L, L, P, S, P]),
        "tp_row_linear_bwd_fp8": (I, [P, P, P, P, P, P, P, I, L, L, L, P, S, P]),
        "tp_route_fwd": (I, [P, P, P, P, P, P, L, L, L, I, P]),
        "tp_route_bwd": (I, [P, P, P, P, P, L, L, L, I, P]),
        "tp_experts_rows": (L, [L, L, L]),
        "tp_experts_plan_size": (S, [L, L, L]),
        "tp_experts_workspace_size": (S, [I, L, L, L, L, L, I]),
        "tp_experts_fwd_fp8": (I, [P, P, P, P, P, P, P, I, L, L, L, L, L, P, S, P]),
        "tp_experts_bwd_fp8": (I, [P, P, P, P, P, P, P, P, P, P, I, L, L, L, L, L, P, S, P]),
        "tp_pipeline_time": (ctypes.c_double, [ctypes.c_double, ctypes.c_double, L]),
        "tp_num_chunks": (L, [L, L]),
        "tp_choose_chunk_m": (L, [I, I, L, L, L]),
        "tp_choose_chunk_m_measured": (L, [L, ctypes.POINTER(L), ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_double), I]),
        "tp_get_device_status": (I, [P, P]),
        "tp_status_string": (ctypes.c_char_p, [I]),
        "tp_debug_set": (I, [I, L]),
        "tp_trace_set": (I, [P, L]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


# ------------------------------------------------------------------ marshalling

def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous (row-major)")
    return t.data_ptr()


def _arr(ts) -> ctypes.Array | None:
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return TP_BF16
    if t.dtype == torch.float32:
        return TP_FP32
    raise ValueError(f"unsupported output dtype {t.dtype}")


def _out_dtype(*groups) -> int:
    """The single output dtype of a call: every output tensor must share it."""
    codes = {_dtype_code(t) for g in groups if g is not None
             for t in (g if isinstance(g, (list, tuple)) else [g])}
    if len(codes) != 1:
        raise ValueError("all outputs of one call must have the same dtype (bfloat16 or float32)")
    return codes.pop()


def _ws(ws):
    return _ptr(ws), ws.nbytes


def _check(status: int, where: str) -> None:
    if status != TP_OK:
        raise TPError(status, where)


# ------------------------------------------------------------------ argument checks
#
# The C ABI takes one M, N, K for all shards and plain pointers: it cannot see
# how large a buffer is, so a shard of the wrong shape would be read or
# written out of bounds on the device.  The binding knows every tensor's
# shape and checks them on the host before anything is enqueued: shape,
# bfloat16 for inputs, row-major layout, and the calling thread's current
# CUDA device (the device the library runs the call on).  None stands for a
# NULL pointer; the library decides where NULL is allowed.

_GET_DEVICE = None


def _current_device() -> int:
    global _GET_DEVICE
    if _GET_DEVICE is None:
        import torch
        dev = torch.cuda.current_device()  # initialises CUDA
        _GET_DEVICE = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        return dev
    return _GET_DEVICE()


def _need(where: str, name: str, t, shape, bf16: bool, dev: int) -> None:
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if bf16:
        import torch
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{where}: {name} must be bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous (row-major)")
    if t.get_device() != dev:
        raise TypeError(f"{where}: {name} is on {t.device}; the call runs on cuda:{dev}, "
                        "the calling thread's current device")


def _need_all(where: str, name: str, ts, counts, shape, bf16: bool, dev: int) -> None:
    if ts is None:
        return
    if len(ts) not in counts:
        raise ValueError(f"{where}: {name} holds {len(ts)} tensors, expected "
                         + " or ".join(str(c) for c in counts))
    for i, t in enumerate(ts):
        _need(where, f"{name}[{i}]", t, shape, bf16, dev)


def _need_ws(where: str, ws, dev: int) -> None:
    if ws.get_device() != dev:
        raise TypeError(f"{where}: the workspace is on {ws.device}; the call runs on cuda:{dev}")


# ------------------------------------------------------------------ host-only calls

def tp_status_string(status: int) -> str:
    return _lib.tp_status_string(int(status)).decode()


def tp_workspace_size(op: int, p: int, M: int, N: int, K: int, chunk_m: int = 0,
                      out_dtype: int = TP_BF16) -> int:
    return int(_lib.tp_workspace_size(op, p, M, N, K, chunk_m, out_dtype))


def tp_pipeline_time(c: float, m: float, n_chunks: int) -> float:
    return float(_lib.tp_pipeline_time(c, m, n_chunks))


def tp_num_chunks(M: int, chunk_m: int) -> int:
    return int(_lib.tp_num_chunks(M, chunk_m))


def tp_choose_chunk_m(op: int, p: int, M: int, N: int, K: int) -> int:
    return int(_lib.tp_choose_chunk_m(op, p, M, N, K))


def tp_choose_chunk_m_measured(M: int, chunks: Sequence[int], c: Sequence[float], m: Sequence[float]) -> int:
    """The candidate chunk_m whose timeline from measured per-chunk c and m is shortest."""
    n = len(chunks)
    if not (len(c) == len(m) == n):
        raise ValueError("one c and one m per candidate chunk")
    return int(_lib.tp_choose_chunk_m_measured(M, (ctypes.c_int64 * n)(*chunks), (ctypes.c_double * n)(*c),
                                               (ctypes.c_double * n)(*m), n))


def workspace(op: int, p: int, M: int, N: int, K: int, chunk_m: int = 0, device="cuda",
              out_dtype: int = TP_BF16):
    """A zero-filled device workspace of tp_workspace_size(...) bytes (torch-allocated)."""
    import torch
    n = tp_workspace_size(op, p, M, N, K, chunk_m, out_dtype)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tp_trace_set(buf, cap_units: int = 0) -> None:
    """Trace the GEMM launches that follow into ``buf`` (a zeroed CUDA
    int64 tensor of cap_units x 4), or stop tracing with ``buf=None``."""
    _check(_lib.tp_trace_set(_ptr(buf), cap_units if buf is not None else 0), "tp_trace_set")


def tp_debug_set(key: int, value: int) -> int:
    """Test hook of the failure-detection path (see tp_fused.h)."""
    return int(_lib.tp_debug_set(key, value))


def tp_get_device_status(ws, stream=None) -> int:
    """Latched device status of ``ws`` (synchronises the stream, clears it)."""
    return int(_lib.tp_get_device_status(_ptr(ws), _stream(stream)))


# ------------------------------------------------------------------ the sharded Linear

def tp_row_linear_fwd_allreduce(x: Sequence, w: Sequence, y: Sequence, ws, chunk_m: int = 0,
                                stream=None, bias=None) -> None:
    """Y = sum_r X_r W_r (+ bias) written once (len(y) == 1) or as p replicas (len(y) == p)."""
    p = len(x)
    M, K = x[0].shape
    N = w[0].shape[1]
    W, dev = "tp_row_linear_fwd_allreduce", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "y", y, (1, p), (M, N), False, dev)
    _need(W, "bias", bias, (N,), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_fwd_allreduce(_arr(x), _arr(w), _ptr(bias), _arr(y), len(y), p, M, N, K, chunk_m,
                                            _dtype_code(y[0]), wp, wb, _stream(stream)),
           "tp_row_linear_fwd_allreduce")


def tp_row_linear_fwd_reducescatter(x: Sequence, w: Sequence, y: Sequence, ws, chunk_m: int = 0,
                                    stream=None, bias=None) -> None:
    """Rank j's y[j] = rows [j M/p, (j+1) M/p) of sum_r X_r W_r (+ bias)."""
    p = len(x)
    M, K = x[0].shape
    N = w[0].shape[1]
    W, dev = "tp_row_linear_fwd_reducescatter", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "y", y, (p,), (M // p, N), False, dev)
    _need(W, "bias", bias, (N,), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_fwd_reducescatter(_arr(x), _arr(w), _ptr(bias), _arr(y), p, M, N, K, chunk_m,
                                                _dtype_code(y[0]), wp, wb, _stream(stream)),
           "tp_row_linear_fwd_reducescatter")


def tp_col_linear_fwd(x, w: Sequence, y: Sequence, ws, epi: int = TP_EPI_NONE, preact=None,
                      chunk_m: int = 0, stream=None, bias=None) -> None:
    """y[k] = X A_k + b_k (or GeLU of it, with H_k into preact[k]); bias[k] = b_k or bias None."""
    p = len(w)
    M, K = x.shape
    N = w[0].shape[1]
    W, dev = "tp_col_linear_fwd", _current_device()
    _need(W, "x", x, (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "y", y, (p,), (M, N), False, dev)
    _need_all(W, "preact", preact, (p,), (M, N), False, dev)
    _need_all(W, "bias", bias, (p,), (N,), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_col_linear_fwd(_ptr(x), _arr(w), _arr(bias), _arr(y), _arr(preact), epi, p, M, N, K, chunk_m,
                                  _out_dtype(y, preact), wp, wb, _stream(stream)), "tp_col_linear_fwd")


def tp_col_linear_bwd(x, w: Sequence, dy: Sequence, dx, dw, ws, chunk_m: int = 0,
                      stream=None, db=None) -> None:
    """dX = sum_k dY_k A_k^T; dw[k] = X^T dY_k; db[k] = row sum of dY_k (dx, dw, db may be None)."""
    p = len(w)
    K, N = w[0].shape
    M = dy[0].shape[0]
    W, dev = "tp_col_linear_bwd", _current_device()
    _need(W, "x", x, (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "dy", dy, (p,), (M, N), True, dev)
    _need(W, "dx", dx, (M, K), False, dev)
    _need_all(W, "dw", dw, (p,), (K, N), False, dev)
    _need_all(W, "db", db, (p,), (N,), False, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_col_linear_bwd(_ptr(x), _arr(w), _arr(dy), _ptr(dx), _arr(dw), _arr(db), p, M, N, K,
                                  chunk_m, _out_dtype(dx, dw, db), wp, wb, _stream(stream)), "tp_col_linear_bwd")


def tp_row_linear_bwd(x, w: Sequence, dy, dx, dw, ws, preact=None, chunk_m: int = 0,
                      stream=None, db=None) -> None:
    """dx[k] = dY A_k^T (times GeLU'(preact[k])); dw[k] = X_k^T dY; db = row sum of dY."""
    p = len(w)
    K, N = w[0].shape
    M = dy.shape[0]
    W, dev = "tp_row_linear_bwd", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need(W, "dy", dy, (M, N), True, dev)
    _need_all(W, "dx", dx, (p,), (M, K), False, dev)
    _need_all(W, "dw", dw, (p,), (K, N), False, dev)
    _need(W, "db", db, (N,), False, dev)
    _need_all(W, "preact", preact, (p,), (M, K), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_bwd(_arr(x), _arr(w), _ptr(dy), _arr(dx), _arr(dw), _ptr(db), _arr(preact), p,
                                  M, N, K, chunk_m, _out_dtype(dx, dw, db), wp, wb, _stream(stream)),
           "tp_row_linear_bwd")


def tp_ag_matmul(x: Sequence, w: Sequence, y: Sequence, ws, x_gathered=None,
                 epi: int = TP_EPI_NONE, preact=None, chunk_m: int = 0, stream=None, bias=None) -> None:
    """y[k] = [X_0; ...; X_{p-1}] A_k + b_k (optionally GeLU, H_k, gathered X)."""
    p = len(x)
    Mp, K = x[0].shape
    N = w[0].shape[1]
    W, dev = "tp_ag_matmul", _current_device()
    _need_all(W, "x", x, (p,), (Mp, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "y", y, (p,), (Mp * p, N), False, dev)
    _need(W, "x_gathered", x_gathered, (Mp * p, K), True, dev)
    _need_all(W, "preact", preact, (p,), (Mp * p, N), False, dev)
    _need_all(W, "bias", bias, (p,), (N,), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_ag_matmul(_arr(x), _arr(w), _arr(bias), _arr(y), _ptr(x_gathered), epi, _arr(preact), p,
                             Mp * p, N, K, chunk_m, _out_dtype(y, preact), wp, wb, _stream(stream)),
           "tp_ag_matmul")


def tp_ag_matmul_bwd(x, w: Sequence, dy: Sequence, dx, dw, ws, chunk_m: int = 0, stream=None,
                     db=None) -> None:
    """dx[s] = rows of sum_k dY_k A_k^T (ReduceScatter); dw[k] = [X_0;...]^T dY_k; db[k] = row sum of dY_k."""
    p = len(w)
    K, N = w[0].shape
    M = dy[0].shape[0]
    W, dev = "tp_ag_matmul_bwd", _current_device()
    _need_all(W, "x", x, (p,), (M // p, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "dy", dy, (p,), (M, N), True, dev)
    _need_all(W, "dx", dx, (p,), (M // p, K), False, dev)
    _need_all(W, "dw", dw, (p,), (K, N), False, dev)
    _need_all(W, "db", db, (p,), (N,), False, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_ag_matmul_bwd(_arr(x), _arr(w), _arr(dy), _arr(dx), _arr(dw), _arr(db), p, M, N, K, chunk_m,
                                 _out_dtype(dx, dw, db), wp, wb, _stream(stream)), "tp_ag_matmul_bwd")


def tp_row_linear_bwd_reducescatter(x, w: Sequence, dy: Sequence, dx, dw, ws, preact=None, chunk_m: int = 0,
                                    stream=None, db=None) -> None:
    """dx[r] = [dY_0;...] A_r^T (* GeLU'(preact[r])) (AllGather); dw[r] = X_r^T [dY_0;...];
    db = row sum of all the dY shards."""
    p = len(w)
    K, N = w[0].shape
    M = dy[0].shape[0] * p
    W, dev = "tp_row_linear_bwd_reducescatter", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "dy", dy, (p,), (M // p, N), True, dev)
    _need_all(W, "dx", dx, (p,), (M, K), False, dev)
    _need_all(W, "dw", dw, (p,), (K, N), False, dev)
    _need(W, "db", db, (N,), False, dev)
    _need_all(W, "preact", preact, (p,), (M, K), True, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_bwd_reducescatter(_arr(x), _arr(w), _arr(dy), _arr(dx), _arr(dw), _ptr(db),
                                                _arr(preact), p, M, N, K, chunk_m, _out_dtype(dx, dw, db), wp, wb,
                                                _stream(stream)), "tp_row_linear_bwd_reducescatter")


def tp_row_linear_fwd_unfused(x: Sequence, w: Sequence, y, ws, chunk_m: int = 0, phases: int = 3,
                              flags: int = 0, stream=None) -> None:
    """Unfused baseline: per-rank fp32 partials (phase 1), rank-order reduce into y (phase 2);
    flags=TP_UNFUSED_BF16_COLLECTIVE sums bf16-rounded partials with a bf16 running sum."""
    p = len(x)
    M, K = x[0].shape
    N = w[0].shape[1]
    W, dev = "tp_row_linear_fwd_unfused", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need(W, "y", y, (M, N), False, dev)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_fwd_unfused(_arr(x), _arr(w), _ptr(y), p, M, N, K, chunk_m, _dtype_code(y),
                                          phases, flags, wp, wb, _stream(stream)), "tp_row_linear_fwd_unfused")


def tp_row_linear_fwd_allreduce_noalloc(x: Sequence, w: Sequence, y: Sequence, chunk_m: int = 0,
                                        stream=None) -> None:
    """tp_row_linear_fwd_allreduce without a workspace: for callers that
    cannot allocate device memory (the library uses its static scratch)."""
    fn = _lib.tp_row_linear_fwd_allreduce_noalloc
    fn.restype = ctypes.c_int
    PP = ctypes.POINTER(ctypes.c_void_p)
    L = ctypes.c_int64
    fn.argtypes = [PP, PP, PP, ctypes.c_int, ctypes.c_int, L, L, L, L, ctypes.c_int, ctypes.c_void_p]
    p = len(x)
    M, K = x[0].shape
    N = w[0].shape[1]
    W, dev = "tp_row_linear_fwd_allreduce_noalloc", _current_device()
    _need_all(W, "x", x, (p,), (M, K), True, dev)
    _need_all(W, "w", w, (p,), (K, N), True, dev)
    _need_all(W, "y", y, (1, p), (M, N), False, dev)
    _check(fn(_arr(x), _arr(w), _arr(y), len(y), p, M, N, K, chunk_m, _dtype_code(y[0]), _stream(stream)),
           "tp_row_linear_fwd_allreduce_noalloc")


def tp_noalloc_device_status(stream=None) -> int:
    """Read and clear the status word of the allocation-free entry point's
    static scratch (synchronises the stream): TP_OK or TP_ERR_DEVICE_TIMEOUT."""
    fn = _lib.tp_noalloc_device_status
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p]
    return fn(_stream(stream))


# ------------------------------------------------------------------ around the sharded Linear
#
# The calls below take few microseconds on the device when they serve single
# tokens, so their checks read each property of a tensor once and go through
# _refuse, which finds the words, only when something is wrong.

_ARRAY = tuple(ctypes.c_void_p * n for n in range(65))  # the C array types, looked up once
_BF16 = _FP32 = _INT8 = _UINT8 = _INT32 = _E4M3 = _RAW_STREAM = None


def _begin() -> int:
    """The current device; the first call fetches torch's dtypes and stream getter."""
    global _BF16, _FP32, _INT8, _UINT8, _INT32, _E4M3, _RAW_STREAM
    if _BF16 is None:
        import torch
        _FP32, _INT8, _UINT8, _INT32, _E4M3 = torch.float32, torch.int8, torch.uint8, torch.int32, torch.float8_e4m3fn
        # the current stream's handle without a Stream object around it, where torch has it
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _BF16 = torch.bfloat16
    return _current_device()


def _on(stream, dev: int) -> int:
    return _RAW_STREAM(dev) if stream is None else _stream(stream)


def _list(where: str, name: str, ts, count: int, shape, dtype, dev: int):
    """The C array of `count` tensors of one shape and dtype (None: NULL)."""
    if ts is None:
        return None
    if len(ts) != count:
        raise ValueError(f"{where}: {name} holds {len(ts)} tensors, expected {count}")
    arr = _ARRAY[count]()
    i = 0
    for t in ts:
        if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            _refuse(where, f"{name}[{i}]", t, shape, dtype, dev)
        arr[i] = t.data_ptr()
        i += 1
    return arr


def _one(where: str, name: str, t, shape, dtype, dev: int):
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(where, name, t, shape, dtype, dev)
    return t.data_ptr()


def _refuse(where: str, name: str, t, shape, dtype, dev: int) -> None:
    _need(where, name, t, shape, False, dev)
    raise TypeError(f"{where}: {name} must be {str(dtype).replace('torch.', '')}, got {t.dtype}")


def _norm_args(where, h, post, w_post, b_post, pre, w_pre, b_pre, gate, alpha, eps, dev):
    rows, v, bf = 0, (h,), _BF16
    if gate is not None:
        if gate.dim() != 2:
            raise ValueError(f"{where}: gate is [rows, h], got {tuple(gate.shape)}")
        rows = gate.shape[0]
        gate = _one(where, "gate", gate, (rows, h), bf, dev)
    return _NormDesc(post, pre, w_post if w_post is None else _one(where, "w_post", w_post, v, bf, dev),
                     b_post if b_post is None else _one(where, "b_post", b_post, v, bf, dev),
                     w_pre if w_pre is None else _one(where, "w_pre", w_pre, v, bf, dev),
                     b_pre if b_pre is None else _one(where, "b_pre", b_pre, v, bf, dev), gate, rows, alpha, eps)


def _residual(where, t):
    if t.dim() != 2:
        raise ValueError(f"{where}: a token shard is [tokens, h], got {tuple(t.shape)}")
    m, h = t.shape
    dtype = t.dtype
    if dtype is _BF16:
        return m, h, dtype, TP_BF16
    if dtype is _FP32:
        return m, h, dtype, TP_FP32
    raise TypeError(f"{where}: the residual stream is bfloat16 or float32, got {dtype}")


def tp_block_norm_fwd(x: Sequence, z, y, n, *, post: int = TP_NORM_NONE, w_post=None, b_post=None,
                      pre: int = TP_NORM_NONE, w_pre=None, b_pre=None, gate=None, alpha: float = 1.0,
                      eps: float = 1e-5, stream=None) -> None:
    """y[s] = x[s] + alpha gate N_post(z[s]); n[s] = N_pre(y[s]), over p row shards.

    z None (then y None): n[s] = N_pre(x[s]).  n None: y alone.  x and y are
    bfloat16 or float32, z and n bfloat16; gate is [rows, h], its row i / (M / rows)
    for token i of the M = p * len(x[0]) tokens.  y[s] may be x[s]."""
    W, dev, p = "tp_block_norm_fwd", _begin(), len(x)
    m, h, dtype, code = _residual(W, x[0])
    shape, bf = (m, h), _BF16
    d = _norm_args(W, h, post, w_post, b_post, pre, w_pre, b_pre, gate, alpha, eps, dev)
    _check(_lib.tp_block_norm_fwd(_list(W, "x", x, p, shape, dtype, dev), _list(W, "z", z, p, shape, bf, dev),
                                  _list(W, "y", y, p, shape, dtype, dev), _list(W, "n", n, p, shape, bf, dev),
                                  ctypes.byref(d), p, p * m, h, code, _on(stream, dev)), W)


def tp_block_norm_bwd(z, y, dn, dy, dx, dz, ws, *, post: int = TP_NORM_NONE, w_post=None, b_post=None,
                      pre: int = TP_NORM_NONE, w_pre=None, b_pre=None, gate=None, alpha: float = 1.0,
                      eps: float = 1e-5, dw_post=None, db_post=None, dw_pre=None, db_pre=None, dgate=None,
                      stream=None) -> None:
    """Gradients of tp_block_norm_fwd: dx[s], dz[s] and those of the vectors.

    y: the stream after the boundary (the forward x when z is None), needed
    with dn; dn, dy: gradients of n and (from its later uses) of y, either may
    be None; dx, dz and each vector's gradient may be None.  dy, y, dx share
    one dtype; the vectors' gradients share one (bfloat16 or float32).
    dx[s] may be dy[s].  ws: workspace(TP_OP_BLOCK_NORM_BWD, p, M, h, 0)."""
    W, dev = "tp_block_norm_bwd", _begin()
    first = y or dy or dx
    if not first:
        raise ValueError(f"{W}: one of y, dy and dx is given")
    p = len(first)
    m, h, dtype, code = _residual(W, first[0])
    shape, v, bf = (m, h), (h,), _BF16
    d = _norm_args(W, h, post, w_post, b_post, pre, w_pre, b_pre, gate, alpha, eps, dev)
    out = _FP32
    for t in (dw_post, db_post, dw_pre, db_pre, dgate):
        if t is not None:
            out = t.dtype
            break
    if out is not _BF16 and out is not _FP32:
        raise TypeError(f"{W}: gradients are bfloat16 or float32, got {out}")
    g = _NormGrads(_one(W, "dw_post", dw_post, v, out, dev), _one(W, "db_post", db_post, v, out, dev),
                   _one(W, "dw_pre", dw_pre, v, out, dev), _one(W, "db_pre", db_pre, v, out, dev),
                   dgate if dgate is None else _one(W, "dgate", dgate, gate.shape if gate is not None else (0, h), out, dev))
    _need_ws(W, ws, dev)
    _check(_lib.tp_block_norm_bwd(_list(W, "z", z, p, shape, bf, dev), _list(W, "y", y, p, shape, dtype, dev),
                                  _list(W, "dn", dn, p, shape, bf, dev), _list(W, "dy", dy, p, shape, dtype, dev),
                                  _list(W, "dx", dx, p, shape, dtype, dev), _list(W, "dz", dz, p, shape, bf, dev),
                                  ctypes.byref(d), ctypes.byref(g), p, p * m, h, code, TP_FP32 if out is _FP32 else TP_BF16,
                                  *_ws(ws), _on(stream, dev)), W)


def ckpt_shapes(M: int, N: int) -> tuple:
    """Shapes of a checkpoint of an [M, N] activation: (q int8, e uint8)."""
    return (M, N), (M, (N + 31) // 32)


def tp_ckpt_pack(x: Sequence, q: Sequence, e: Sequence, stream=None) -> None:
    """(q[i], e[i]) = x[i] in 8 bits: int8 [M, N] and a power of two per 32 columns, uint8 [M, ceil(N/32)]."""
    W, dev, p = "tp_ckpt_pack", _begin(), len(x)
    M, N = x[0].shape
    qs, es = ckpt_shapes(M, N)
    _check(_lib.tp_ckpt_pack(_list(W, "x", x, p, (M, N), _BF16, dev), _list(W, "q", q, p, qs, _INT8, dev),
                             _list(W, "e", e, p, es, _UINT8, dev), p, M, N, _on(stream, dev)), W)


def tp_ckpt_unpack(q: Sequence, e: Sequence, y: Sequence, epi: int = TP_EPI_NONE, stream=None) -> None:
    """y[i] = the value of (q[i], e[i]), or its GeLU (epi=TP_EPI_GELU), in bfloat16."""
    W, dev, p = "tp_ckpt_unpack", _begin(), len(q)
    M, N = q[0].shape
    qs, es = ckpt_shapes(M, N)
    _check(_lib.tp_ckpt_unpack(_list(W, "q", q, p, qs, _INT8, dev), _list(W, "e", e, p, es, _UINT8, dev),
                               _list(W, "y", y, p, (M, N), _BF16, dev), epi, p, M, N, _on(stream, dev)), W)


def tp_col_linear_bwd_ckpt(q, e, w: Sequence, dy: Sequence, dx, dw, ws, chunk_m: int = 0, stream=None, db=None) -> None:
    """tp_col_linear_bwd with X given as a checkpoint (q, e) (both None without dw)."""
    W, dev, p, bf = "tp_col_linear_bwd_ckpt", _begin(), len(w), _BF16
    (K, N), M = w[0].shape, dy[0].shape[0]
    qs, es = ckpt_shapes(M, K)
    out = _out_dtype(dx, dw, db)
    od = _FP32 if out == TP_FP32 else bf
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_col_linear_bwd_ckpt(
        _one(W, "q", q, qs, _INT8, dev), _one(W, "e", e, es, _UINT8, dev), _list(W, "w", w, p, (K, N), bf, dev),
        _list(W, "dy", dy, p, (M, N), bf, dev), _one(W, "dx", dx, (M, K), od, dev), _list(W, "dw", dw, p, (K, N), od, dev),
        _list(W, "db", db, p, (N,), od, dev), p, M, N, K, chunk_m, out, wp, wb, _on(stream, dev)), W)


def tp_row_linear_bwd_ckpt(q, e, w: Sequence, dy, dx, dw, ws, epi: int = TP_EPI_DGELU, chunk_m: int = 0, stream=None,
                           db=None) -> None:
    """tp_row_linear_bwd from checkpoints: of the pre-activations H_k (epi=TP_EPI_DGELU: dx[k] = dY A_k^T * GeLU'(H_k),
    dw[k] = GeLU(H_k)^T dY) or of the layer's inputs X_k (epi=TP_EPI_NONE)."""
    W, dev, p, bf = "tp_row_linear_bwd_ckpt", _begin(), len(w), _BF16
    (K, N), M = w[0].shape, dy.shape[0]
    qs, es = ckpt_shapes(M, K)
    out = _out_dtype(dx, dw, db)
    od = _FP32 if out == TP_FP32 else bf
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_bwd_ckpt(
        _list(W, "q", q, p, qs, _INT8, dev), _list(W, "e", e, p, es, _UINT8, dev),
        _list(W, "w", w, p, (K, N), bf, dev), _one(W, "dy", dy, (M, N), bf, dev), _list(W, "dx", dx, p, (M, K), od, dev),
        _list(W, "dw", dw, p, (K, N), od, dev), _one(W, "db", db, (N,), od, dev), epi, p, M, N, K, chunk_m, out, wp, wb,
        _on(stream, dev)), W)


def tp_ag_matmul_bwd_ckpt(q, e, w: Sequence, dy: Sequence, dx, dw, ws, chunk_m: int = 0, stream=None, db=None) -> None:
    """tp_ag_matmul_bwd with the token shards X_s given as checkpoints (None without dw)."""
    W, dev, p, bf = "tp_ag_matmul_bwd_ckpt", _begin(), len(w), _BF16
    (K, N), M = w[0].shape, dy[0].shape[0]
    qs, es = ckpt_shapes(M // p, K)
    out = _out_dtype(dx, dw, db)
    od = _FP32 if out == TP_FP32 else bf
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_ag_matmul_bwd_ckpt(
        _list(W, "q", q, p, qs, _INT8, dev), _list(W, "e", e, p, es, _UINT8, dev),
        _list(W, "w", w, p, (K, N), bf, dev), _list(W, "dy", dy, p, (M, N), bf, dev),
        _list(W, "dx", dx, p, (M // p, K), od, dev), _list(W, "dw", dw, p, (K, N), od, dev),
        _list(W, "db", db, p, (N,), od, dev), p, M, N, K, chunk_m, out, wp, wb, _on(stream, dev)), W)


def tp_row_linear_bwd_reducescatter_ckpt(q, e, w: Sequence, dy: Sequence, dx, dw, ws, epi: int = TP_EPI_DGELU,
                                         chunk_m: int = 0, stream=None, db=None) -> None:
    """tp_row_linear_bwd_reducescatter from checkpoints, as tp_row_linear_bwd_ckpt; dy[s] are row shards."""
    W, dev, p, bf = "tp_row_linear_bwd_reducescatter_ckpt", _begin(), len(w), _BF16
    (K, N), M = w[0].shape, dy[0].shape[0] * len(w)
    qs, es = ckpt_shapes(M, K)
    out = _out_dtype(dx, dw, db)
    od = _FP32 if out == TP_FP32 else bf
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_bwd_reducescatter_ckpt(
        _list(W, "q", q, p, qs, _INT8, dev), _list(W, "e", e, p, es, _UINT8, dev),
        _list(W, "w", w, p, (K, N), bf, dev), _list(W, "dy", dy, p, (M // p, N), bf, dev),
        _list(W, "dx", dx, p, (M, K), od, dev), _list(W, "dw", dw, p, (K, N), od, dev),
        _one(W, "db", db, (N,), od, dev), epi, p, M, N, K, chunk_m, out, wp, wb, _on(stream, dev)), W)


def w4_shapes(K: int, N: int, group: int) -> tuple:
    """Shapes of a 4-bit weight [K, N]: (q uint8, s bfloat16)."""
    return ((N + 31) // 32, (K + 63) // 64, 1024), ((N + 31) // 32, (K + group - 1) // group, 32)


def _group(where: str, group: int) -> int:
    if group not in (32, 64, 128):
        raise ValueError(f"{where}: group is 32, 64 or 128 rows, got {group}")
    return group


def tp_col_linear_fwd_w4(x, q: Sequence, s: Sequence, y: Sequence, ws, group: int = 128, epi: int = TP_EPI_NONE,
                         stream=None, bias=None) -> None:
    """y[k] = X W_k + b_k (or its GeLU) with 4-bit weights (q[k], s[k]); up to TP_W4_MAX_M tokens."""
    W, dev, p, bf = "tp_col_linear_fwd_w4", _begin(), len(q), _BF16
    (M, K), N, dtype = x.shape, y[0].shape[1], y[0].dtype
    qs, ss = w4_shapes(K, N, _group(W, group))
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_col_linear_fwd_w4(
        _one(W, "x", x, (M, K), bf, dev), _list(W, "q", q, p, qs, _UINT8, dev), _list(W, "s", s, p, ss, bf, dev),
        _list(W, "bias", bias, p, (N,), bf, dev), _list(W, "y", y, p, (M, N), dtype, dev), epi, p, M, N, K, group,
        _dtype_code(y[0]), wp, wb, _on(stream, dev)), W)


def tp_row_linear_fwd_w4(x: Sequence, q: Sequence, s: Sequence, y, ws, group: int = 128, stream=None, bias=None) -> None:
    """y = sum_r X_r W_r (+ bias) with 4-bit weights (q[r], s[r]); up to TP_W4_MAX_M tokens."""
    W, dev, p, bf = "tp_row_linear_fwd_w4", _begin(), len(q), _BF16
    (M, K), N, dtype = x[0].shape, y.shape[1], y.dtype
    qs, ss = w4_shapes(K, N, _group(W, group))
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_fwd_w4(
        _list(W, "x", x, p, (M, K), bf, dev), _list(W, "q", q, p, qs, _UINT8, dev), _list(W, "s", s, p, ss, bf, dev),
        _one(W, "bias", bias, (N,), bf, dev), _one(W, "y", y, (M, N), dtype, dev), p, M, N, K, group, _dtype_code(y), wp, wb,
        _on(stream, dev)), W)


def tp_w4_pack(w: Sequence, q: Sequence, s: Sequence, group: int = 128, stream=None) -> None:
    """(q[r], s[r]) = w[r] [K, N] in 4 bits, a scale max|w| / 7 for each column and group of rows."""
    W, dev, p, bf = "tp_w4_pack", _begin(), len(w), _BF16
    K, N = w[0].shape
    qs, ss = w4_shapes(K, N, _group(W, group))
    _check(_lib.tp_w4_pack(_list(W, "w", w, p, (K, N), bf, dev), _list(W, "q", q, p, qs, _UINT8, dev),
                           _list(W, "s", s, p, ss, bf, dev), p, N, K, group, _on(stream, dev)), W)


def tp_w4_unpack(q: Sequence, s: Sequence, w: Sequence, group: int = 128, stream=None) -> None:
    """w[r] [K, N] in bfloat16 of the 4-bit weights (q[r], s[r])."""
    W, dev, p, bf = "tp_w4_unpack", _begin(), len(w), _BF16
    K, N = w[0].shape
    qs, ss = w4_shapes(K, N, _group(W, group))
    _check(_lib.tp_w4_unpack(_list(W, "q", q, p, qs, _UINT8, dev), _list(W, "s", s, p, ss, bf, dev),
                             _list(W, "w", w, p, (K, N), bf, dev), p, N, K, group, _on(stream, dev)), W)


# ------------------------------------------------------------------ 8-bit operands

class Fp8(NamedTuple):
    """An operand in 8 bits: a matrix [rows, cols] whose products sum over its columns.

    q: float8_e4m3fn [rows, cols rounded up to 128], zeros past cols; e: uint8 [ceil(rows/128), ceil(cols/512), 512],
    the exponents of a power of two for each row and 128 columns.  Both may have a leading dimension of matrices."""
    q: object
    e: object


def fp8_shapes(rows: int, cols: int) -> tuple:
    """Shapes of the operand of a matrix [rows, cols]: (q float8_e4m3fn, e uint8)."""
    return (rows, (cols + 127) // 128 * 128), ((rows + 127) // 128, (cols + 511) // 512, 512)


def fp8_empty(rows: int, cols: int, batch: int | None = None, device="cuda") -> Fp8:
    """An operand (or `batch` of them, one after the other) to be packed into."""
    import torch
    qs, es = fp8_shapes(rows, cols)
    lead = () if batch is None else (batch,)
    return Fp8(torch.empty(lead + qs, dtype=torch.float8_e4m3fn, device=device),
               torch.empty(lead + es, dtype=torch.uint8, device=device))


def _fp8s(where: str, name: str, ts, count: int, rows: int, cols: int, dev: int, lead: tuple = ()):
    """The C array of `count` operands of [rows, cols] (None: NULL)."""
    if ts is None:
        return None
    if len(ts) != count:
        raise ValueError(f"{where}: {name} holds {len(ts)} operands, expected {count}")
    qs, es = (*lead, rows, (cols + 127) // 128 * 128), (*lead, (rows + 127) // 128, (cols + 511) // 512, 512)
    arr, i = _ARRAY[2 * count](), 0
    for q, e in ts:
        if (q.shape != qs or e.shape != es or q.dtype is not _E4M3 or e.dtype is not _UINT8 or q.get_device() != dev
                or e.get_device() != dev or not q.is_contiguous() or not e.is_contiguous()):
            for part, t, shape, dtype in (("q", q, qs, _E4M3), ("e", e, es, _UINT8)):
                if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
                    _refuse(where, f"{name}[{i // 2}].{part}", t, shape, dtype, dev)
        arr[i] = q.data_ptr()
        arr[i + 1] = e.data_ptr()
        i += 2
    return arr


def _matrices(where: str, t) -> tuple:
    """(leading shape, matrices, rows, cols) of a tensor [M, N] or [batch, M, N]."""
    if t.dim() == 2:
        return (), 1, t.shape[0], t.shape[1]
    if t.dim() == 3:
        return (t.shape[0],), t.shape[0], t.shape[1], t.shape[2]
    raise ValueError(f"{where}: a matrix [M, N] or matrices [batch, M, N], got {tuple(t.shape)}")


def tp_fp8_pack(x: Sequence, q=None, qt=None, tiles: bool = False, epi: int = TP_EPI_NONE, stream=None) -> None:
    """q[i] = the operand of x[i] ([M, N] or [batch, M, N]), qt[i] = that of its transpose; either may be None.

    An exponent for each 128 columns of a row (of the operand), or with `tiles` for each 128 x 128, as weights have it;
    epi=TP_EPI_GELU packs GeLU(x[i])."""
    W, dev, p = "tp_fp8_pack", _begin(), len(x)
    lead, batch, M, N = _matrices(W, x[0])
    _check(_lib.tp_fp8_pack(_list(W, "x", x, p, lead + (M, N), _BF16, dev), _fp8s(W, "q", q, p, M, N, dev, lead),
                            _fp8s(W, "qt", qt, p, N, M, dev, lead), int(tiles), epi, p, batch, M, N, _on(stream, dev)), W)


def tp_fp8_unpack(q: Sequence, y: Sequence, stream=None) -> None:
    """y[i] = the values of the operand q[i], in bfloat16."""
    W, dev, p = "tp_fp8_unpack", _begin(), len(q)
    lead, batch, M, N = _matrices(W, y[0])
    _check(_lib.tp_fp8_unpack(_fp8s(W, "q", q, p, M, N, dev, lead), _list(W, "y", y, p, lead + (M, N), _BF16, dev), p, batch, M, N,
                              _on(stream, dev)), W)


def tp_col_linear_fwd_fp8(x: Fp8, w: Sequence, y, ws, epi: int = TP_EPI_NONE, preact=None, z=None, stream=None, bias=None) -> None:
    """y[k] = X A_k + b_k (or its GeLU, with H_k into preact[k]) on 8-bit operands: x [M, K], w[k] [N, K], the packed
    transpose of A_k.  With y None the results go to the operands z[k] [M, N]."""
    W, dev, p, bf = "tp_col_linear_fwd_fp8", _begin(), len(w), _BF16
    if (y is None) == (z is None):
        raise ValueError(f"{W}: one of y and z is given")
    (M, K), N = x.q.shape, w[0].q.shape[0]
    if y is not None and y[0].shape[1] != N:
        raise ValueError(f"{W}: y[0] has {y[0].shape[1]} columns, w[0] has {N} rows")
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_col_linear_fwd_fp8(
        _fp8s(W, "x", (x,), 1, M, K, dev), _fp8s(W, "w", w, p, N, K, dev), _list(W, "bias", bias, p, (N,), bf, dev),
        _list(W, "y", y, p, (M, N), bf, dev), _fp8s(W, "z", z, p, M, N, dev), _list(W, "preact", preact, p, (M, N), bf, dev), epi, p, M,
        N, K, wp, wb, _on(stream, dev)), W)


def tp_row_linear_fwd_fp8(x: Sequence, w: Sequence, y, ws, stream=None, bias=None) -> None:
    """y = sum_r X_r A_r (+ bias) on 8-bit operands: x[r] [M, K], w[r] [N, K], the packed transpose of A_r."""
    W, dev, p, bf = "tp_row_linear_fwd_fp8", _begin(), len(w), _BF16
    (M, K), N = x[0].q.shape, w[0].q.shape[0]
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    _check(_lib.tp_row_linear_fwd_fp8(
        _fp8s(W, "x", x, p, M, K, dev), _fp8s(W, "w", w, p, N, K, dev), _one(W, "bias", bias, (N,), bf, dev),
        _one(W, "y", y, (M, N), bf, dev), p, M, N, K, wp, wb, _on(stream, dev)), W)


def _bwd_sizes(where: str, dx, dw, dy, dyt, w, xt, p=None) -> tuple:
    """(M, N, K, p) of a backward call.  An operand's rows are exact, its columns rounded up to 128: with dw alone, M
    is what the operands hold, a multiple of 128."""
    if dx is not None:
        if w is None or dy is None or dy[0] is None:
            raise ValueError(f"{where}: dx needs w and dy")
        (M, K), N = dx.shape, dw[0].shape[1] if dw is not None else w[0].q.shape[1]
    elif dw is not None:
        if xt is None or dyt is None or dyt[0] is None:
            raise ValueError(f"{where}: dw needs xt and dyt")
        (K, N), M = dw[0].shape, dyt[0].q.shape[1]
    else:
        raise ValueError(f"{where}: dx or dw is given")
    if dw is not None and (xt is None or dyt is None or dyt[0] is None):
        raise ValueError(f"{where}: dw needs xt and dyt")
    return M, N, K, len(dw if dw is not None else w) if p is None else p


def tp_col_linear_bwd_fp8(xt, w, dy, dyt, dx, dw, ws, stream=None) -> None:
    """dx = sum_k dY_k A_k^T from w[k] [K, N] (packed A_k) and dy[k] [M, N]; dw[k] = X^T dY_k from xt [K, M] and dyt[k] [N, M].

    dx (with w, dy) or dw (with xt, dyt) may be None."""
    W, dev, bf = "tp_col_linear_bwd_fp8", _begin(), _BF16
    M, N, K, p = _bwd_sizes(W, dx, dw, dy, dyt, w, xt)
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    need_x, need_w = dx is not None, dw is not None
    _check(_lib.tp_col_linear_bwd_fp8(
        _fp8s(W, "xt", (xt,) if need_w else None, 1, K, M, dev), _fp8s(W, "w", w if need_x else None, p, K, N, dev),
        _fp8s(W, "dy", dy if need_x else None, p, M, N, dev), _fp8s(W, "dyt", dyt if need_w else None, p, N, M, dev),
        _one(W, "dx", dx, (M, K), bf, dev), _list(W, "dw", dw, p, (K, N), bf, dev), p, M, N, K, wp, wb, _on(stream, dev)), W)


def tp_row_linear_bwd_fp8(xt, w, dy, dyt, dx, dw, ws, preact=None, stream=None) -> None:
    """dx[k] = dY A_k^T (times GeLU'(preact[k])) from w[k] [K, N] (packed A_k) and dy [M, N]; dw[k] = X_k^T dY from xt[k] [K, M]
    and dyt [N, M].

    dx (with w, dy) or dw (with xt, dyt) may be None."""
    W, dev, bf = "tp_row_linear_bwd_fp8", _begin(), _BF16
    M, N, K, p = _bwd_sizes(W, dx and dx[0], dw, (dy,), (dyt,), w, xt and xt[0], len(dx or dw or ()))
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    need_x, need_w = dx is not None, dw is not None
    _check(_lib.tp_row_linear_bwd_fp8(
        _fp8s(W, "xt", xt if need_w else None, p, K, M, dev), _fp8s(W, "w", w if need_x else None, p, K, N, dev),
        _fp8s(W, "dy", (dy,) if need_x else None, 1, M, N, dev), _fp8s(W, "dyt", (dyt,) if need_w else None, 1, N, M, dev),
        _list(W, "dx", dx, p, (M, K), bf, dev), _list(W, "dw", dw, p, (K, N), bf, dev),
        _list(W, "preact", preact if need_x else None, p, (M, K), bf, dev), p, M, N, K, wp, wb, _on(stream, dev)), W)


# ------------------------------------------------------------------ routing to experts

def _logits(where: str, t) -> tuple:
    if t.dim() != 2:
        raise ValueError(f"{where}: logits are [tokens, experts], got {tuple(t.shape)}")
    if t.dtype is not _BF16 and t.dtype is not _FP32:
        raise TypeError(f"{where}: logits are bfloat16 or float32, got {t.dtype}")
    return t.shape[0], t.shape[1], TP_BF16 if t.dtype is _BF16 else TP_FP32


def _slots(where: str, name: str, t, T: int) -> int:
    if t.dim() != 2 or t.shape[0] != T:
        raise ValueError(f"{where}: {name} is [{T}, k], got {tuple(t.shape)}")
    return t.shape[1]


def tp_route_fwd(logits, experts, weights, counts=None, *, bias=None, score: int = TP_ROUTE_SOFTMAX, groups: int = 1,
                 top_groups: int = 1, group_best: int = 1, renorm: bool = False, scale: float = 1.0, stream=None) -> None:
    """experts[t] (int32 [T, k]) and weights[t] (float32 [T, k]) of the k best of logits[t] ([T, E], bfloat16 or float32).

    The choice is by s + bias, s the softmax or sigmoid of the logits, among the top_groups groups with the largest sums
    of their group_best best; weights = scale * s, with renorm over the sum of the chosen.  An expert with a logit of -inf
    or NaN is closed; a slot without an open expert gets -1 and 0.  counts (int32 [E]): how often each was chosen."""
    W, dev = "tp_route_fwd", _begin()
    T, E, code = _logits(W, logits)
    k = _slots(W, "experts", experts, T)
    d = _RouteDesc(score, groups, top_groups, group_best, int(renorm), scale)
    _check(_lib.tp_route_fwd(_one(W, "logits", logits, (T, E), logits.dtype, dev), _one(W, "bias", bias, (E,), _FP32, dev),
                             _one(W, "experts", experts, (T, k), _INT32, dev), _one(W, "weights", weights, (T, k), _FP32, dev),
                             _one(W, "counts", counts, (E,), _INT32, dev), ctypes.byref(d), T, E, k, code, _on(stream, dev)), W)


def tp_route_bwd(logits, experts, dweights, dlogits, *, score: int = TP_ROUTE_SOFTMAX, renorm: bool = False, scale: float = 1.0,
                 stream=None) -> None:
    """dlogits ([T, E], the logits' dtype) from dweights (float32 [T, k]) and the experts that tp_route_fwd chose."""
    W, dev = "tp_route_bwd", _begin()
    T, E, code = _logits(W, logits)
    k = _slots(W, "experts", experts, T)
    d = _RouteDesc(score, 1, 1, 1, int(renorm), scale)
    _check(_lib.tp_route_bwd(_one(W, "logits", logits, (T, E), logits.dtype, dev), _one(W, "experts", experts, (T, k), _INT32, dev),
                             _one(W, "dweights", dweights, (T, k), _FP32, dev), _one(W, "dlogits", dlogits, (T, E), logits.dtype, dev),
                             ctypes.byref(d), T, E, k, code, _on(stream, dev)), W)


# ------------------------------------------------------------------ routed experts

class ExpertsSaved(NamedTuple):
    """What tp_experts_fwd_fp8 leaves for tp_experts_bwd_fp8 (see experts_saved)."""
    plan: object
    preact: object
    out: object


def tp_experts_rows(E: int, T: int, k: int) -> int:
    return int(_lib.tp_experts_rows(E, T, k))


def tp_experts_plan_size(E: int, T: int, k: int) -> int:
    return int(_lib.tp_experts_plan_size(E, T, k))


def tp_experts_workspace_size(p: int, E: int, T: int, k: int, h: int, f: int, backward: bool = False) -> int:
    return int(_lib.tp_experts_workspace_size(p, E, T, k, h, f, int(backward)))


def experts_workspace(p: int, E: int, T: int, k: int, h: int, f: int, backward: bool = False, device="cuda"):
    """A zero-filled workspace of the forward call, with `backward` of both."""
    import torch
    return torch.zeros((tp_experts_workspace_size(p, E, T, k, h, f, backward) + 15) // 16 * 16, dtype=torch.uint8, device=device)


def experts_saved(E: int, T: int, k: int, h: int, f: int, device="cuda") -> ExpertsSaved:
    """Memory for what a forward call leaves for its backward call."""
    import torch
    rows = tp_experts_rows(E, T, k)
    bf = dict(dtype=torch.bfloat16, device=device)
    return ExpertsSaved(torch.empty(tp_experts_plan_size(E, T, k) // 4, dtype=torch.int32, device=device),
                        torch.empty((rows, f), **bf), torch.empty((rows, h), **bf))


def _saved(where: str, s, E: int, T: int, k: int, h: int, f: int, dev: int):
    rows = tp_experts_rows(E, T, k)
    return _ExpertsSaved(_one(where, "saved.plan", s.plan, (tp_experts_plan_size(E, T, k) // 4,), _INT32, dev),
                         _one(where, "saved.preact", s.preact, (rows, f), _BF16, dev), _one(where, "saved.out", s.out, (rows, h), _BF16, dev))


def _expert_sizes(where: str, x, name: str, t) -> tuple:
    if x.dim() != 2:
        raise ValueError(f"{where}: tokens are [T, h], got {tuple(x.shape)}")
    return x.shape[0], x.shape[1], _slots(where, name, t, x.shape[0])


def tp_experts_fwd_fp8(x, experts, weights, w1: Sequence, w2: Sequence, y, ws, saved=None, stream=None) -> None:
    """y[t] = sum_j weights[t, j] GeLU(x[t] W1_e) W2_e, e = experts[t, j] (int32 [T, k], weights float32 [T, k]).

    w1[r], w2[r]: the E/p operands [f, h] and [h, f] of shard r, packed transposes of W1_e [h, f] and W2_e [f, h] with a
    leading dimension.  A slot with a number outside 0..E-1 has no part in it.  saved (experts_saved) for the backward call."""
    W, dev, p, bf = "tp_experts_fwd_fp8", _begin(), len(w1), _BF16
    T, h, k = _expert_sizes(W, x, "experts", experts)
    if w1[0].q.dim() != 3:
        raise ValueError(f"{W}: w1[0] is operands [experts, f, h], got {tuple(w1[0].q.shape)}")
    per, f = w1[0].q.shape[:2]
    E = per * p
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    sv = None if saved is None else ctypes.byref(_saved(W, saved, E, T, k, h, f, dev))
    _check(_lib.tp_experts_fwd_fp8(
        _one(W, "x", x, (T, h), bf, dev), _one(W, "experts", experts, (T, k), _INT32, dev), _one(W, "weights", weights, (T, k), _FP32, dev),
        _fp8s(W, "w1", w1, p, f, h, dev, (per,)), _fp8s(W, "w2", w2, p, h, f, dev, (per,)), _one(W, "y", y, (T, h), bf, dev), sv, p, E, T, k,
        h, f, wp, wb, _on(stream, dev)), W)


def tp_experts_bwd_fp8(x, weights, dy, w1t, w2t, dx, dweights, dw1, dw2, saved, ws, stream=None) -> None:
    """Gradients of tp_experts_fwd_fp8 from what it saved: dx [T, h], dweights (bfloat16 [T, k]), dw1[r] [E/p, h, f], dw2[r] [E/p, f, h].

    w1t[r] (read for dx) and w2t[r] (for dx and dw1): operands [h, f] of W1_e and [f, h] of W2_e.  Each output may be None."""
    W, dev, bf = "tp_experts_bwd_fp8", _begin(), _BF16
    T, h, k = _expert_sizes(W, dy, "weights", weights)
    first = dw1 if dw1 is not None else dw2 if dw2 is not None else w2t if w2t is not None else w1t
    if first is None:
        raise ValueError(f"{W}: one of dw1, dw2, w1t and w2t is given")
    p, one = len(first), first[0]
    per, f = (one.q.shape[0] if isinstance(one, Fp8) else one.shape[0]), saved.preact.shape[1]
    E = per * p
    _need_ws(W, ws, dev)
    wp, wb = _ws(ws)
    need_h = dx is not None or dw1 is not None
    _check(_lib.tp_experts_bwd_fp8(
        _one(W, "x", x if dw1 is not None else None, (T, h), bf, dev), _one(W, "weights", weights, (T, k), _FP32, dev),
        _one(W, "dy", dy, (T, h), bf, dev), _fp8s(W, "w1t", w1t if dx is not None else None, p, h, f, dev, (per,)),
        _fp8s(W, "w2t", w2t if need_h else None, p, f, h, dev, (per,)), _one(W, "dx", dx, (T, h), bf, dev),
        _one(W, "dweights", dweights, (T, k), bf, dev), _list(W, "dw1", dw1, p, (per, h, f), bf, dev),
        _list(W, "dw2", dw2, p, (per, f, h), bf, dev), ctypes.byref(_saved(W, saved, E, T, k, h, f, dev)), p, E, T, k, h, f, wp, wb,
        _on(stream, dev)), W)
