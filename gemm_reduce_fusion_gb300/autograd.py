"""PyTorch autograd wrappers over the sharded-Linear C-ABI.

The TP tutorial (§6.3, the autograd view of the duality) pairs the two
layouts with two communication regions:

* the column-parallel Linear copies its input to every rank in the forward
  pass (identity) and all-reduces the input gradient in the backward pass;
* the row-parallel Linear all-reduces the partial outputs in the forward
  pass and passes the output gradient through unchanged in the backward
  pass (each rank's dX_k is already its own shard).

Here all p ranks live in one GPU's memory and every reduction is fused into
the GEMM that produces it, so each layer is one ``torch.autograd.Function``
whose forward and backward are single library calls:

==========================  ===================================  ==========================================
Function                    forward                              backward
==========================  ===================================  ==========================================
column (copy region)        tp_col_linear_fwd                    tp_col_linear_bwd (fused dX reduce, dA_k)
row (reduce region)         tp_row_linear_fwd_allreduce          tp_row_linear_bwd (no reduction)
MLP block (§7.1)            column + GeLU, then row + AllReduce  row bwd with GeLU' epilogue, column bwd
sequence-parallel column    tp_ag_matmul (AllGather+MatMul)      tp_ag_matmul_bwd (ReduceScatter of dX)
sequence-parallel row       tp_row_linear_fwd_reducescatter      tp_row_linear_bwd_reducescatter (AllGather)
sequence-parallel MLP       AG+MatMul+GeLU, row + ReduceScatter  both sequence-parallel backwards
==========================  ===================================  ==========================================

GeLU exists only inside the MLP functions: its derivative is applied in the
epilogue of FC2's backward GEMM, so no separate elementwise kernel is
needed.  ``parallel_mlp_fp8`` is the MLP on 8-bit operands; ``route`` and
``routed_experts`` choose experts for each token and run them, on 8-bit
operands too.  Biases are optional: a column layer adds rank k's block b_k before
the activation, a row layer adds its b once after the reduction (TP §三/§四),
and their gradients are the row sums of the output gradient, computed by
the backward call.  Tensors are bf16 CUDA tensors; weights are ``[in, out]``
row-major shards (rank k's column block for column layers, row block for
row layers).  Gradients are produced in bf16.  Nothing here computes: every
arithmetic step runs in the library's kernels.
"""
from __future__ import annotations

from typing import Sequence

import torch
from torch.autograd.function import once_differentiable

from . import (TP_EPI_GELU, TP_OP_AG_MM, TP_OP_AG_MM_BWD, TP_OP_BLOCK_NORM_BWD, TP_OP_COL_BWD, TP_OP_COL_BWD_FP8, TP_OP_COL_FP8,
               TP_OP_COL_FWD, TP_OP_COL_W4, TP_OP_ROW_AR, TP_OP_ROW_BWD, TP_OP_ROW_BWD_FP8, TP_OP_ROW_FP8, TP_OP_ROW_RS,
               TP_OP_ROW_RS_BWD, TP_OP_ROW_W4, TP_ROUTE_SIGMOID, TP_ROUTE_SOFTMAX, ExpertsSaved, Fp8, experts_saved, fp8_empty, tp_ag_matmul,
               tp_ag_matmul_bwd, tp_col_linear_bwd, tp_col_linear_bwd_fp8, tp_col_linear_fwd, tp_col_linear_fwd_fp8,
               tp_experts_bwd_fp8, tp_experts_fwd_fp8, tp_experts_workspace_size, tp_fp8_pack, tp_route_bwd, tp_route_fwd,
               tp_row_linear_bwd, tp_row_linear_bwd_fp8, tp_row_linear_bwd_reducescatter, tp_row_linear_fwd_allreduce,
               tp_row_linear_fwd_fp8, tp_row_linear_fwd_reducescatter, tp_workspace_size)

_WS: dict[tuple[int, int], torch.Tensor] = {}  # by device and stream
_HEAD = 16384  # a workspace's status word and slice counters lie in its first bytes
_COUNT_NOTHING = {TP_OP_BLOCK_NORM_BWD, TP_OP_COL_W4, TP_OP_ROW_W4, TP_OP_COL_FP8, TP_OP_ROW_FP8, TP_OP_COL_BWD_FP8, TP_OP_ROW_BWD_FP8}


def _workspace(device: torch.device, calls, least: int = 256) -> torch.Tensor:
    """A workspace for every call in ``calls`` (tuples of tp_workspace_size
    arguments), of at least ``least`` bytes: the current stream's, whose calls
    are ordered, grown (zero-filled) where it is too small.

    A call that is captured into a CUDA graph gets one of the graph's own,
    from the graph's memory: the stream's may be outgrown and freed while the
    graph still points to it, and graphs may be replayed side by side.  What
    has to start at zero is cleared in the graph."""
    need = (max([least, *(tp_workspace_size(*c) for c in calls)]) + 255) // 256 * 256
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        if any(c[0] not in _COUNT_NOTHING for c in calls):
            ws[:_HEAD].zero_()
        return ws
    key = idx, torch.cuda.current_stream(idx).cuda_stream
    ws = _WS.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _WS[key] = ws
    return ws


def _bf16(t: torch.Tensor, what: str) -> torch.Tensor:
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{what}: expected a bfloat16 CUDA tensor, got {t.dtype} on {t.device}")
    return t if t.is_contiguous() else t.contiguous()


def _grad(g, like: torch.Tensor) -> torch.Tensor:
    """An output gradient as a contiguous bf16 tensor (zeros when autograd passes None)."""
    if g is None:
        return torch.zeros_like(like)
    return _bf16(g, "output gradient")


def _empty(shape, like):
    return torch.empty(shape, dtype=torch.bfloat16, device=like.device)


# ------------------------------------------------------------------ column parallel (copy region)

def _opt(ts):
    """A list of optional tensors -> None when absent, else bf16 contiguous."""
    if not ts or ts[0] is None:
        return None
    return [_bf16(t, "bias") for t in ts]


class _ColumnFn(torch.autograd.Function):
    """Y_k = X A_k + b_k for k < p.  Backward: dX = sum_k dY_k A_k^T (fused
    reduce), dA_k = X^T dY_k, db_k = row sum of dY_k."""

    @staticmethod
    def forward(ctx, p, x, *wb):
        x = _bf16(x, "x")
        w = [_bf16(a, "weight shard") for a in wb[:p]]
        b = _opt(wb[p:])
        (M, K), N = x.shape, w[0].shape[1]
        ws = _workspace(x.device, [(TP_OP_COL_FWD, p, M, N, K, 0), (TP_OP_COL_BWD, p, M, N, K, 0)])
        y = [_empty((M, N), x) for _ in range(p)]
        tp_col_linear_fwd(x, w, y, ws, bias=b)
        ctx.p = p
        ctx.save_for_backward(x, *w)
        return tuple(y)

    @staticmethod
    def backward(ctx, *dy):
        p = ctx.p
        x, *w = ctx.saved_tensors
        (M, K), N = x.shape, w[0].shape[1]
        dy = [_grad(g, x.new_empty((M, N))) for g in dy]
        need_x = ctx.needs_input_grad[1]
        need_w = any(ctx.needs_input_grad[2:2 + p])
        need_b = any(ctx.needs_input_grad[2 + p:])
        dx = _empty((M, K), x) if need_x else None
        dw = [_empty((K, N), x) for _ in range(p)] if need_w else None
        db = [_empty((N,), x) for _ in range(p)] if need_b else None
        if need_x or need_w or need_b:
            ws = _workspace(x.device, [(TP_OP_COL_BWD, p, M, N, K, 0)])
            tp_col_linear_bwd(x, w, dy, dx, dw, ws, db=db)
        return (None, dx, *(dw or [None] * p), *(db or [None] * p))


# ------------------------------------------------------------------ row parallel (reduce region)

class _RowFn(torch.autograd.Function):
    """Y = sum_r X_r A_r + b (fused AllReduce, b once).  Backward: dX_r = dY A_r^T,
    dA_r = X_r^T dY (no reduction), db = row sum of dY."""

    @staticmethod
    def forward(ctx, p, bias, *xw):
        x = [_bf16(a, "input shard") for a in xw[:p]]
        w = [_bf16(a, "weight shard") for a in xw[p:]]
        b = _bf16(bias, "bias") if bias is not None else None
        (M, K), N = x[0].shape, w[0].shape[1]
        ws = _workspace(x[0].device, [(TP_OP_ROW_AR, p, M, N, K, 0), (TP_OP_ROW_BWD, p, M, N, K, 0)])
        y = _empty((M, N), x[0])
        tp_row_linear_fwd_allreduce(x, w, [y], ws, bias=b)
        ctx.p = p
        ctx.save_for_backward(*x, *w)
        return y

    @staticmethod
    def backward(ctx, dy):
        p = ctx.p
        saved = ctx.saved_tensors
        x, w = list(saved[:p]), list(saved[p:])
        (M, K), N = x[0].shape, w[0].shape[1]
        dy = _grad(dy, x[0].new_empty((M, N)))
        need_b = ctx.needs_input_grad[1]
        need_x = any(ctx.needs_input_grad[2:2 + p])
        need_w = any(ctx.needs_input_grad[2 + p:])
        dx = [_empty((M, K), dy) for _ in range(p)] if need_x else None
        dw = [_empty((K, N), dy) for _ in range(p)] if need_w else None
        db = _empty((N,), dy) if need_b else None
        if need_x or need_w or need_b:
            ws = _workspace(dy.device, [(TP_OP_ROW_BWD, p, M, N, K, 0)])
            tp_row_linear_bwd(x, w, dy, dx, dw, ws, db=db)
        return (None, db, *(dx or [None] * p), *(dw or [None] * p))


# ------------------------------------------------------------------ the MLP block

class _MLPFn(torch.autograd.Function):
    """Y = sum_k GeLU(X A1_k + b1_k) A2_k + b2: column FC1 with GeLU, row FC2
    with the fused AllReduce (biases optional).

    Backward: dH_k = (dY A2_k^T) * GeLU'(H_k) in FC2's backward epilogue,
    dA2_k = Z_k^T dY, db2 = row sum of dY, then FC1's dX = sum_k dH_k A1_k^T
    (fused), dA1_k = X^T dH_k and db1_k = row sum of dH_k.  Saves X,
    Z_k = GeLU(H_k) and H_k (bf16)."""

    @staticmethod
    def forward(ctx, p, b2, x, *wb):
        x = _bf16(x, "x")
        w1 = [_bf16(a, "FC1 weight shard") for a in wb[:p]]
        w2 = [_bf16(a, "FC2 weight shard") for a in wb[p:2 * p]]
        b1 = _opt(wb[2 * p:])
        b2 = _bf16(b2, "FC2 bias") if b2 is not None else None
        (M, h), nk = x.shape, w1[0].shape[1]
        ws = _workspace(x.device, [(TP_OP_COL_FWD, p, M, nk, h, 0), (TP_OP_ROW_AR, p, M, h, nk, 0),
                                   (TP_OP_ROW_BWD, p, M, h, nk, 0), (TP_OP_COL_BWD, p, M, nk, h, 0)])
        z = [_empty((M, nk), x) for _ in range(p)]
        hh = [_empty((M, nk), x) for _ in range(p)]
        tp_col_linear_fwd(x, w1, z, ws, epi=TP_EPI_GELU, preact=hh, bias=b1)
        y = _empty((M, h), x)
        tp_row_linear_fwd_allreduce(z, w2, [y], ws, bias=b2)
        ctx.p = p
        ctx.save_for_backward(x, *w1, *w2, *z, *hh)
        return y

    @staticmethod
    def backward(ctx, dy):
        p = ctx.p
        s = ctx.saved_tensors
        x, w1, w2 = s[0], list(s[1:1 + p]), list(s[1 + p:1 + 2 * p])
        z, hh = list(s[1 + 2 * p:1 + 3 * p]), list(s[1 + 3 * p:])
        (M, h), nk = x.shape, w1[0].shape[1]
        dy = _grad(dy, x)
        need_b2 = ctx.needs_input_grad[1]
        need_b1 = any(ctx.needs_input_grad[3 + 2 * p:])
        ws = _workspace(x.device, [(TP_OP_ROW_BWD, p, M, h, nk, 0), (TP_OP_COL_BWD, p, M, nk, h, 0)])
        dz = [_empty((M, nk), x) for _ in range(p)]
        dw2 = [_empty((nk, h), x) for _ in range(p)]
        db2 = _empty((h,), x) if need_b2 else None
        tp_row_linear_bwd(z, w2, dy, dz, dw2, ws, preact=hh, db=db2)
        dx = _empty((M, h), x) if ctx.needs_input_grad[2] else None
        dw1 = [_empty((h, nk), x) for _ in range(p)]
        db1 = [_empty((nk,), x) for _ in range(p)] if need_b1 else None
        tp_col_linear_bwd(x, w1, dz, dx, dw1, ws, db=db1)
        return (None, db2, dx, *dw1, *dw2, *(db1 or [None] * p))


# ------------------------------------------------------------------ sequence parallel (§11.3)

class _AllGatherColumnFn(torch.autograd.Function):
    """Y_k = [X_0; ...; X_{p-1}] A_k + b_k.  Backward: dX_s = rows s of
    sum_k dY_k A_k^T (ReduceScatter), dA_k = X_gathered^T dY_k, db_k = row sum of dY_k."""

    @staticmethod
    def forward(ctx, p, *xwb):
        x = [_bf16(a, "token shard") for a in xwb[:p]]
        w = [_bf16(a, "weight shard") for a in xwb[p:2 * p]]
        b = _opt(xwb[2 * p:])
        (Mp, K), N = x[0].shape, w[0].shape[1]
        M = Mp * p
        ws = _workspace(x[0].device, [(TP_OP_AG_MM, p, M, N, K, 0), (TP_OP_AG_MM_BWD, p, M, N, K, 0)])
        y = [_empty((M, N), x[0]) for _ in range(p)]
        tp_ag_matmul(x, w, y, ws, bias=b)
        ctx.p = p
        ctx.save_for_backward(*x, *w)
        return tuple(y)

    @staticmethod
    def backward(ctx, *dy):
        p = ctx.p
        s = ctx.saved_tensors
        x, w = list(s[:p]), list(s[p:])
        (Mp, K), N = x[0].shape, w[0].shape[1]
        M = Mp * p
        dy = [_grad(g, x[0].new_empty((M, N))) for g in dy]
        need_x = any(ctx.needs_input_grad[1:1 + p])
        need_w = any(ctx.needs_input_grad[1 + p:1 + 2 * p])
        need_b = any(ctx.needs_input_grad[1 + 2 * p:])
        dx = [_empty((Mp, K), x[0]) for _ in range(p)] if need_x else None
        dw = [_empty((K, N), x[0]) for _ in range(p)] if need_w else None
        db = [_empty((N,), x[0]) for _ in range(p)] if need_b else None
        if need_x or need_w or need_b:
            ws = _workspace(x[0].device, [(TP_OP_AG_MM_BWD, p, M, N, K, 0)])
            tp_ag_matmul_bwd(x, w, dy, dx, dw, ws, db=db)
        return (None, *(dx or [None] * p), *(dw or [None] * p), *(db or [None] * p))


class _RowReduceScatterFn(torch.autograd.Function):
    """Y_j = rows j of sum_r X_r A_r + b (ReduceScatter).  Backward: dX_r = [dY_0; ...] A_r^T
    (AllGather of dY), dA_r = X_r^T [dY_0; ...], db = row sum of all dY shards."""

    @staticmethod
    def forward(ctx, p, bias, *xw):
        x = [_bf16(a, "input shard") for a in xw[:p]]
        w = [_bf16(a, "weight shard") for a in xw[p:]]
        b = _bf16(bias, "bias") if bias is not None else None
        (M, K), N = x[0].shape, w[0].shape[1]
        if M % p:
            raise ValueError(f"ReduceScatter needs M % p == 0 (M={M}, p={p})")
        ws = _workspace(x[0].device, [(TP_OP_ROW_RS, p, M, N, K, 0), (TP_OP_ROW_RS_BWD, p, M, N, K, 0)])
        y = [_empty((M // p, N), x[0]) for _ in range(p)]
        tp_row_linear_fwd_reducescatter(x, w, y, ws, bias=b)
        ctx.p = p
        ctx.save_for_backward(*x, *w)
        return tuple(y)

    @staticmethod
    def backward(ctx, *dy):
        p = ctx.p
        s = ctx.saved_tensors
        x, w = list(s[:p]), list(s[p:])
        (M, K), N = x[0].shape, w[0].shape[1]
        dy = [_grad(g, x[0].new_empty((M // p, N))) for g in dy]
        need_b = ctx.needs_input_grad[1]
        need_x = any(ctx.needs_input_grad[2:2 + p])
        need_w = any(ctx.needs_input_grad[2 + p:])
        dx = [_empty((M, K), x[0]) for _ in range(p)] if need_x else None
        dw = [_empty((K, N), x[0]) for _ in range(p)] if need_w else None
        db = _empty((N,), x[0]) if need_b else None
        if need_x or need_w or need_b:
            ws = _workspace(x[0].device, [(TP_OP_ROW_RS_BWD, p, M, N, K, 0)])
            tp_row_linear_bwd_reducescatter(x, w, dy, dx, dw, ws, db=db)
        return (None, db, *(dx or [None] * p), *(dw or [None] * p))


class _SequenceParallelMLPFn(torch.autograd.Function):
    """Token shards in, token shards out: Y_j = rows j of
    sum_k GeLU([X_0;...] A1_k + b1_k) A2_k + b2.

    Forward: AllGather+MatMul with GeLU, then the row layer with the fused
    ReduceScatter.  Backward: the row layer's AllGather of dY with GeLU' in
    the epilogue, then the AllGather+MatMul backward (ReduceScatter of dX)."""

    @staticmethod
    def forward(ctx, p, b2, *args):
        x = [_bf16(a, "token shard") for a in args[:p]]
        w1 = [_bf16(a, "FC1 weight shard") for a in args[p:2 * p]]
        w2 = [_bf16(a, "FC2 weight shard") for a in args[2 * p:3 * p]]
        b1 = _opt(args[3 * p:])
        b2 = _bf16(b2, "FC2 bias") if b2 is not None else None
        (Mp, h), nk = x[0].shape, w1[0].shape[1]
        M = Mp * p
        ws = _workspace(x[0].device, [(TP_OP_AG_MM, p, M, nk, h, 0), (TP_OP_ROW_RS, p, M, h, nk, 0),
                                      (TP_OP_ROW_RS_BWD, p, M, h, nk, 0), (TP_OP_AG_MM_BWD, p, M, nk, h, 0)])
        z = [_empty((M, nk), x[0]) for _ in range(p)]
        hh = [_empty((M, nk), x[0]) for _ in range(p)]
        tp_ag_matmul(x, w1, z, ws, epi=TP_EPI_GELU, preact=hh, bias=b1)
        y = [_empty((Mp, h), x[0]) for _ in range(p)]
        tp_row_linear_fwd_reducescatter(z, w2, y, ws, bias=b2)
        ctx.p = p
        ctx.save_for_backward(*x, *w1, *w2, *z, *hh)
        return tuple(y)

    @staticmethod
    def backward(ctx, *dy):
        p = ctx.p
        s = ctx.saved_tensors
        x, w1, w2 = list(s[:p]), list(s[p:2 * p]), list(s[2 * p:3 * p])
        z, hh = list(s[3 * p:4 * p]), list(s[4 * p:])
        (Mp, h), nk = x[0].shape, w1[0].shape[1]
        M = Mp * p
        dy = [_grad(g, x[0]) for g in dy]
        need_b2 = ctx.needs_input_grad[1]
        need_b1 = any(ctx.needs_input_grad[2 + 3 * p:])
        ws = _workspace(x[0].device, [(TP_OP_ROW_RS_BWD, p, M, h, nk, 0), (TP_OP_AG_MM_BWD, p, M, nk, h, 0)])
        dz = [_empty((M, nk), x[0]) for _ in range(p)]
        dw2 = [_empty((nk, h), x[0]) for _ in range(p)]
        db2 = _empty((h,), x[0]) if need_b2 else None
        tp_row_linear_bwd_reducescatter(z, w2, dy, dz, dw2, ws, preact=hh, db=db2)
        dx = [_empty((Mp, h), x[0]) for _ in range(p)]
        dw1 = [_empty((h, nk), x[0]) for _ in range(p)]
        db1 = [_empty((nk,), x[0]) for _ in range(p)] if need_b1 else None
        tp_ag_matmul_bwd(x, w1, dz, dx, dw1, ws, db=db1)
        return (None, db2, *dx, *dw1, *dw2, *(db1 or [None] * p))


# ------------------------------------------------------------------ 8-bit operands

def _operands(ts, rows=None, cols=None, tiles=False, epi=0):
    """Packed from the matrices ``ts`` ([M, N], or [B, M, N]): their operands if
    ``rows``, those of their transposes if ``cols``."""
    *lead, M, N = ts[0].shape
    make = lambda r, c: [fp8_empty(r, c, *lead, device=ts[0].device) for _ in ts]  # noqa: E731
    q, qt = make(M, N) if rows else None, make(N, M) if cols else None
    for i in range(0, len(ts), 8):  # shards a call
        tp_fp8_pack(ts[i:i + 8], q and q[i:i + 8], qt and qt[i:i + 8], tiles=tiles, epi=epi)
    return q, qt


def _flat(ops):
    return [t for op in ops for t in op]


def _paired(ts):
    return [Fp8(q, e) for q, e in zip(ts[::2], ts[1::2])]


class _Fp8MLPFn(torch.autograd.Function):
    """sum_k GeLU(X A1_k) A2_k with every product on 8-bit operands, a power of
    two for each block of 128: X and the activations packed in rows, the
    weights in 128 x 128 (so that they and their transposes hold the same
    values).

    Backward: dH_k = (dY A2_k^T) GeLU'(H_k), dX = sum_k dH_k A1_k^T,
    dA2_k = GeLU(H_k)^T dY, dA1_k = X^T dH_k, each on operands of its factors.
    Saves H in bf16, and X and the weights as the operands that the backward
    products take; without ``grad`` (the mode of the call: inside it is always
    off) nothing is saved or packed for them."""

    @staticmethod
    def forward(ctx, p, grad, x, *wb):
        x = _bf16(x, "x")
        w1 = [_bf16(a, "FC1 weight shard") for a in wb[:p]]
        w2 = [_bf16(a, "FC2 weight shard") for a in wb[p:]]
        (M, h), nk = x.shape, w1[0].shape[1]
        train = grad and any(ctx.needs_input_grad)
        ws = _workspace(x.device, [(TP_OP_COL_FP8, p, M, nk, h), (TP_OP_ROW_FP8, p, M, h, nk)])
        back1, fwd1 = _operands(w1, train, True, tiles=True)
        back2, fwd2 = _operands(w2, train, True, tiles=True)
        xq, xt = _operands([x], True, train)
        hh = [_empty((M, nk), x) for _ in range(p)] if train else None
        z = [fp8_empty(M, nk, device=x.device) for _ in range(p)]
        tp_col_linear_fwd_fp8(xq[0], fwd1, None, ws, epi=TP_EPI_GELU, preact=hh, z=z)
        y = _empty((M, h), x)
        tp_row_linear_fwd_fp8(z, fwd2, y, ws)
        if train:
            ctx.p = p
            ctx.save_for_backward(*hh, *_flat(xt), *_flat(back1), *_flat(back2))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        p, s = ctx.p, list(ctx.saved_tensors)
        hh, xt = s[:p], _paired(s[p:p + 2])[0]
        back1, back2 = _paired(s[p + 2:3 * p + 2]), _paired(s[3 * p + 2:])
        M, nk = hh[0].shape
        h = back1[0].q.shape[0]
        dy = _grad(dy, hh[0].new_empty((M, h)))
        ws = _workspace(dy.device, [(TP_OP_ROW_BWD_FP8, p, M, h, nk), (TP_OP_COL_BWD_FP8, p, M, nk, h)])
        dyq, dyt = _operands([dy], True, True)
        _, zt = _operands(hh, False, True, epi=TP_EPI_GELU)
        dh = [_empty((M, nk), dy) for _ in range(p)]
        dw1, dw2 = [_empty((h, nk), dy) for _ in range(p)], [_empty((nk, h), dy) for _ in range(p)]
        tp_row_linear_bwd_fp8(zt, back2, dyq[0], dyt[0], dh, dw2, ws, preact=hh)
        dhq, dht = _operands(dh, True, True)
        dx = _empty((M, h), dy)
        tp_col_linear_bwd_fp8(xt, back1, dhq, dht, dx, dw1, ws)
        return (None, None, dx, *dw1, *dw2)


class _RouteFn(torch.autograd.Function):
    """(weights, experts, counts) of the k experts of each row of logits; the
    weights are differentiable in the logits, the choice is not."""

    @staticmethod
    def forward(ctx, logits, k, how, bias, groups):
        if not logits.is_cuda or logits.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"logits: expected a bfloat16 or float32 CUDA tensor, got {logits.dtype} on {logits.device}")
        logits = logits.contiguous()
        T, E = logits.shape
        on = dict(device=logits.device)
        experts, weights = torch.empty((T, k), dtype=torch.int32, **on), torch.empty((T, k), dtype=torch.float32, **on)
        counts = torch.empty(E, dtype=torch.int32, **on)
        tp_route_fwd(logits, experts, weights, counts=counts, bias=bias, **groups, **how)
        ctx.how = how
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts, counts)
        return weights, experts, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, *_):
        logits, experts = ctx.saved_tensors
        if dweights is None:
            return torch.zeros_like(logits), None, None, None, None
        dlogits = torch.empty_like(logits)
        tp_route_bwd(logits, experts, dweights.contiguous(), dlogits, **ctx.how)
        return dlogits, None, None, None, None


class _ExpertsFn(torch.autograd.Function):
    """y[t] = sum_j weights[t, j] GeLU(x[t] W1_e) W2_e on 8-bit operands; the
    p shards hold E/p experts each.  Saves x, dispatched slots, pre-activations
    and the experts' outputs, and the weights as operands; nothing without
    ``grad``, the mode of the call, and a few tokens then take smaller tiles."""

    @staticmethod
    def forward(ctx, p, grad, x, experts, weights, *wb):
        x, experts, weights = _bf16(x, "x"), experts.contiguous(), weights.contiguous()
        w1 = [_bf16(a, "FC1 weights of the experts") for a in wb[:p]]
        w2 = [_bf16(a, "FC2 weights of the experts") for a in wb[p:]]
        (T, h), (per, _, f), k = x.shape, w1[0].shape, experts.shape[1]
        train = grad and any(ctx.needs_input_grad)
        ws = _workspace(x.device, [], tp_experts_workspace_size(p, p * per, T, k, h, f, train))
        back1, fwd1 = _operands(w1, train, True, tiles=True)
        back2, fwd2 = _operands(w2, train, True, tiles=True)
        saved = experts_saved(p * per, T, k, h, f, device=x.device) if train else None
        y = _empty((T, h), x)
        tp_experts_fwd_fp8(x, experts, weights, fwd1, fwd2, y, ws, saved=saved)
        if train:
            ctx.p = p
            ctx.save_for_backward(x, weights, *saved, *_flat(back1), *_flat(back2))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        p, s = ctx.p, ctx.saved_tensors
        x, weights, saved = s[0], s[1], ExpertsSaved(*s[2:5])
        back1, back2 = _paired(s[5:5 + 2 * p]), _paired(s[5 + 2 * p:])
        (T, h), k, (per, f) = x.shape, weights.shape[1], back2[0].q.shape[:2]
        dy = _grad(dy, x)
        ws = _workspace(x.device, [], tp_experts_workspace_size(p, p * per, T, k, h, f, True))
        need = ctx.needs_input_grad
        dx = _empty((T, h), x) if need[2] else None
        dw = _empty((T, k), x) if need[4] else None
        dw1 = [_empty((per, h, f), x) for _ in range(p)] if any(need[5:5 + p]) else None
        dw2 = [_empty((per, f, h), x) for _ in range(p)] if any(need[5 + p:]) else None
        tp_experts_bwd_fp8(x, weights, dy, back1, back2, dx, dw, dw1, dw2, saved, ws)
        return (None, None, dx, None, dw.float() if dw is not None else None, *(dw1 or [None] * p), *(dw2 or [None] * p))


# ------------------------------------------------------------------ functional API

def _blocks(b, p):
    return list(b) if b is not None else [None] * p


def column_parallel_linear(x: torch.Tensor, weights: Sequence[torch.Tensor], biases=None) -> tuple:
    """(Y_0, ..., Y_{p-1}) with Y_k = X A_k (+ b_k); differentiable in X, every A_k and b_k."""
    p = len(weights)
    return _ColumnFn.apply(p, x, *weights, *_blocks(biases, p))


def row_parallel_linear(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor], bias=None) -> torch.Tensor:
    """Y = sum_r X_r A_r (+ b) (fused AllReduce); differentiable in every X_r, A_r and b."""
    if len(xs) != len(weights):
        raise ValueError("one input shard per weight shard")
    return _RowFn.apply(len(xs), bias, *xs, *weights)


def parallel_mlp(x: torch.Tensor, w1: Sequence[torch.Tensor], w2: Sequence[torch.Tensor],
                 b1=None, b2=None) -> torch.Tensor:
    """Y = sum_k GeLU(X A1_k + b1_k) A2_k + b2 (the TP tutorial's §7.1 block)."""
    if len(w1) != len(w2):
        raise ValueError("FC1 and FC2 need the same number of shards")
    p = len(w1)
    return _MLPFn.apply(p, b2, x, *w1, *w2, *_blocks(b1, p))


def allgather_column_parallel_linear(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                                     biases=None) -> tuple:
    """(Y_0, ..., Y_{p-1}) with Y_k = [X_0; ...; X_{p-1}] A_k (+ b_k) (AllGather+MatMul)."""
    if len(xs) != len(weights):
        raise ValueError("one token shard per weight shard")
    p = len(xs)
    return _AllGatherColumnFn.apply(p, *xs, *weights, *_blocks(biases, p))


def row_parallel_linear_reducescatter(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                                      bias=None) -> tuple:
    """(Y_0, ..., Y_{p-1}): rank j's rows of sum_r X_r A_r (+ b) (MatMul+ReduceScatter)."""
    if len(xs) != len(weights):
        raise ValueError("one input shard per weight shard")
    return _RowReduceScatterFn.apply(len(xs), bias, *xs, *weights)


def sequence_parallel_mlp(xs: Sequence[torch.Tensor], w1: Sequence[torch.Tensor],
                          w2: Sequence[torch.Tensor], b1=None, b2=None) -> tuple:
    """Token shards of sum_k GeLU([X_0; ...] A1_k + b1_k) A2_k + b2 (the TP tutorial's §11.3 pair)."""
    if not (len(xs) == len(w1) == len(w2)):
        raise ValueError("one token shard and one FC1/FC2 shard per rank")
    p = len(xs)
    return _SequenceParallelMLPFn.apply(p, b2, *xs, *w1, *w2, *_blocks(b1, p))


def parallel_mlp_fp8(x: torch.Tensor, w1: Sequence[torch.Tensor], w2: Sequence[torch.Tensor]) -> torch.Tensor:
    """Y = sum_k GeLU(X A1_k) A2_k, every product on 8-bit operands (see _Fp8MLPFn).

    Each call packs the weights, for a backward pass in both orientations."""
    if len(w1) != len(w2):
        raise ValueError("FC1 and FC2 need the same number of shards")
    return _Fp8MLPFn.apply(len(w1), torch.is_grad_enabled(), x, *w1, *w2)


SCORES = {"softmax": TP_ROUTE_SOFTMAX, "sigmoid": TP_ROUTE_SIGMOID}


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
          group_best: int = 1, renorm: bool = False, scale: float = 1.0) -> tuple:
    """(weights [T, k], experts [T, k], counts [E]) of the k best experts of each row of logits [T, E]
    (see tp_route_fwd); the weights are differentiable in the logits."""
    if score not in SCORES:
        raise ValueError(f"score is one of {sorted(SCORES)}, got {score!r}")
    return _RouteFn.apply(logits, k, dict(score=SCORES[score], renorm=renorm, scale=scale), bias,
                          dict(groups=groups, top_groups=top_groups, group_best=group_best))


def routed_experts(x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, w1: Sequence[torch.Tensor],
                   w2: Sequence[torch.Tensor]) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] GeLU(x[t] W1_e) W2_e with e = experts[t, j]; shard r of w1 [E/p, h, f] and
    w2 [E/p, f, h] holds E/p experts.  Differentiable in x, the weights and every shard.

    Each call packs the experts' weights, for a backward pass in both orientations.  Where no gradient is recorded the
    outputs of few tokens' experts stay fp32 until they are added up, instead of bfloat16."""
    if len(w1) != len(w2):
        raise ValueError("FC1 and FC2 need the same number of shards")
    return _ExpertsFn.apply(len(w1), torch.is_grad_enabled(), x, experts, weights, *w1, *w2)


# ------------------------------------------------------------------ modules

def _shards(weight: torch.Tensor, p: int, dim: int) -> list:
    n = weight.shape[dim]
    if n % p:
        raise ValueError(f"dimension {dim} of size {n} does not split into {p} shards")
    return [c.contiguous() for c in torch.split(weight, n // p, dim=dim)]


def _params(ts):
    return torch.nn.ParameterList(torch.nn.Parameter(t) for t in ts)


class ColumnParallelLinear(torch.nn.Module):
    """X [M, in] -> p outputs Y_k [M, out/p]; weight [in, out] split into
    contiguous column blocks A_k (TP tutorial §2.3), and the optional bias
    [out] into the matching blocks b_k."""

    def __init__(self, weight: torch.Tensor, p: int, bias: torch.Tensor | None = None):
        super().__init__()
        self.p = p
        self.weights = _params(_shards(weight, p, 1))
        self.biases = _params(_shards(bias, p, 0)) if bias is not None else None

    def forward(self, x: torch.Tensor) -> tuple:
        return column_parallel_linear(x, list(self.weights), list(self.biases) if self.biases else None)


class RowParallelLinear(torch.nn.Module):
    """p input shards X_r [M, in/p] -> Y [M, out] = sum_r X_r A_r (+ b);
    weight [in, out] split into contiguous row blocks A_r (TP tutorial
    §2.4); the bias [out] is added once, after the reduction.  With
    ``sequence_parallel`` the output is the p token shards of Y
    (ReduceScatter) instead of the full Y."""

    def __init__(self, weight: torch.Tensor, p: int, bias: torch.Tensor | None = None,
                 sequence_parallel: bool = False):
        super().__init__()
        self.p = p
        self.sequence_parallel = sequence_parallel
        self.weights = _params(_shards(weight, p, 0))
        self.bias = torch.nn.Parameter(bias.contiguous()) if bias is not None else None

    def forward(self, xs: Sequence[torch.Tensor]):
        if self.sequence_parallel:
            return row_parallel_linear_reducescatter(xs, list(self.weights), self.bias)
        return row_parallel_linear(xs, list(self.weights), self.bias)


class ParallelMLP(torch.nn.Module):
    """Column FC1 [h, ffn] (+ b1 [ffn]) + GeLU, row FC2 [ffn, h] (+ b2 [h]),
    p shards each (TP tutorial §7.1).  Input X [M, h] -> Y [M, h]; with
    ``sequence_parallel`` the input and output are p token shards [M/p, h]
    (§11.3)."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, p: int, b1: torch.Tensor | None = None,
                 b2: torch.Tensor | None = None, sequence_parallel: bool = False):
        super().__init__()
        self.p = p
        self.sequence_parallel = sequence_parallel
        self.w1 = _params(_shards(w1, p, 1))
        self.w2 = _params(_shards(w2, p, 0))
        self.b1 = _params(_shards(b1, p, 0)) if b1 is not None else None
        self.b2 = torch.nn.Parameter(b2.contiguous()) if b2 is not None else None

    def forward(self, x):
        b1 = list(self.b1) if self.b1 is not None else None
        if self.sequence_parallel:
            return sequence_parallel_mlp(x, list(self.w1), list(self.w2), b1, self.b2)
        return parallel_mlp(x, list(self.w1), list(self.w2), b1, self.b2)
