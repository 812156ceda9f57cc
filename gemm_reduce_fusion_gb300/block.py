"""The MLP block of a transformer as it stands in a model: the sharded MLP
between two norms, with its gate and residual connection.

A block takes the residual stream x and its normalised form n, which the
boundary before it has written, and ends with the boundary after it:

    z = sum_k GeLU(n A1_k) A2_k                      (the sharded MLP)
    y = x + alpha * gate * N_post(z),  n' = N_pre(y)  (one fused call)

so that blocks chain as ``x, n = block(x, n)``; the stream begins with
``n = pre_norm(x, ...)``.

``MLPBlock`` trains: the MLP saves its input X and its pre-activations H in
8 bits, 33/32 bytes an FFN element where H and Z = GeLU(H) in bfloat16 take 4
(Z is restored from H); with ``fp8`` its products run on 8-bit floating-point
operands instead.  ``W4MLPBlock``
serves it: 4-bit weights, single tokens and small batches straight from
them, prompts through weights unpacked for the call.

``RoutedMLPBlock`` has experts in the MLP's place, each token sent to k of
them by a router, their products on 8-bit operands; ``serve()`` gives the
block for serving, its weights packed once.

Tensors are [tokens, h], or lists of p token shards [tokens / p, h] with
``sequence_parallel`` (the ReduceScatter layouts).  The stream is bfloat16 or
float32; everything else is bfloat16.  All arithmetic runs in the library's
kernels.
"""
from __future__ import annotations

from typing import Sequence

import torch
from torch.autograd.function import once_differentiable

from . import (TP_EPI_GELU, TP_NORM_LAYER, TP_NORM_NONE, TP_NORM_RMS, TP_OP_AG_MM, TP_OP_AG_MM_BWD_CKPT,
               TP_OP_BLOCK_NORM_BWD, TP_OP_COL_BWD_CKPT, TP_OP_COL_FWD, TP_OP_COL_W4, TP_OP_ROW_AR, TP_OP_ROW_BWD_CKPT,
               TP_OP_ROW_RS, TP_OP_ROW_RS_BWD_CKPT, TP_OP_ROW_W4, TP_W4_MAX_M, ckpt_shapes, tp_ag_matmul,
               tp_ag_matmul_bwd_ckpt, tp_block_norm_bwd, tp_block_norm_fwd, tp_ckpt_pack, tp_col_linear_bwd_ckpt,
               tp_col_linear_fwd, tp_col_linear_fwd_w4, tp_experts_fwd_fp8, tp_experts_workspace_size, tp_route_fwd,
               tp_row_linear_bwd_ckpt, tp_row_linear_bwd_reducescatter_ckpt, tp_row_linear_fwd_allreduce,
               tp_row_linear_fwd_reducescatter, tp_row_linear_fwd_w4, tp_w4_pack, tp_w4_unpack, w4_shapes)
from .autograd import (SCORES, _bf16, _empty, _grad, _operands, _params, _shards, _workspace, column_parallel_linear, parallel_mlp_fp8, route,
                       routed_experts)

NORMS = {"none": TP_NORM_NONE, "rms": TP_NORM_RMS, "layer": TP_NORM_LAYER}


def _kind(norm: str) -> int:
    if norm not in NORMS:
        raise ValueError(f"norm is one of {sorted(NORMS)}, got {norm!r}")
    return NORMS[norm]


def _stream_grad(g, like):
    if g is None:
        return torch.zeros_like(like)
    if g.dtype != like.dtype:
        raise TypeError(f"gradient of the stream: expected {like.dtype}, got {g.dtype}")
    return g.contiguous()


# ------------------------------------------------------------------ the boundary

class _BoundaryFn(torch.autograd.Function):
    """(y..., n...) of x + alpha gate N_post(z) and N_pre of it; n alone without z."""

    @staticmethod
    def forward(ctx, p, how, w_post, b_post, w_pre, b_pre, gate, *xz):
        x = [t.contiguous() for t in xz[:p]]
        z = [_bf16(t, "block output") for t in xz[p:]] or None
        y = [torch.empty_like(t) for t in x] if z else None
        n = [_empty(t.shape, t) for t in x] if how["pre"] else None
        vec = dict(w_post=w_post, b_post=b_post, w_pre=w_pre, b_pre=b_pre, gate=gate)
        tp_block_norm_fwd(x, z, y, n, **how, **vec)
        ctx.p, ctx.how, ctx.has_z = p, how, z is not None
        ctx.save_for_backward(*vec.values(), *(y or x), *(z or []))
        return tuple((y or []) + (n or []))

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        p, how = ctx.p, ctx.how
        s = ctx.saved_tensors
        vec = dict(zip(("w_post", "b_post", "w_pre", "b_pre", "gate"), s[:5]))
        y, z = list(s[5:5 + p]), list(s[5 + p:]) or None
        dy = [_stream_grad(g, t) for g, t in zip(grads[:p], y)] if ctx.has_z else None
        dn = [_grad(g, _empty(t.shape, t)) for g, t in zip(grads[p if ctx.has_z else 0:], y)] if how["pre"] else None
        need = ctx.needs_input_grad
        names = ("w_post", "b_post", "w_pre", "b_pre", "gate")
        g = {"d" + k: torch.empty_like(v) if v is not None and n else None for (k, v), n in zip(vec.items(), need[2:7])}
        dx = [torch.empty_like(t) for t in y]
        dz = [_empty(t.shape, t) for t in z] if z else None
        M, h = p * y[0].shape[0], y[0].shape[1]
        ws = _workspace(y[0].device, [(TP_OP_BLOCK_NORM_BWD, p, M, h, 0)])
        tp_block_norm_bwd(z, y if dn else None, dn, dy, dx, dz, ws, **g, **how, **vec)
        return (None, None, *[g["d" + k] for k in names], *dx, *(dz or []))


def block_boundary(xs: Sequence[torch.Tensor], zs: Sequence[torch.Tensor], *, post: str = "rms", w_post=None, b_post=None,
                   pre: str = "rms", w_pre=None, b_pre=None, gate=None, alpha: float = 1.0, eps: float = 1e-5) -> tuple:
    """(ys, ns): y = x + alpha gate N_post(z) and n = N_pre(y) over p token shards (ns empty with pre="none");
    differentiable in xs, zs and every vector."""
    p = len(xs)
    how = dict(post=_kind(post), pre=_kind(pre), alpha=alpha, eps=eps)
    out = _BoundaryFn.apply(p, how, w_post, b_post, w_pre, b_pre, gate, *xs, *zs)
    return list(out[:p]), list(out[p:])


def pre_norm(xs: Sequence[torch.Tensor], *, pre: str = "rms", w_pre=None, b_pre=None, eps: float = 1e-5) -> list:
    """n = N_pre(x) over p token shards: the beginning of a stream."""
    how = dict(post=TP_NORM_NONE, pre=_kind(pre), alpha=1.0, eps=eps)
    return list(_BoundaryFn.apply(len(xs), how, None, None, w_pre, b_pre, None, *xs))


# ------------------------------------------------------------------ the MLP on 8-bit checkpoints

def _packed(ts):
    """8-bit checkpoints of bf16 tensors of one shape: (q list, e list)."""
    qs, es = ckpt_shapes(*ts[0].shape)
    q = [torch.empty(qs, dtype=torch.int8, device=ts[0].device) for _ in ts]
    e = [torch.empty(es, dtype=torch.uint8, device=ts[0].device) for _ in ts]
    tp_ckpt_pack(ts, q, e)
    return q, e


class _CkptMLPFn(torch.autograd.Function):
    """sum_k GeLU(X A1_k) A2_k, saving X and H_k in 8 bits: as the MLP of
    autograd.py, with the backward products taken from the checkpoints.  With
    sp, X and Y are p token shards (AllGather in, ReduceScatter out)."""

    @staticmethod
    def forward(ctx, p, sp, *xw):
        nx = p if sp else 1
        x = [_bf16(t, "x") for t in xw[:nx]]
        w1 = [_bf16(t, "FC1 weight shard") for t in xw[nx:nx + p]]
        w2 = [_bf16(t, "FC2 weight shard") for t in xw[nx + p:]]
        (m, h), nk = x[0].shape, w1[0].shape[1]
        M = m * nx
        ws = _workspace(x[0].device, [(TP_OP_AG_MM if sp else TP_OP_COL_FWD, p, M, nk, h, 0),
                                      (TP_OP_ROW_RS if sp else TP_OP_ROW_AR, p, M, h, nk, 0)])
        z = [_empty((M, nk), x[0]) for _ in range(p)]
        hh = [_empty((M, nk), x[0]) for _ in range(p)]
        y = [_empty((m, h), x[0]) for _ in range(nx)]
        if sp:
            tp_ag_matmul(x, w1, z, ws, epi=TP_EPI_GELU, preact=hh)
            tp_row_linear_fwd_reducescatter(z, w2, y, ws)
        else:
            tp_col_linear_fwd(x[0], w1, z, ws, epi=TP_EPI_GELU, preact=hh)
            tp_row_linear_fwd_allreduce(z, w2, y, ws)
        (qx, ex), (qh, eh) = _packed(x), _packed(hh)
        ctx.p, ctx.sp = p, sp
        ctx.save_for_backward(*qx, *ex, *qh, *eh, *w1, *w2)
        return tuple(y)

    @staticmethod
    @once_differentiable
    def backward(ctx, *dy):
        p, sp = ctx.p, ctx.sp
        nx = p if sp else 1
        s = list(ctx.saved_tensors)
        take = lambda n: [s.pop(0) for _ in range(n)]  # noqa: E731
        qx, ex, qh, eh, w1, w2 = take(nx), take(nx), take(p), take(p), take(p), take(p)
        (m, h), nk = qx[0].shape, w1[0].shape[1]
        M, like = m * nx, w1[0]
        dy = [_grad(g, _empty((m, h), like)) for g in dy]
        ops = (TP_OP_ROW_RS_BWD_CKPT, TP_OP_AG_MM_BWD_CKPT) if sp else (TP_OP_ROW_BWD_CKPT, TP_OP_COL_BWD_CKPT)
        ws = _workspace(like.device, [(ops[0], p, M, h, nk, 0), (ops[1], p, M, nk, h, 0)])
        dh = [_empty((M, nk), like) for _ in range(p)]
        dw1, dw2 = [torch.empty_like(t) for t in w1], [torch.empty_like(t) for t in w2]
        dx = [_empty((m, h), like) for _ in range(nx)]
        if sp:
            tp_row_linear_bwd_reducescatter_ckpt(qh, eh, w2, dy, dh, dw2, ws)
            tp_ag_matmul_bwd_ckpt(qx, ex, w1, dh, dx, dw1, ws)
        else:
            tp_row_linear_bwd_ckpt(qh, eh, w2, dy[0], dh, dw2, ws)
            tp_col_linear_bwd_ckpt(qx[0], ex[0], w1, dh, dx[0], dw1, ws)
        return (None, None, *dx, *dw1, *dw2)


def parallel_mlp_ckpt(x, w1: Sequence[torch.Tensor], w2: Sequence[torch.Tensor]):
    """The sharded MLP with its activations saved in 8 bits; x is [M, h], or a list of p token shards."""
    if len(w1) != len(w2):
        raise ValueError("FC1 and FC2 need the same number of shards")
    sp = isinstance(x, (list, tuple))
    if sp and len(x) != len(w1):
        raise ValueError("one token shard per weight shard")
    y = _CkptMLPFn.apply(len(w1), sp, *(x if sp else [x]), *w1, *w2)
    return list(y) if sp else y[0]


# ------------------------------------------------------------------ modules

def _boundary_params(block, h, device, post, pre, gate, alpha, eps) -> None:
    """The vectors of a block's boundary, as its parameters."""
    like = dict(dtype=torch.bfloat16, device=device)
    block.post, block.pre, block.alpha, block.eps = post, pre, alpha, eps
    vec = lambda on, make: torch.nn.Parameter(make(h, **like)) if on else None  # noqa: E731
    block.w_post, block.b_post = vec(_kind(post), torch.ones), vec(post == "layer", torch.zeros)
    block.w_pre, block.b_pre = vec(_kind(pre), torch.ones), vec(pre == "layer", torch.zeros)
    block.gate = torch.nn.Parameter(gate.to(torch.bfloat16).contiguous()) if gate is not None else None


def _boundary_of(block) -> dict:
    return dict(post=block.post, w_post=block.w_post, b_post=block.b_post, pre=block.pre, w_pre=block.w_pre, b_pre=block.b_pre,
                gate=block.gate, alpha=block.alpha, eps=block.eps)


class MLPBlock(torch.nn.Module):
    """A trained block: ``y, n = block(x, n)``.

    w1 [h, ffn] and w2 [ffn, h] are split into p shards.  ``post`` / ``pre``
    name the norms of the boundary ("none", "rms" or "layer"; layer norms have
    biases), ``gate`` is an optional [rows, h] gate (one row: per channel),
    ``alpha`` the residual scale.  ``fp8``: the products on 8-bit
    floating-point operands (whole token tensors only)."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, p: int, *, post: str = "rms", pre: str = "rms", gate=None,
                 alpha: float = 1.0, eps: float = 1e-5, sequence_parallel: bool = False, fp8: bool = False):
        super().__init__()
        if fp8 and sequence_parallel:
            raise ValueError("the 8-bit products take whole token tensors, not shards")
        self.p, self.sequence_parallel, self.fp8 = p, sequence_parallel, fp8
        self.w1, self.w2 = _params(_shards(w1, p, 1)), _params(_shards(w2, p, 0))
        _boundary_params(self, w1.shape[0], w1.device, post, pre, gate, alpha, eps)

    def boundary(self) -> dict:
        return _boundary_of(self)

    def forward(self, x, n):
        z = (parallel_mlp_fp8 if self.fp8 else parallel_mlp_ckpt)(n, list(self.w1), list(self.w2))
        if self.sequence_parallel:
            return block_boundary(x, z, **self.boundary())
        ys, ns = block_boundary([x], [z], **self.boundary())
        return ys[0], (ns[0] if ns else None)

    def serve(self, group: int = 128) -> "W4MLPBlock":
        """This block for serving, its weights in 4 bits with a scale per `group` rows."""
        return W4MLPBlock(self, group)


class W4MLPBlock:
    """A block that serves: ``y, n = block(x, n)`` on [tokens, h] tensors,
    also where the trained block takes token shards.

    It keeps copies of what the block holds when it is made.  Up to
    TP_W4_MAX_M tokens take their products from the 4-bit weights, more from
    weights unpacked for the call (rounded to bfloat16, so that 64 and 65
    tokens differ by that rounding).  The stream x is updated in place.  A
    gate of several rows serves multiples of them only."""

    def __init__(self, block: MLPBlock, group: int = 128):
        self.p, self.group = block.p, group
        with torch.no_grad():
            self.how = {k: v.detach().clone() if torch.is_tensor(v) else v for k, v in block.boundary().items()}
            self.fc1, self.fc2 = self._pack(block.w1), self._pack(block.w2)
        self.how.update(post=_kind(self.how["post"]), pre=_kind(self.how["pre"]))

    def _pack(self, ws):
        K, N = ws[0].shape
        qs, ss = w4_shapes(K, N, self.group)
        q = [torch.empty(qs, dtype=torch.uint8, device=ws[0].device) for _ in ws]
        s = [torch.empty(ss, dtype=torch.bfloat16, device=ws[0].device) for _ in ws]
        tp_w4_pack([w.detach() for w in ws], q, s, group=self.group)
        return q, s, K, N

    def _unpack(self, fc):
        q, s, K, N = fc
        w = [torch.empty((K, N), dtype=torch.bfloat16, device=q[0].device) for _ in q]
        tp_w4_unpack(q, s, w, group=self.group)
        return w

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, n: torch.Tensor) -> tuple:
        p, M = self.p, n.shape[0]
        (q1, s1, h, nk), (q2, s2, _, _) = self.fc1, self.fc2
        a, z = [_empty((M, nk), n) for _ in range(p)], _empty((M, h), n)
        if M <= TP_W4_MAX_M:
            ws = _workspace(n.device, [(TP_OP_COL_W4, p, M, nk, h), (TP_OP_ROW_W4, p, M, h, nk)])
            tp_col_linear_fwd_w4(n, q1, s1, a, ws, group=self.group, epi=TP_EPI_GELU)
            tp_row_linear_fwd_w4(a, q2, s2, z, ws, group=self.group)
        else:
            ws = _workspace(n.device, [(TP_OP_COL_FWD, p, M, nk, h), (TP_OP_ROW_AR, p, M, h, nk)])
            tp_col_linear_fwd(n, self._unpack(self.fc1), a, ws, epi=TP_EPI_GELU)
            tp_row_linear_fwd_allreduce(a, self._unpack(self.fc2), [z], ws)
        out = _empty((M, h), n) if self.how["pre"] else None
        tp_block_norm_fwd([x], [z], [x], [out] if out is not None else None, **self.how)
        return x, out


def _whole_eights(router: torch.Tensor) -> torch.Tensor:
    """A router [h, E] with columns of zeros up to a multiple of 8, as the column layer takes them."""
    return torch.nn.functional.pad(router, (0, -router.shape[1] % 8)) if router.shape[1] % 8 else router


class RoutedMLPBlock(torch.nn.Module):
    """A trained block with experts in the MLP's place: ``y, n = block(x, n)``.

        z[t] = sum_j weights[t, j] GeLU(n[t] W1_e) W2_e,  e = experts[t, j]

    router [h, E], w1 [E, h, f] and w2 [E, f, h] bfloat16, the experts split
    into p shards (h and f multiples of 8).  The logits are bfloat16, as every
    column layer's outputs here; the choice is that of exact arithmetic on
    them, and equal ones go to the lower expert.  ``k`` experts a token; ``score``, ``groups``,
    ``top_groups``, ``group_best``, ``renorm`` and ``scale`` as in ``route``.
    ``bias`` (float32 [E], zeros at first, no parameter) moves the choice only:
    a program balances the load by it, from ``counts``, how often each expert
    was chosen in the last call.  The boundary is MLPBlock's."""

    def __init__(self, router: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, p: int, k: int, *, score: str = "softmax",
                 groups: int = 1, top_groups: int = 1, group_best: int = 1, renorm: bool = False, scale: float = 1.0,
                 post: str = "rms", pre: str = "rms", gate=None, alpha: float = 1.0, eps: float = 1e-5):
        super().__init__()
        E, h, f = w1.shape
        if tuple(router.shape) != (h, E) or tuple(w2.shape) != (E, f, h):
            raise ValueError(f"router [h, E], w1 [E, h, f], w2 [E, f, h]: got {tuple(router.shape)}, {tuple(w1.shape)}, {tuple(w2.shape)}")
        for name, t in (("router", router), ("w1", w1), ("w2", w2)):
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name}: expected bfloat16, got {t.dtype}")
        if score not in SCORES:
            raise ValueError(f"score is one of {sorted(SCORES)}, got {score!r}")
        self.p, self.k = p, k
        self.routing = dict(score=score, groups=groups, top_groups=top_groups, group_best=group_best, renorm=renorm, scale=scale)
        self.router = torch.nn.Parameter(router.contiguous())
        self.w1, self.w2 = _params(_shards(w1, p, 0)), _params(_shards(w2, p, 0))
        self.register_buffer("bias", torch.zeros(E, dtype=torch.float32, device=w1.device))
        self.counts = None
        _boundary_params(self, h, w1.device, post, pre, gate, alpha, eps)

    def forward(self, x, n):
        logits, = column_parallel_linear(n, [_whole_eights(self.router)])
        weights, experts, self.counts = route(logits[:, :self.router.shape[1]], self.k, bias=self.bias, **self.routing)
        z = routed_experts(n, experts, weights, list(self.w1), list(self.w2))
        ys, ns = block_boundary([x], [z], **_boundary_of(self))
        return ys[0], (ns[0] if ns else None)

    def serve(self) -> "ServedRoutedMLPBlock":
        """This block for serving, its experts' weights packed once."""
        return ServedRoutedMLPBlock(self)


class ServedRoutedMLPBlock:
    """A routed block that serves: ``y, n = block(x, n)`` on [tokens, h]
    tensors.  It keeps copies of what the block holds when it is made, the
    experts' weights in 8 bits.  The stream x is updated in place.  A gate of
    several rows serves multiples of them only."""

    def __init__(self, block: RoutedMLPBlock):
        self.p, self.k, self.routing = block.p, block.k, {**block.routing, "score": SCORES[block.routing["score"]]}
        with torch.no_grad():
            copy = lambda v: v.detach().clone() if torch.is_tensor(v) else v  # noqa: E731
            self.how = {k: copy(v) for k, v in _boundary_of(block).items()}
            self.router, self.bias = copy(_whole_eights(block.router)), copy(block.bias)
            _, self.w1 = _operands([w.detach() for w in block.w1], False, True, tiles=True)
            _, self.w2 = _operands([w.detach() for w in block.w2], False, True, tiles=True)
        self.how.update(post=_kind(self.how["post"]), pre=_kind(self.how["pre"]))

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, n: torch.Tensor) -> tuple:
        p, (T, h), (per, f) = self.p, n.shape, self.w1[0].q.shape[:2]
        E, wide = p * per, self.router.shape[1]
        ws = _workspace(n.device, [(TP_OP_COL_FWD, 1, T, wide, h)], tp_experts_workspace_size(p, E, T, self.k, h, f))
        logits, z = _empty((T, wide), n), _empty((T, h), n)
        tp_col_linear_fwd(n, [self.router], [logits], ws)
        logits = logits[:, :E].contiguous()
        experts = torch.empty((T, self.k), dtype=torch.int32, device=n.device)
        weights = torch.empty((T, self.k), dtype=torch.float32, device=n.device)
        tp_route_fwd(logits, experts, weights, bias=self.bias, **self.routing)
        tp_experts_fwd_fp8(n, experts, weights, self.w1, self.w2, z, ws)
        out = _empty((T, h), n) if self.how["pre"] else None
        tp_block_norm_fwd([x], [z], [x], [out] if out is not None else None, **self.how)
        return x, out
