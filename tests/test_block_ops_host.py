"""Refusals of the operators around the sharded Linear, on the host: by the
binding before the library is reached, and by the library's own checks (fake
pointers: nothing is launched)."""
import ctypes

import pytest
import torch

import gemm_reduce_fusion_gb300 as tp
from test_binding_checks import BF, F32, WS, lib, z, zs  # noqa: F401

I8, U8 = torch.int8, torch.uint8
p, M, h = 2, 6, 64


def test_the_documented_shapes_pass(lib):  # noqa: F811
    x, n = zs(p, M, h), zs(p, M, h)
    tp.tp_block_norm_fwd(x, zs(p, M, h), zs(p, M, h), n, post=tp.TP_NORM_LAYER, w_post=z(h), b_post=z(h), pre=tp.TP_NORM_RMS,
                         w_pre=z(h), gate=z(4, h), alpha=0.5, stream=0)
    tp.tp_block_norm_fwd(zs(p, M, h, dtype=F32), None, None, n, pre=tp.TP_NORM_RMS, stream=0)
    tp.tp_block_norm_bwd(zs(p, M, h), zs(p, M, h, dtype=F32), n, None, zs(p, M, h, dtype=F32), zs(p, M, h), WS, pre=tp.TP_NORM_RMS,
                         post=tp.TP_NORM_RMS, gate=z(1, h), dgate=z(1, h, dtype=F32), dw_pre=z(h, dtype=F32), stream=0)
    tp.tp_ckpt_pack(zs(p, M, 40), zs(p, M, 40, dtype=I8), zs(p, M, 2, dtype=U8), stream=0)
    tp.tp_ckpt_unpack(zs(p, M, 40, dtype=I8), zs(p, M, 2, dtype=U8), zs(p, M, 40), epi=tp.TP_EPI_GELU, stream=0)
    K, N = 40, 24
    q, e = z(M, K, dtype=I8), z(M, 2, dtype=U8)
    tp.tp_col_linear_bwd_ckpt(q, e, zs(p, K, N), zs(p, M, N), z(M, K), zs(p, K, N), WS, stream=0, db=zs(p, N))
    tp.tp_col_linear_bwd_ckpt(None, None, zs(p, K, N), zs(p, M, N), z(M, K), None, WS, stream=0)
    tp.tp_row_linear_bwd_ckpt([q] * p, [e] * p, zs(p, K, N), z(M, N), zs(p, M, K), zs(p, K, N), WS, stream=0, db=z(N))
    tp.tp_ag_matmul_bwd_ckpt([z(3, K, dtype=I8)] * p, [z(3, 2, dtype=U8)] * p, zs(p, K, N), zs(p, M, N), zs(p, 3, K),
                             zs(p, K, N), WS, stream=0)
    tp.tp_row_linear_bwd_reducescatter_ckpt([q] * p, [e] * p, zs(p, K, N), zs(p, 3, N), zs(p, M, K), zs(p, K, N), WS, stream=0)
    qs, ss = tp.w4_shapes(K, N, 32)
    q4, s4 = zs(p, *qs, dtype=U8), zs(p, *ss)
    tp.tp_col_linear_fwd_w4(z(M, K), q4, s4, zs(p, M, N), WS, group=32, epi=tp.TP_EPI_GELU, bias=zs(p, N), stream=0)
    tp.tp_row_linear_fwd_w4(zs(p, M, K), q4, s4, z(M, N, dtype=F32), WS, group=32, bias=z(N), stream=0)
    tp.tp_w4_pack(zs(p, K, N), q4, s4, group=32, stream=0)
    tp.tp_w4_unpack(q4, s4, zs(p, K, N), group=32, stream=0)
    assert len(lib.calls) == 14


def _qs(K, N, G):
    qs, ss = tp.w4_shapes(K, N, G)
    return zs(p, *qs, dtype=U8), zs(p, *ss)


WRONG = {
    "short shard": lambda: tp.tp_block_norm_fwd([z(M, h), z(M - 1, h)], None, None, zs(p, M, h), pre=1, stream=0),
    "wide z": lambda: tp.tp_block_norm_fwd(zs(p, M, h), zs(p, M, h + 8), zs(p, M, h), zs(p, M, h), pre=1, stream=0),
    "missing n shard": lambda: tp.tp_block_norm_fwd(zs(p, M, h), None, None, zs(1, M, h), pre=1, stream=0),
    "weight length": lambda: tp.tp_block_norm_fwd(zs(p, M, h), None, None, zs(p, M, h), pre=1, w_pre=z(h + 8), stream=0),
    "gate width": lambda: tp.tp_block_norm_fwd(zs(p, M, h), zs(p, M, h), zs(p, M, h), zs(p, M, h), pre=1, gate=z(1, 8), stream=0),
    "gate vector": lambda: tp.tp_block_norm_fwd(zs(p, M, h), zs(p, M, h), zs(p, M, h), zs(p, M, h), pre=1, gate=z(h), stream=0),
    "dgate rows": lambda: tp.tp_block_norm_bwd(zs(p, M, h), zs(p, M, h), zs(p, M, h), None, zs(p, M, h), None, WS, pre=1,
                                               gate=z(2, h), dgate=z(1, h), stream=0),
    "no stream": lambda: tp.tp_block_norm_bwd(None, None, zs(p, M, h), None, None, None, WS, pre=1, stream=0),
    "exponents": lambda: tp.tp_ckpt_pack(zs(p, M, 40), zs(p, M, 40, dtype=I8), zs(p, M, 1, dtype=U8), stream=0),
    "restored": lambda: tp.tp_ckpt_unpack(zs(p, M, 40, dtype=I8), zs(p, M, 2, dtype=U8), zs(p, M, 48), stream=0),
    "col ckpt": lambda: tp.tp_col_linear_bwd_ckpt(z(M, 48, dtype=I8), z(M, 2, dtype=U8), zs(p, 40, 24), zs(p, M, 24), z(M, 40),
                                                  None, WS, stream=0),
    "row ckpt": lambda: tp.tp_row_linear_bwd_ckpt(zs(1, M, 40, dtype=I8), zs(1, M, 2, dtype=U8), zs(p, 40, 24), z(M, 24),
                                                  zs(p, M, 40), None, WS, stream=0),
    "w4 tiles": lambda: tp.tp_row_linear_fwd_w4(zs(p, M, 72), *_qs(64, 24, 32), z(M, 24), WS, group=32, stream=0),
    "w4 scales": lambda: tp.tp_row_linear_fwd_w4(zs(p, M, 72), *_qs(72, 24, 64), z(M, 24), WS, group=32, stream=0),
    "w4 group": lambda: tp.tp_row_linear_fwd_w4(zs(p, M, 72), *_qs(72, 24, 16), z(M, 24), WS, group=16, stream=0),
    "w4 output": lambda: tp.tp_col_linear_fwd_w4(z(M, 72), *_qs(72, 24, 32), [z(M, 24), z(M, 32)], WS, group=32, stream=0),
}


@pytest.mark.parametrize("case", WRONG)
def test_wrong_shapes_are_refused_before_the_library(lib, case):  # noqa: F811
    with pytest.raises(ValueError):
        WRONG[case]()
    assert lib.calls == []


def test_wrong_dtypes_layouts_and_devices_are_refused(lib, monkeypatch):  # noqa: F811
    x = zs(p, M, h)
    with pytest.raises(TypeError):
        tp.tp_block_norm_fwd(zs(p, M, h, dtype=torch.float16), None, None, x, pre=1, stream=0)
    with pytest.raises(TypeError):
        tp.tp_block_norm_fwd(x, None, None, zs(p, M, h, dtype=F32), pre=1, stream=0)
    with pytest.raises(TypeError):
        tp.tp_block_norm_bwd(None, x, x, None, x, None, WS, pre=1, dw_pre=z(h, dtype=torch.float16), stream=0)
    with pytest.raises(TypeError):
        tp.tp_ckpt_pack(zs(p, M, 40), zs(p, M, 40, dtype=U8), zs(p, M, 2, dtype=U8), stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        tp.tp_ckpt_pack([z(40, M).t()] * p, zs(p, M, 40, dtype=I8), zs(p, M, 2, dtype=U8), stream=0)
    with pytest.raises(TypeError):
        tp.tp_w4_pack(zs(p, 72, 24, dtype=F32), *_qs(72, 24, 32), group=32, stream=0)
    monkeypatch.setattr(tp, "_current_device", lambda: 0)
    with pytest.raises(TypeError, match="cuda:0"):
        tp.tp_block_norm_fwd(x, None, None, x, pre=1, stream=0)
    assert lib.calls == []


# ------------------------------------------------------------------ the library's own checks

L = tp._lib
BASE = 1 << 32


def arr(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def at(i):
    """A fake, aligned device pointer; different i never overlap."""
    return BASE + i * (1 << 24)


def norm_fwd(x=arr(at(0)), zz=arr(at(1)), y=arr(at(2)), n=arr(at(3)), p=1, M=8, h=64, res=0, **d):
    d = {**dict(post=1, pre=1, alpha=1.0, eps=1e-5), **d}
    desc = tp._NormDesc(**d)
    return L.tp_block_norm_fwd(x, zz, y, n, ctypes.byref(desc), p, M, h, res, None)


BAD, ALIGN, SHAPE, SMALL = tp.TP_ERR_INVALID_ARG, tp.TP_ERR_ALIGNMENT, tp.TP_ERR_UNSUPPORTED_SHAPE, tp.TP_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("status,kw", [
    (BAD, dict(p=0)), (BAD, dict(p=9)), (BAD, dict(M=-1)), (BAD, dict(res=2)), (BAD, dict(post=3)), (BAD, dict(pre=-1)),
    (BAD, dict(eps=-1.0)), (BAD, dict(eps=float("nan"))), (BAD, dict(alpha=float("inf"))), (BAD, dict(zz=None)),
    (BAD, dict(y=None)), (BAD, dict(n=None)), (BAD, dict(pre=0)), (BAD, dict(x=None)), (BAD, dict(x=arr(None))),
    (BAD, dict(b_post=at(9))), (BAD, dict(post=0, w_post=at(9))), (BAD, dict(gate=at(9), gate_rows=0)),
    (BAD, dict(y=arr(at(1)))), (BAD, dict(n=arr(at(0)))), (BAD, dict(y=arr(at(3)))), (BAD, dict(y=arr(at(0) + 16))),
    (BAD, dict(w_pre=at(3))), (SHAPE, dict(h=16392)), (SHAPE, dict(p=3, M=8)), (SHAPE, dict(gate=at(9), gate_rows=3)),
    (ALIGN, dict(h=60)), (ALIGN, dict(x=arr(at(0) + 8))), (ALIGN, dict(w_pre=at(9) + 2))])
def test_norm_forward_refusals(status, kw):
    assert norm_fwd(**kw) == status


def test_norm_backward_refusals():
    def call(zz=arr(at(0)), y=arr(at(1)), dn=arr(at(2)), dy=arr(at(3)), dx=arr(at(4)), dz=arr(at(5)), ws=at(7), n=None, out=1,
             g=None, **d):
        d = {**dict(post=1, pre=1, alpha=1.0, eps=1e-5), **d}
        grads = tp._NormGrads(**(g or {}))
        need = tp.tp_workspace_size(tp.TP_OP_BLOCK_NORM_BWD, 1, 8, 64, 0)
        return L.tp_block_norm_bwd(zz, y, dn, dy, dx, dz, ctypes.byref(tp._NormDesc(**d)), ctypes.byref(grads), 1, 8, 64, 0, out,
                                   ws, need if n is None else n, None)
    for kw in (dict(dn=None), dict(dn=None, dy=None, pre=0), dict(y=None), dict(dx=None, dz=None), dict(zz=None, post=0),
               dict(out=2), dict(g=dict(dgate=at(8))), dict(g=dict(db_pre=at(8))), dict(post=0, g=dict(dw_post=at(8))),
               dict(ws=None), dict(dz=arr(at(3))), dict(dx=arr(at(1))), dict(ws=at(2)), dict(g=dict(dw_pre=at(7)))):
        assert call(**kw) == BAD, kw
    assert call(n=256) == SMALL
    assert call(ws=at(7) + 8) == ALIGN
    assert call(g=dict(dw_pre=at(8) + 8)) == ALIGN


def test_checkpoint_refusals():
    x, q, e = arr(at(0)), arr(at(1)), arr(at(2))
    assert L.tp_ckpt_pack(x, q, e, 0, 8, 64, None) == BAD
    assert L.tp_ckpt_pack(None, q, e, 1, 8, 64, None) == BAD
    assert L.tp_ckpt_pack(x, q, None, 1, 8, 64, None) == BAD
    assert L.tp_ckpt_pack(x, arr(at(0) + 64), e, 1, 8, 64, None) == BAD
    assert L.tp_ckpt_pack(x, q, e, 1, 8, 60, None) == ALIGN
    assert L.tp_ckpt_pack(x, arr(at(1) + 8), e, 1, 8, 64, None) == ALIGN
    assert L.tp_ckpt_unpack(q, e, x, 2, 1, 8, 64, None) == BAD
    assert L.tp_ckpt_unpack(q, e, arr(at(2)), 0, 1, 8, 64, None) == BAD
    P, N, K = 2, 64, 32
    need = {op: tp.tp_workspace_size(op, P, 8, N, K) for op in range(10, 14)}
    w, dy, dw = arr(at(3), at(4)), arr(at(5), at(6)), arr(at(7), at(8))

    def col(q=at(1), e=at(2), dx=at(9), dw=dw, ws=at(10), n=need[10]):
        return L.tp_col_linear_bwd_ckpt(q, e, w, dy, dx, dw, None, P, 8, N, K, 0, 0, ws, n, None)
    assert col(q=None) == BAD and col(e=None) == BAD and col(dx=None, dw=None) == BAD
    assert col(dx=at(1)) == BAD and col(ws=at(2)) == BAD and col(n=need[10] - 1) == SMALL and col(q=at(1) + 8) == ALIGN
    assert L.tp_ag_matmul_bwd_ckpt(w, w, w, dy, None, dw, None, P, 9, N, K, 0, 0, at(10), 1 << 22, None) == SHAPE

    def row(q=arr(at(11), at(12)), e=arr(at(13), at(14)), dx=arr(at(9), at(15)), epi=2, n=need[11]):
        return L.tp_row_linear_bwd_ckpt(q, e, w, at(5), dx, dw, None, epi, P, 8, N, K, 0, 0, at(10), n, None)
    assert row(epi=1) == BAD and row(q=None) == BAD and row(e=arr(at(13), None)) == BAD and row(n=need[11] - 1) == SMALL
    assert row(dx=arr(at(9), at(9))) == BAD and row(dx=arr(at(9), at(13))) == BAD


def test_4_bit_refusals():
    P, M, N, K = 2, 4, 64, 128
    x, q, s = arr(at(0), at(1)), arr(at(2), at(3)), arr(at(4), at(5))
    need = tp.tp_workspace_size(tp.TP_OP_ROW_W4, P, M, N, K)

    def row(x=x, q=q, s=s, y=at(6), bias=None, p=P, M=M, N=N, K=K, G=64, dt=0, ws=at(7), n=need):
        return L.tp_row_linear_fwd_w4(x, q, s, bias, y, p, M, N, K, G, dt, ws, n, None)
    for kw in (dict(x=None), dict(q=None), dict(s=arr(at(4), None)), dict(y=None), dict(p=9), dict(G=0), dict(G=96), dict(dt=3),
               dict(ws=None), dict(y=at(2)), dict(ws=at(1)), dict(y=at(7) + 64), dict(M=-1)):
        assert row(**kw) == BAD, kw
    assert row(M=65) == SHAPE and row(n=need - 1) == SMALL
    assert row(K=12) == ALIGN and row(y=at(6) + 8) == ALIGN and row(bias=at(8) + 2) == ALIGN
    assert L.tp_col_linear_fwd_w4(at(0), q, s, None, arr(at(6), at(8)), 2, P, M, N, K, 64, 0, at(7), 1 << 22, None) == BAD
    assert L.tp_col_linear_fwd_w4(at(0), q, s, None, arr(at(6), at(6)), 0, P, M, N, K, 64, 0, at(7), 1 << 22, None) == BAD
    assert L.tp_w4_pack(q, q, s, P, N, K, 64, None) == BAD
    assert L.tp_w4_unpack(q, s, arr(at(6), None), P, N, K, 64, None) == BAD
    assert L.tp_w4_unpack(q, s, arr(at(6), at(8)), P, N, K, 48, None) == BAD
