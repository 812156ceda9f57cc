"""Refusals of the 8-bit products, on the host: by the binding before the
library is reached, and by the library's own checks (made-up pointers, nothing
is launched)."""
import ctypes

import pytest
import torch

import gemm_reduce_fusion_gb300 as tp
from test_binding_checks import BF, WS, lib, z, zs  # noqa: F401
from test_block_ops_host import ALIGN, BAD, SHAPE, SMALL, arr, at

p, M, N, K = 2, 8, 40, 256


def op(rows, cols, batch=None):
    return tp.fp8_empty(rows, cols, batch, device="cpu")


def ops(n, rows, cols):
    return [op(rows, cols) for _ in range(n)]


def test_shapes():
    assert tp.fp8_shapes(300, 1000) == ((300, 1024), (3, 2, 512))
    assert tp.fp8_shapes(1, 8) == ((1, 128), (1, 1, 512))
    assert tp.fp8_empty(1, 8, 3, device="cpu").e.shape == (3, 1, 1, 512)


def test_the_documented_shapes_pass(lib):  # noqa: F811
    tp.tp_fp8_pack(zs(p, M, 200), ops(p, M, 200), ops(p, 200, M), stream=0)
    tp.tp_fp8_pack([z(3, M, 200)], [op(M, 200, 3)], tiles=True, stream=0)
    tp.tp_fp8_pack(zs(p, M, 200), None, ops(p, 200, M), epi=tp.TP_EPI_GELU, stream=0)
    tp.tp_fp8_unpack(ops(p, M, 200), zs(p, M, 200), stream=0)
    tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), zs(p, M, N), WS, epi=tp.TP_EPI_GELU, preact=zs(p, M, N), bias=zs(p, N), stream=0)
    tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), None, WS, z=ops(p, M, N), stream=0)
    tp.tp_row_linear_fwd_fp8(ops(p, M, 200), ops(p, N, 200), z(M, N), WS, bias=z(N), stream=0)
    tp.tp_col_linear_bwd_fp8(op(K, M), ops(p, K, N), ops(p, M, N), ops(p, N, M), z(M, K), zs(p, K, N), WS, stream=0)
    tp.tp_col_linear_bwd_fp8(None, ops(p, K, N), ops(p, M, N), None, z(M, K), None, WS, stream=0)
    tp.tp_row_linear_bwd_fp8(ops(p, K, M), ops(p, K, N), op(M, N), op(N, M), zs(p, M, K), zs(p, K, N), WS, preact=zs(p, M, K), stream=0)
    tp.tp_row_linear_bwd_fp8(ops(p, K, M), None, None, op(N, M), None, zs(p, K, N), WS, stream=0)
    assert len(lib.calls) == 11


WRONG = {
    "pack rows": lambda: tp.tp_fp8_pack(zs(p, M, 200), ops(p, M + 1, 200), stream=0),
    "pack columns": lambda: tp.tp_fp8_pack(zs(p, M, 200), ops(p, M, 264), stream=0),
    "pack transpose": lambda: tp.tp_fp8_pack(zs(p, M, 200), None, ops(p, M, 200), stream=0),
    "pack batch": lambda: tp.tp_fp8_pack([z(3, M, 200)], [op(M, 200, 2)], stream=0),
    "pack vector": lambda: tp.tp_fp8_pack([z(200)], [op(1, 200)], stream=0),
    "pack count": lambda: tp.tp_fp8_pack(zs(p, M, 200), ops(1, M, 200), stream=0),
    "unpack": lambda: tp.tp_fp8_unpack(ops(p, M, 200), zs(p, M, 300), stream=0),
    "col depth": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 300), zs(p, M, N), WS, stream=0),
    "col columns": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), zs(p, M, N + 8), WS, stream=0),
    "col both": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), zs(p, M, N), WS, z=ops(p, M, N), stream=0),
    "col none": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), None, WS, stream=0),
    "col z": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), None, WS, z=ops(p, M + 1, N), stream=0),
    "col preact": lambda: tp.tp_col_linear_fwd_fp8(op(M, 200), ops(p, N, 200), zs(p, M, N), WS, epi=1, preact=zs(p, M, 8), stream=0),
    "row exponents": lambda: tp.tp_row_linear_fwd_fp8([tp.Fp8(op(M, 200).q, op(200, 200).e)], ops(1, N, 200), z(M, N), WS, stream=0),
    "row bias": lambda: tp.tp_row_linear_fwd_fp8(ops(p, M, 200), ops(p, N, 200), z(M, N), WS, bias=z(M), stream=0),
    "bwd none": lambda: tp.tp_col_linear_bwd_fp8(op(K, M), ops(p, K, N), ops(p, M, N), ops(p, N, M), None, None, WS, stream=0),
    "bwd without dy": lambda: tp.tp_col_linear_bwd_fp8(op(K, M), ops(p, K, N), None, ops(p, N, M), z(M, K), None, WS, stream=0),
    "bwd without xt": lambda: tp.tp_row_linear_bwd_fp8(None, ops(p, K, N), op(M, N), op(N, M), zs(p, M, K), zs(p, K, N), WS, stream=0),
    "bwd weights": lambda: tp.tp_row_linear_bwd_fp8(None, ops(p, N, K), op(M, N), None, zs(p, M, K), None, WS, stream=0),
    "bwd shards": lambda: tp.tp_col_linear_bwd_fp8(op(K, M), ops(p, K, N), ops(1, M, N), ops(p, N, M), z(M, K), None, WS, stream=0),
}


@pytest.mark.parametrize("case", WRONG)
def test_wrong_shapes_are_refused_before_the_library(lib, case):  # noqa: F811
    with pytest.raises(ValueError):
        WRONG[case]()
    assert lib.calls == []


def test_wrong_dtypes_layouts_and_devices_are_refused(lib, monkeypatch):  # noqa: F811
    with pytest.raises(TypeError):
        tp.tp_fp8_pack(zs(p, M, 200, dtype=torch.float32), ops(p, M, 200), stream=0)
    with pytest.raises(TypeError):
        tp.tp_fp8_pack(zs(1, M, 200), [tp.Fp8(op(M, 200).q.view(torch.uint8), op(M, 200).e)], stream=0)
    with pytest.raises(TypeError):
        tp.tp_fp8_pack(zs(1, M, 200), [tp.Fp8(op(M, 200).q, op(M, 200).e.view(torch.int8))], stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        tp.tp_fp8_pack([z(200, M).t()], [op(M, 200)], stream=0)
    monkeypatch.setattr(tp, "_current_device", lambda: 0)
    with pytest.raises(TypeError, match="cuda:0"):
        tp.tp_fp8_pack(zs(1, M, 200), [op(M, 200)], stream=0)
    assert lib.calls == []


# ------------------------------------------------------------------ the library's own checks

L = tp._lib


def pairs(*ptrs):
    """A C array of operands: q at each pointer, e far behind it."""
    return (ctypes.c_void_p * (2 * len(ptrs)))(*[v for q in ptrs for v in (q, None if q is None else q + (1 << 23))])


def test_packing_refusals():
    def call(x=arr(at(0), at(1)), q=pairs(at(2), at(3)), qt=pairs(at(4), at(5)), tiles=0, epi=0, p=2, batch=1, M=64, N=128):
        return L.tp_fp8_pack(x, q, qt, tiles, epi, p, batch, M, N, None)
    for kw in (dict(x=None), dict(x=arr(at(0), None)), dict(q=None, qt=None), dict(q=pairs(at(2), None)), dict(tiles=2), dict(epi=2),
               dict(p=0), dict(p=9), dict(batch=-1), dict(M=-1), dict(q=pairs(at(0), at(3))), dict(qt=pairs(at(2), at(5))),
               dict(qt=pairs(at(4), at(4)))):
        assert call(**kw) == BAD, kw
    assert call(N=60) == ALIGN and call(q=pairs(at(2) + 8, at(3))) == ALIGN and call(x=arr(at(0) + 2, at(1))) == ALIGN
    assert call(batch=40000) == SHAPE and call(M=1 << 24) == SHAPE
    assert call(M=0) == tp.TP_OK and call(batch=0) == tp.TP_OK and call(N=0) == tp.TP_OK
    assert L.tp_fp8_unpack(pairs(at(0)), arr(at(0)), 1, 1, 64, 128, None) == BAD
    assert L.tp_fp8_unpack(pairs(None), arr(at(0)), 1, 1, 64, 128, None) == BAD
    assert L.tp_fp8_unpack(pairs(at(0)), arr(at(1) + 8), 1, 1, 64, 128, None) == ALIGN


def test_forward_refusals():
    need = tp.tp_workspace_size(tp.TP_OP_COL_FP8, 2, 16, 64, 8192)
    assert need > 256

    def col(x=pairs(at(0)), w=pairs(at(1), at(2)), bias=None, y=arr(at(3), at(4)), z=None, pre=None, epi=0, p=2, M=16, N=64, K=8192, ws=at(7),
            n=need):
        return L.tp_col_linear_fwd_fp8(x, w, bias, y, z, pre, epi, p, M, N, K, ws, n, None)
    for kw in (dict(x=None), dict(w=None), dict(w=pairs(at(1), None)), dict(y=None), dict(z=pairs(at(5), at(6))), dict(epi=2),
               dict(pre=arr(at(5), at(6))), dict(y=arr(at(3), None)), dict(y=arr(at(3), at(3))), dict(y=arr(at(0), at(3))), dict(ws=at(1)),
               dict(ws=None), dict(p=9), dict(M=-1), dict(y=None, z=pairs(at(5), at(0))), dict(epi=1, pre=arr(at(5), at(3)))):
        assert col(**kw) == BAD, kw
    assert col(n=need - 1) == SMALL and col(N=60) == ALIGN and col(x=pairs(at(0) + 8)) == ALIGN and col(bias=arr(at(8) + 2, None)) == ALIGN
    assert col(ws=at(7) + 8) == ALIGN

    need = tp.tp_workspace_size(tp.TP_OP_ROW_FP8, 2, 16, 64, 8192)

    def row(x=pairs(at(0), at(1)), w=pairs(at(2), at(3)), bias=None, y=at(4), p=2, M=16, N=64, K=8192, ws=at(7), n=need):
        return L.tp_row_linear_fwd_fp8(x, w, bias, y, p, M, N, K, ws, n, None)
    for kw in (dict(x=None), dict(w=pairs(None, at(2))), dict(y=None), dict(y=at(1)), dict(ws=at(2))):
        assert row(**kw) == BAD, kw
    assert row(n=need - 1) == SMALL and row(bias=at(8) + 8) == ALIGN
    assert row(M=0) == tp.TP_OK


def test_backward_refusals():
    def col(xt=pairs(at(0)), w=pairs(at(1), at(2)), dy=pairs(at(3), at(4)), dyt=pairs(at(5), at(6)), dx=at(8), dw=arr(at(9), at(10)), ws=at(11),
            n=1 << 23, N=64):
        return L.tp_col_linear_bwd_fp8(xt, w, dy, dyt, dx, dw, 2, 16, N, 128, ws, n, None)
    for kw in (dict(dx=None, dw=None), dict(xt=None), dict(w=None), dict(dy=None), dict(dyt=pairs(at(5), None)), dict(dw=arr(at(9), at(9))),
               dict(dx=at(3)), dict(dw=arr(at(5), at(10))), dict(ws=at(0)), dict(ws=None)):
        assert col(**kw) == BAD, kw
    assert col(n=128) == SMALL and col(N=60) == ALIGN and col(dx=at(8) + 2) == ALIGN

    def row(xt=pairs(at(0), at(1)), w=pairs(at(2), at(3)), dy=pairs(at(4)), dyt=pairs(at(5)), dx=arr(at(6), at(7)), dw=arr(at(8), at(9)),
            pre=arr(at(10), at(11)), ws=at(12)):
        return L.tp_row_linear_bwd_fp8(xt, w, dy, dyt, dx, dw, pre, 2, 16, 64, 128, ws, 1 << 23, None)
    for kw in (dict(dx=None, dw=None), dict(xt=None), dict(w=None), dict(dy=None), dict(dyt=None), dict(pre=arr(at(10), None)),
               dict(dx=arr(at(6), at(10)))):
        assert row(**kw) == BAD, kw
