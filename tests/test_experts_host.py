"""Refusals of the routed experts' calls, on the host."""
import ctypes

import pytest
import torch

import gemm_reduce_fusion_gb300 as tp
from test_binding_checks import BF, F32, WS, lib, z, zs  # noqa: F401
from test_block_ops_host import ALIGN, BAD, SHAPE, SMALL, arr, at
from test_fp8_host import pairs

I32 = torch.int32
p, E, T, k, h, f = 2, 4, 6, 2, 64, 136
ROWS, PLAN = tp.tp_experts_rows(E, T, k), tp.tp_experts_plan_size(E, T, k) // 4


def ops(rows, cols, n=p, per=E // p):
    return [tp.fp8_empty(rows, cols, per, device="cpu") for _ in range(n)]


def saved(rows=ROWS, plan=PLAN):
    return tp.ExpertsSaved(z(plan, dtype=I32), z(rows, f), z(rows, h))


@pytest.fixture
def sizes(monkeypatch):
    """The recorder answers every call with 0: the sizes come from the library."""
    monkeypatch.setattr(tp, "tp_experts_rows", lambda *a: ROWS)
    monkeypatch.setattr(tp, "tp_experts_plan_size", lambda *a: PLAN * 4)


def test_sizes():
    # 12 slots of at most 4 experts: each expert's last tile may be nearly empty
    assert ROWS == (12 + 127 * 4) // 128 * 128
    assert PLAN * 4 >= 4 * (1 + (E + 1) + ROWS // 128 + ROWS + T * k)
    assert tp.tp_experts_rows(E, 0, k) == 0 and tp.tp_experts_rows(0, 1, 1) == 0 and tp.tp_experts_rows(513, 1, 1) == 0
    assert tp.tp_experts_workspace_size(1, 4, 1, 2, 64, 64) > 256
    assert tp.tp_experts_workspace_size(1, 4, 99, 2, 64, 64, True) > tp.tp_experts_workspace_size(1, 4, 99, 2, 64, 64)
    assert tp.tp_experts_workspace_size(3, 4, 99, 2, 64, 64) == 256


def test_the_documented_shapes_pass(lib, sizes):  # noqa: F811
    e, w = z(T, k, dtype=I32), z(T, k, dtype=F32)
    tp.tp_experts_fwd_fp8(z(T, h), e, w, ops(f, h), ops(h, f), z(T, h), WS, stream=0)
    tp.tp_experts_fwd_fp8(z(T, h), e, w, ops(f, h), ops(h, f), z(T, h), WS, saved=saved(), stream=0)
    d1, d2 = zs(p, E // p, h, f), zs(p, E // p, f, h)
    tp.tp_experts_bwd_fp8(z(T, h), w, z(T, h), ops(h, f), ops(f, h), z(T, h), z(T, k), d1, d2, saved(), WS, stream=0)
    tp.tp_experts_bwd_fp8(None, w, z(T, h), ops(h, f), ops(f, h), z(T, h), None, None, None, saved(), WS, stream=0)
    tp.tp_experts_bwd_fp8(None, w, z(T, h), None, None, None, z(T, k), None, d2, saved(), WS, stream=0)
    assert len(lib.calls) == 5


def test_wrong_arguments_are_refused_before_the_library(lib, sizes):  # noqa: F811
    e, w, a, b = z(T, k, dtype=I32), z(T, k, dtype=F32), ops(f, h), ops(h, f)
    d1 = zs(p, E // p, h, f)

    def fwd(x=z(T, h), e=e, w=w, a=a, b=b, y=z(T, h), s=None):
        tp.tp_experts_fwd_fp8(x, e, w, a, b, y, WS, saved=s, stream=0)

    def bwd(x=z(T, h), w=w, dy=z(T, h), a=ops(h, f), b=ops(f, h), dx=z(T, h), dw=z(T, k), d1=d1, d2=None, s=saved()):
        tp.tp_experts_bwd_fp8(x, w, dy, a, b, dx, dw, d1, d2, s, WS, stream=0)
    for call in (lambda: fwd(x=z(T * h)), lambda: fwd(e=z(T + 1, k, dtype=I32)), lambda: fwd(w=z(T, k + 1, dtype=F32)),
                 lambda: fwd(a=ops(f, h + 128)), lambda: fwd(b=ops(h, f, n=1)), lambda: fwd(b=ops(h, f, per=1)),
                 lambda: fwd(a=[tp.fp8_empty(f, h, device="cpu")] * 2), lambda: fwd(y=z(T, h + 8)), lambda: fwd(s=saved(rows=ROWS - 128)),
                 lambda: fwd(s=saved(plan=PLAN - 64)), lambda: bwd(dy=z(T + 1, h)), lambda: bwd(x=z(T, h + 8)), lambda: bwd(a=ops(f, h)),
                 lambda: bwd(b=ops(h, f)), lambda: bwd(dw=z(T, k + 1)), lambda: bwd(d1=zs(p, E // p, f, h)), lambda: bwd(d2=zs(1, E // p, f, h)),
                 lambda: bwd(a=None, b=None, d1=None), lambda: bwd(s=saved(rows=ROWS + 128))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fwd(x=z(T, h, dtype=F32)), lambda: fwd(e=z(T, k, dtype=torch.int64)), lambda: fwd(w=z(T, k)), lambda: fwd(y=z(T, h, dtype=F32)),
                 lambda: bwd(dw=z(T, k, dtype=F32)), lambda: bwd(dy=z(T, h, dtype=F32))):
        with pytest.raises(TypeError):
            call()
    assert lib.calls == []


L = tp._lib
SV = tp._ExpertsSaved


def test_forward_refusals():
    need = tp.tp_experts_workspace_size(p, E, T, k, h, f)

    def fwd(x=at(0), e=at(1), w=at(2), a=pairs(at(3), at(4)), b=pairs(at(5), at(6)), y=at(7), s=None, p=p, E=E, T=T, k=k, h=h, f=f, ws=at(8), n=need):
        return L.tp_experts_fwd_fp8(x, e, w, a, b, y, ctypes.byref(s) if s else None, p, E, T, k, h, f, ws, n, None)
    for kw in (dict(x=None), dict(e=None), dict(w=None), dict(a=None), dict(b=pairs(at(5), None)), dict(y=None), dict(p=0), dict(p=9), dict(E=0),
               dict(T=-1), dict(k=0), dict(h=0), dict(f=0), dict(y=at(0)), dict(y=at(5)), dict(ws=at(1)), dict(ws=None),
               dict(s=SV(at(9), at(10), None), n=1 << 26, ws=at(30)), dict(s=SV(at(9), at(10), at(0)), n=1 << 26, ws=at(30))):
        assert fwd(**kw) == BAD, kw
    assert fwd(n=need - 1) == SMALL
    assert fwd(p=3) == SHAPE and fwd(E=514) == SHAPE and fwd(k=33) == SHAPE and fwd(T=1 << 30, k=4) == SHAPE
    assert fwd(h=60) == ALIGN and fwd(x=at(0) + 8) == ALIGN and fwd(e=at(1) + 2) == ALIGN and fwd(ws=at(8) + 8) == ALIGN
    assert fwd(T=0) == tp.TP_OK


def test_backward_refusals():
    n = tp.tp_experts_workspace_size(p, E, T, k, h, f, True)
    s = SV(at(20), at(21), at(22))

    def bwd(x=at(0), w=at(1), dy=at(2), a=pairs(at(3), at(4)), b=pairs(at(5), at(6)), dx=at(7), dw=at(8), d1=arr(at(9), at(10)), d2=arr(at(11), at(12)),
            s=s, ws=at(30), n=n, **o):
        o = {**dict(p=p, E=E, T=T, k=k, h=h, f=f), **o}
        return L.tp_experts_bwd_fp8(x, w, dy, a, b, dx, dw, d1, d2, ctypes.byref(s) if s else None, *o.values(), ws, n, None)
    for kw in (dict(dx=None, dw=None, d1=None, d2=None), dict(x=None), dict(w=None), dict(dy=None), dict(a=None), dict(b=None), dict(s=None),
               dict(d1=arr(at(9), None)), dict(d2=arr(at(11), at(11))), dict(dx=at(2)), dict(dw=at(1)), dict(d1=arr(at(9), at(21))), dict(ws=None),
               dict(s=SV(at(20), None, at(22)))):
        assert bwd(**kw) == BAD, kw
    assert bwd(n=n - 1) == SMALL and bwd(p=3) == SHAPE and bwd(f=60) == ALIGN and bwd(dw=at(8) + 1) == ALIGN
