"""Refusals of the routing calls, on the host."""
import ctypes

import pytest
import torch

import gemm_reduce_fusion_gb300 as tp
from test_binding_checks import BF, F32, lib, z  # noqa: F401
from test_block_ops_host import ALIGN, BAD, SHAPE, at

I32 = torch.int32
T, E, k = 6, 40, 3


def test_the_documented_shapes_pass(lib):  # noqa: F811
    tp.tp_route_fwd(z(T, E), z(T, k, dtype=I32), z(T, k, dtype=F32), counts=z(E, dtype=I32), bias=z(E, dtype=F32), groups=4, top_groups=2,
                    group_best=2, renorm=True, scale=2.5, score=tp.TP_ROUTE_SIGMOID, stream=0)
    tp.tp_route_fwd(z(T, E, dtype=F32), z(T, k, dtype=I32), z(T, k, dtype=F32), stream=0)
    tp.tp_route_bwd(z(T, E), z(T, k, dtype=I32), z(T, k, dtype=F32), z(T, E), renorm=True, stream=0)
    assert len(lib.calls) == 3


def test_wrong_arguments_are_refused_before_the_library(lib):  # noqa: F811
    e, w = z(T, k, dtype=I32), z(T, k, dtype=F32)
    for call in (lambda: tp.tp_route_fwd(z(T * E), e, w, stream=0), lambda: tp.tp_route_fwd(z(T, E), e, z(T, k + 1, dtype=F32), stream=0),
                 lambda: tp.tp_route_fwd(z(T, E), z(T + 1, k, dtype=I32), w, stream=0),
                 lambda: tp.tp_route_fwd(z(T, E), e, w, bias=z(E + 1, dtype=F32), stream=0),
                 lambda: tp.tp_route_fwd(z(T, E), e, w, counts=z(k, dtype=I32), stream=0),
                 lambda: tp.tp_route_fwd(z(E, T).t(), e, w, stream=0),
                 lambda: tp.tp_route_bwd(z(T, E), e, w, z(T, E + 1), stream=0),
                 lambda: tp.tp_route_bwd(z(T, E), e, z(T, k + 1, dtype=F32), z(T, E), stream=0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tp.tp_route_fwd(z(T, E, dtype=torch.float16), e, w, stream=0),
                 lambda: tp.tp_route_fwd(z(T, E), z(T, k, dtype=torch.int64), w, stream=0), lambda: tp.tp_route_fwd(z(T, E), e, z(T, k), stream=0),
                 lambda: tp.tp_route_fwd(z(T, E), e, w, bias=z(E), stream=0),
                 lambda: tp.tp_route_bwd(z(T, E), e, w, z(T, E, dtype=F32), stream=0)):
        with pytest.raises(TypeError):
            call()
    assert lib.calls == []


L = tp._lib


def fwd(logits=at(0), bias=at(1), experts=at(2), weights=at(3), counts=at(4), T=T, E=E, k=k, dt=0, desc=True, **d):
    d = tp._RouteDesc(**{**dict(score=0, groups=1, top_groups=1, group_best=1, renorm=0, scale=1.0), **d})
    return L.tp_route_fwd(logits, bias, experts, weights, counts, ctypes.byref(d) if desc else None, T, E, k, dt, None)


@pytest.mark.parametrize("status,kw", [
    (BAD, dict(desc=False)), (BAD, dict(T=-1)), (BAD, dict(E=0, k=0)), (BAD, dict(k=0)), (BAD, dict(k=41)), (BAD, dict(dt=2)), (BAD, dict(score=2)),
    (BAD, dict(groups=0)), (BAD, dict(top_groups=0)), (BAD, dict(groups=4, top_groups=5)), (BAD, dict(group_best=0)), (BAD, dict(group_best=3)),
    (BAD, dict(renorm=2)), (BAD, dict(scale=float("nan"))), (BAD, dict(scale=float("inf"))), (BAD, dict(logits=None)), (BAD, dict(experts=None)),
    (BAD, dict(weights=None)), (BAD, dict(weights=at(2))), (BAD, dict(experts=at(0))), (BAD, dict(counts=at(1))),
    (SHAPE, dict(E=513)), (SHAPE, dict(k=33)), (SHAPE, dict(groups=33, E=66)), (SHAPE, dict(groups=3)),
    (ALIGN, dict(logits=at(0) + 1)), (ALIGN, dict(bias=at(1) + 2)), (ALIGN, dict(experts=at(2) + 2)), (ALIGN, dict(dt=1, logits=at(0) + 2))])
def test_forward_refusals(status, kw):
    assert fwd(**kw) == status


def test_backward_refusals():
    def bwd(logits=at(0), experts=at(1), dweights=at(2), dlogits=at(3), E=E, k=k, dt=0, **d):
        d = tp._RouteDesc(**{**dict(score=0, groups=1, top_groups=1, group_best=1, renorm=0, scale=1.0), **d})
        return L.tp_route_bwd(logits, experts, dweights, dlogits, ctypes.byref(d), T, E, k, dt, None)
    for kw in (dict(logits=None), dict(experts=None), dict(dweights=None), dict(dlogits=None), dict(dlogits=at(0)), dict(dlogits=at(2)),
               dict(k=41), dict(score=-1), dict(dt=5)):
        assert bwd(**kw) == BAD, kw
    assert bwd(E=1024) == SHAPE and bwd(dlogits=at(3) + 1) == ALIGN
