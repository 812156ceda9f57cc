"""Routed experts where a tile of rows, a pair of tiles or the number of slots
ends: counts around multiples of 16, 32, 128 and 256, closed experts between
them, many experts, tokens that are not finite, calls beside each other."""
import math

import pytest
import torch

import fp8_ref as ref
from fp8_ref import D, assert_within
from test_gpu_experts import BF, Problem, forward_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def with_counts(tp, p, counts, h, f, seed):
    """A problem of one choice a token in which expert e has counts[e] tokens, in a mixed order."""
    E, T = len(counts), sum(counts)
    P = Problem(tp, p, E, T, 1, h, f, seed)
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    P.experts = e[torch.randperm(T, generator=torch.Generator().manual_seed(seed))][:, None].to(torch.int32).cuda().contiguous()
    return P


COUNTS = [
    [1, 0, 15, 16, 17, 3, 0, 1],                                 # tiles of 16 rows
    [31, 32, 33, 1, 0, 16, 17, 2],                               # 32
    [63, 64, 65, 1, 15, 48, 49, 0],                              # 64
    [127, 128, 129, 1, 0, 16, 113, 255],                         # 128, one by one
    [256, 257, 1, 128, 129, 240, 241, 224],                      # pairs
    [225, 0, 512, 513, 96, 97, 385, 32],
    [1000, 0, 0, 0, 0, 0, 0, 7],
]


@pytest.mark.parametrize("p,h,f", [(2, 264, 392), (1, 136, 520), (4, 128, 72)])
@pytest.mark.parametrize("counts", COUNTS)
def test_counts_at_the_edges(tp, counts, p, h, f):
    P = with_counts(tp, p, counts, h, f, sum(counts) + h)
    E, T = P.E, P.T
    want, slack, per_expert = forward_reference(P)
    nan = lambda *s: torch.full(s, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    ws = tp.experts_workspace(p, E, T, 1, h, f, backward=True)
    ws[256:] = 0xFF
    y = nan(T, h)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    assert_within(y, want, slack, "y")
    # a training step's tiles, and gradients that rows without a token have no part in
    saved = tp.experts_saved(E, T, 1, h, f)
    saved.preact.fill_(float("nan"))
    saved.out.fill_(float("nan"))
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws, saved=saved)
    assert_within(y, want, slack, "y, trained")
    ws[256:] = 0xFF
    dx, dw = nan(T, h), nan(T, 1)
    d1, d2 = [nan(E // p, h, f) for _ in range(p)], [nan(E // p, f, h) for _ in range(p)]
    tp.tp_experts_bwd_fp8(P.x, P.weights, P.dy, P.t1, P.t2, dx, dw, d1, d2, saved, ws)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    assert all(bool(torch.isfinite(t).all()) for t in [dx, dw] + d1 + d2)
    for e in range(E):
        a2 = d2[e // (E // p)][e % (E // p)]
        t, _ = P.slots(e)
        if not t.numel():
            assert bool((a2 == 0).all())
            continue
        # dW2 = GeLU(H)^T dO: each factor rounded to e4m3 once, by blocks of 128 rows (a block's smallest step is
        # 2^-9 of its power of two, at most 2^-17 of twice its largest value), H within the error of the forward pass
        # and its rounding to bf16, products of at most 256 in magnitude summed in fp32
        hh, eh = per_expert[e][0], per_expert[e][1]
        z = ref.gelu(hh)
        do = P.weights[t, 0][:, None].to(D) * P.dy[t].to(D)
        before = 1.13 * (eh + ref.HALF_BF16 * hh.abs()) + 1e-6 * (1 + hh.abs())
        ez = (1 + ref.HALF_E4M3) * before + ref.HALF_E4M3 * z.abs() + 2.0 ** -16 * (z.abs() + before).amax(0)
        ed = (ref.HALF_E4M3 + 2.0 ** -23) * do.abs() + 2.0 ** -16 * do.abs().amax(0)
        err = ez.t() @ (do.abs() + ed) + z.abs().t() @ ed + ref.sum_error(z.t().abs() + ez.t(), do.t().abs() + ed.t())
        assert_within(a2, z.t() @ do, err * 1.01, "dW2")


@pytest.mark.parametrize("p,E,T,k,h,f", [
    (1, 512, 128, 4, 64, 72), (1, 512, 171, 3, 64, 72),          # 512 and 513 slots: packed with their dispatch, and after it
    (4, 512, 16, 32, 72, 64), (1, 64, 1, 32, 520, 136), (2, 6, 1024, 6, 136, 136), (1, 1, 512, 1, 1160, 8)])
def test_many_experts_and_choices(tp, p, E, T, k, h, f):
    P = Problem(tp, p, E, T, k, h, f, E + T + k, closed=T > 200)
    want, slack, _ = forward_reference(P)
    ws = tp.experts_workspace(p, E, T, k, h, f)
    ws[256:] = 0xFF
    # slots that begin at any element
    flat = torch.empty(T * k + 1, dtype=torch.int32, device="cuda")
    flat[1:] = P.experts.flatten()
    y = torch.full((T, h), float("nan"), dtype=BF, device="cuda")
    tp.tp_experts_fwd_fp8(P.x, flat[1:].view(T, k), P.weights, P.o1, P.o2, y, ws)
    assert_within(y, want, slack, "y")


@pytest.mark.parametrize("T,E,k", [(3, 4, 2), (40, 4, 2), (700, 4, 1), (700, 16, 3)])
def test_tokens_that_are_not_finite_stay_alone(tp, T, E, k):
    p, h, f = 2, 264, 392
    P = Problem(tp, p, E, T, k, h, f, T)
    ws = tp.experts_workspace(p, E, T, k, h, f, backward=True)
    y, y1 = torch.empty_like(P.x), torch.empty_like(P.x)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    P.x[1, 5] = math.nan
    P.x[2, 0] = -math.inf
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y1, ws)
    assert bool(torch.isnan(y1[1:3]).all())
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[1:3] = False
    assert torch.equal(y1[rest], y[rest])
    # gradients: the tokens that are not finite reach their experts' weights only
    saved = tp.experts_saved(E, T, k, h, f)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y1, ws, saved=saved)
    assert bool(torch.isfinite(y1[rest]).all()) and bool(torch.isnan(y1[1:3]).all())
    dx, dw = torch.empty_like(P.x), torch.empty((T, k), dtype=BF, device="cuda")
    d1, d2 = [torch.empty_like(t) for t in P.w1], [torch.empty_like(t) for t in P.w2]
    tp.tp_experts_bwd_fp8(P.x, P.weights, P.dy, P.t1, P.t2, dx, dw, d1, d2, saved, ws)
    assert bool(torch.isfinite(dx[rest]).all()) and bool(torch.isfinite(dw[rest]).all())
    hit = set(P.experts[1:3].flatten().tolist())
    for e in range(E):
        if e not in hit:
            assert bool(torch.isfinite(d1[e // (E // p)][e % (E // p)]).all()) and bool(torch.isfinite(d2[e // (E // p)][e % (E // p)]).all())


def test_calls_beside_each_other(tp):
    """Two streams with a workspace each, and two graphs of them replayed at once."""
    sizes = [(2, 8, 900, 2, 264, 392), (4, 64, 40, 6, 520, 264)]
    Ps = [Problem(tp, *s, 7) for s in sizes]
    wss = [tp.experts_workspace(*s) for s in sizes]
    ys, want = [torch.empty_like(P.x) for P in Ps], []
    for P, ws, y in zip(Ps, wss, ys):
        tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
        want.append(y.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ps]
    for _ in range(20):
        for P, ws, y, s in zip(Ps, wss, ys, streams):
            with torch.cuda.stream(s):
                y.fill_(9)
                tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
    graphs = []
    for P, ws, y in zip(Ps, wss, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
        graphs.append(g)
        y.fill_(9)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_rows_behind_the_backward_limit_are_refused(tp):
    """More rows than the backward call packs: refused by the forward call that saves for it, before a launch."""
    E, T, k, h, f = 1, 65536 * 128 // 32, 32, 8, 8
    P = Problem(tp, 1, 1, 2, 1, h, f, 1)
    meta = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    ws = torch.zeros(tp.tp_experts_workspace_size(1, E, T, k, h, f, 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(tp.TPError):
        tp.tp_experts_fwd_fp8(meta(T, h), meta(T, k, dtype=torch.int32).fill_(-1), meta(T, k, dtype=torch.float32), P.o1, P.o2, meta(T, h), ws,
                              saved=tp.experts_saved(E, T, k, h, f))


@pytest.mark.parametrize("p,E,T,k,h,f", [(1, 4, 20, 2, 1160, 264), (2, 4, 900, 1, 1160, 520)])
def test_a_wait_that_runs_out_is_reported(tp, p, E, T, k, h, f):
    """Single CTAs and pairs: a stage that is never handed over ends the call with a status, and the next call is right."""
    P = Problem(tp, p, E, T, k, h, f, 3)
    ws, y = tp.experts_workspace(p, E, T, k, h, f), torch.empty_like(P.x)
    try:
        assert tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 50) == tp.TP_OK and tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, 2) == tp.TP_OK
        tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
        assert tp.tp_get_device_status(ws) == tp.TP_ERR_DEVICE_TIMEOUT
    finally:
        tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 0)
        tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, -1)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    want, slack, _ = forward_reference(P)
    assert_within(y, want, slack, "y")
