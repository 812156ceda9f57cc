"""Routing to experts against its definition in 64 bits: the choice exactly,
weights and gradients within the roundings of fp32."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, D = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def route(logits, k, bias, sigmoid, groups, tops, best, renorm, scale):
    """(experts, weights, scores, gradient function) of the definition, row by row in 64 bits, on the CPU."""
    T, E = logits.shape
    l = logits.to(D).clamp(max=float(torch.finfo(F32).max))
    open_ = l > -math.inf
    if sigmoid:
        s = torch.where(open_, torch.sigmoid(l), torch.zeros_like(l))
    else:
        top = torch.where(open_, l, torch.full_like(l, -math.inf)).amax(1, keepdim=True).clamp(min=-1e300)
        e = torch.where(open_, torch.exp(l - top), torch.zeros_like(l))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    experts, size = torch.full((T, k), -1, dtype=torch.int32), E // groups
    for t in range(T):
        v = [(float(s[t, e]) + (float(bias[e]) if bias is not None else 0.0)) if open_[t, e] else None for e in range(E)]
        if bias is None:  # both scores grow with the logit
            order = {e: float(l[t, e]) for e in range(E) if open_[t, e]}
        else:
            order = {e: v[e] for e in range(E) if open_[t, e]}
        if groups > 1:
            score = []
            for g in range(groups):
                mine = sorted((order[e] if best == 1 else v[e] for e in range(g * size, (g + 1) * size) if open_[t, e]), reverse=True)
                if mine:
                    score.append((-math.fsum(mine[:best]), g))
            kept = {g for _, g in sorted(score)[:tops]}
            order = {e: x for e, x in order.items() if e // size in kept}
        for j, e in enumerate(sorted(order, key=lambda e: (-order[e], e))[:k]):
            experts[t, j] = e
    there = experts >= 0
    w = torch.where(there, s.gather(1, experts.clamp(min=0).long()), torch.zeros((), dtype=D))
    n = w.sum(1, keepdim=True).clamp(min=float(torch.finfo(F32).tiny)) if renorm else torch.ones((T, 1), dtype=D)
    return experts, scale * w / n, s


def gradient(logits, experts, dweights, sigmoid, renorm, scale):
    """The gradient by automatic differentiation of the definition in 64 bits, with the choice held."""
    l = logits.to(D).clamp(max=float(torch.finfo(F32).max)).clone().requires_grad_()
    open_ = logits > -math.inf
    if sigmoid:
        s = torch.where(open_, torch.sigmoid(l), torch.zeros_like(l))
    else:
        some = open_.any(1, keepdim=True)
        s = torch.softmax(torch.where(open_ | ~some, torch.where(open_, l, torch.zeros_like(l)), torch.full_like(l, -math.inf)), 1)
        s = torch.where(open_, s, torch.zeros_like(s))
    there = (experts >= 0) & (experts < logits.shape[1])
    w = torch.where(there, s.gather(1, torch.where(there, experts, torch.zeros_like(experts)).long()), torch.zeros((), dtype=D))
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=float(torch.finfo(F32).tiny))
    (scale * w * dweights.to(D)).sum().backward()
    return torch.where(open_, l.grad, torch.zeros_like(l))


CASES = [  # T, E, k, bias, sigmoid, groups, tops, best, renorm, scale, f32
    (1, 1, 1, False, False, 1, 1, 1, False, 1.0, False),
    (1, 64, 6, False, False, 1, 1, 1, False, 1.0, False),
    (3, 7, 7, True, True, 1, 1, 1, True, 2.5, True),
    (130, 60, 4, False, False, 1, 1, 1, True, 1.0, True),
    (257, 64, 8, True, True, 8, 3, 2, True, 2.5, False),
    (64, 256, 8, True, True, 8, 4, 2, True, 2.5, False),
    (64, 256, 32, True, False, 32, 5, 1, False, 1.0, True),
    (40, 96, 5, False, True, 3, 2, 2, False, 1.0, False),
    (40, 96, 5, False, True, 3, 2, 1, True, 1.0, False),
    (33, 130, 3, False, False, 2, 1, 2, True, 1.0, True),
    (20, 512, 16, True, False, 1, 1, 1, True, 1.0, False),
    (20, 500, 10, False, True, 4, 1, 2, True, 1.0, True),
]


def inputs(T, E, bias, f32, seed):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * 1.5).to(F32 if f32 else BF)
    if T > 8:
        l[torch.rand(T, E, generator=g) < 0.05] = -math.inf
        l[2] = -math.inf
        l[3, 1:] = -math.inf
        l[4] = float("nan")
        l[5, 0], l[6, -1], l[7, E // 2] = math.inf, float("nan"), -0.0
        l[8] = 0.0
        l[8, ::2] = -0.0
    return l, torch.randn(E, generator=g) * 0.1 if bias else None


@pytest.mark.parametrize("T,E,k,bias,sigmoid,groups,tops,best,renorm,scale,f32", CASES)
def test_forward_and_backward(tp, T, E, k, bias, sigmoid, groups, tops, best, renorm, scale, f32):
    l, b = inputs(T, E, bias, f32, T + E + k)
    experts, weights, s = route(l, k, b, sigmoid, groups, tops, best, renorm, scale)
    how = dict(score=tp.TP_ROUTE_SIGMOID if sigmoid else tp.TP_ROUTE_SOFTMAX, renorm=renorm, scale=scale)
    ld = l.cuda()
    e = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    n = torch.full((E,), 77, dtype=torch.int32, device="cuda")
    tp.tp_route_fwd(ld, e, w, counts=n, bias=b.cuda() if bias else None, groups=groups, top_groups=tops, group_best=best, **how)
    assert torch.equal(e.cpu(), experts)
    # exp, sum, division and two products: fewer than 64 roundings of 2^-24 (E / 32 + 5 of them in the sum)
    assert bool(((w.cpu().to(D) - weights).abs() <= 64 * 2.0 ** -24 * weights.abs()).all())
    assert torch.equal(n.cpu(), torch.bincount(experts.flatten().long() + 1, minlength=E + 1)[1:].to(torch.int32))
    g = torch.Generator().manual_seed(E)
    dw = torch.randn(T, k, generator=g)
    d = torch.full((T, E), float("nan"), dtype=l.dtype, device="cuda")
    tp.tp_route_bwd(ld, e, dw.cuda(), d, **how)
    want = gradient(l, experts, dw, sigmoid, renorm, scale)
    got = d.cpu().to(D)
    # the largest term that is added up in a row: scale * |dw| (twice over the sum of the chosen scores with renorm)
    big = scale * dw.abs().to(D).sum(1, keepdim=True)
    if renorm:
        big = 2 * big / (s.gather(1, experts.clamp(min=0).long()) * (experts >= 0)).sum(1, keepdim=True).clamp(min=1e-30)
    slack = 128 * 2.0 ** -24 * s * big
    half = 2.0 ** -24 if f32 else 2.0 ** -8
    assert bool(torch.isfinite(got).all())
    assert bool(((got - want).abs() <= half * want.abs() + slack + 1e-38).all())
    assert bool((got[~(l > -math.inf)] == 0).all())


def test_gradient_against_differences(tp):
    T, E, k = 4, 12, 3
    g = torch.Generator().manual_seed(3)
    l, dw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    for sigmoid in (False, True):
        for renorm in (False, True):
            how = dict(score=int(sigmoid), renorm=renorm, scale=1.5)
            e, w, d = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty((T, E), device="cuda")
            tp.tp_route_fwd(l.cuda(), e, w, **how)
            tp.tp_route_bwd(l.cuda(), e, dw.cuda(), d, **how)
            h = 2.0 ** -6
            for i in range(E):
                both = []
                for step in (h, -h):
                    m = l.clone()
                    m[:, i] += step
                    x, _, s = route(m, k, None, sigmoid, 1, 1, 1, renorm, 1.5)
                    y = s.gather(1, e.cpu().long())
                    both.append((1.5 * (y / y.sum(1, keepdim=True) if renorm else y) * dw).sum(1))
                # central differences: h^2 / 6 of a third derivative, here below 10
                assert bool((((both[0] - both[1]) / (2 * h) - d.cpu()[:, i].to(D)).abs() <= 10 * h * h).all())


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,tops,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_scores_that_fp32_does_not_tell_apart(tp, sigmoid, groups, tops, best):
    """Logits some 1e-7 apart with a bias: fp32 scores coincide or swap, the choice is that of 64 bits."""
    T, E, k = 300, 256, 8
    g = torch.Generator().manual_seed(11)
    l = torch.randn(T, E, generator=g) * 1e-6
    b = torch.zeros(E)
    b[::3] = 2.0 ** -20
    b[1::7] = 1e-7
    experts, _, _ = route(l, k, b, sigmoid, groups, tops, best, False, 1.0)
    e, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    tp.tp_route_fwd(l.cuda(), e, w, bias=b.cuda(), score=int(sigmoid), groups=groups, top_groups=tops, group_best=best)
    assert torch.equal(e.cpu(), experts)


def test_equal_scores_go_to_the_lower_expert(tp):
    T, E, k = 50, 128, 6
    g = torch.Generator().manual_seed(12)
    l = torch.randint(-2, 3, (T, E), generator=g).to(BF)
    for bias in (None, torch.zeros(E), torch.full((E,), -0.25)):
        for sigmoid in (False, True):
            experts, _, _ = route(l, k, bias, sigmoid, 1, 1, 1, False, 1.0)
            e, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
            tp.tp_route_fwd(l.cuda(), e, w, bias=bias.cuda() if bias is not None else None, score=int(sigmoid))
            assert torch.equal(e.cpu(), experts)


def test_rows_do_not_see_each_other(tp):
    """A row alone, among others, with the last of many, and no row at all."""
    T, E, k = 10007, 64, 4
    l = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    b = torch.randn(E, device="cuda") * 0.1

    def call(x):
        n = torch.empty(E, dtype=torch.int32, device="cuda")
        e, w = torch.empty((x.shape[0], k), dtype=torch.int32, device="cuda"), torch.empty((x.shape[0], k), device="cuda")
        tp.tp_route_fwd(x, e, w, counts=n, bias=b, score=tp.TP_ROUTE_SIGMOID, renorm=True)
        return e, w, n
    e, w, n = call(l)
    assert int(n.sum()) == T * k
    assert torch.equal(n, torch.bincount(e.flatten(), minlength=E).to(torch.int32))
    for t in (0, 5000, T - 1):
        e1, w1, _ = call(l[t:t + 1].clone())
        assert torch.equal(e1[0], e[t]) and torch.equal(w1[0], w[t])
    assert int(call(l[:0].clone())[2].abs().sum()) == 0
    # an odd row of a larger tensor: logits at any element's alignment
    flat = torch.randn(7 * 33 + 1, device="cuda").to(BF)
    x = flat[1:].view(7, 33)
    e1, w1 = torch.empty((7, k), dtype=torch.int32, device="cuda"), torch.empty((7, k), device="cuda")
    tp.tp_route_fwd(x, e1, w1)
    e2, w2 = torch.empty_like(e1), torch.empty_like(w1)
    tp.tp_route_fwd(x.clone(), e2, w2)
    assert torch.equal(e1, e2) and torch.equal(w1, w2)


def test_backward_passes_over_numbers_out_of_range(tp):
    T, E, k = 5, 40, 4
    l = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    e = torch.tensor([[0, 39, -1, 40]] * T, dtype=torch.int32, device="cuda")
    dw = torch.randn((T, k), device="cuda")
    d = torch.empty_like(l)
    tp.tp_route_bwd(l, e, dw, d, renorm=True)
    want = gradient(l.cpu(), e.cpu(), dw.cpu(), False, True, 1.0)
    assert bool(((d.cpu().to(D) - want).abs() <= 1e-5 * (1 + want.abs())).all())


def test_captured_and_replayed(tp):
    T, E, k = 600, 64, 4
    xs = [torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in range(3)]
    x, n = xs[0].clone(), torch.empty(E, dtype=torch.int32, device="cuda")
    e, w, d = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty_like(x)

    def call():
        tp.tp_route_fwd(x, e, w, counts=n, renorm=True)
        tp.tp_route_bwd(x, e, w, d, renorm=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for y in xs[::-1]:
        x.copy_(y)
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (e, w, n, d)]
        for t in (e, w, n, d):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((e, w, n, d), want))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_of_weights_that_add_up_to_one(tp, sigmoid):
    T, E, k = 64, 40, 4
    g = torch.Generator().manual_seed(9)
    l, dw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    how = dict(score=int(sigmoid), renorm=True)

    def call(l, k, bias=None):
        T, E = l.shape
        e, w, d = (torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"),
                   torch.full((T, E), float("nan"), device="cuda"))
        tp.tp_route_fwd(l.cuda(), e, w, bias=bias, **how)
        tp.tp_route_bwd(l.cuda(), e, dw[:T, :k].contiguous().cuda(), d, **how)
        return e, w, d

    # a single choice: its weight is the scale, whatever the logits
    assert bool((call(l, 1)[2] == 0).all())
    alone = torch.full_like(l, -math.inf)
    alone[:, 7] = l[:, 7]
    assert bool((call(alone, k)[2] == 0).all())
    # one score far above (softmax), or all others far below: the small differences keep their digits
    l[:, 3] = 12.0
    l[:, :3] -= 9.0
    l[:, 4:] -= 9.0
    e, w, d = call(l, k)
    want = gradient(l, e.cpu(), dw, sigmoid, True, 1.0)
    share, v = route(l, k, None, sigmoid, 1, 1, 1, True, 1.0)[1], dw.to(D)
    # d_i = w_i c_i sum_j w_j (v_i - v_j), c_i <= 1: fewer than 64 roundings of each weight and of c_i, one or two of the rest
    size = share * (share[:, None, :] * (v[:, :, None] - v[:, None, :]).abs()).sum(2)
    slack = torch.zeros(T, E, dtype=D).scatter_(1, e.cpu().long(), 160 * 2.0 ** -24 * size)
    # (the definition itself leaves 2^-50 of the terms where the sum is 0)
    assert bool(((d.cpu().to(D) - want).abs() <= slack + 2.0 ** -50).all())
    # scores that leave the range of fp32, chosen for their bias
    low = torch.full((4, E), -120.0)
    low[:, 0] = 100.0
    bias = torch.zeros(E, device="cuda")
    bias[1:] = 10.0
    e, w, d = call(low, k, bias)
    assert bool((e > 0).all()) and bool(torch.isfinite(w).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,f32", [(40, True), (37, False), (256, False)])
def test_backward_adds_up_a_number_that_comes_twice(tp, sigmoid, renorm, E, f32):
    T, k = 9, 5
    g = torch.Generator().manual_seed(E)
    l, dw = torch.randn(T, E, generator=g).to(F32 if f32 else BF), torch.randn(T, k, generator=g)
    e = torch.tensor([[3, 0, 3, -1, 3], [1, 1, 2, 2, E]] + [[0, E - 1, 5, E - 1, 7]] * (T - 2), dtype=torch.int32)
    flat = torch.full((T * E + 1,), float("nan"), dtype=l.dtype, device="cuda")
    d = flat[1:].view(T, E)  # rows that begin at any element
    tp.tp_route_bwd(l.cuda(), e.cuda(), dw.cuda(), d, score=int(sigmoid), renorm=renorm)
    want = gradient(l, e, dw, sigmoid, renorm, 1.0)
    # at most a dozen terms below 2 |dw|, each within 64 roundings of 2^-24, and the result's own
    slack = 12 * 2 * float(dw.abs().max()) * 64 * 2.0 ** -24
    assert bool(((d.cpu().to(D) - want).abs() <= (2.0 ** -24 if f32 else 2.0 ** -8) * want.abs() + slack).all())
    assert bool(torch.isnan(flat[0]))
