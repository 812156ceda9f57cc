"""Routing where fp32 scores say nothing: large biases that cancel in a group's
sum, biases of the type's lowest value, scores far below one, choices that
leave next to nothing for the others.  The choice is compared with decimal
arithmetic of 120 digits."""
import decimal
import math

import pytest
import torch

from test_gpu_route import gradient, route

pytestmark = pytest.mark.gpu
BF, F32, D = torch.bfloat16, torch.float32, torch.float64
LOWEST = float(torch.finfo(F32).min)


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def choose(l, bias, k, sigmoid, groups, tops, best):
    """(experts, gap) of one row in decimals.  gap: the smallest difference that the choice turns on, in units of the larger
    of 1 and what was added up (2^20 at most), or without a bias of the values (inf: none but exact ties)."""
    with decimal.localcontext(decimal.Context(prec=120)):
        one, dec = decimal.Decimal(1), [decimal.Decimal(float(x)) if x > -math.inf else None for x in l.tolist()]
        top = max((x for x in dec if x is not None), default=None)
        if sigmoid:
            s = [None if x is None else one / (one + (-x).exp()) for x in dec]
        else:
            e = [None if x is None else (x - top).exp() for x in dec]
            total = sum((x for x in e if x is not None), decimal.Decimal(0))
            s = [None if x is None else x / total for x in e]
        b = [decimal.Decimal(0)] * len(dec) if bias is None else [decimal.Decimal(float(x)) for x in bias.tolist()]
        v = [None if x is None else x + y for x, y in zip(s, b)]
        size = len(dec) // groups
        gaps = []

        def gap(x, y, parts):
            if x != y:
                gaps.append((x - y) / (x if bias is None else max(one, *(min(abs(t), decimal.Decimal(2 ** 20)) for t in parts))))
        kept = set(range(groups))
        if groups > 1:
            sums = []
            for g in range(groups):
                mine = sorted((x for x in v[g * size:(g + 1) * size] if x is not None), reverse=True)[:best]
                if mine:
                    sums.append((-sum(mine), g, mine))
            sums.sort(key=lambda t: t[:2])
            if len(sums) > tops:
                gap(-sums[tops - 1][0], -sums[tops][0], sums[tops - 1][2] + sums[tops][2])
            kept = {g for _, g, _ in sums[:tops]}
        order = sorted((e for e in range(len(dec)) if v[e] is not None and e // size in kept), key=lambda e: (-v[e], e))
        if bias is not None:  # without one the logits tell them apart
            for x, y in zip(order[:k], order[1:]):
                gap(v[x], v[y], [v[x], v[y]])
        return order[:k] + [-1] * (k - len(order)), float(min(gaps, default=decimal.Decimal("inf")))


def check(tp, l, bias, k, sigmoid, groups, tops, best):
    rows = [choose(r, bias, k, sigmoid, groups, tops, best) for r in l]
    sure = torch.tensor([gap > 2.0 ** -40 for _, gap in rows])  # some times what is documented to be told apart
    assert int(sure.sum()) >= 0.97 * len(rows)
    want, l = torch.tensor([e for e, _ in rows], dtype=torch.int32)[sure], l[sure]
    e, w = torch.empty((l.shape[0], k), dtype=torch.int32, device="cuda"), torch.empty((l.shape[0], k), device="cuda")
    tp.tp_route_fwd(l.cuda(), e, w, bias=None if bias is None else bias.cuda(), score=int(sigmoid), groups=groups, top_groups=tops, group_best=best)
    assert torch.equal(e.cpu(), want)


def opposite(size, m, sigmoid, seed, T):
    """Eight groups with biases of +m and -m (a third expert is closed) whose two scores add up to nearly the same."""
    g = torch.Generator().manual_seed(seed)
    l, bias = torch.full((T, 8, size), -math.inf, dtype=D), torch.zeros(8, size)
    l[:, :, 0] = torch.rand(T, 8, generator=g, dtype=D) * 1.5 - 1
    l[:, :, 1] = -l[:, :, 0] if sigmoid else torch.log(2.5 - l[:, :, 0].exp())
    l[:, :, 1] += torch.randn(T, 8, generator=g, dtype=D) * (2e-6 if sigmoid else 1e-5)
    bias[:, 0], bias[:, 1] = m, -m
    bias[::2, :2] = bias[::2, :2].flip(1)
    return l.view(T, -1).to(F32), bias.view(-1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [2, 3])  # groups that end between lanes, and groups that do not
@pytest.mark.parametrize("m", [16.0, 64.0])
def test_sums_of_large_biases(tp, m, size, sigmoid):
    """Each value carries the rounding of a number of m, their sum is near 1: fp32 would take the wrong group."""
    check(tp, *opposite(size, m, sigmoid, 5, 2500), 4, sigmoid, 8, 4, 2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [2, 3])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("some", [False, True])
def test_biases_of_the_lowest_value(tp, some, best, size, sigmoid):
    """Experts put last by the lowest bias that there is: still open, and two of them do not add up to -infinity."""
    g = torch.Generator().manual_seed(6)
    l, bias = torch.randn(40, 4, size, generator=g), torch.full((4, size), LOWEST)
    if some:
        bias[2] = 0.25
    check(tp, l.view(40, -1), bias.view(-1), 2 * size, sigmoid, 4, 2, best)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [4, 5])
@pytest.mark.parametrize("low", [60.0, 90.0, 150.0, 2000.0])
def test_sums_of_scores_far_below_one(tp, low, size, sigmoid):
    """Without a bias, groups of scores below what fp32 holds are told apart."""
    g = torch.Generator().manual_seed(7)
    l = torch.randn(200, 8, size, generator=g) * 3 - low
    l[:100, 5, 1] = 1.0  # one group far above, or all of them down there
    l[::7, 3, 1:] = -math.inf  # a sum of one
    check(tp, l.view(200, -1), None, 6, sigmoid, 8, 3, 2)


@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_weights_below_the_normal_range(tp, renorm):
    T, E, k = 64, 8, 4
    l = -86 - 17 * torch.rand(T, E, generator=torch.Generator().manual_seed(8))
    experts, want, _ = route(l, k, None, True, 1, 1, 1, renorm, 1.0)
    e, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    tp.tp_route_fwd(l.cuda(), e, w, score=tp.TP_ROUTE_SIGMOID, renorm=renorm)
    assert torch.equal(e.cpu(), experts)
    # 64 roundings, and where numbers are that small steps of 2^-149 (of each of k scores, over a sum of 2^-126 or more)
    step = 2.0 ** -149 * (2 * k / 2.0 ** -126 if renorm else 2)
    assert bool(((w.cpu().to(D) - want).abs() <= 64 * 2.0 ** -24 * want + step).all())


@pytest.mark.parametrize("E,k,f32", [(64, 1, True), (64, 1, False), (60, 3, True), (200, 8, True), (512, 32, True)])
def test_softmax_gradient_of_a_score_near_one(tp, E, k, f32):
    """The largest score is 1 but for what its logit leads by: its gradient keeps its digits."""
    lead = torch.tensor([8.0, 10.0, 12.0, 14.0, 17.0, 20.0]).repeat_interleave(16)
    T = lead.numel()
    g = torch.Generator().manual_seed(E + k)
    l, dw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    l[torch.arange(T), torch.randint(0, E, (T,), generator=g)] = l.amax(1) + lead
    l = l.to(F32 if f32 else BF)
    e, w, d = (torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"),
               torch.full((T, E), float("nan"), dtype=l.dtype, device="cuda"))
    tp.tp_route_fwd(l.cuda(), e, w, scale=1.5)
    tp.tp_route_bwd(l.cuda(), e, dw.cuda(), d, scale=1.5)
    want = gradient(l, e.cpu(), dw, False, False, 1.5)
    s, v, at = torch.softmax(l.to(D), 1), 1.5 * dw.to(D), e.cpu().long()
    sc = s.gather(1, at)
    rest = s.clone().scatter_(1, at, 0.0).sum(1, keepdim=True)
    # s_i (v_i rest + sum_j s_j (v_i - v_j)) of the chosen, -s_i sum_j s_j v_j of the others.  A score is within 64 roundings
    # of 2^-24: up to 23 in its exponent's difference (of at most 26: half a step is 2^-20), exp, the sum, a division and a product.
    terms = s * (sc * v.abs()).sum(1, keepdim=True)
    terms.scatter_(1, at, sc * (v.abs() * rest + (sc[:, None, :] * (v[:, :, None] - v[:, None, :]).abs()).sum(2)))
    slack = 160 * 2.0 ** -24 * terms + 2.0 ** -50 * v.abs().sum(1, keepdim=True)  # (the second: the definition's own in 64 bits)
    assert bool(((d.cpu().to(D) - want).abs() <= (2.0 ** -24 if f32 else 2.0 ** -8) * want.abs() + slack).all())
