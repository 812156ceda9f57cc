"""Routed experts against their definition in 64 bits.

A value that is packed on the way is known within the error of the sum before
it; `packed` follows both ends of that range through the roundings (they are
monotone), so that the bounds of the outputs hold without a margin."""
import pytest
import torch

import fp8_ref as ref
from fp8_ref import D, assert_within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def packed(v, slack, via_bf16=False):
    """(value, how far off) of the operand of a matrix that is within `slack` of v."""
    lo, hi = v - slack, v + slack
    if via_bf16:
        lo, hi, v = (t.to(torch.float32).to(BF).to(D) for t in (lo - 2.0 ** -24 * lo.abs(), hi + 2.0 ** -24 * hi.abs(), v))
    R, C = v.shape
    B = -(-C // 128)
    pad = lambda t: torch.nn.functional.pad(t, (0, B * 128 - C)).view(R, B, 128)  # noqa: E731
    most = torch.maximum(lo.abs(), hi.abs())
    least = torch.where((lo < 0) & (hi > 0), torch.zeros_like(v), torch.minimum(lo.abs(), hi.abs()))
    k_lo, k_hi = ref.exponents(pad(least).amax(2)), ref.exponents(pad(most).amax(2))
    val, _ = ref.pack(v)
    s = ref.two_to(k_hi)[..., None]
    at = lambda t: (ref.round_e4m3((pad(t) / s).clamp(-448, 448)) * s).view(R, -1)[:, :C]  # noqa: E731
    off = torch.maximum((at(hi) - val).abs(), (at(lo) - val).abs())
    unsure = (k_lo != k_hi).repeat_interleave(128, 1)[:, :C]
    coarse = slack + 2 * ref.HALF_E4M3 * most + 2 * ref.two_to(k_hi).repeat_interleave(128, 1)[:, :C] * 2.0 ** -10
    return val, torch.where(unsure, coarse, off)


def product(a, ea, b, eb=None):
    """(a b^T, its error) where a and b are known within ea and eb, summed in fp32."""
    err = ref.sum_error(a.abs() + ea, b) + ea @ b.abs().t()
    if eb is not None:
        err = err + (a.abs() + ea) @ eb.t()
    return a @ b.t(), err


def operands(tp, ws, transposed):
    out = []
    for w in ws:
        B, M, N = w.shape
        op = tp.fp8_empty(*((N, M) if transposed else (M, N)), B)
        tp.tp_fp8_pack([w], None if transposed else [op], [op] if transposed else None, tiles=True)
        out.append(op)
    return out


class Problem:
    def __init__(self, tp, p, E, T, k, h, f, seed, closed=False, skew=0.0, same=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.p, self.E, self.T, self.k, self.h, self.f = p, E, T, k, h, f
        self.x, self.dy = rnd(T, h).to(BF), rnd(T, h).to(BF)
        self.x[:, ::37] *= 8
        score = rnd(T, E) + skew * torch.arange(E, device="cuda").flip(0)
        self.experts = score.topk(k, 1).indices.to(torch.int32).contiguous()
        self.weights = torch.rand((T, k), generator=g, device="cuda")
        if closed and T > 2:
            none = torch.rand((T, k), generator=g, device="cuda") < 0.2
            self.experts[none] = -1
            self.experts[1] = -1
            self.experts[0, 0] = E  # out of range: as closed
        if same:
            self.experts[:, :] = self.experts[:, :1]
        per = E // p
        self.w1 = [(rnd(per, h, f) * 0.7 / h ** 0.5).to(BF) for _ in range(p)]
        self.w2 = [rnd(per, f, h).to(BF) for _ in range(p)]
        self.o1, self.o2 = operands(tp, self.w1, True), operands(tp, self.w2, True)
        self.t1, self.t2 = operands(tp, self.w1, False), operands(tp, self.w2, False)

    def expert(self, e, ops, cols):
        """The values of expert e's operand."""
        per = self.E // self.p
        op = ops[e // per]
        return ref.values((op.q[e % per], op.e[e % per]), cols)

    def slots(self, e):
        return (self.experts == e).nonzero(as_tuple=True)


def forward_reference(P):
    """(y, slack, {expert: (H, slack, O, slack)})."""
    y = torch.zeros((P.T, P.h), dtype=D, device="cuda")
    err, size, per_expert = torch.zeros_like(y), torch.zeros_like(y), {}
    for e in range(P.E):
        t, j = P.slots(e)
        if not t.numel():
            continue
        hh, eh = product(ref.pack(P.x[t])[0], torch.zeros((), dtype=D, device="cuda").expand(t.numel(), P.h), P.expert(e, P.o1, P.h))
        z, ez = packed(ref.gelu(hh), 1.13 * eh + 1e-6 * (1 + hh.abs()))
        o, eo = product(z, ez, P.expert(e, P.o2, P.f))
        w = P.weights[t, j][:, None].to(D)
        y.index_add_(0, t, w * o)
        # the expert's output may be rounded to bf16, and the sums over the choices are in fp32
        err.index_add_(0, t, w * (eo + ref.HALF_BF16 * (o.abs() + eo)))
        size.index_add_(0, t, w * (o.abs() + eo))
        per_expert[e] = (hh, eh, o, eo)
    return y, err + (P.k + 2) * 2.0 ** -23 * size, per_expert


SHAPES = [  # p, E, T, k, h, f
    (1, 1, 1, 1, 8, 8), (1, 4, 1, 2, 128, 136), (2, 8, 3, 2, 264, 520), (4, 64, 1, 6, 1024, 256), (2, 64, 48, 6, 520, 264),
    (1, 16, 100, 3, 136, 392), (2, 4, 150, 1, 1032, 264), (4, 8, 300, 2, 392, 1032), (1, 2, 700, 2, 520, 136), (8, 32, 555, 4, 264, 264),
    (1, 3, 129, 3, 2056, 128)]


@pytest.mark.parametrize("closed,skew", [(False, 0.0), (True, 0.4)])
@pytest.mark.parametrize("p,E,T,k,h,f", SHAPES)
def test_forward(tp, p, E, T, k, h, f, closed, skew):
    P = Problem(tp, p, E, T, k, h, f, T + E + h, closed, skew)
    want, slack, _ = forward_reference(P)
    ws = tp.experts_workspace(p, E, T, k, h, f)
    ws[256:] = 0xFF  # what lies in it does not matter
    y, y2 = (torch.full((T, h), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    assert_within(y, want, slack, "y")
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y2, ws)
    assert torch.equal(y, y2), "the order of the sums is fixed"
    if closed and T > 2:
        assert bool((y[1] == 0).all())
    assert tp.tp_get_device_status(ws) == tp.TP_OK


@pytest.mark.parametrize("closed,skew", [(False, 0.0), (True, 0.4)])
@pytest.mark.parametrize("p,E,T,k,h,f", SHAPES)
def test_training_step(tp, p, E, T, k, h, f, closed, skew):
    P = Problem(tp, p, E, T, k, h, f, T + E + h + 1, closed, skew)
    ws = tp.experts_workspace(p, E, T, k, h, f, backward=True)
    ws[256:] = 0xFF
    saved = tp.experts_saved(E, T, k, h, f)
    saved.preact.fill_(float("nan"))
    saved.out.fill_(float("nan"))
    saved.plan.fill_(-1)
    nan = lambda *s: torch.full(s, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    y = nan(T, h)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws, saved=saved)
    want, slack, per_expert = forward_reference(P)
    assert_within(y, want, slack, "y")
    dx, dw = nan(T, h), nan(T, k)
    d1, d2 = [nan(E // p, h, f) for _ in range(p)], [nan(E // p, f, h) for _ in range(p)]
    tp.tp_experts_bwd_fp8(P.x, P.weights, P.dy, P.t1, P.t2, dx, dw, d1, d2, saved, ws)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    # the plan: tiles of 128 rows of one expert, slots in their order
    n, pairs, first = int(saved.plan[0]), int(saved.plan[1]), saved.plan[2:E + 3].tolist()
    row_of = torch.full((T * k,), -1, dtype=torch.int64)
    rows = 0
    for e in range(E):
        t, j = P.slots(e)
        assert first[e] == rows // 128
        row_of[(t * k + j).cpu()] = rows + torch.arange(t.numel())
        rows += -(-t.numel() // 128) * 128
    assert n == first[E] == rows // 128
    assert pairs == sum((b - a + 1) // 2 for a, b in zip(first, first[1:]))
    row_of = row_of.cuda()
    zero = torch.zeros((), dtype=D, device="cuda")
    gx, ex, sx = (torch.zeros((T, h), dtype=D, device="cuda") for _ in range(3))
    gw, ew = (torch.zeros((T, k), dtype=D, device="cuda") for _ in range(2))
    for e in range(E):
        a1, a2 = d1[e // (E // p)][e % (E // p)], d2[e // (E // p)][e % (E // p)]
        t, j = P.slots(e)
        if not t.numel():
            assert bool((a1 == 0).all()) and bool((a2 == 0).all())
            continue
        r = row_of[t * k + j]
        hh, out = saved.preact[r].to(D), saved.out[r].to(D)
        assert_within(saved.preact[r], per_expert[e][0], per_expert[e][1], "H")
        assert_within(saved.out[r], per_expert[e][2], per_expert[e][3], "O")
        gw[t, j] = (out * P.dy[t].to(D)).sum(1)
        ew[t, j] = (h + 8) * 2.0 ** -23 * (out * P.dy[t].to(D)).abs().sum(1)
        do = P.weights[t, j][:, None] * P.dy[t].float()
        g, eg = product(ref.pack(do)[0], zero.expand(t.numel(), h), P.expert(e, P.t2, h))
        s = ref.gelu_prime(hh)
        g, eg = g * s, eg * s.abs() + (g.abs() + eg) * 2e-6
        dh, edh = packed(g, eg, True)
        o, eo = product(dh, edh, P.expert(e, P.t1, f))
        gx.index_add_(0, t, o)
        ex.index_add_(0, t, eo + ref.HALF_BF16 * (o.abs() + eo))
        sx.index_add_(0, t, o.abs() + eo)
        dht, edht = packed(g.t().contiguous(), eg.t().contiguous(), True)
        want, slack = product(ref.pack(P.x[t].t())[0], zero.expand(h, t.numel()), dht, edht)
        assert_within(a1, want, slack, "dW1")
        zt, ezt = packed(ref.gelu(hh).t().contiguous(), 1e-6 * (1 + hh.abs()).t())
        want, slack = product(zt, ezt, ref.pack(do.t())[0])
        assert_within(a2, want, slack, "dW2")
    assert_within(dx, gx, ex + (k + 2) * 2.0 ** -23 * sx, "dx")
    assert_within(dw, gw, ew, "dweights")
    # each output alone
    alone = nan(T, h)
    tp.tp_experts_bwd_fp8(None, P.weights, P.dy, P.t1, P.t2, alone, None, None, None, saved, ws)
    assert torch.equal(alone, dx)
    a1, a2, aw = [nan(E // p, h, f) for _ in range(p)], [nan(E // p, f, h) for _ in range(p)], nan(T, k)
    tp.tp_experts_bwd_fp8(P.x, P.weights, P.dy, None, P.t2, None, None, a1, None, saved, ws)
    tp.tp_experts_bwd_fp8(None, P.weights, P.dy, None, None, None, None, None, a2, saved, ws)
    tp.tp_experts_bwd_fp8(None, P.weights, P.dy, None, P.t2, None, aw, None, None, saved, ws)
    assert all(torch.equal(a, b) for a, b in zip(a1 + a2 + [aw], d1 + d2 + [dw]))


def test_the_same_expert_twice(tp):
    """Both slots count, forward and backward."""
    P = Problem(tp, 1, 4, 20, 3, 136, 264, 5, same=True)
    ws, saved = tp.experts_workspace(1, 4, 20, 3, 136, 264, backward=True), tp.experts_saved(4, 20, 3, 136, 264)
    y, y1 = torch.empty_like(P.x), torch.empty_like(P.x)
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y, ws)
    want, slack, _ = forward_reference(P)
    assert_within(y, want, slack, "y")
    tp.tp_experts_fwd_fp8(P.x, P.experts, P.weights, P.o1, P.o2, y1, ws, saved=saved)
    assert_within(y1, want, slack, "y")
    dw = torch.empty((20, 3), dtype=BF, device="cuda")
    tp.tp_experts_bwd_fp8(None, P.weights, P.dy, None, P.t2, None, dw, None, None, saved, ws)
    assert torch.equal(dw[:, 0], dw[:, 1]) and torch.equal(dw[:, 0], dw[:, 2])


def test_no_token(tp):
    E, k, h, f = 4, 2, 64, 128
    P = Problem(tp, 2, E, 3, k, h, f, 1)
    ws, saved = tp.experts_workspace(2, E, 0, k, h, f, backward=True), tp.experts_saved(E, 0, k, h, f)
    none = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    tp.tp_experts_fwd_fp8(none(0, h), none(0, k, dtype=torch.int32), none(0, k, dtype=torch.float32), P.o1, P.o2, none(0, h), ws, saved=saved)
    d1, d2 = [none(2, h, f).fill_(1) for _ in range(2)], [none(2, f, h).fill_(1) for _ in range(2)]
    tp.tp_experts_bwd_fp8(none(0, h), none(0, k, dtype=torch.float32), none(0, h), P.t1, P.t2, none(0, h), none(0, k), d1, d2, saved, ws)
    assert all(bool((t == 0).all()) for t in d1 + d2)
    # every slot closed: nothing to add up
    ws, saved = tp.experts_workspace(2, E, 3, k, h, f, backward=True), tp.experts_saved(E, 3, k, h, f)
    shut, y, dx, dw = torch.full((3, k), -1, dtype=torch.int32, device="cuda"), none(3, h), none(3, h), none(3, k)
    for s in (None, saved):
        y.fill_(7)
        tp.tp_experts_fwd_fp8(P.x, shut, P.weights, P.o1, P.o2, y, ws, saved=s)
        assert bool((y == 0).all())
    [t.fill_(1) for t in d1 + d2]
    tp.tp_experts_bwd_fp8(P.x, P.weights, P.dy, P.t1, P.t2, dx, dw, d1, d2, saved, ws)
    assert all(bool((t == 0).all()) for t in [dx, dw] + d1 + d2)


def test_gradient_against_differences(tp):
    """Values that no rounding touches: one-hot tokens, even whole weights between 8 and 14 (whose GeLU is themselves), and
    second weights with one power of two a row.  A difference of the loss is then its gradient exactly."""
    E, T, k, h, f = 4, 8, 2, 16, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    w1 = (8 + 2 * torch.randint(0, 4, (E, h, f), generator=g, device="cuda")).to(BF)
    w2 = torch.zeros((E, f, h), device="cuda", dtype=BF)
    hot = torch.arange(f, device="cuda")
    w2[:, hot, hot % h] = torch.pow(2.0, torch.randint(0, 3, (E, f), generator=g, device="cuda")).to(BF)
    o1, o2, t1, t2 = operands(tp, [w1], True), operands(tp, [w2], True), operands(tp, [w1], False), operands(tp, [w2], False)
    at = torch.randint(0, h, (T,), generator=g, device="cuda")
    x = torch.zeros((T, h), device="cuda", dtype=BF)
    x[torch.arange(T), at] = 1
    dy = torch.randint(-1, 2, (T, h), generator=g, device="cuda").to(BF)
    experts = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32).contiguous()
    weights = torch.full((T, k), 0.5, device="cuda")
    ws, saved = tp.experts_workspace(1, E, T, k, h, f, backward=True), tp.experts_saved(E, T, k, h, f)

    def loss(x, w1=o1, w2=o2, weights=weights, saved=None):
        y = torch.empty_like(x)
        tp.tp_experts_fwd_fp8(x, experts, weights, w1, w2, y, ws, saved=saved)
        return (y.to(D) * dy.to(D)).sum(1)
    base = loss(x, saved=saved)
    dx, dw, d1, d2 = torch.empty_like(x), torch.empty((T, k), device="cuda", dtype=BF), [torch.empty_like(w1)], [torch.empty_like(w2)]
    tp.tp_experts_bwd_fp8(x, weights, dy, t1, t2, dx, dw, d1, d2, saved, ws)
    assert torch.equal(loss(2 * x) - base, dx[torch.arange(T), at].to(D))
    more = weights.clone()
    more[:, 1] = 1.5
    assert torch.equal(loss(x, weights=more) - base, dw[:, 1].to(D))
    for e in range(E):
        b = w2.clone()
        b[e] *= 2  # along w2[e] itself
        assert float((loss(x, w2=operands(tp, [b], True)) - base).sum()) == float((d2[0][e].to(D) * w2[e].to(D)).sum())
        a = w1.clone()
        a[e] += 2 * (a[e] < 14)
        assert float((loss(x, w1=operands(tp, [a], True)) - base).sum()) == float((d1[0][e].to(D) * (a[e] - w1[e]).to(D)).sum())


def test_captured_and_replayed(tp):
    """A step captured once and replayed on other tokens and another routing, which only the device sees."""
    p, E, T, k, h, f = 2, 8, 200, 2, 264, 136
    P, Q = Problem(tp, p, E, T, k, h, f, 1), Problem(tp, p, E, T, k, h, f, 2, closed=True, skew=0.8)
    ws, saved = tp.experts_workspace(p, E, T, k, h, f, backward=True), tp.experts_saved(E, T, k, h, f)
    x, e, w, dy = P.x.clone(), P.experts.clone(), P.weights.clone(), P.dy.clone()
    out = [torch.empty_like(x), torch.empty_like(x), torch.empty((T, k), device="cuda", dtype=BF)]
    d1, d2 = [torch.empty_like(t) for t in P.w1], [torch.empty_like(t) for t in P.w2]

    def step():
        tp.tp_experts_fwd_fp8(x, e, w, P.o1, P.o2, out[0], ws, saved=saved)
        tp.tp_experts_bwd_fp8(x, w, dy, P.t1, P.t2, out[1], out[2], d1, d2, saved, ws)
        return [t.clone() for t in out + d1 + d2]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_experts_fwd_fp8(x, e, w, P.o1, P.o2, out[0], ws, saved=saved)
        tp.tp_experts_bwd_fp8(x, w, dy, P.t1, P.t2, out[1], out[2], d1, d2, saved, ws)
    for R in (Q, P):
        for a, b in ((x, R.x), (e, R.experts), (w, R.weights), (dy, R.dy)):
            a.copy_(b)
        want = step()
        for t in out + d1 + d2:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out + d1 + d2, want))
