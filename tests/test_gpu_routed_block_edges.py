"""The routed block with any number of experts, blocks on 8-bit operands where no
gradient is recorded, and their captured training steps."""
import pytest
import torch

from test_gpu_routed_block import BF, D, GRAD, OUT, ROUTING, blk, gen, leaf, norm, off, reference, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("routing", [ROUTING[0], dict(score="sigmoid", renorm=True, scale=2.5)])
@pytest.mark.parametrize("p,E,T,k,h,f", [(4, 60, 300, 4, 264, 136), (2, 4, 33, 2, 136, 264), (1, 1, 5, 1, 64, 128), (3, 9, 1, 3, 64, 72)])
def test_any_number_of_experts(blk, p, E, T, k, h, f, routing):  # noqa: F811
    """Numbers of experts that are not multiples of 8: trained, served, captured."""
    from gemm_reduce_fusion_gb300.autograd import column_parallel_linear, route
    g = gen(E + T)
    router, w1, w2 = rnd(g, h, E, scale=h ** -0.5), rnd(g, E, h, f, scale=h ** -0.5), rnd(g, E, f, h, scale=f ** -0.5)
    b = blk.RoutedMLPBlock(router, w1, w2, p, k, alpha=0.5, **routing)
    b.bias.copy_(0.05 * torch.randn(E, generator=g, device="cuda"))
    x0, n0, dy, dn = (rnd(g, T, h) for _ in range(4))
    x, n = x0.clone().requires_grad_(), n0.clone().requires_grad_()
    y, m = b(x, n)
    torch.autograd.backward([y, m], [dy, dn])
    assert b.router.grad.shape == (h, E)
    # the logits of a router with columns of zeros behind its own are those of its own
    wide = torch.zeros((h, E + 7), dtype=BF, device="cuda")[:, :(E + 7) // 8 * 8].contiguous()
    wide[:, :E] = router
    _, experts, counts = route(column_parallel_linear(n0, [wide])[0][:, :E], k, bias=b.bias, **routing)
    assert torch.equal(counts, b.counts) and int(counts.sum()) == T * k
    xr, nr, rr, r1, r2 = leaf(x0), leaf(n0), leaf(router), leaf(w1), leaf(w2)
    yr = xr + 0.5 * norm(reference(nr, rr, r1, r2, experts.long(), routing), 1.0)
    mr = norm(yr, 1.0)
    torch.autograd.backward([yr, mr], [dy.to(D), dn.to(D)])
    assert off(y, yr) < OUT and off(m, mr) < OUT
    assert off(x.grad, xr.grad) < GRAD and off(n.grad, nr.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w1]), r1.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w2]), r2.grad) < GRAD
    if T > 30:
        assert off(b.router.grad, rr.grad) < GRAD
    served, xs = b.serve(), x0.clone()
    ys, ms = served(xs, n0)
    assert off(ys, y.detach().to(D)) < 2.0 ** -7 and off(ms, m.detach().to(D)) < 2.0 ** -7
    graph, out = torch.cuda.CUDAGraph(), x0.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        yc, mc = served(out, n0)
    out.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yc, ys) and torch.equal(mc, ms)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_gradients_nothing_is_kept_for_them(blk, mode, monkeypatch):  # noqa: F811
    """Parameters that require gradients, in an evaluation pass: one orientation of the weights, no saved rows."""
    from gemm_reduce_fusion_gb300 import autograd as ag
    g = gen(1)
    p, E, T, k, h, f = 2, 8, 5, 2, 264, 392
    w1, w2 = [rnd(g, h, f, scale=h ** -0.5).requires_grad_() for _ in range(p)], [rnd(g, f, h, scale=f ** -0.5).requires_grad_() for _ in range(p)]
    e1, e2 = ([rnd(g, E // p, *s, scale=s[0] ** -0.5).requires_grad_() for _ in range(p)] for s in ((h, f), (f, h)))
    x = rnd(g, T, h)
    experts = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, k), generator=g, device="cuda")
    want = ag.parallel_mlp_fp8(x, w1, w2), ag.routed_experts(x, experts, weights, e1, e2)
    assert all(y.requires_grad for y in want)
    both, pack = [], ag.tp_fp8_pack
    monkeypatch.setattr(ag, "tp_fp8_pack", lambda x, q=None, qt=None, **kw: (both.append(q is not None and qt is not None), pack(x, q, qt, **kw)))
    monkeypatch.setattr(ag, "experts_saved", lambda *a, **kw: pytest.fail("memory for a backward pass"))
    with mode():
        y, z = ag.parallel_mlp_fp8(x, w1, w2), ag.routed_experts(x, experts, weights, e1, e2)
        assert not y.requires_grad and not z.requires_grad
        direct = torch.empty_like(x)
        ops = [ag._operands(list(w), False, True, tiles=True)[1] for w in (e1, e2)]
        ag.tp_experts_fwd_fp8(x, experts, weights, *ops, direct, ag._workspace(x.device, [], ag.tp_experts_workspace_size(p, E, T, k, h, f)))
    assert both and not any(both)
    assert torch.equal(y, want[0])
    assert torch.equal(z, direct)  # tiles by the tokens that there are
    assert off(z, want[1].to(D)) < 2.0 ** -7  # the experts' outputs in fp32 instead of bf16


@pytest.mark.parametrize("E", [None, 16, 60])
def test_a_captured_training_step_replays(blk, E):  # noqa: F811
    """Forward and backward in one graph, replayed on other tokens with another routing; None: the MLP block."""
    g = gen(2)
    p, T, h, f = 2, 700, 264, 528
    if E is None:
        b = blk.MLPBlock(rnd(g, h, f, scale=h ** -0.5), rnd(g, f, h, scale=f ** -0.5), p, fp8=True)
    else:
        b = blk.RoutedMLPBlock(rnd(g, h, E, scale=h ** -0.5), rnd(g, E, h, f, scale=h ** -0.5), rnd(g, E, f, h, scale=f ** -0.5), p, 2)
    xs, gy, gm = [rnd(g, T, h) for _ in range(3)], rnd(g, T, h), rnd(g, T, h)
    x = xs[0].clone().requires_grad_()

    def step():
        y, m = b(x, blk.pre_norm([x])[0])
        return [y, m, *torch.autograd.grad([y, m], [x, *b.parameters()], [gy, gm])]

    def put(t):
        with torch.no_grad():
            x.copy_(t)
    side, want = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in xs:
            put(t)
            want.append([r.clone() for r in step()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for i in (1, 0, 2):
        put(xs[i])
        for t in got:
            t.detach().fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, want[i]))
