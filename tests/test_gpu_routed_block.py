"""Blocks on 8-bit operands as they stand in a model: the MLP block and the
routed block, trained and served, against 64-bit arithmetic on the same values.

A value in e4m3 is off by at most 2^-4 of itself, 2^-4 / sqrt(3) = 3.6 % in the
mean square; a product has two such factors, 5.1 %, and in a sum of many
products with errors of either sign the 2-norm keeps that.  An output lies
behind two such sums (7.2 %), a gradient behind up to four (10.2 %) and one
GeLU' of a value that is itself off by the first sum's error: at a slope of at
most 0.8 of |GeLU''| that adds at most 5.1 % x 0.8 (11 %)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64
OUT, GRAD = 0.072, 0.11


@pytest.fixture(scope="module")
def blk():
    import gemm_reduce_fusion_gb300.block as blk
    return blk


def off(got, want):
    return float((got.detach().to(D) - want.detach()).norm() / want.detach().norm())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def norm(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w


def leaf(t):
    return t.detach().to(D).requires_grad_()


@pytest.mark.parametrize("p,M,h,f", [(1, 1, 64, 128), (2, 192, 264, 528), (4, 700, 520, 1056)])
def test_the_mlp_block_trains_on_8_bit_operands(blk, p, M, h, f):
    g = gen(M)
    w1, w2 = rnd(g, h, f, scale=h ** -0.5), rnd(g, f, h, scale=f ** -0.5)
    x0, n0, dy, dn = (rnd(g, M, h) for _ in range(4))
    b = blk.MLPBlock(w1, w2, p, alpha=0.5, fp8=True)
    x, n = x0.clone().requires_grad_(), n0.clone().requires_grad_()
    y, m = b(x, n)
    torch.autograd.backward([y, m], [dy, dn])
    xr, nr, r1, r2 = leaf(x0), leaf(n0), leaf(w1), leaf(w2)
    z = torch.nn.functional.gelu(nr @ r1) @ r2
    yr = xr + 0.5 * norm(z, 1.0)
    mr = norm(yr, 1.0)
    torch.autograd.backward([yr, mr], [dy.to(D), dn.to(D)])
    assert off(y, yr) < OUT and off(m, mr) < OUT
    assert off(x.grad, xr.grad) < GRAD and off(n.grad, nr.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w1], 1), r1.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w2], 0), r2.grad) < GRAD


ROUTING = [dict(score="softmax"), dict(score="sigmoid", groups=4, top_groups=2, group_best=2, renorm=True, scale=2.5)]


def routed(blk, p, E, h, f, k, routing, seed):
    g = gen(seed)
    router, w1, w2 = rnd(g, h, E, scale=h ** -0.5), rnd(g, E, h, f, scale=h ** -0.5), rnd(g, E, f, h, scale=f ** -0.5)
    b = blk.RoutedMLPBlock(router, w1, w2, p, k, alpha=0.5, **routing)
    b.bias.copy_(0.05 * torch.randn(E, generator=g, device="cuda"))
    return b, router, w1, w2, g


def reference(n, router, w1, w2, experts, routing):
    """z of the routed MLP with the choice given, in 64 bits, with autograd."""
    logits = n @ router
    s = torch.sigmoid(logits) if routing["score"] == "sigmoid" else torch.softmax(logits, 1)
    w = s.gather(1, experts)
    if routing.get("renorm"):
        w = w / w.sum(1, keepdim=True)
    w = w * routing.get("scale", 1.0)
    z = torch.zeros_like(n)
    for e in range(w1.shape[0]):
        t, j = (experts == e).nonzero(as_tuple=True)
        if t.numel():
            z = z.index_add(0, t, w[t, j][:, None] * (torch.nn.functional.gelu(n[t] @ w1[e]) @ w2[e]))
    return z


def choice(blk, b, n):
    from gemm_reduce_fusion_gb300.autograd import column_parallel_linear, route
    with torch.no_grad():
        _, experts, counts = route(column_parallel_linear(n, [b.router])[0], b.k, bias=b.bias, **b.routing)
    return experts.long(), counts


@pytest.mark.parametrize("routing", ROUTING)
@pytest.mark.parametrize("p,E,T,k,h,f", [(1, 8, 1, 2, 64, 128), (2, 16, 150, 2, 264, 392), (4, 16, 700, 3, 520, 264)])
def test_the_routed_block_trains_and_serves(blk, p, E, T, k, h, f, routing):
    b, router, w1, w2, g = routed(blk, p, E, h, f, k, routing, T)
    x0, n0, dy, dn = (rnd(g, T, h) for _ in range(4))
    x, n = x0.clone().requires_grad_(), n0.clone().requires_grad_()
    y, m = b(x, n)
    torch.autograd.backward([y, m], [dy, dn])
    experts, counts = choice(blk, b, n0)
    assert torch.equal(counts, b.counts) and int(counts.sum()) == T * k
    xr, nr, rr, r1, r2 = leaf(x0), leaf(n0), leaf(router), leaf(w1), leaf(w2)
    z = reference(nr, rr, r1, r2, experts, routing)
    yr = xr + 0.5 * norm(z, 1.0)
    mr = norm(yr, 1.0)
    torch.autograd.backward([yr, mr], [dy.to(D), dn.to(D)])
    assert off(y, yr) < OUT and off(m, mr) < OUT
    assert off(x.grad, xr.grad) < GRAD and off(n.grad, nr.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w1]), r1.grad) < GRAD
    assert off(torch.cat([t.grad for t in b.w2]), r2.grad) < GRAD
    if T > 1:
        assert off(b.router.grad, rr.grad) < GRAD
    # served from weights packed once: the same products, experts' outputs in fp32 instead of bf16 at most
    served = b.serve()
    xs = x0.clone()
    ys, ms = served(xs, n0)
    assert ys.data_ptr() == xs.data_ptr()
    assert off(ys, y.detach().to(D)) < 2.0 ** -7 and off(ms, m.detach().to(D)) < 2.0 ** -7
    # what the trained block's weights become does not reach the served one
    with torch.no_grad():
        for t in list(b.w1) + list(b.w2) + [b.router]:
            t.zero_()
    again = served(x0.clone(), n0)
    assert torch.equal(again[0], ys) and torch.equal(again[1], ms)


def test_a_served_step_captured_and_replayed(blk):
    """One token at a time through two blocks, captured once; each replay routes its own token."""
    p, E, k, h, f = 2, 16, 2, 264, 128
    one, *_ = routed(blk, p, E, h, f, k, ROUTING[1], 1)
    two, *_ = routed(blk, p, E, h, f, k, ROUTING[0], 2)
    blocks = [one.serve(), two.serve()]
    g = gen(3)
    tokens = [rnd(g, 1, h) for _ in range(5)]
    w = torch.ones(h, dtype=BF, device="cuda")

    def step(x):
        with torch.no_grad():
            n, = blk.pre_norm([x], w_pre=w)
            for b in blocks:
                x, n = b(x, n)
        return x, n
    want = [tuple(t.clone() for t in step(x.clone())) for x in tokens]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    inp = tokens[0].clone()
    with torch.cuda.stream(side):
        step(inp.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(inp.clone())
    for i in (3, 0, 4, 1, 2):
        inp.copy_(tokens[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


def test_two_streams_at_once(blk):
    p, E, k, h, f = 2, 8, 2, 264, 392
    b, *_, g = routed(blk, p, E, h, f, k, ROUTING[0], 5)
    served = b.serve()
    ns = [rnd(g, 300, h) for _ in range(4)]
    want = [served(torch.zeros_like(n), n)[0].clone() for n in ns]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None] * 4
    for i, n in enumerate(ns):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = served(torch.zeros_like(n), n)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_refusals(blk):
    z = lambda *s: torch.zeros(s, dtype=BF)  # noqa: E731
    with pytest.raises(ValueError, match="router"):
        blk.RoutedMLPBlock(z(8, 4), z(4, 8, 16), z(4, 8, 16), 2, 2)
    with pytest.raises(ValueError, match="shards"):
        blk.RoutedMLPBlock(z(8, 5), z(5, 8, 16), z(5, 16, 8), 2, 2)
    with pytest.raises(ValueError, match="token tensors"):
        blk.MLPBlock(z(8, 8), z(8, 8), 2, fp8=True, sequence_parallel=True)
    with pytest.raises(ValueError, match="score is one of"):
        blk.route(z(2, 4).cuda(), 2, score="max")
    with pytest.raises(TypeError, match="CUDA"):
        blk.route(z(2, 4), 2)
    with pytest.raises(ValueError, match="same number"):
        blk.parallel_mlp_fp8(z(2, 8), [z(8, 8)], [])
    with pytest.raises(RuntimeError):  # second derivatives
        n = rnd(gen(1), 4, 64).requires_grad_()
        y = blk.parallel_mlp_fp8(n, [rnd(gen(2), 64, 64)], [rnd(gen(3), 64, 64)])
        g, = torch.autograd.grad(y.float().square().sum(), n, create_graph=True)
        g.float().sum().backward()


def test_no_token_and_strided_inputs():
    from gemm_reduce_fusion_gb300.autograd import parallel_mlp_fp8, route, routed_experts
    h, f, E, p, k = 64, 128, 4, 2, 2
    g = torch.Generator(device="cuda").manual_seed(8)
    mk = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.1).to(torch.bfloat16).requires_grad_()  # noqa: E731
    x = torch.empty((0, h), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    shards = [mk(h, f) for _ in range(p)], [mk(f, h) for _ in range(p)]
    parallel_mlp_fp8(x, *shards).sum().backward()
    experts = [mk(E // p, h, f) for _ in range(p)], [mk(E // p, f, h) for _ in range(p)]
    logits = torch.empty((0, E), device="cuda", requires_grad=True)
    w, e, counts = route(logits, k, renorm=True)
    routed_experts(x, e, w, *experts).sum().backward()
    assert all(bool((t.grad == 0).all()) for t in (*shards[0], *shards[1], *experts[0], *experts[1]))
    assert x.grad.shape == x.shape and logits.grad.shape == logits.shape and int(counts.abs().sum()) == 0
    # views that are not contiguous give what their copies give
    x, l = mk(40, 2 * h).detach(), torch.randn((E, 40), generator=g, device="cuda")
    got = []
    for copy in (False, True):
        xs, ls = (t.contiguous().requires_grad_() if copy else t.requires_grad_() for t in (x.clone()[:, ::2], l.clone().t()))
        w, e, _ = route(ls, k)
        y = routed_experts(xs, e if copy else e.t().contiguous().t(), w if copy else w.t().contiguous().t(), *experts)
        y.float().square().sum().backward()
        got.append((y, xs.grad, ls.grad))
    assert all(torch.equal(a, b) for a, b in zip(*got))
