"""A served block beside others: it keeps the weights that it was made of, and
no other stream, graph or later call shares its workspace."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def blk():
    import gemm_reduce_fusion_gb300.block as blk
    return blk


def make(blk, h=264, f=528, p=2, seed=1, kind="layer"):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF).cuda()  # noqa: E731
    b = blk.MLPBlock(rnd(h, f, scale=h ** -0.5), rnd(f, h, scale=f ** -0.5), p, post=kind, pre=kind, gate=1 + rnd(1, h, scale=0.1),
                     alpha=0.5)
    return b, rnd


def test_training_on_leaves_a_served_block_as_it_was(blk):
    b, rnd = make(blk)
    served = b.serve(group=64)
    x, n = rnd(3, 264), rnd(3, 264)
    first = [t.clone() for t in served(x.clone(), n)]
    with torch.no_grad():
        for t in b.parameters():
            t.add_(1.0)
    again = served(x.clone(), n)
    assert all(torch.equal(s, t) for s, t in zip(first, again))


def test_second_derivatives_are_refused(blk):
    """The gradients come from kernels that autograd cannot differentiate
    again: a penalty on them is refused, not taken for a constant."""
    b, rnd = make(blk)
    for apply in (lambda t: blk.parallel_mlp_ckpt(t, list(b.w1), list(b.w2)), lambda t: blk.pre_norm([t])[0],
                  lambda t: blk.block_boundary([t], [t])[0][0]):
        t = rnd(16, 264).requires_grad_()
        (g,) = torch.autograd.grad(apply(t).float().square().sum(), t, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.float().square().sum() + t.float().sum()).backward()


def test_streams_and_graphs_have_workspaces_of_their_own(blk):
    from gemm_reduce_fusion_gb300.autograd import _workspace
    dev, call = torch.device("cuda", torch.cuda.current_device()), [(blk.TP_OP_ROW_W4, 2, 4, 264, 528)]
    here = _workspace(dev, call)
    assert _workspace(dev, call).data_ptr() == here.data_ptr()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        there = _workspace(dev, call)
    a, b = here.data_ptr(), there.data_ptr()
    assert a + here.numel() <= b or b + there.numel() <= a
    kept = []
    torch.cuda.synchronize()
    for stream in (side, torch.cuda.Stream()):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            kept.append((graph, _workspace(dev, call).data_ptr()))
    assert len({a, b, kept[0][1], kept[1][1]}) == 4
    assert _workspace(dev, call).data_ptr() == a


def test_a_captured_step_keeps_its_memory(blk):
    """A longer prompt and other allocations between capture and replay: the
    replayed step gives the same tokens and writes nothing of theirs."""
    b, rnd = make(blk, h=1032, f=2064)
    served = b.serve(group=64)
    x0, n0 = rnd(1, 1032), rnd(1, 1032)
    want = [t.clone() for t in served(x0.clone(), n0)]
    x, n = x0.clone(), n0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m = served(x, n)
    served(rnd(300, 1032), rnd(300, 1032))
    others = [torch.full((1 << k,), 77, dtype=torch.uint8, device="cuda") for k in range(8, 24) for _ in range(4)]
    for _ in range(2):
        x.copy_(x0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(m, want[1])
    assert all(bool((t == 77).all()) for t in others)


def test_a_captured_training_step_replays(blk):
    """Forward and backward in one graph, whose products count their slices in the graph's workspace."""
    b, rnd = make(blk, h=1032, f=4128, kind="rms")
    x = rnd(3000, 1032).requires_grad_()
    gy, gm = rnd(3000, 1032), rnd(3000, 1032)
    leaves = [x, *b.parameters()]

    def step():
        y, m = b(x, blk.pre_norm([x])[0])
        return [y, m, *torch.autograd.grad([y, m], leaves, [gy, gm])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(3):
        for t in got:
            t.detach().fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, want))
