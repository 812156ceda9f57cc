"""The MLP block as it stands in a model: two blocks chained, trained on 8-bit
checkpoints and served from 4-bit weights, against 64-bit arithmetic on the
same values.

Each bf16 tensor that passes from one call to the next is rounded once (2^-9
of its size) and a sum over it keeps that relative error; about eight such
roundings lie between the inputs and the gradients of the first block, and the
checkpoints add an error of at most 1/127 of their group's largest value, 1 % of
a product's size when it is random.  Outputs are held to 1 % and gradients to
3 % in the 2-norm."""
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def blk():
    import gemm_reduce_fusion_gb300.block as blk
    return blk


def off(got, want):
    return float((got.detach().cpu().to(D) - want).norm() / want.norm())


def rnd(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF)


def reference_block(x, n, w1, w2, d):
    """y, n' of the plain block in 64 bits, with autograd."""
    def norm(v, kind, w):
        if kind == "layer":
            v = v - v.mean(1, keepdim=True)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w
    z = torch.nn.functional.gelu(n @ w1) @ w2
    y = x + d["alpha"] * d["gate"] * norm(z, d["post"], d["w_post"])
    return y, norm(y, d["pre"], d["w_pre"])


@pytest.mark.parametrize("sp", [False, True])
@pytest.mark.parametrize("res", [BF, torch.float32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_two_blocks_train(blk, sp, res, kind):
    p, M, h, f = 2, 192, 264, 528
    g = torch.Generator().manual_seed(11)
    ws = [(rnd(g, h, f, scale=h ** -0.5), rnd(g, f, h, scale=f ** -0.5)) for _ in range(2)]
    gates = [1 + rnd(g, 1, h, scale=0.1) for _ in range(2)]
    x0, dy, dn = rnd(g, M, h).to(res), rnd(g, M, h).to(res), rnd(g, M, h)
    blocks = [blk.MLPBlock(a.cuda(), b.cuda(), p, post=kind, pre=kind, gate=t.cuda(), alpha=0.5, sequence_parallel=sp)
              for (a, b), t in zip(ws, gates)]
    w_in = (1 + rnd(g, h, scale=0.1)).cuda().requires_grad_()
    x = x0.cuda().requires_grad_()
    xs = list(x.chunk(p)) if sp else [x]
    ns = blk.pre_norm(xs, pre=kind, w_pre=w_in)
    s, n = (xs, ns) if sp else (xs[0], ns[0])
    for b in blocks:
        s, n = b(s, n)
    s, n = (torch.cat(s), torch.cat(n)) if sp else (s, n)
    torch.autograd.backward([s, n], [dy.cuda(), dn.cuda()])

    leaf = lambda t: t.detach().cpu().to(D).requires_grad_()  # noqa: E731
    xr, wr = leaf(x0), leaf(w_in)
    par = [dict(w1=leaf(a), w2=leaf(b), gate=leaf(t), w_post=leaf(m.w_post), w_pre=leaf(m.w_pre), alpha=0.5, post=kind, pre=kind)
           for (a, b), t, m in zip(ws, gates, blocks)]
    c = xr - xr.mean(1, keepdim=True) if kind == "layer" else xr
    nr, sr = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * wr, xr
    for q in par:
        sr, nr = reference_block(sr, nr, q["w1"], q["w2"], q)
    torch.autograd.backward([sr, nr], [dy.to(D), dn.to(D)])
    assert off(s, sr.detach()) < 0.01 and off(n, nr.detach()) < 0.01
    assert off(x.grad, xr.grad) < 0.03 and off(w_in.grad, wr.grad) < 0.03
    for m, q in zip(blocks, par):
        assert off(torch.cat([t.grad for t in m.w1], 1), q["w1"].grad) < 0.03
        assert off(torch.cat([t.grad for t in m.w2], 0), q["w2"].grad) < 0.03
        for k in ("gate", "w_post", "w_pre"):
            assert off(getattr(m, k).grad, q[k].grad) < 0.03, k


def test_what_is_saved_takes_half(blk):
    """X [M, h] and H [M, ffn] in 8 bits and a byte per 32, against X, H and Z in bf16."""
    p, M, h, f = 2, 256, 256, 1024
    g = torch.Generator().manual_seed(1)
    n = rnd(g, M, h).cuda().requires_grad_()
    w1, w2 = [rnd(g, h, f // p, scale=0.05).cuda() for _ in range(p)], [rnd(g, f // p, h, scale=0.05).cuda() for _ in range(p)]
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        blk.parallel_mlp_ckpt(n, w1, w2)
    held = sum(t.numel() * t.element_size() for t in kept if t.data_ptr() not in {w.data_ptr() for w in w1 + w2})
    assert held == M * (h + f) * 33 // 32
    assert held < 0.3 * 2 * M * (h + 2 * f)


@pytest.mark.parametrize("M", [1, 5, 64, 65, 300])
def test_a_served_block_is_the_block_with_its_4_bit_weights(blk, M):
    p, h, f, G = 2, 264, 528, 64
    g = torch.Generator().manual_seed(M)
    w1, w2 = rnd(g, h, f, scale=h ** -0.5), rnd(g, f, h, scale=f ** -0.5)
    b = blk.MLPBlock(w1.cuda(), w2.cuda(), p, gate=(1 + rnd(g, 1, h, scale=0.1)).cuda(), alpha=0.5)
    served = b.serve(group=G)
    values = []
    for q, s, K, N in (served.fc1, served.fc2):
        values.append([ref.w4_value(a, c, K, N, G) for a, c in zip(q, s)])
    assert off(torch.cat(values[0], 1), w1.to(D)) < 0.15  # 4 bits: a step of max / 7, 1 / sqrt(12) of it at random
    x, n = rnd(g, M, h), rnd(g, M, h)
    xd = x.cuda()
    y, m = served(xd, n.cuda())
    assert y.data_ptr() == xd.data_ptr()
    d = dict(alpha=0.5, gate=b.gate.detach().cpu().to(D), post="rms", pre="rms", w_post=1.0, w_pre=1.0)
    yr, nr = reference_block(x.to(D), n.to(D), torch.cat(values[0], 1), torch.cat(values[1], 0), d)
    assert off(y, yr) < 0.01 and off(m, nr) < 0.01


def test_refusals(blk):
    w = [torch.zeros(8, 8, dtype=BF) for _ in range(2)]
    with pytest.raises(ValueError, match="norm is one of"):
        blk.block_boundary([w[0]], [w[1]], post="batch")
    with pytest.raises(ValueError, match="same number"):
        blk.parallel_mlp_ckpt(w[0], w, w[:1])
    with pytest.raises(ValueError, match="token shard"):
        blk.parallel_mlp_ckpt(w[:1], w, w)
