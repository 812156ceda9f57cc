"""The sharded Linear with 4-bit weights: packing bit for bit, products
against the definition in 64 bits.  The products keep the library's bounds:
1e-5 of the largest value for fp32 outputs, 5e-3 for bf16."""
import pytest
import torch

import ops_ref as ref
from gpu_util import assert_close, host_f64, poisoned

pytestmark = pytest.mark.gpu
BF, F32, D = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def random_w4(tp, K, N, G, g, garbage=False):
    """A 4-bit weight of random nibbles and scales; garbage: whatever lies past K and N is random too."""
    qs, ss = tp.w4_shapes(K, N, G)
    q = torch.randint(0, 256, qs, generator=g, dtype=torch.uint8)
    s = (0.01 * (0.5 + torch.rand(ss, generator=g))).to(BF)
    if garbage:  # scales of columns past N are never used: NaN must not leak
        n = torch.arange(ss[0] * 32).view(ss[0], 2, 2, 8).permute(0, 1, 3, 2).reshape(ss[0], 1, 32).expand(ss)
        s[n >= N] = float("nan")
    return q, s


SHAPES = [(1, 1, 8, 8), (1, 1, 32, 64), (2, 1, 264, 1000), (1, 7, 40, 72), (3, 8, 520, 200), (2, 9, 256, 512), (8, 16, 264, 136),
          (1, 17, 2056, 1160), (2, 33, 520, 264), (1, 48, 96, 2048), (2, 64, 264, 1032), (4, 3, 1000, 4104)]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("p,M,N,K", SHAPES)
def test_row(tp, p, M, N, K, G):
    g = torch.Generator().manual_seed(M + N + K)
    w = [random_w4(tp, K, N, G, g, garbage=True) for _ in range(p)]
    x = [torch.randn(M, K, generator=g).to(BF) for _ in range(p)]
    b = torch.randn(N, generator=g).to(BF)
    want = sum(a.to(D) @ ref.w4_value(q, s, K, N, G) for a, (q, s) in zip(x, w))
    ws = tp.workspace(tp.TP_OP_ROW_W4, p, M, N, K)
    q, s, xd = [a.cuda() for a, _ in w], [a.cuda() for _, a in w], [a.cuda() for a in x]
    for f32 in (True, False):
        y = poisoned((M, N), f32)
        tp.tp_row_linear_fwd_w4(xd, q, s, y, ws, group=G)
        assert_close(host_f64(y), want.numpy(), f32, "Y")
        y2 = poisoned((M, N), f32)
        tp.tp_row_linear_fwd_w4(xd, q, s, y2, ws, group=G)
        assert torch.equal(y, y2), "the sum's order is fixed"
        tp.tp_row_linear_fwd_w4(xd, q, s, y2, ws, group=G, bias=b.cuda())
        assert_close(host_f64(y2), (want + b.to(D)).numpy(), f32, "Y + b")


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("p,M,N,K", SHAPES)
def test_column(tp, p, M, N, K, G):
    g = torch.Generator().manual_seed(M + N + K + 1)
    w = [random_w4(tp, K, N, G, g, garbage=True) for _ in range(p)]
    x = torch.randn(M, K, generator=g).to(BF)
    b = [torch.randn(N, generator=g).to(BF) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_COL_W4, p, M, N, K)
    q, s = [a.cuda() for a, _ in w], [a.cuda() for _, a in w]
    for f32 in (True, False):
        for bias, act in ((False, False), (True, True)):
            y = [poisoned((M, N), f32) for _ in range(p)]
            tp.tp_col_linear_fwd_w4(x.cuda(), q, s, y, ws, group=G, epi=tp.TP_EPI_GELU if act else tp.TP_EPI_NONE,
                                    bias=[a.cuda() for a in b] if bias else None)
            for k in range(p):
                want = x.to(D) @ ref.w4_value(*w[k], K, N, G)
                want = want + b[k].to(D) if bias else want
                assert_close(host_f64(y[k]), (ref.gelu(want) if act else want).numpy(), f32, f"Y_{k}")


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 12, 24, 31, 32, 40, 41, 56, 63])
def test_every_token_tile(tp, M):
    g = torch.Generator().manual_seed(M)
    K, N, G = 328, 296, 64
    q, s = random_w4(tp, K, N, G, g)
    x = torch.randn(M, K, generator=g).to(BF)
    y = poisoned((M, N), True)
    tp.tp_row_linear_fwd_w4([x.cuda()], [q.cuda()], [s.cuda()], y, tp.workspace(tp.TP_OP_ROW_W4, 1, M, N, K), group=G)
    assert_close(host_f64(y), (x.to(D) @ ref.w4_value(q, s, K, N, G)).numpy(), True, "Y")


@pytest.mark.parametrize("G", [32, 128])
@pytest.mark.parametrize("p,N,K", [(1, 8, 8), (2, 40, 72), (1, 264, 1000), (3, 520, 160)])
def test_pack_and_unpack(tp, p, N, K, G):
    g = torch.Generator().manual_seed(N * K)
    w = [(torch.randn(K, N, generator=g) * 0.02).to(BF) for _ in range(p)]
    w[0][:, 0] = 0
    w[0][0, 1] = float("nan")
    w[0][K - 1, 2] = float("inf")
    w[0][:, 3] = (torch.arange(K) % 8).to(BF) - 3.5  # quotients half-way between whole numbers
    qs, ss = tp.w4_shapes(K, N, G)
    q = [torch.full(qs, 0xEE, dtype=torch.uint8, device="cuda") for _ in w]
    s = [torch.full(ss, 3.0, dtype=BF, device="cuda") for _ in w]
    tp.tp_w4_pack([a.cuda() for a in w], q, s, group=G)
    out = [torch.empty((K, N), dtype=BF, device="cuda") for _ in w]
    tp.tp_w4_unpack(q, s, out, group=G)
    word, nib = ref.w4_place(K, N)
    for i in range(p):
        n, sc = ref.w4_quant(w[i], G)
        words = q[i].cpu().view(torch.int32).view(-1).to(torch.int64)
        assert torch.equal((words[word] >> (4 * nib)) & 15, n)
        got = s[i].cpu().view(-1)[ref.w4_scale_place(K, N, G)[::G]]
        assert torch.equal(torch.isnan(got), torch.isnan(sc)) and torch.equal(got.nan_to_num(), sc.nan_to_num())
        # past the edges: nibbles that stand for zero
        used = torch.zeros(words.numel() * 8, dtype=torch.bool)
        used[(word * 8 + nib).view(-1)] = True
        all_nibbles = torch.stack([(words >> (4 * b)) & 15 for b in range(8)], 1).view(-1)
        assert (all_nibbles[~used] == 8).all()
        want = ref.w4_value(q[i], s[i], K, N, G).to(BF)
        assert torch.equal(torch.isnan(out[i].cpu()), torch.isnan(want))
        assert torch.equal(out[i].cpu().nan_to_num(), want.nan_to_num())


def test_unpacked_weights_serve_long_prompts(tp):
    """The products of many tokens: unpack, then the sharded Linear in bf16."""
    p, M, N, K, G = 2, 300, 264, 520, 64
    g = torch.Generator().manual_seed(9)
    w = [random_w4(tp, K, N, G, g) for _ in range(p)]
    x = [torch.randn(M, K, generator=g).to(BF) for _ in range(p)]
    full = [torch.empty((K, N), dtype=BF, device="cuda") for _ in range(p)]
    tp.tp_w4_unpack([a.cuda() for a, _ in w], [a.cuda() for _, a in w], full, group=G)
    y = poisoned((M, N))
    tp.tp_row_linear_fwd_allreduce([a.cuda() for a in x], full, [y], tp.workspace(tp.TP_OP_ROW_AR, p, M, N, K))
    want = sum(a.to(D) @ ref.w4_value(q, s, K, N, G).to(BF).to(D) for a, (q, s) in zip(x, w))
    assert_close(host_f64(y), want.numpy(), False, "Y")


def test_broken_tokens_and_columns_keep_to_themselves(tp):
    p, M, N, K, G = 2, 11, 296, 1000, 32
    g = torch.Generator().manual_seed(4)
    w = [random_w4(tp, K, N, G, g) for _ in range(p)]
    x = [torch.randn(M, K, generator=g).to(BF) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_ROW_W4, p, M, N, K)
    call = lambda x, w, y: tp.tp_row_linear_fwd_w4([a.cuda() for a in x], [a.cuda() for a, _ in w],  # noqa: E731
                                                   [a.cuda() for _, a in w], y, ws, group=G)
    y0, y1 = poisoned((M, N), True), poisoned((M, N), True)
    call(x, w, y0)
    x[1][3, K - 1], x[0][9, 0] = float("nan"), float("inf")
    place = ref.w4_scale_place(K, N, G)
    w[1][1].view(-1)[place[5, 17]] = float("nan")
    call(x, w, y1)
    rows, cols = [i for i in range(M) if i not in (3, 9)], [i for i in range(N) if i != 17]
    assert torch.equal(y0[rows][:, cols], y1[rows][:, cols])
    assert torch.isnan(y1[3]).all() and not torch.isfinite(y1[9]).any() and torch.isnan(y1[:, 17]).all()


def test_a_shared_workspace_empty_sizes_and_graph_replay(tp):
    p, M, N, K, G = 2, 5, 520, 1000, 128
    g = torch.Generator().manual_seed(6)
    w = [random_w4(tp, K, N, G, g) for _ in range(p)]
    x = [torch.randn(M, K, generator=g).to(BF).cuda() for _ in range(p)]
    q, s = [a.cuda() for a, _ in w], [a.cuda() for _, a in w]
    want = sum(a.cpu().to(D) @ ref.w4_value(b, c, K, N, G) for a, (b, c) in zip(x, w)).numpy()
    n = max(tp.tp_workspace_size(tp.TP_OP_ROW_W4, p, M, N, K), tp.tp_workspace_size(tp.TP_OP_ROW_AR, 8, 16, 2048, 512, 16))
    ws = torch.zeros((n + 255) // 256 * 256, dtype=torch.uint8, device="cuda")
    y = poisoned((M, N), True)
    tp.tp_row_linear_fwd_w4(x, q, s, y, ws, group=G)
    assert_close(host_f64(y), want, True, "Y")
    xs = [torch.randn(16, 512, device="cuda").to(BF) for _ in range(8)]
    fs = [torch.randn(512, 2048, device="cuda").to(BF) for _ in range(8)]
    tp.tp_row_linear_fwd_allreduce(xs, fs, [torch.empty((16, 2048), dtype=BF, device="cuda")], ws, chunk_m=16)
    y2 = poisoned((M, N), True)
    tp.tp_row_linear_fwd_w4(x, q, s, y2, ws, group=G)
    assert torch.equal(y, y2) and tp.tp_get_device_status(ws) == tp.TP_OK
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_row_linear_fwd_w4(x, q, s, y2, ws, group=G)
    for _ in range(3):
        y2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
    # no rows to add up: the epilogue of zero; no tokens, no columns: nothing
    z = [torch.empty((3, 0), dtype=BF, device="cuda")] * p
    b = torch.randn(N, generator=g).to(BF).cuda()
    qs, ss = tp.w4_shapes(0, N, G)
    e, f = [torch.empty(qs, dtype=torch.uint8, device="cuda")] * p, [torch.empty(ss, dtype=BF, device="cuda")] * p
    y3 = poisoned((3, N), True)
    tp.tp_row_linear_fwd_w4(z, e, f, y3, ws, group=G, bias=b)
    assert torch.equal(y3, b.float().expand(3, N))
    tp.tp_row_linear_fwd_w4([t[:0] for t in x], q, s, poisoned((0, N)), ws, group=G)
