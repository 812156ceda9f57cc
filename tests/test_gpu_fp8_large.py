"""Tensors of more than 2^31 elements through the 8-bit operators, on values
that no rounding touches: what lies behind 32-bit offsets is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GB of free memory")
    yield
    torch.cuda.empty_cache()


def test_products_and_packing(tp):
    M, N, K = 40000, 65536, 128  # 2.6e9 elements
    a = (1 + torch.arange(M, device="cuda") % 3).to(BF)
    b = (1 + torch.arange(N, device="cuda") % 2).to(BF)
    x, w = a[:, None].expand(M, K).contiguous(), b[:, None].expand(N, K).contiguous()
    xq, wq = tp.fp8_empty(M, K), tp.fp8_empty(N, K)
    tp.tp_fp8_pack([x], [xq])
    tp.tp_fp8_pack([w], [wq], tiles=True)
    y, ws = torch.empty((M, N), dtype=BF, device="cuda"), tp.workspace(tp.TP_OP_COL_FP8, 1, M, N, K)
    tp.tp_col_linear_fwd_fp8(xq, [wq], [y], ws)
    row = lambda i, j: (K * a[i:j, None].float() * b[None].float()).to(BF)  # noqa: E731
    assert all(torch.equal(y[i:i + 4000], row(i, i + 4000)) for i in range(0, M, 4000))
    q, qt = tp.fp8_empty(M, N), tp.fp8_empty(N, M)
    tp.tp_fp8_pack([y], [q], [qt])
    back = torch.empty_like(y)
    tp.tp_fp8_unpack([q], [back])
    assert torch.equal(back, y)
    back = back.view(N, M)
    tp.tp_fp8_unpack([qt], [back])
    assert all(torch.equal(back[i:i + 8192], y[:, i:i + 8192].t()) for i in range(0, N, 8192))
    # the result in 8 bits, from the epilogue
    z = tp.fp8_empty(M, N)
    z.q.view(torch.uint8).fill_(0xFF)
    tp.tp_col_linear_fwd_fp8(xq, [wq], None, ws, z=[z])
    back = back.view(M, N).fill_(7)
    tp.tp_fp8_unpack([z], [back])
    assert torch.equal(back, y)
    # a contraction over all of it, and a gradient of its size
    dx = torch.empty((N, K), dtype=BF, device="cuda")
    ones = torch.ones((K, M), dtype=BF, device="cuda")
    oq = tp.fp8_empty(K, M)
    tp.tp_fp8_pack([ones], [oq])
    tp.tp_row_linear_fwd_fp8([qt], [oq], dx, tp.workspace(tp.TP_OP_ROW_FP8, 1, N, K, M))
    # (multiples of K, a power of two, below 2^24 K: sums in fp32 are exact)
    want = (K * b.float() * float(a.float().sum())).to(BF)
    assert float(a.float().sum()) * 2 < 2 ** 24 and torch.equal(dx, want[:, None].expand(N, K))


def test_experts(tp):
    """One-hot tokens, whole first weights of 8 to 14 (whose GeLU is themselves), second weights with one power of two a row."""
    E, T, k, h, f = 3, 270000, 2, 4096, 16  # 540000 rows, 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(4)
    w1 = (8 + 2 * torch.randint(0, 4, (E, h, f), generator=g, device="cuda")).to(BF)
    w2 = torch.zeros((E, f, h), device="cuda", dtype=BF)
    hot = torch.arange(f, device="cuda") * 255
    w2[:, torch.arange(f, device="cuda"), hot] = torch.pow(2.0, torch.randint(0, 3, (E, f), generator=g, device="cuda")).to(BF)

    def packed(w, transposed):
        op = tp.fp8_empty(*((w.shape[2], w.shape[1]) if transposed else w.shape[1:]), E)
        tp.tp_fp8_pack([w], None if transposed else [op], [op] if transposed else None, tiles=True)
        return [op]
    at = torch.randint(0, h, (T,), generator=g, device="cuda")
    x = torch.zeros((T, h), dtype=BF, device="cuda")
    x[torch.arange(T, device="cuda"), at] = 1
    dy = torch.zeros((T, h), dtype=BF, device="cuda")
    dy[:, hot] = torch.randint(-1, 2, (T, f), generator=g, device="cuda").to(BF)
    experts = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32).contiguous()
    weights = torch.full((T, k), 0.5, device="cuda")
    ws, saved = tp.experts_workspace(1, E, T, k, h, f, backward=True), tp.experts_saved(E, T, k, h, f)
    assert tp.tp_experts_rows(E, T, k) * h > 2 ** 31
    e = experts.long()
    first = w1[e, at[:, None]].float()                       # [T, k, f]
    power = w2[:, torch.arange(f, device="cuda"), hot].float()  # [E, f]
    want = (0.5 * first * power[e]).sum(1)                   # at the columns `hot`
    for s in (None, saved):
        y = torch.full((T, h), 9.0, dtype=BF, device="cuda")
        tp.tp_experts_fwd_fp8(x, experts, weights, packed(w1, True), packed(w2, True), y, ws, saved=s)
        assert torch.equal(y[:, hot].float(), want.to(BF).float())
        y[:, hot] = 0
        assert all(int(y[i:i + 30000].count_nonzero()) == 0 for i in range(0, T, 30000))
    del y
    dx, dw, d1, d2 = torch.empty_like(x), torch.empty((T, k), device="cuda", dtype=BF), [torch.empty_like(w1)], [torch.empty_like(w2)]
    tp.tp_experts_bwd_fp8(x, weights, dy, packed(w1, False), packed(w2, False), dx, dw, d1, d2, saved, ws)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    assert torch.equal(dw.float(), (first * power[e] * dy[:, None, hot].float()).sum(2).to(BF).float())
    dh = 0.5 * dy[:, None, hot].float() * power[e]           # [T, k, f], exact
    for i in list(range(0, T, 90000)) + [T - 500]:
        rows = slice(i, i + 500)
        each = torch.einsum("tkf,tkhf->tkh", dh[rows], w1[e[rows]].float()).to(BF).float()
        assert torch.equal(dx[rows].float(), (each[:, 0] + each[:, 1]).to(BF).float())
    # weights' gradients: dW2 at (f, hot) adds up whole halves below 2^24, exactly
    for n in range(E):
        t, j = (experts == n).nonzero(as_tuple=True)
        full = first[t, j].t().double() @ (0.5 * dy[t][:, hot].double())
        assert torch.equal(d2[0][n][:, hot].double(), full.to(BF).double())
        sums = torch.zeros((h, f), dtype=torch.float64, device="cuda").index_add_(0, at[t], dh[t, j].double())
        assert torch.equal(d1[0][n].double(), sums.to(BF).double())
