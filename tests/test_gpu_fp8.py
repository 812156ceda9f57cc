"""The sharded Linear on 8-bit operands: packing bit for bit, products against
the definition in 64 bits, exactly where all sums are whole numbers."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def activation(g, shape):
    x = torch.randn(shape, generator=g, device="cuda")
    x[:, torch.rand(shape[1], generator=g, device="cuda") < 0.02] *= 30
    return x.to(BF)


def poisoned(tp, rows, cols, batch=None):
    op = tp.fp8_empty(rows, cols, batch)
    op.q.view(torch.uint8).fill_(0x7F)
    op.e.fill_(0xFF)
    return op


def check_operand(op, R, C, want, k):
    """The operand's bits: exponents, values, and zeros past the columns."""
    same = torch.equal(ref.exponents_of(op[1], R, k.shape[1]), k)
    assert same, "exponents"
    same = torch.equal(ref.values(op, C).nan_to_num(12345.0), want.nan_to_num(12345.0))
    assert same, "values"
    assert bool((op[0][:, C:].contiguous().view(torch.uint8) == 0).all())


PACKED = [(1, 8), (1, 1000), (16, 128), (77, 520), (128, 512), (129, 136), (256, 1032), (300, 2056), (1100, 264)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("M,N", PACKED)
def test_pack_rows_and_transpose(tp, M, N, tiles):
    x = [activation(gen(M + N + i), (M, N)) for i in range(2)]
    x[1][M // 2] = 0
    x[1][:, N // 2] = 0
    q, qt = [poisoned(tp, M, N) for _ in x], [poisoned(tp, N, M) for _ in x]
    only, only_t = [poisoned(tp, M, N) for _ in x], [poisoned(tp, N, M) for _ in x]
    tp.tp_fp8_pack(x, q, qt, tiles=tiles)
    tp.tp_fp8_pack(x, only, tiles=tiles)
    tp.tp_fp8_pack(x, None, only_t, tiles=tiles)
    for i, a in enumerate(x):
        v, k = ref.pack(a, tiles)
        vt, kt = ref.pack(a.t(), tiles)
        for op in (q[i], only[i]):
            check_operand(op, M, N, v, k)
        for op in (qt[i], only_t[i]):
            check_operand(op, N, M, vt, kt)
        if tiles:
            assert torch.equal(v, vt.t())
    y = [torch.empty_like(a) for a in x]
    tp.tp_fp8_unpack(q, y)
    for i in range(2):
        assert torch.equal(y[i].to(D), ref.values(q[i], N))


def test_pack_extremes(tp):
    """Infinities, NaN, the type's largest and smallest values, blocks of zeros, and values on the border of an exponent."""
    M, N = 130, 520
    x = torch.randn((M, N), generator=gen(1), device="cuda").to(BF)
    x[0, 3], x[1, 130], x[2, 400] = float("inf"), float("-inf"), float("nan")
    x[3, :128] = float("inf")
    x[4] = torch.finfo(BF).max
    x[5] = -torch.finfo(BF).max
    x[6] = 2.0 ** -133
    x[7] = torch.finfo(BF).tiny
    x[8] = 0
    for i, v in enumerate((448.0, 450.0, 447.0, 1.75, 1.7578125, 1.7421875)):
        x[9 + i] = 0.001
        x[9 + i, ::128] = v
    q, qt, few = poisoned(tp, M, N), poisoned(tp, N, M), poisoned(tp, M, N)
    tp.tp_fp8_pack([x], [q], [qt])
    tp.tp_fp8_pack([x], [few])
    for op in (q, few):
        check_operand(op, M, N, *ref.pack(x))
    check_operand(qt, N, M, *ref.pack(x.t()))
    tile = poisoned(tp, M, N)
    tp.tp_fp8_pack([x], [tile], tiles=True)
    check_operand(tile, M, N, *ref.pack(x, True))


def test_pack_gelu_and_batches(tp):
    B, M, N = 3, 200, 264
    x = torch.randn((B, M, N), generator=gen(2), device="cuda").to(BF)
    q, qt = poisoned(tp, M, N, B), poisoned(tp, N, M, B)
    tp.tp_fp8_pack([x], [q], [qt], tiles=True)
    for b in range(B):
        check_operand((q.q[b], q.e[b]), M, N, *ref.pack(x[b], True))
        check_operand((qt.q[b], qt.e[b]), N, M, *ref.pack(x[b].t(), True))
    back = torch.empty_like(x)
    tp.tp_fp8_unpack([q], [back])
    assert torch.equal(back.to(D), torch.stack([ref.values((q.q[b], q.e[b]), N) for b in range(B)]))
    op, opt = poisoned(tp, M, N), poisoned(tp, N, M)
    tp.tp_fp8_pack([x[0]], [op], [opt], epi=tp.TP_EPI_GELU)
    g = ref.gelu(x[0].to(D))
    for o, R, C, w in ((op, M, N, g), (opt, N, M, g.t())):
        k = ref.exponents_of(o.e, R, -(-C // 128))
        step = ref.two_to(k).repeat_interleave(128, 1)[:, :C]
        # GeLU is within 3e-7 (1 + |h|) in fp32; then half a step of e4m3, which below 2^-6 of the scale is 2^-10 of it
        off = (ref.values(o, C) - w).abs()
        assert bool((off <= ref.HALF_E4M3 * w.abs() + step * 2.0 ** -10 + 1e-6 * (1 + w.abs())).all())


def operands(tp, xs, transposed=False, tiles=False):
    out = []
    for x in xs:
        M, N = x.shape
        op = tp.fp8_empty(*((N, M) if transposed else (M, N)))
        tp.tp_fp8_pack([x], None if transposed else [op], [op] if transposed else None, tiles=tiles)
        out.append(op)
    return out


SHAPES = [(1, 1, 8, 8), (1, 1, 136, 128), (2, 1, 264, 1000), (1, 7, 40, 72), (8, 3, 520, 200), (2, 16, 256, 512), (3, 17, 264, 136),
          (1, 33, 2056, 1160), (4, 77, 520, 1000), (2, 128, 1000, 264), (1, 129, 128, 4104), (2, 300, 384, 640), (5, 1030, 520, 264),
          (2, 1100, 2056, 1160), (8, 513, 1032, 392), (1, 2049, 2056, 2568)]


@pytest.mark.parametrize("p,M,N,K", SHAPES)
def test_row(tp, p, M, N, K):
    g = gen(M + N + K)
    x, w = [activation(g, (M, K)) for _ in range(p)], [(torch.randn((K, N), generator=g, device="cuda") * 0.05).to(BF) for _ in range(p)]
    b = torch.randn(N, generator=g, device="cuda").to(BF)
    xq, wq = operands(tp, x), operands(tp, w, True, True)
    a = torch.cat([ref.values(o, K) for o in xq], 1)
    v = torch.cat([ref.values(o, K) for o in wq], 1)
    want, slack = a @ v.t(), ref.sum_error(a, v)
    ws = tp.workspace(tp.TP_OP_ROW_FP8, p, M, N, K)
    y, y2 = (torch.full((M, N), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    tp.tp_row_linear_fwd_fp8(xq, wq, y, ws)
    assert_within(y, want, slack, "Y")
    tp.tp_row_linear_fwd_fp8(xq, wq, y2, ws)
    assert torch.equal(y, y2), "the sum's order is fixed"
    tp.tp_row_linear_fwd_fp8(xq, wq, y, ws, bias=b)
    assert_within(y, want + b.to(D), slack + 2.0 ** -23 * (want.abs() + b.to(D).abs()), "Y + b")
    assert tp.tp_get_device_status(ws) == tp.TP_OK


@pytest.mark.parametrize("p,M,N,K", SHAPES)
def test_column(tp, p, M, N, K):
    g = gen(M + N + K + 1)
    x, w = activation(g, (M, K)), [(torch.randn((K, N), generator=g, device="cuda") * 0.05).to(BF) for _ in range(p)]
    b = [torch.randn(N, generator=g, device="cuda").to(BF) for _ in range(p)]
    (xq,), wq = operands(tp, [x]), operands(tp, w, True, True)
    ws = tp.workspace(tp.TP_OP_COL_FP8, p, M, N, K)
    nan = lambda: [torch.full((M, N), float("nan"), dtype=BF, device="cuda") for _ in range(p)]  # noqa: E731
    y, hh, y2 = nan(), nan(), nan()
    tp.tp_col_linear_fwd_fp8(xq, wq, y, ws)
    tp.tp_col_linear_fwd_fp8(xq, wq, y2, ws, epi=tp.TP_EPI_GELU, preact=hh, bias=b)
    z = [poisoned(tp, M, N) for _ in range(p)]
    h2 = nan()
    tp.tp_col_linear_fwd_fp8(xq, wq, None, ws, epi=tp.TP_EPI_GELU, preact=h2, bias=b, z=z)
    plain = [poisoned(tp, M, N) for _ in range(p)]
    tp.tp_col_linear_fwd_fp8(xq, wq, None, ws, z=plain)
    a = ref.values(xq, K)
    for k in range(p):
        v = ref.values(wq[k], K)
        want, slack = a @ v.t(), ref.sum_error(a, v)
        assert_within(y[k], want, slack, "Y")
        check_near(plain[k], want, slack)
        want = want + b[k].to(D)
        slack = slack + 2.0 ** -23 * want.abs()
        assert_within(hh[k], want, slack, "H")
        assert torch.equal(hh[k], h2[k])
        g1 = ref.gelu(want)
        # |GeLU'| <= 1.13; GeLU itself is within 3e-7 (1 + |h|) in fp32
        assert_within(y2[k], g1, 1.13 * slack + 1e-6 * (1 + want.abs()), "GeLU")
        check_near(z[k], g1, 1.13 * slack + 1e-6 * (1 + want.abs()))
    assert tp.tp_get_device_status(ws) == tp.TP_OK


def check_near(op, want, slack):
    """An operand packed from values within `slack` of want."""
    R, C = want.shape
    B = -(-C // 128)
    k = ref.exponents_of(op.e, R, B)
    pad = lambda t: torch.nn.functional.pad(t, (0, B * 128 - C)).view(R, B, 128)  # noqa: E731
    lo, hi = pad(want.abs() - slack).amax(2), pad(want.abs() + slack).amax(2)
    assert bool((k <= ref.exponents(hi)).all()) and bool((k >= ref.exponents(lo.clamp(min=0))).all())
    step = ref.two_to(k).repeat_interleave(128, 1)[:, :C]
    off = (ref.values(op, C) - want).abs()
    assert bool((off <= ref.HALF_E4M3 * (want.abs() + slack) + step * 2.0 ** -10 + slack).all())
    assert bool((op[0][:, C:].contiguous().view(torch.uint8) == 0).all())


@pytest.mark.parametrize("p,M,N,K", [(1, 1, 8, 8), (2, 5, 264, 136), (1, 129, 256, 384), (3, 300, 520, 264), (2, 513, 2056, 1160),
                                     (4, 1100, 1000, 520)])
def test_backward(tp, p, M, N, K):
    g = gen(M + N + K + 2)
    rnd = lambda n, *s: [torch.randn(s, generator=g, device="cuda").to(BF) for _ in range(n)]  # noqa: E731
    w = rnd(p, K, N)
    wq = operands(tp, w, tiles=True)
    wv = [ref.values(o, N) for o in wq]
    nan = lambda *s: torch.full(s, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    # column: dX = sum_k dY_k A_k^T, dA_k = X^T dY_k
    x, dy = rnd(1, M, K)[0], rnd(p, M, N)
    (xt,), dyq, dyt = operands(tp, [x], True), operands(tp, dy), operands(tp, dy, True)
    ws = tp.workspace(tp.TP_OP_COL_BWD_FP8, p, M, N, K)
    dx, dw, dx2, dw2 = nan(M, K), [nan(K, N) for _ in range(p)], nan(M, K), [nan(K, N) for _ in range(p)]
    tp.tp_col_linear_bwd_fp8(xt, wq, dyq, dyt, dx, dw, ws)
    tp.tp_col_linear_bwd_fp8(None, wq, dyq, None, dx2, None, ws)
    tp.tp_col_linear_bwd_fp8(xt, None, None, dyt, None, dw2, ws)
    a, b = torch.cat([ref.values(o, N) for o in dyq], 1), torch.cat(wv, 1)
    assert_within(dx, a @ b.t(), ref.sum_error(a, b), "dX")
    assert torch.equal(dx, dx2)
    a = ref.values(xt, M)
    for k in range(p):
        b = ref.values(dyt[k], M)
        assert_within(dw[k], a @ b.t(), ref.sum_error(a, b), "dA")
        assert_within(dw2[k], a @ b.t(), ref.sum_error(a, b), "dA alone")
    # row: dX_k = dY A_k^T * GeLU'(H_k), dA_k = X_k^T dY
    x, dy, hh = rnd(p, M, K), rnd(1, M, N)[0], rnd(p, M, K)
    xt, (dyq,), (dyt,) = operands(tp, x, True), operands(tp, [dy]), operands(tp, [dy], True)
    ws = tp.workspace(tp.TP_OP_ROW_BWD_FP8, p, M, N, K)
    dx, dg, dw = [nan(M, K) for _ in range(p)], [nan(M, K) for _ in range(p)], [nan(K, N) for _ in range(p)]
    tp.tp_row_linear_bwd_fp8(xt, wq, dyq, dyt, dx, dw, ws)
    tp.tp_row_linear_bwd_fp8(None, wq, dyq, None, dg, None, ws, preact=hh)
    a, t = ref.values(dyq, N), ref.values(dyt, M)
    for k in range(p):
        want, slack = a @ wv[k].t(), ref.sum_error(a, wv[k])
        assert_within(dx[k], want, slack, "dX")
        s = ref.gelu_prime(hh[k].to(D))
        # GeLU' is within 1e-6 in fp32, and its product rounded once
        assert_within(dg[k], want * s, slack * s.abs() + (want.abs() + slack) * 2e-6, "dX GeLU'")
        b = ref.values(xt[k], M)
        assert_within(dw[k], b @ t.t(), ref.sum_error(b, t), "dA")
    assert tp.tp_get_device_status(ws) == tp.TP_OK


@pytest.mark.parametrize("p,M,N,K", [(2, 5, 264, 1000), (4, 300, 520, 640), (2, 1100, 2056, 1160)])
def test_whole_numbers_are_exact(tp, p, M, N, K):
    """Whole numbers up to 8 with a power of two a row: no product or sum is rounded, and the outputs are whole."""
    g = gen(M + N + K + 3)
    whole = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, w = [whole(M, K) for _ in range(p)], [whole(K, N) for _ in range(p)]
    scale = torch.pow(2.0, torch.randint(-20, 20, (M, 1), generator=g, device="cuda")).to(BF)
    xq, wq = operands(tp, [a * scale for a in x], False), operands(tp, w, True, True)
    y = torch.empty((M, N), dtype=BF, device="cuda")
    ws = tp.workspace(tp.TP_OP_ROW_FP8, p, M, N, K)
    tp.tp_row_linear_fwd_fp8(xq, wq, y, ws)
    want = sum(a.to(D) @ b.to(D) for a, b in zip(x, w)) * scale.to(D)
    assert torch.equal(y, want.to(BF))
    # a difference of the outputs is the product of a difference of the inputs: here exactly
    x2 = [a.clone() for a in x]
    x2[0][:, 0] += 1
    d = [b.to(D)[0] for b in w][0]
    want2 = want / scale.to(D) + d
    xq2 = operands(tp, [a * scale for a in x2], False)
    tp.tp_row_linear_fwd_fp8(xq2, wq, y, ws)
    assert torch.equal(y, (want2 * scale.to(D)).to(BF))


def test_empty_and_nan(tp):
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    x, w = operands(tp, [torch.ones((4, 128), dtype=BF, device="cuda")])[0], operands(tp, [torch.ones((128, 64), dtype=BF, device="cuda")], True)
    y = torch.full((0, 64), 1.0, dtype=BF, device="cuda")
    tp.tp_row_linear_fwd_fp8([tp.fp8_empty(0, 128)], w, y, ws)
    # an empty contraction: the bias and its activation
    b = torch.randn(64, generator=gen(5), device="cuda").to(BF)
    y = torch.full((4, 64), float("nan"), dtype=BF, device="cuda")
    tp.tp_row_linear_fwd_fp8([tp.fp8_empty(4, 0)], [tp.fp8_empty(64, 0)], y, ws, bias=b)
    assert torch.equal(y, b.expand(4, 64))
    # a NaN or infinity in a row stays in that row
    for bad in (float("nan"), float("inf")):
        a = torch.ones((200, 256), dtype=BF, device="cuda")
        a[3, 200] = bad
        y = torch.empty((200, 64), dtype=BF, device="cuda")
        tp.tp_row_linear_fwd_fp8(operands(tp, [a]), operands(tp, [torch.ones((256, 64), dtype=BF, device="cuda")], True), y, ws)
        assert bool(torch.isnan(y[3]).all()) and bool((y[:3] == 256).all()) and bool((y[4:] == 256).all())


def test_streams_graphs_and_workspaces(tp):
    """Two streams with a workspace each, and a captured call that is replayed on new inputs."""
    M, N, K = 40, 264, 1000
    g = gen(9)
    w = operands(tp, [torch.randn((K, N), generator=g, device="cuda").to(BF)], True, True)
    xs = [torch.randn((M, K), generator=g, device="cuda").to(BF) for _ in range(4)]
    want = []
    ws = tp.workspace(tp.TP_OP_ROW_FP8, 1, M, N, K)
    for x in xs:
        y = torch.empty((M, N), dtype=BF, device="cuda")
        tp.tp_row_linear_fwd_fp8(operands(tp, [x]), w, y, ws)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            own = tp.workspace(tp.TP_OP_ROW_FP8, 1, M, N, K)
            for x in xs[2 * i:2 * i + 2]:
                y = torch.empty((M, N), dtype=BF, device="cuda")
                tp.tp_row_linear_fwd_fp8(operands(tp, [x]), w, y, own)
                got.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, y, op = xs[0].clone(), torch.empty((M, N), dtype=BF, device="cuda"), tp.fp8_empty(M, K)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_fp8_pack([x], [op])
        tp.tp_row_linear_fwd_fp8([op], w, y, ws)
    for i in (2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_a_wait_that_runs_out_is_reported(tp):
    """A stage that is never handed over ends the call with a status, not with a hang."""
    for M, N in ((16, 264), (2100, 1500 // 8 * 8)):
        K = 1024
        x, w = operands(tp, [torch.ones((M, K), dtype=BF, device="cuda")]), operands(tp, [torch.ones((K, N), dtype=BF, device="cuda")], True)
        y = torch.empty((M, N), dtype=BF, device="cuda")
        ws = tp.workspace(tp.TP_OP_ROW_FP8, 1, M, N, K)
        try:
            assert tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 50) == tp.TP_OK and tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, 2) == tp.TP_OK
            tp.tp_row_linear_fwd_fp8(x, w, y, ws)
            assert tp.tp_get_device_status(ws) == tp.TP_ERR_DEVICE_TIMEOUT
        finally:
            tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 0)
            tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, -1)
        tp.tp_row_linear_fwd_fp8(x, w, y, ws)
        assert tp.tp_get_device_status(ws) == tp.TP_OK
        assert bool((y == K).all())


@pytest.mark.parametrize("p,K,N", [(2, 136, 264), (4, 1032, 2056)])
def test_gradients_of_empty_contractions_are_zero(tp, p, K, N):
    """Without tokens the weights' gradients are zero, without outputs the inputs'."""
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    nan = lambda *s: torch.full(s, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    dw, dx = [nan(K, N) for _ in range(p)], nan(0, K)
    weights = [tp.fp8_empty(K, N) for _ in range(p)]
    tp.tp_col_linear_bwd_fp8(tp.fp8_empty(K, 0), weights, [tp.fp8_empty(0, N) for _ in range(p)], [tp.fp8_empty(N, 0) for _ in range(p)], dx, dw, ws)
    assert all(bool((t == 0).all()) for t in dw)
    dw = [nan(K, N) for _ in range(p)]
    tp.tp_row_linear_bwd_fp8([tp.fp8_empty(K, 0) for _ in range(p)], weights, tp.fp8_empty(0, N), tp.fp8_empty(N, 0),
                             [nan(0, K) for _ in range(p)], dw, ws)
    assert all(bool((t == 0).all()) for t in dw)
    M = 300
    dx, dw = nan(M, K), [nan(K, 0) for _ in range(p)]
    tp.tp_col_linear_bwd_fp8(tp.fp8_empty(K, M), [tp.fp8_empty(K, 0) for _ in range(p)], [tp.fp8_empty(M, 0) for _ in range(p)],
                             [tp.fp8_empty(0, M) for _ in range(p)], dx, dw, ws)
    assert bool((dx == 0).all())
    assert tp.tp_get_device_status(ws) == tp.TP_OK
