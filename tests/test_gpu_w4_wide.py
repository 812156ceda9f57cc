"""The sharded Linear with 4-bit weights for more tokens on large weights
(tcgen05): against the definition in 64 bits, with the library's bounds (1e-5
of the largest value for fp32 outputs, 5e-3 for bf16).  The shapes have eight
stages (256 columns x 128 rows) an SM, the least that takes this path, with
columns, rows and scale groups that end inside a tile."""
import pytest
import torch

import ops_ref as ref
from gpu_util import assert_close, host_f64, poisoned
from test_gpu_w4 import random_w4

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


_weights = {}


def weights(tp, p, K, N, G):
    """(q, s, values) of each shard, made once."""
    if (p, K, N, G) not in _weights:
        _weights.clear()
        g = torch.Generator().manual_seed(K + N + G)
        w = [random_w4(tp, K, N, G, g, garbage=True) for _ in range(p)]
        _weights[p, K, N, G] = [a.cuda() for a, _ in w], [a.cuda() for _, a in w], [ref.w4_value(q, s, K, N, G).float() for q, s in w]
    return _weights[p, K, N, G]


SHAPES = [(8, 2056, 2056), (1, 155400, 136), (3, 16, 57000)]  # p, N, K; blocks that runs share, that one run has whole, that many share


@pytest.mark.parametrize("p,N,K", SHAPES)
@pytest.mark.parametrize("G,M", [(32, 49), (32, 64), (64, 17), (64, 47), (128, 24), (128, 33), (128, 64)])
def test_row(tp, p, N, K, G, M):
    q, s, w = weights(tp, p, K, N, G)
    g = torch.Generator().manual_seed(M)
    x = [torch.randn(M, K, generator=g).to(BF) for _ in range(p)]
    want = sum(a.to(D) @ v.to(D) for a, v in zip(x, w))
    b = torch.randn(N, generator=g).to(BF)
    ws, xd = tp.workspace(tp.TP_OP_ROW_W4, p, M, N, K), [a.cuda() for a in x]
    for f32 in (True, False):
        y, again = poisoned((M, N), f32), poisoned((M, N), f32)
        tp.tp_row_linear_fwd_w4(xd, q, s, y, ws, group=G)
        assert_close(host_f64(y), want.numpy(), f32, "Y")
        tp.tp_row_linear_fwd_w4(xd, q, s, again, ws, group=G)
        assert torch.equal(y, again), "the sum's order is fixed"
    tp.tp_row_linear_fwd_w4(xd, q, s, y, ws, group=G, bias=b.cuda())
    assert_close(host_f64(y), (want + b.to(D)).numpy(), False, "Y + b")
    assert tp.tp_get_device_status(ws) == tp.TP_OK


@pytest.mark.parametrize("p,N,K", SHAPES[:2])
@pytest.mark.parametrize("G,M", [(32, 64), (64, 17), (128, 48)])
def test_column(tp, p, N, K, G, M):
    q, s, w = weights(tp, p, K, N, G)
    g = torch.Generator().manual_seed(M + 1)
    x = torch.randn(M, K, generator=g).to(BF)
    b = [torch.randn(N, generator=g).to(BF) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_COL_W4, p, M, N, K)
    for f32 in (True, False):
        y = [poisoned((M, N), f32) for _ in range(p)]
        tp.tp_col_linear_fwd_w4(x.cuda(), q, s, y, ws, group=G, epi=tp.TP_EPI_GELU, bias=[a.cuda() for a in b])
        for k in range(p):
            assert_close(host_f64(y[k]), ref.gelu(x.to(D) @ w[k].to(D) + b[k].to(D)).numpy(), f32, f"Y_{k}")


def test_a_token_keeps_its_infinities_to_itself(tp):
    p, N, K = SHAPES[0]
    M, G = 40, 128
    q, s, w = weights(tp, p, K, N, G)
    x = [torch.randn(M, K, generator=torch.Generator().manual_seed(5)).to(BF) for _ in range(p)]
    x[0][3, 7], x[p - 1][39, K - 1] = float("inf"), float("nan")
    y = poisoned((M, N), True)
    tp.tp_row_linear_fwd_w4([a.cuda() for a in x], q, s, y, tp.workspace(tp.TP_OP_ROW_W4, p, M, N, K), group=G)
    got, clean = y.cpu(), [i for i in range(M) if i not in (3, 39)]
    assert not torch.isfinite(got[3]).any() and torch.isnan(got[39]).all()
    want = sum(a.to(D) @ v.to(D) for a, v in zip(x, w))
    assert_close(got[clean].to(D).numpy(), want[clean].numpy(), True, "the other tokens")


def test_a_wait_that_runs_out_is_reported_and_the_next_call_works(tp):
    p, N, K = SHAPES[0]
    M, G = 33, 64
    q, s, w = weights(tp, p, K, N, G)
    x = [torch.randn(M, K, generator=torch.Generator().manual_seed(6)).to(BF) for _ in range(p)]
    xd, ws, y = [a.cuda() for a in x], tp.workspace(tp.TP_OP_ROW_W4, p, M, N, K), poisoned((M, N), True)
    assert tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 200) == tp.TP_OK
    assert tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, 2) == tp.TP_OK
    try:
        tp.tp_row_linear_fwd_w4(xd, q, s, y, ws, group=G)
        status = tp.tp_get_device_status(ws)
    finally:
        tp.tp_debug_set(tp.TP_DEBUG_DROP_LOAD, -1)
        tp.tp_debug_set(tp.TP_DEBUG_TIMEOUT_MS, 0)
    assert status == tp.TP_ERR_DEVICE_TIMEOUT
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    tp.tp_row_linear_fwd_w4(xd, q, s, y, ws, group=G)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    assert_close(host_f64(y), sum(a.to(D) @ v.to(D) for a, v in zip(x, w)).numpy(), True, "after recovery")
