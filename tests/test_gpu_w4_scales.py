"""The sharded Linear with 4-bit weights over the whole range of scales: packed
from weights up to the largest bfloat16, and down to the smallest scale, with
tokens that bring the products back into range.  Bounds as in test_gpu_w4.py."""
import pytest
import torch

import ops_ref as ref
from gpu_util import assert_close, host_f64, poisoned

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


# one to 64 tokens on mma.sync, and the tcgen05 kernel (17 tokens or more, eight stages an SM)
@pytest.mark.parametrize("power", [127, -125])
@pytest.mark.parametrize("M,N,K,G", [(1, 72, 264, 32), (5, 264, 200, 64), (16, 40, 520, 128), (24, 264, 200, 128), (48, 72, 264, 32),
                                     (64, 264, 136, 64), (33, 16384, 2560, 128), (64, 16384, 2560, 32)])
def test_every_scale(tp, M, N, K, G, power):
    g = torch.Generator().manual_seed(M)
    w = ((torch.rand(K, N, generator=g, dtype=D) * 3.98 - 1.99) * 2.0 ** power).to(BF)
    x = (torch.randn(M, K, generator=g) * 2.0 ** (-60 if power > 0 else 60)).to(BF)
    assert torch.isfinite(w.float()).all() and (w != 0).any(0).all()
    q, s = (torch.empty(t, dtype=d, device="cuda") for t, d in zip(tp.w4_shapes(K, N, G), (torch.uint8, BF)))
    tp.tp_w4_pack([w.cuda()], [q], [s], group=G)
    want = x.to(D) @ ref.w4_value(q, s, K, N, G)
    b = torch.zeros(N, dtype=BF, device="cuda")
    for f32 in (True, False):
        y = poisoned((M, N), f32)
        tp.tp_row_linear_fwd_w4([x.cuda()], [q], [s], y, tp.workspace(tp.TP_OP_ROW_W4, 1, M, N, K), group=G, bias=b)
        assert_close(host_f64(y), want.numpy(), f32, "row")
        y = poisoned((M, N), f32)
        tp.tp_col_linear_fwd_w4(x.cuda(), [q], [s], [y], tp.workspace(tp.TP_OP_COL_W4, 1, M, N, K), group=G)
        assert_close(host_f64(y), want.numpy(), f32, "column")
