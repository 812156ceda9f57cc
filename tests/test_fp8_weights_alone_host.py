"""The 8-bit row backward call for the weights' gradients alone, on the host."""
import gemm_reduce_fusion_gb300 as tp
from test_binding_checks import WS, lib, zs  # noqa: F401
from test_fp8_host import K, M, N, op, ops, p


def test_weights_alone_take_no_preactivation(lib):  # noqa: F811
    """H is read for the inputs' gradients: with the weights' alone it may be given and is not looked at."""
    tp.tp_row_linear_bwd_fp8(ops(p, K, M), None, None, op(N, M), None, zs(p, K, N), WS, preact=zs(p, M, K), stream=0)
    assert len(lib.calls) == 1
