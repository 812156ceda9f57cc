"""Products of several ranks without a contraction: what is added to nothing is
the bias, or zero, on every kind of tile."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("p", [2, 8])
@pytest.mark.parametrize("M,N", [(1, 8), (33, 264), (100, 520), (300, 136), (2049, 2056)])  # rows as N, as M, pairs
def test_no_contraction(p, M, N):
    import gemm_reduce_fusion_gb300 as tp
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    b = torch.randn(N, generator=torch.Generator(device="cuda").manual_seed(M), device="cuda").to(BF)
    none = lambda n, rows: [tp.fp8_empty(rows, 0) for _ in range(n)]  # noqa: E731
    for bias in (None, b):
        y = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
        tp.tp_row_linear_fwd_fp8(none(p, M), none(p, N), y, ws, bias=bias)
        assert torch.equal(y, (torch.zeros_like(b) if bias is None else b).expand(M, N))
    y = [torch.full((M, N), float("nan"), dtype=BF, device="cuda") for _ in range(p)]
    tp.tp_col_linear_fwd_fp8(none(1, M)[0], none(p, N), y, ws, bias=[b] * p)
    assert all(torch.equal(t, b.expand(M, N)) for t in y)
    dx = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
    tp.tp_col_linear_bwd_fp8(None, none(p, N), none(p, M), None, dx, None, ws)
    assert bool((dx == 0).all())
    assert tp.tp_get_device_status(ws) == tp.TP_OK
