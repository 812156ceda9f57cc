"""An infinity among the vectors of the block boundary stays in its column."""
import pytest
import torch

from test_gpu_block_norm import BF, F32, call_args, make, nan_like

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["w_post", "gate"])
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("h", [8, 264, 1032, 1160, 4104])
def test_an_infinite_weight_of_the_last_column(h, res, where):
    """y is infinite in that column alone.  The row's mean square is then
    infinite and its reciprocal root zero: n = y * 0 is zero in the other
    columns and NaN in that one."""
    import gemm_reduce_fusion_gb300 as tp
    x, z, _, _, d = make(5, h, "rms", "rms", 1, res)
    clean = [t.cuda() for t in (x, z)]
    y0 = nan_like([clean[0]])
    tp.tp_block_norm_fwd([clean[0]], [clean[1]], y0, nan_like([clean[0]], BF), **call_args(tp, d))
    d[where].view(-1)[h - 1] = float("inf")
    ys, ns = nan_like([clean[0]]), nan_like([clean[0]], BF)
    tp.tp_block_norm_fwd([clean[0]], [clean[1]], ys, ns, **call_args(tp, d))
    y, n = ys[0].cpu(), ns[0].cpu()
    assert torch.equal(y[:, :-1], y0[0].cpu()[:, :-1]) and torch.isinf(y[:, -1]).all()
    assert bool((n[:, :-1] == 0).all()) and torch.isnan(n[:, -1]).all()
