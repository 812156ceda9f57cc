"""The block boundary's kernels where a worker (a warp, a thread block or a
cluster of them) has several rows: the prefetch of the next row, the reduction
buffers that take turns, the walk over shards, column sums of several rows and
gate groups that end inside a worker's rows and between workers.  Bounds as in
test_gpu_block_norm.py."""
import pytest
import torch

from test_gpu_block_norm import BF, F32, call_args, cat, check_bwd, check_fwd, make, nan_like, shards

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


# rows for every form's resident thread blocks several times over
FWD = [(4, 6000, 1160), (2, 3000, 4096), (8, 1600, 12288), (1, 900, 16384)]


@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("p,M,h", FWD)
def test_forward(tp, p, M, h, res):
    check_fwd(tp, p, M, h, "rms", "rms", 1, res)
    check_fwd(tp, p, M, h, "layer", "layer", M, res)


# h > 4096: clusters of two thread blocks (up to 8192) and of four
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("h", [4104, 6152, 8200, 12288])
def test_backward_by_clusters(tp, h, res):
    M = 700
    check_bwd(tp, 1, M, h, "rms", "rms", 1, res)
    check_bwd(tp, 4, M, h, "layer", "layer", 1, res)
    check_bwd(tp, 2, M, h, "none", "layer", 0, res, weights=False)
    check_bwd(tp, 7, M, h, "layer", "rms", 0, res, BF, has_dy=False)


@pytest.mark.parametrize("groups", [2, 7, 100, 350, 700])
@pytest.mark.parametrize("h", [4104, 12288])
def test_gate_groups_that_end_inside_and_between_clusters(tp, h, groups):
    check_bwd(tp, 2, 700, h, "rms", "rms", groups, BF)
    check_bwd(tp, 1, 700, h, "layer", "layer", groups, F32)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("h", [1160, 4104, 12288])
def test_the_same_bits_every_time(tp, h, kind):
    p, M = 4, 1200
    x, z, dn, dy, d = make(M, h, kind, kind, 3, BF)
    a, xs, zs, dns, dys = call_args(tp, d), shards(x, p), shards(z, p), shards(dn, p), shards(dy, p)
    names = ["dw_post", "dw_pre"] + (["db_post", "db_pre"] if kind == "layer" else [])
    first = None
    for _ in range(5):
        ys, ns, dx, dz = nan_like(xs), nan_like(xs, BF), nan_like(xs), nan_like(xs, BF)
        g = {k: torch.full((h,), float("nan"), device="cuda") for k in names}
        g["dgate"] = torch.full((3, h), float("nan"), device="cuda")
        tp.tp_block_norm_fwd(xs, zs, ys, ns, **a)
        tp.tp_block_norm_bwd(zs, ys, dns, dys, dx, dz, tp.workspace(tp.TP_OP_BLOCK_NORM_BWD, p, M, h, 0), **g, **a)
        got = [cat(t) for t in (ys, ns, dx, dz)] + [t.cpu() for t in g.values()]
        first = first or got
        assert all(torch.equal(s, t) for s, t in zip(first, got))
