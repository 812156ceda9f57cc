"""8-bit activation checkpoints: packing and restoring bit for bit against the
definition, and the backward calls on them against the fp64 oracle.

Packing and restoring have no tolerance: every step is an exact scaling by a
power of two and one rounding to a whole number.  GeLU of a restored value is
rounded to bf16 once (2^-8 of its size, plus 1e-6 for the fp32 function).
The backward calls keep the library's bound of 5e-3 of the largest value."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import oracle
import synth
from gpu_util import assert_close, dev, host_f64, poisoned

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


def pack(tp, xs):
    M, N = xs[0].shape
    qs, es = tp.ckpt_shapes(M, N)
    q = [torch.full(qs, 77, dtype=torch.int8, device="cuda") for _ in xs]
    e = [torch.full(es, 200, dtype=torch.uint8, device="cuda") for _ in xs]
    tp.tp_ckpt_pack(xs, q, e)
    return q, e


def same(a, b):
    """Bit for bit, any NaN like any other."""
    a, b = a.cpu(), b.cpu()
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# N: part of a group, whole groups, groups and a rest; M: one row to many
SHAPES = [(1, 1, 8), (2, 3, 24), (1, 1, 32), (3, 5, 40), (1, 7, 1000), (8, 33, 96), (2, 129, 2048), (1, 1025, 136), (4, 300, 4104)]


@pytest.mark.parametrize("p,M,N", SHAPES)
def test_pack_and_unpack_are_exact(tp, p, M, N):
    g = torch.Generator().manual_seed(M * N)
    xs = [torch.randn(M, N, generator=g).to(BF) for _ in range(p)]
    for x in xs:  # sizes over the whole exponent range, zeros, and halves that tie
        x *= (2.0 ** torch.randint(-60, 60, (M, 1), generator=g).float()).to(BF)
        x[torch.rand(M, N, generator=g) < 0.05] = 0
        x[:, : N // 2] = (x[:, : N // 2].float() * 8).round().to(BF) / 8
    q, e = pack(tp, [x.cuda() for x in xs])
    y = [torch.full((M, N), float("nan"), dtype=BF, device="cuda") for _ in xs]
    tp.tp_ckpt_unpack(q, e, y)
    z = [torch.full((M, N), float("nan"), dtype=BF, device="cuda") for _ in xs]
    tp.tp_ckpt_unpack(q, e, z, epi=tp.TP_EPI_GELU)
    for i, x in enumerate(xs):
        qr, er = ref.ckpt_pack(x)
        assert torch.equal(q[i].cpu(), qr) and torch.equal(e[i].cpu(), er)
        v = ref.ckpt_value(qr, er)
        assert torch.equal(v.to(BF).to(D), v), "a restored value is a bf16"
        assert same(y[i], v.to(BF))
        want = ref.gelu(v)
        assert ((z[i].cpu().to(D) - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6 * v.abs().clamp(max=8.0)).all()


def test_every_exponent_and_the_edges_of_a_group(tp):
    """Largest values from the smallest subnormal to the largest bf16, every
    mantissa of the top value, and quotients that lie half-way."""
    rows = []
    for bits in list(range(1, 0x100)) + list(range(0x3F80, 0x4080)) + list(range(0x7E00, 0x7F80)):
        top = torch.tensor([bits], dtype=torch.int16).view(BF)
        row = torch.zeros(32, dtype=BF)
        row[0] = top
        row[1:] = (top.float() * torch.arange(1, 32) / 62).to(BF)
        row[2::3] *= -1
        rows.append(row)
    x = torch.stack(rows)
    q, e = pack(tp, [x.cuda()])
    qr, er = ref.ckpt_pack(x)
    assert torch.equal(q[0].cpu(), qr) and torch.equal(e[0].cpu(), er)
    y = torch.empty_like(x, device="cuda")
    tp.tp_ckpt_unpack(q, e, [y])
    assert same(y, ref.ckpt_value(qr, er).to(BF))


@pytest.mark.parametrize("N", [64, 72])
def test_infinities_and_nan_mark_their_group_alone(tp, N):
    x = torch.randn(6, N, generator=torch.Generator().manual_seed(1)).to(BF)
    x[1, 3], x[2, 40], x[4, N - 1], x[5] = float("inf"), float("nan"), float("-inf"), 0
    q, e = pack(tp, [x.cuda()])
    qr, er = ref.ckpt_pack(x)
    assert torch.equal(q[0].cpu(), qr) and torch.equal(e[0].cpu(), er)
    y, z = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    tp.tp_ckpt_unpack(q, e, [y])
    tp.tp_ckpt_unpack(q, e, [z], epi=tp.TP_EPI_GELU)
    v = ref.ckpt_value(qr, er)
    assert same(y, v.to(BF)) and torch.equal(torch.isnan(z.cpu()), torch.isnan(v))
    assert torch.isnan(v).sum() == 2 * 32 + (32 if N % 32 == 0 else N % 32)


def test_empty_and_other_streams(tp):
    for M, N in ((0, 64), (5, 0)):
        x = torch.empty((M, N), dtype=BF, device="cuda")
        q, e = pack(tp, [x])
        tp.tp_ckpt_unpack(q, e, [torch.empty_like(x)])
    x = torch.randn(300, 520, device="cuda").to(BF)
    q, e = pack(tp, [x])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        q2, e2 = pack(tp, [x])
    st.synchronize()
    assert torch.equal(q[0], q2[0]) and torch.equal(e[0], e2[0])


# ------------------------------------------------------------------ the backward calls

def saved(tp, M, K, n, seed):
    """Packed tensors and the bf16 bit patterns they stand for."""
    xs = [dev(synth.normal_bf16((M, K), synth.seed_for(seed, i))) for i in range(n)]
    q, e = pack(tp, xs)
    bits = [ref.ckpt_value(a.cpu(), b.cpu()).to(BF).view(torch.int16).numpy().view(np.uint16) for a, b in zip(q, e)]
    return q, e, bits


def normals(shape, c, t, sigma=1.0):
    return synth.normal_bf16(shape, synth.seed_for(c, t), sigma)


CASES = [(1, 1, 8, 8), (2, 300, 264, 136), (4, 64, 256, 512), (2, 1030, 520, 1160), (3, 96, 40, 72)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("p,M,N,K", CASES)
def test_column_backward(tp, p, M, N, K, f32):
    q, e, x = saved(tp, M, K, 1, 120)
    w, dy = [normals((K, N), 121, k, 0.05) for k in range(p)], [normals((M, N), 122, k) for k in range(p)]
    dx, dw, db = poisoned((M, K), f32), [poisoned((K, N), f32) for _ in range(p)], [poisoned((N,), f32) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_COL_BWD_CKPT, p, M, N, K, out_dtype=tp.TP_FP32 if f32 else tp.TP_BF16)
    tp.tp_col_linear_bwd_ckpt(q[0], e[0], [dev(a) for a in w], [dev(a) for a in dy], dx, dw, ws, db=db)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    assert_close(host_f64(dx), oracle.col_bwd_dx(w, dy), f32, "dX")
    for k, r in enumerate(oracle.col_bwd_dw(x[0], dy)):
        assert_close(host_f64(dw[k]), r, f32, f"dA_{k}")
        assert_close(host_f64(db[k]), oracle.bias_grad(dy[k]), f32, f"db_{k}")


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("p,M,N,K", CASES)
def test_row_backward(tp, p, M, N, K, act):
    q, e, h = saved(tp, M, K, p, 123)
    w, dy = [normals((K, N), 124, k, 0.05) for k in range(p)], normals((M, N), 125, 0)
    dx, dw, db = [poisoned((M, K)) for _ in range(p)], [poisoned((K, N)) for _ in range(p)], poisoned((N,))
    ws = tp.workspace(tp.TP_OP_ROW_BWD_CKPT, p, M, N, K)
    epi = tp.TP_EPI_DGELU if act else tp.TP_EPI_NONE
    tp.tp_row_linear_bwd_ckpt(q, e, [dev(a) for a in w], dev(dy), dx, dw, ws, epi=epi, db=db)
    x = [oracle.round_bf16(ref.gelu(torch.from_numpy(oracle.widen(a))).numpy()) for a in h] if act else h
    for k, r in enumerate(oracle.row_bwd_dx(w, dy, preacts=h if act else None)):
        assert_close(host_f64(dx[k]), r, False, f"dX_{k}")
    for k, r in enumerate(oracle.row_bwd_dw(x, dy)):
        assert_close(host_f64(dw[k]), r, False, f"dA_{k}")
    assert_close(host_f64(db), oracle.bias_grad(dy), False, "db")
    # one product alone gives the same bits
    d2 = [poisoned((M, K)) for _ in range(p)]
    tp.tp_row_linear_bwd_ckpt(q, e, [dev(a) for a in w], dev(dy), d2, None, ws, epi=epi)
    d3 = [poisoned((K, N)) for _ in range(p)]
    tp.tp_row_linear_bwd_ckpt(q, e, [dev(a) for a in w], dev(dy), None, d3, ws, epi=epi)
    for k in range(p):
        assert_close(host_f64(d2[k]), host_f64(dx[k]), False, "dX alone")
        assert_close(host_f64(d3[k]), host_f64(dw[k]), False, "dA alone")


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("p,Mp,N,K", [(2, 150, 264, 136), (4, 64, 256, 512), (1, 5, 8, 40)])
def test_sequence_parallel_backward(tp, p, Mp, N, K, act):
    M = Mp * p
    q, e, x = saved(tp, Mp, K, p, 126)
    w, dy = [normals((K, N), 127, k, 0.05) for k in range(p)], [normals((M, N), 128, k) for k in range(p)]
    dx, dw, db = [poisoned((Mp, K)) for _ in range(p)], [poisoned((K, N)) for _ in range(p)], [poisoned((N,)) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_AG_MM_BWD_CKPT, p, M, N, K)
    tp.tp_ag_matmul_bwd_ckpt(q, e, [dev(a) for a in w], [dev(a) for a in dy], dx, dw, ws, db=db)
    for s, r in enumerate(oracle.ag_matmul_bwd_dx(w, dy)):
        assert_close(host_f64(dx[s]), r, False, f"dX_{s}")
    for k, r in enumerate(oracle.ag_matmul_bwd_dw(x, dy)):
        assert_close(host_f64(dw[k]), r, False, f"dA_{k}")
        assert_close(host_f64(db[k]), oracle.bias_grad(dy[k]), False, f"db_{k}")
    q, e, h = saved(tp, M, K, p, 129)
    dy = [normals((Mp, N), 130, s) for s in range(p)]
    dx, dw = [poisoned((M, K)) for _ in range(p)], [poisoned((K, N)) for _ in range(p)]
    ws = tp.workspace(tp.TP_OP_ROW_RS_BWD_CKPT, p, M, N, K)
    tp.tp_row_linear_bwd_reducescatter_ckpt(q, e, [dev(a) for a in w], [dev(a) for a in dy], dx, dw, ws,
                                            epi=tp.TP_EPI_DGELU if act else tp.TP_EPI_NONE)
    z = [oracle.round_bf16(ref.gelu(torch.from_numpy(oracle.widen(a))).numpy()) for a in h] if act else h
    for k, r in enumerate(oracle.row_rs_bwd_dx(w, dy, preacts=h if act else None)):
        assert_close(host_f64(dx[k]), r, False, f"dX_{k}")
    for k, r in enumerate(oracle.row_rs_bwd_dw(z, dy)):
        assert_close(host_f64(dw[k]), r, False, f"dA_{k}")
