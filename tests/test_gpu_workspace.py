"""What calls that share a workspace may leave in it for one another: the
counters of a sliced last wave never mistake other data for a count, and the
calls around the sharded Linear keep off them."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


# 84 tiles of 256 x 256 for 76 clusters: the last 8 run as slices.  Every
# counter starts as data: the first launch's number above the low 16 bits, as
# four bfloat16 values of a restored activation can make up.
FORGED = """
import torch
import gemm_reduce_fusion_gb300 as tp
p, M, N, K = 2, 3584, 1536, 512
g = torch.Generator().manual_seed(1)
x = [torch.randint(-3, 4, (M, K), generator=g).to(torch.bfloat16).cuda() for _ in range(p)]
w = [torch.randint(-3, 4, (K, N), generator=g).to(torch.bfloat16).cuda() for _ in range(p)]
want = sum(a.double() @ b.double() for a, b in zip(x, w))
ws = tp.workspace(tp.TP_OP_ROW_AR, p, M, N, K)
assert ws.numel() > 256 + 8 * 2 * 8 * 8, "no slices"
words = ws[256:256 + 8 * 2 * 8 * 8].view(torch.int64)
for launch in range(1, 9):
    words.fill_(launch << 16 | launch % 4)
    y = torch.full((M, N), float("nan"), device="cuda")
    tp.tp_row_linear_fwd_allreduce(x, w, [y], ws)
    assert tp.tp_get_device_status(ws) == tp.TP_OK
    assert torch.equal(y.double(), want), launch
"""


def test_data_in_the_workspace_is_not_taken_for_a_count(tp):
    """A workspace's second use finds the first one's data where a sliced
    launch counts.  In a process of its own, whose launches are numbered from 1."""
    r = subprocess.run([sys.executable, "-c", FORGED], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT}, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


COUNTERS = 75 * 2 * 8 * 8  # of the largest last wave: tiles x CTAs x epilogue warps, 8 bytes each


def test_the_calls_around_the_linear_keep_off_the_counters(tp):
    """Column sums, 4-bit partials and restored activations lie behind them."""
    def check(ws, what):
        assert tp.tp_get_device_status(ws) == tp.TP_OK
        assert bool((ws[256:256 + COUNTERS] == 0x5A).all()), what

    def space(op, p, M, N, K):
        n = max(tp.tp_workspace_size(op, p, M, N, K), 256 + COUNTERS)
        ws = torch.full(((n + 15) // 16 * 16,), 0x5A, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        return ws

    rnd = lambda *s: torch.randn(*s, device="cuda").to(BF)  # noqa: E731
    for h in (520, 1160, 8192):
        M = 300
        ws = space(tp.TP_OP_BLOCK_NORM_BWD, 1, M, h, 0)
        t = [rnd(M, h) for _ in range(6)]
        tp.tp_block_norm_bwd([t[0]], [t[1]], [t[2]], [t[3]], [t[4]], [t[5]], ws, post=tp.TP_NORM_RMS, pre=tp.TP_NORM_RMS,
                             gate=rnd(3, h), dw_pre=torch.empty(h, device="cuda"), dgate=torch.empty(3, h, device="cuda"))
        check(ws, "norm backward")
    p, K, N = 4, 4096, 2048
    q, s = ([torch.zeros(t, dtype=d, device="cuda") for _ in range(p)] for t, d in zip(tp.w4_shapes(K, N, 128), (torch.uint8, BF)))
    for M in (1, 48):
        ws = space(tp.TP_OP_COL_W4, p, M, N, K)
        tp.tp_col_linear_fwd_w4(rnd(M, K), q, s, [rnd(M, N) for _ in range(p)], ws)
        check(ws, "4 bits, column")
        ws = space(tp.TP_OP_ROW_W4, p, M, N, K)
        tp.tp_row_linear_fwd_w4([rnd(M, K) for _ in range(p)], q, s, rnd(M, N), ws)
        check(ws, "4 bits, row")
    p, M, N, K = 2, 300, 520, 200  # products too small for partials of their own
    qs, es = tp.ckpt_shapes(M, K)
    q = [torch.ones(qs, dtype=torch.int8, device="cuda") for _ in range(p)]
    e = [torch.full(es, 120, dtype=torch.uint8, device="cuda") for _ in range(p)]
    w, dw = [rnd(K, N) for _ in range(p)], [rnd(K, N) for _ in range(p)]
    for base, op in ((tp.TP_OP_COL_BWD, tp.TP_OP_COL_BWD_CKPT), (tp.TP_OP_ROW_BWD, tp.TP_OP_ROW_BWD_CKPT),
                     (tp.TP_OP_AG_MM_BWD, tp.TP_OP_AG_MM_BWD_CKPT), (tp.TP_OP_ROW_RS_BWD, tp.TP_OP_ROW_RS_BWD_CKPT)):
        assert tp.tp_workspace_size(base, p, M, N, K) == 256
        ws = space(op, p, M, N, K)
        if op == tp.TP_OP_COL_BWD_CKPT:
            tp.tp_col_linear_bwd_ckpt(q[0], e[0], w, [rnd(M, N) for _ in range(p)], rnd(M, K), dw, ws)
        elif op == tp.TP_OP_ROW_BWD_CKPT:
            tp.tp_row_linear_bwd_ckpt(q, e, w, rnd(M, N), [rnd(M, K) for _ in range(p)], dw, ws)
        elif op == tp.TP_OP_AG_MM_BWD_CKPT:
            half = [t[:M // p].contiguous() for t in q], [t[:M // p].contiguous() for t in e]
            tp.tp_ag_matmul_bwd_ckpt(*half, w, [rnd(M, N) for _ in range(p)], [rnd(M // p, K) for _ in range(p)], dw, ws)
        else:
            tp.tp_row_linear_bwd_reducescatter_ckpt(q, e, w, [rnd(M // p, N) for _ in range(p)], [rnd(M, K) for _ in range(p)], dw, ws)
        check(ws, op)
