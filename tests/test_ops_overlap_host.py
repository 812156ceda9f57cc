"""Overlaps that the operators around the sharded Linear refuse, on the host:
made-up pointers, nothing is launched.  A call that passes these checks goes
on to the device query, which fails without a GPU."""
import ctypes
import os
import subprocess

import pytest

import gemm_reduce_fusion_gb300 as tp
from test_block_ops_host import BAD, arr, at

L = tp._lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers would reach the GPU")


def desc(**d):
    return ctypes.byref(tp._NormDesc(**{**dict(post=1, pre=1, alpha=1.0, eps=1e-5), **d}))


def norm_fwd(x, z, y, n, p, M=8, res=0, **d):
    return L.tp_block_norm_fwd(arr(*x), arr(*z), arr(*y), arr(*n), desc(**d), p, M, 64, res, None)


def test_in_place_is_for_the_shard_itself_alone():
    a, b, c, d, e, f, g, h = (at(i) for i in range(8))
    z, n = [c, d], [e, f]
    # y[s] == x[s], for all shards or some
    for y in ([a, b], [a, g], [g, b], [g, h]):
        assert norm_fwd([a, b], z, y, n, 2) not in (tp.TP_OK, BAD)
        assert norm_fwd([a, b], z, y, n, 2, res=1) not in (tp.TP_OK, BAD)
    # another shard's x, any shard's z, or a vector, where a shard is written
    assert norm_fwd([a, a], z, [a, b], n, 2) == BAD
    assert norm_fwd([a, b], z, [b, a], n, 2) == BAD
    assert norm_fwd([a, b], z, [b, g], n, 2) == BAD
    assert norm_fwd([a, b], [c, a], [a, b], n, 2) == BAD
    assert norm_fwd([a, b], [a, c], [a, b], n, 2) == BAD
    assert norm_fwd([a], [c], [a], [e], 1, M=1, w_pre=a) == BAD
    assert norm_fwd([a], [c], [a], [e], 1, M=1, gate=a, gate_rows=1) == BAD
    assert norm_fwd([a + 16], [c], [a], [e], 1) == BAD


def test_in_place_in_the_backward_pass():
    z, y, dn, dy, dz, other = ([at(2 * i), at(2 * i + 1)] for i in range(6))
    ws, need = at(20), tp.tp_workspace_size(tp.TP_OP_BLOCK_NORM_BWD, 2, 8, 64, 0)

    def call(dx, dy=dy, y=y, dn=dn, **d):
        return L.tp_block_norm_bwd(arr(*z), arr(*y), arr(*dn), arr(*dy), arr(*dx), arr(*dz), desc(**d), None, 2, 8, 64, 0, 1, ws, need,
                                   None)
    for dx in (dy, other, [dy[0], other[1]]):
        assert call(dx) not in (tp.TP_OK, BAD)
    assert call(dy, dy=[dy[0], dy[0]]) == BAD
    assert call([dy[0], other[1]], dy=[dy[0], dy[0]]) == BAD
    assert call([dy[1], dy[0]]) == BAD
    assert call(dy, y=dy) == BAD and call(dy, dn=dy) == BAD and call(dy, y=[y[0], dy[0]]) == BAD


def test_the_restored_part_of_a_workspace_overlaps_no_operand():
    P, M, N, K = 2, 8, 64, 32
    q, e, w, dy, dx, dw = ([at(2 * i), at(2 * i + 1)] for i in range(6))
    ws = at(20)

    def need(op):
        return tp.tp_workspace_size(op, P, M, N, K)

    def col(w=w, dy=dy):
        return L.tp_col_linear_bwd_ckpt(q[0], e[0], arr(*w), arr(*dy), dx[0], arr(*dw), None, P, M, N, K, 0, 0, ws, need(10), None)

    def row(w=w, dy=dy):
        return L.tp_row_linear_bwd_ckpt(arr(*q), arr(*e), arr(*w), dy[0], arr(*dx), arr(*dw), None, 2, P, M, N, K, 0, 0, ws, need(11), None)

    def ag(w=w, dy=dy):
        return L.tp_ag_matmul_bwd_ckpt(arr(*q), arr(*e), arr(*w), arr(*dy), arr(*dx), arr(*dw), None, P, M, N, K, 0, 0, ws, need(12), None)

    def rs(w=w, dy=dy):
        return L.tp_row_linear_bwd_reducescatter_ckpt(arr(*q), arr(*e), arr(*w), arr(*dy), arr(*dx), arr(*dw), None, 2, P, M, N, K, 0, 0,
                                                      ws, need(13), None)
    for call, op in ((col, 10), (row, 11), (ag, 12), (rs, 13)):
        assert call() not in (tp.TP_OK, BAD)
        last = ws + need(op) - 16  # the last restored tensor's end
        assert call(w=[w[0], last]) == BAD and call(w=[ws + 256, w[1]]) == BAD, op
        assert call(dy=[last, dy[1]]) == BAD, op
        if call is not row:
            assert call(dy=[dy[0], last]) == BAD, op


def test_a_full_list_of_ranges_refuses(tmp_path):
    """What a list of ranges has no room for counts as an overlap."""
    src = tmp_path / "ranges.cpp"
    src.write_text('''
#include "host_util.h"
int main() {
  tpf::RangeList outs, few, many;
  outs.push_back({reinterpret_cast<void*>(1 << 20), 16});
  for (int i = 0; i < 64; ++i) few.push_back({reinterpret_cast<void*>((2 << 20) + 32 * i), 16});
  for (int i = 0; i < 65; ++i) many.push_back({reinterpret_cast<void*>((2 << 20) + 32 * i), 16});
  if (tpf::any_overlap(outs, few)) return 1;
  if (!tpf::any_overlap(outs, many) || !tpf::any_overlap(many, outs)) return 2;
  return 0;
}
''')
    from gemm_reduce_fusion_gb300.build import nvcc
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    csrc = os.path.join(ROOT, "gemm_reduce_fusion_gb300", "csrc")
    exe = tmp_path / "ranges"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, "-I", cuda, str(src), "-o", str(exe)], check=True, capture_output=True)
    assert subprocess.run([str(exe)]).returncode == 0
