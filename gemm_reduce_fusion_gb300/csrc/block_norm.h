// Launchers of the block boundary's backward kernels, one translation unit
// for each residual type and kind of norm so that they compile in parallel.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

#include "../../include/tp_fused.h"

namespace tpf {

struct NormParams;
struct NormBwdLaunch {
  int kind;               // WorkerKind
  int nv, threads;
  int cluster, ctas;      // CTAs of a cluster; CTAs, or clusters of them (lowered to what fits)
  size_t smem;
  bool groups;  // the gate has several rows
  bool full;    // nothing optional is left out
};

tp_status block_norm_bwd_run_bf16_rms(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_bf16_ln(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_f32_rms(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_f32_ln(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream);

// Clusters of `cluster` blocks that the current device holds at a time (asked
// once for each kernel and shape).
tp_status resident_clusters(const void* kernel, int cluster, int threads, size_t smem, int* out);

// Workspace of tp_block_norm_bwd: the column sums of every CTA.
size_t block_norm_bwd_workspace(int64_t M, int64_t h);

}  // namespace tpf
