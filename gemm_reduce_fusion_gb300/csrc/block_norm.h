// Launchers of the block boundary's backward kernels, one translation unit
// for each residual type and kind of norm so that they compile in parallel.
#pragma once
#include <cuda_runtime.h>

#include "../../include/tp_fused.h"

namespace tpf {

struct NormParams;
struct NormBwdLaunch {
  bool warp;
  int nv, threads, ctas;
  bool groups, ln;
};

tp_status block_norm_bwd_run_bf16_rms(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_bf16_ln(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_f32_rms(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream);
tp_status block_norm_bwd_run_f32_ln(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream);

// Workspace of tp_block_norm_bwd: the column sums of every CTA.
size_t block_norm_bwd_workspace(int64_t M, int64_t h);

}  // namespace tpf
