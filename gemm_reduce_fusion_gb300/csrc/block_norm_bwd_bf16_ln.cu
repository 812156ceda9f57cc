#include "block_norm_bwd.cuh"

namespace tpf {

tp_status block_norm_bwd_run_bf16_ln(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  return dispatch_bwd_groups<false, true>(P, L, stream);
}

}  // namespace tpf
