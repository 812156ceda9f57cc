#include "block_norm_bwd.cuh"

namespace tpf {

tp_status block_norm_bwd_run_f32_ln(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  return dispatch_bwd_groups<true, true>(P, L, stream);
}

}  // namespace tpf
