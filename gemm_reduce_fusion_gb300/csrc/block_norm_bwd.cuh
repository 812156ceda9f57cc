// Launch of block_norm_bwd_kernel<..., RES32, LN, ...> for one residual type
// and kind of norm; included once by each of block_norm_bwd_*.cu.
#pragma once
#include "block_norm.cuh"
#include "block_norm.h"
#include "host_util.h"

namespace tpf {

template <int NV, bool RES32, bool LN, bool GROUPS, bool WARP, int MAXT>
tp_status run_bwd(const NormParams& P0, const NormBwdLaunch& L, cudaStream_t stream) {
  static KernelInfo info;
  void (*k)(NormParams) = block_norm_bwd_kernel<NV, RES32, LN, GROUPS, WARP, MAXT>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  NormParams P = P0;
  const size_t stage = static_cast<size_t>(L.threads) * NV * (2 * (RES32 ? 2 : 1) + 2) * 16;
  P.stages = 2 * stage <= 100 * 1024 ? 2 : 1;
  return launch_dependent(k, dim3(static_cast<unsigned>(L.ctas)), static_cast<unsigned>(L.threads), P.stages * stage, stream, P);
}

template <bool RES32, bool LN, bool GROUPS>
tp_status dispatch_bwd(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream) {
  if (L.warp) {
    return L.nv == 2 ? run_bwd<2, RES32, LN, GROUPS, true, 256>(P, L, stream)
                     : run_bwd<4, RES32, LN, GROUPS, true, 256>(P, L, stream);
  }
  if (L.threads <= 256) return run_bwd<2, RES32, LN, GROUPS, false, 256>(P, L, stream);
  if (L.threads <= 512) return run_bwd<2, RES32, LN, GROUPS, false, 512>(P, L, stream);
  if (L.threads <= 768) return run_bwd<2, RES32, LN, GROUPS, false, 768>(P, L, stream);
  return run_bwd<2, RES32, LN, GROUPS, false, 1024>(P, L, stream);
}

template <bool RES32, bool LN>
tp_status dispatch_bwd_groups(const NormParams& P, const NormBwdLaunch& L, cudaStream_t stream) {
  return L.groups ? dispatch_bwd<RES32, LN, true>(P, L, stream) : dispatch_bwd<RES32, LN, false>(P, L, stream);
}

}  // namespace tpf
