// Launch of block_norm_bwd_kernel<..., RES32, LN, ...> for one residual type
// and kind of norm; included once by each of block_norm_bwd_*.cu.
#pragma once
#include "block_norm.cuh"
#include "block_norm.h"
#include "host_util.h"

namespace tpf {

template <int NV, bool RES32, bool LN, bool GROUPS, int KIND, int MAXT, bool FULL>
tp_status run_kernel(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  static KernelInfo info;
  void (*k)(NormParams) = block_norm_bwd_kernel<NV, RES32, LN, GROUPS, KIND, MAXT, FULL>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  if constexpr (KIND == BY_CLUSTER) {
    // clusters stay within a GPC, so that not every SM may find partners: as
    // many clusters as are resident together
    int most = 0;
    TP_TRY(resident_clusters(reinterpret_cast<const void*>(k), L.cluster, L.threads, L.smem, &most));
    if (L.ctas > most) L.ctas = most;
  } else {
    DevInfo di;
    TP_TRY(device_info(&di));
    const int most = di.sms * blocks_per_sm(L.threads, regs, L.smem + sizeof(Totals));
    if (L.ctas > most) L.ctas = most;
  }
  return launch_dependent(k, dim3(static_cast<unsigned>(L.ctas * L.cluster)), static_cast<unsigned>(L.threads), L.smem, stream, P,
                          L.cluster);
}

template <int NV, bool RES32, bool LN, bool GROUPS, int KIND, int MAXT>
tp_status run_bwd(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  if constexpr (!LN && !GROUPS && KIND != BY_WARP) {
    if (L.full) return run_kernel<NV, RES32, LN, GROUPS, KIND, MAXT, true>(P, L, stream);
  }
  return run_kernel<NV, RES32, LN, GROUPS, KIND, MAXT, false>(P, L, stream);
}

template <bool RES32, bool LN, bool GROUPS>
tp_status dispatch_bwd(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  if (L.kind == BY_WARP) {
    return L.nv == 2 ? run_bwd<2, RES32, LN, GROUPS, BY_WARP, 256>(P, L, stream)
                     : run_bwd<4, RES32, LN, GROUPS, BY_WARP, 256>(P, L, stream);
  }
  if (L.kind == BY_CLUSTER) {
    return L.threads <= 192 ? run_bwd<2, RES32, LN, GROUPS, BY_CLUSTER, 192>(P, L, stream)
                            : run_bwd<2, RES32, LN, GROUPS, BY_CLUSTER, 256>(P, L, stream);
  }
  return L.threads <= 128 ? run_bwd<2, RES32, LN, GROUPS, BY_CTA, 128>(P, L, stream)
                          : run_bwd<2, RES32, LN, GROUPS, BY_CTA, 256>(P, L, stream);
}

template <bool RES32, bool LN>
tp_status dispatch_bwd_groups(const NormParams& P, NormBwdLaunch& L, cudaStream_t stream) {
  return L.groups ? dispatch_bwd<RES32, LN, true>(P, L, stream) : dispatch_bwd<RES32, LN, false>(P, L, stream);
}

}  // namespace tpf
