// Internal interface of the 8-bit activation checkpoints (ckpt.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tp_fused.h"

namespace tpf {

// Restores n packed tensors [M, N] into bf16: plain[i] gets the values,
// gelu[i] their GeLU; either array may be null.
tp_status ckpt_restore(const void* const* q, const void* const* e, void* const* plain, void* const* gelu, int n, int64_t M,
                       int64_t N, cudaStream_t stream);

// What a backward call restores from its checkpoints, after its arguments
// have been checked and before its products run.
struct CkptRestore {
  const void* const* q;
  const void* const* e;
  void* const* plain;
  void* const* gelu;
  int n;
  int64_t M, N;
};

inline tp_status ckpt_restore(const CkptRestore& r, cudaStream_t stream) {
  return ckpt_restore(r.q, r.e, r.plain, r.gelu, r.n, r.M, r.N, stream);
}

}  // namespace tpf
