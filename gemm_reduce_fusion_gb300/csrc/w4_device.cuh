// What the kernels of the 4-bit sharded Linear share: their parameters, the
// conversion of nibbles and the places of results.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/tp_fused.h"
#include "gelu.cuh"
#include "vec_util.cuh"

namespace tpf {

struct W4Params {
  const void* x[8];
  const void* q[8];
  const void* s[8];
  const __nv_bfloat16* bias[8];
  void* y[8];
  float* part;                // [2 * runs] slabs: sums of a column block's part
  uint32_t run_stages;        // run r: stages r * run_stages ... (the last run may be shorter)
  uint32_t M, N, K;
  uint32_t ktiles, groups, pairs;  // 64-row tiles, scale groups, 32-column pairs of 16-column strips of a shard
  uint32_t nblocks;                // column blocks of a shard
  uint32_t kstages;                // stages of a shard
  uint32_t spb;                    // stages of a column block: row layout p * kstages, column layout kstages
  uint32_t stages;                 // all
  int32_t row, epi, out_f32;
  uint32_t* status;
  uint64_t timeout_ns;
  int32_t drop;  // test hook of w4_wide_kernel: a stage of tokens that block 0 never hands over, or -1
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  const uint32_t n = valid ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The four fragment registers of a word (see the top), for the columns i
// (q - 8, times 2^-6) and i + 8 (times 2^-2) in turn.
__device__ __forceinline__ void dequant(uint32_t w, uint32_t (&a)[4]) {
  constexpr uint32_t kUp = 0x7F007F00u, kOff0 = 0xBE00BE00u, kOff1 = 0xC000C000u;  // 2^127, -2^-3, -2
  const uint32_t v = w >> 8;
  a[0] = fma_bf16x2(w & 0x000F000Fu, kUp, kOff0);
  a[1] = fma_bf16x2(w & 0x00F000F0u, kUp, kOff1);
  a[2] = fma_bf16x2(v & 0x000F000Fu, kUp, kOff0);
  a[3] = fma_bf16x2(v & 0x00F000F0u, kUp, kOff1);
}

// The operands lack 2^6 (columns i) and 2^2 (columns i + 8).  The scales of
// the latter are multiplied by 2^-4, which is exact for the smallest of them
// too, and the sums by 2^6 at the end: a scale times 2^6 would be infinite
// from 2^122.
constexpr float kLift = 64.f, kEven = 0.0625f;

// The runs that hold stages of a column block.
struct Parts {
  uint32_t first, last;
};
__device__ __forceinline__ Parts parts_of(const W4Params& P, uint32_t block) {
  const uint32_t b0 = block * P.spb;
  return {b0 / P.run_stages, (b0 + P.spb - 1) / P.run_stages};
}

// Bias, activation and rounding of one sum, which lacks a factor of 2^6
// (kLift): token `tok`, column `col` of an output shard.
__device__ __forceinline__ void write_one(const W4Params& P, uint32_t shard, uint32_t tok, uint32_t col, float bias, float v) {
  float y = fmaf(v, kLift, bias);
  if (P.epi == TP_EPI_GELU) y = gelu_f(y);
  const int64_t at = static_cast<int64_t>(tok) * P.N + col;
  if (P.out_f32) static_cast<float*>(P.y[shard])[at] = y;
  else static_cast<__nv_bfloat16*>(P.y[shard])[at] = __float2bfloat16_rn(y);
}

}  // namespace tpf
