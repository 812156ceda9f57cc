// Device helpers shared by the bandwidth-bound kernels: packed bf16 vectors,
// thread-private asynchronous copies and small conversions.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"

namespace tpf {

// The two bf16 values of a 32-bit word (low half first).
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values rounded to nearest even and packed, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
  v[0] = bf_lo(p.x);
  v[1] = bf_hi(p.x);
  v[2] = bf_lo(p.y);
  v[3] = bf_hi(p.y);
  v[4] = bf_lo(p.z);
  v[5] = bf_hi(p.z);
  v[6] = bf_lo(p.w);
  v[7] = bf_hi(p.w);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// 16-byte asynchronous copy global -> shared of the issuing thread (both
// addresses 16-byte aligned); completed by cp_async_wait of that thread.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's latest groups are still in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Global store of 16 bytes that this kernel does not read again.
__device__ __forceinline__ void st_global_cs(void* p, const uint4& v) { __stcs(static_cast<uint4*>(p), v); }

}  // namespace tpf
