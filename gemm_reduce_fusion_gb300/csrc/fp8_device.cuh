// The 8-bit operands on the device: exponents, conversions, and the tcgen05
// forms that read their scales.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace tpf {

// |x|, or 0 of an infinity or NaN, which takes no part in a block's exponent.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __uint_as_float(0x7F800000u) ? a : 0.f;
}

// The byte e of the smallest 2^(e - 127), at least 2^-127, with
// top <= 448 * 2^(e - 127): top = 1.f * 2^(x - 127) reaches 448 = 1.75 * 2^8
// times 2^(x - 8 - 127) unless 1.f > 1.75.  (A denormal top is below
// 448 * 2^-127.)
__device__ __forceinline__ uint32_t fp8_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int32_t e = static_cast<int32_t>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}
// 2^(127 - e), e <= 248: exact, so that a scaled value is rounded once.
__device__ __forceinline__ float fp8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Four finite values in e4m3, rounded to nearest even.
__device__ __forceinline__ uint32_t fp8_pack4_finite(float a, float b, float c, float d, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four values in e4m3, rounded to nearest even; an infinity or NaN is NaN.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float inv) {
  const float inf = __uint_as_float(0x7F800000u), nan = __uint_as_float(0x7FC00000u);
  a = fabsf(a) < inf ? a * inv : nan;
  b = fabsf(b) < inf ? b * inv : nan;
  c = fabsf(c) < inf ? c * inv : nan;
  d = fabsf(d) < inf ? d * inv : nan;
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The values of four e4m3 bytes, by way of f16, which holds each exactly.
__device__ __forceinline__ void fp8_unpack4(uint32_t w, float* f) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
  const __half2 a = *reinterpret_cast<const __half2*>(&lo), b = *reinterpret_cast<const __half2*>(&hi);
  f[0] = __low2float(a);
  f[1] = __high2float(a);
  f[2] = __low2float(b);
  f[3] = __high2float(b);
}

// Place of the exponent of row r and block b of the 512 bytes that hold those
// of 128 rows and four blocks.
__device__ __forceinline__ uint32_t fp8_e_at(uint32_t r, uint32_t b) { return (r & 31) * 16 + (r >> 5) * 4 + b; }

// ------------------------------------------------------------------ PTX
//
// The instructions below take their operands from uniform registers.  A whole
// warp goes through the code around them, so that the compiler knows them to
// be uniform, and the lane with `one` set executes them (in code of one lane
// each of them costs its thread some 120 cycles).

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}

// A tile of a map to shared memory; its bytes count on `bar`, with CTAS = 2 an
// address in the cluster.
template <int CTAS>
__device__ __forceinline__ void load_2d(uint32_t one, uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_3d_pair(uint32_t one, uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one)
      : "memory");
}
__device__ __forceinline__ void load_512(uint32_t one, uint32_t dst, const void* src, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 512, [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bar), "r"(one)
      : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t one, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(one)
      : "memory");
}

// 512 bytes of exponents, shared -> tensor memory: 16 bytes for each of 32
// lanes (four 32-bit columns, rows 32 j + lane in column j), the same in every
// 32 lanes.  The descriptor: no swizzle, groups of 8 rows 128 bytes apart.
template <int CTAS>
__device__ __forceinline__ void tmem_cp_scales(uint32_t one, uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
  if constexpr (CTAS == 2)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc),
                 "r"(one)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc),
                 "r"(one)
                 : "memory");
}

// Instruction descriptor of kind::mxf8f6f4 with e4m3 operands, both K-major,
// and power-of-two scales: bits 4-5 and 29-30 the byte of B's and A's scale
// columns, 7-9 and 10-12 the formats (0: e4m3), 17-22 N >> 3, 23 scale format
// (1: 8-bit exponent), 24-28 M >> 4.
__device__ __forceinline__ uint32_t make_idesc_mxf8(uint32_t M, uint32_t N, uint32_t byte) {
  return (byte << 4) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24) | (byte << 29);
}

// D[tmem] (+)= (A scaled) (B scaled)^T over 32 of the contraction.
template <int CTAS>
__device__ __forceinline__ void umma_mxf8(uint32_t one, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)
        : "memory");
}

// Arrive once on `bar` (CTAS = 2: of the CTAs in `mask`) when every tcgen05 op
// that the thread has issued is done.
template <int CTAS>
__device__ __forceinline__ void commit_to(uint32_t one, uint32_t bar, uint16_t mask) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(mask), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// A staged box to memory; what lies outside the tensor is not written.
__device__ __forceinline__ void store_3d(const void* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

}  // namespace tpf
