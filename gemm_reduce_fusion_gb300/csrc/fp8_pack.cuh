// Packing of a token's row into the rows of its slots (fp8_pack.cu, and
// experts.cu where there are few slots).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fp8_device.cuh"
#include "vec_util.cuh"

namespace tpf {

// The largest magnitude of bf16 pairs, as 15-bit integers (an infinity or NaN
// is at least 0x7F80, and the magnitudes are then looked at one by one).
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7FFF7FFFu); }
constexpr uint32_t kInfinite = 0x7F80u;

struct TokenPack {
  const __nv_bfloat16* x;  // [tokens, cols]
  uint8_t *q, *e;
  int64_t tokens, cols, ldq, e_block;  // bytes of a row of q, of a tile's exponents
  int32_t k, tile_rows;
  const int32_t* row;  // of slot t * k + j, -1: none
};

// A warp's share: 512 columns of token t, packed once and written to the
// rows of its k slots, which the first k lanes have (-1: none).
__device__ __forceinline__ void pack_token(const TokenPack& P, int64_t t, uint32_t four, int32_t my_row, uint32_t lane) {
  const int64_t c = static_cast<int64_t>(four) * 512 + lane * 16;
  const __nv_bfloat16* x = P.x + t * P.cols;
  const uint4 a = c < P.cols ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
  const uint4 b = c + 8 < P.cols ? *reinterpret_cast<const uint4*>(x + c + 8) : make_uint4(0, 0, 0, 0);
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float f[16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = max_abs(m, u[i]);
    f[2 * i] = bf_lo(u[i]);
    f[2 * i + 1] = bf_hi(u[i]);
  }
  m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));  // of 128 columns
  float top = __uint_as_float(m << 16);
  const bool finite = __all_sync(0xFFFFFFFFu, m < kInfinite);
  if (!finite) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, finite_abs(f[i]));
#pragma unroll
    for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  const uint32_t e = fp8_exponent(top);
  const float inv = fp8_inverse(e);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = finite ? fp8_pack4_finite(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], inv)
                  : fp8_pack4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], inv);
  uint32_t es = 0;  // the four blocks' exponents, which lie side by side
#pragma unroll
  for (int i = 0; i < 4; ++i) es |= __shfl_sync(0xFFFFFFFFu, e, i * 8) << (i * 8);
  for (int32_t j = 0; j < P.k; ++j) {
    const int64_t r = __shfl_sync(0xFFFFFFFFu, my_row, j);
    if (r < 0) continue;
    if (c < P.ldq) *reinterpret_cast<uint4*>(P.q + r * P.ldq + c) = make_uint4(q[0], q[1], q[2], q[3]);
    const int64_t block = r / P.tile_rows;
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(P.e + block * P.e_block + four * 512 + fp8_e_at(static_cast<uint32_t>(r - block * P.tile_rows), 0)) = es;
  }
}

}  // namespace tpf
