// 8-bit activation checkpoints: packing, restoring, and the C ABI of both.
//
// A group of 32 columns shares the quantum 2^E, the smallest power of two
// with 127 * 2^E >= max|x| (and E >= -126); q = x / 2^E rounded to nearest
// even, kept with the byte E + 126.  Scaling by a power of two is exact, so
// q is the correctly rounded quotient, and q * 2^E, with seven significant
// bits, is exactly a bf16: a restored activation enters the tensor cores
// without a second rounding.  (One exception, at the end of the range: beside
// the largest finite magnitude, 255/128 * 2^127, it and the next one round to
// 64 * 2^122 and come back as infinity.)  The price against a quantum of max|x| / 127 is
// at most one bit.  The byte 255 marks a group that held an infinity or NaN;
// it is restored as NaN throughout, so that an overflow stays visible.
//
// Both directions are bound by HBM (3.03 bytes an element), restoring with
// GeLU also by its two special functions an element (28 us of the 40 below).
// Measured at 4 x 4096 x 4096: packing 30 us and restoring with GeLU about 40,
// 69 us together, 5.9 TB/s, against 60 us at the copy rate.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "ckpt.h"
#include "gelu.cuh"
#include "host_util.h"
#include "vec_util.cuh"

using namespace tpf;

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // vectors of 8 columns a thread has in flight

struct CkptParams {
  const void* x[8];  // pack: bf16 in
  const void* q[8];
  const void* e[8];
  void* plain[8];    // restore: values, or null
  void* gelu[8];     // restore: GeLU of the values, or null
  int64_t units;     // vectors of 8 columns, each row padded to whole groups of 4
  uint32_t per_row;  // of them in a row (FLAT: not used)
  uint32_t nvec;     // real ones in a row
};

// Place of unit u: its vector in the bf16 (and, halved, int8) tensor, or
// false past the row's end.  FLAT: rows are whole groups, so that the tensor
// is one long row.  A unit's group is always u / 4.
template <bool FLAT>
__device__ __forceinline__ bool place(const CkptParams& P, int64_t u, int64_t& vec) {
  if (u >= P.units) return false;
  vec = u;
  if constexpr (!FLAT) {
    const int64_t row = P.units <= 0xFFFFFFFFll ? static_cast<uint32_t>(u) / P.per_row : u / P.per_row;
    const uint32_t c = static_cast<uint32_t>(u - row * P.per_row);
    vec = row * P.nvec + c;
    return c < P.nvec;
  }
  return true;
}

// max of the magnitudes of two bf16 pairs, as 15-bit integers (an infinity
// or NaN is at least 0x7F80)
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu); }

template <bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt_pack_kernel(const __grid_constant__ CkptParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint4* x = static_cast<const uint4*>(P.x[blockIdx.y]);
  uint2* q = static_cast<uint2*>(const_cast<void*>(P.q[blockIdx.y]));
  uint8_t* e = static_cast<uint8_t*>(const_cast<void*>(P.e[blockIdx.y]));
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 v[kUnroll];
  int64_t at[kUnroll];
  bool ok[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    ok[i] = place<FLAT>(P, u0 + i * kThreads, at[i]);
    v[i] = ok[i] ? __ldcs(x + at[i]) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    uint32_t m = __vmaxu2(max_abs(v[i].x, v[i].y), max_abs(v[i].z, v[i].w));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    // max|x| = 1.f * 2^(E8 - 127) with 7 fraction bits: 127 * 2^E reaches it
    // at E = E8 - 133, or one more where f is all ones (1.f above 127/64)
    const bool bad = m >= 0x7F80u;
    int b = static_cast<int>(m >> 7) - 7 + ((m & 127u) == 127u ? 1 : 0);
    b = max(b, 0);
    const float inv = __uint_as_float(static_cast<uint32_t>(253 - b) << 23);  // 2^-E
    float f[8];
    unpack8(v[i], f);
    // x / 2^E + 1.5 * 2^23 rounds to the whole number whose low byte is q
    uint32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __float_as_uint(fmaf(f[j], inv, 12582912.f));
    uint2 o;
    o.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    if (bad) o = make_uint2(0, 0);
    if (ok[i]) __stcs(q + at[i], o);
    const int64_t u = u0 + i * kThreads;
    if ((threadIdx.x & 3) == 0 && u < P.units) e[u >> 2] = bad ? 255 : static_cast<uint8_t>(b);
  }
}

// q bytes -> fp32: the byte with its sign bit flipped, as the low byte of
// 2^23 + (q + 128), less 2^23 + 128
__device__ __forceinline__ void bytes_to_f(uint32_t w, float* f) {
  w ^= 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + j)) - 8388736.f;
}

template <bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt_restore_kernel(const __grid_constant__ CkptParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint2* q = static_cast<const uint2*>(P.q[blockIdx.y]);
  const uint8_t* e = static_cast<const uint8_t*>(P.e[blockIdx.y]);
  uint4* plain = static_cast<uint4*>(P.plain[blockIdx.y]);
  uint4* gelu = static_cast<uint4*>(P.gelu[blockIdx.y]);
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint2 v[kUnroll];
  uint32_t b[kUnroll];
  int64_t at[kUnroll];
  bool ok[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t u = u0 + i * kThreads;
    ok[i] = place<FLAT>(P, u, at[i]);
    v[i] = ok[i] ? __ldcs(q + at[i]) : make_uint2(0, 0);
    b[i] = ok[i] ? e[u >> 2] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (!ok[i]) continue;
    // 2^E = 2^(b - 126), its exponent field b + 1; 255 gives NaN
    const float s = b[i] == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((b[i] + 1u) << 23);
    float f[8];
    bytes_to_f(v[i].x, f);
    bytes_to_f(v[i].y, f + 4);
    if (gelu) {
      const uint64_t s2 = pk2(s, s), scaled = pk2(s * kTailRoot, s * kTailRoot);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        upk2(gelu_scaled2(f[2 * j], f[2 * j + 1], s2, scaled), lo, hi);
        w[j] = pack_bf16(lo, hi);
      }
      gelu[at[i]] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (plain) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      plain[at[i]] = pack8(f);
    }
  }
}

void fill_units(CkptParams* P, int64_t M, int64_t N) {
  const bool flat = N % 32 == 0;
  P->nvec = static_cast<uint32_t>(N / 8);
  P->per_row = static_cast<uint32_t>(cdiv(N, 32) * 4);
  P->units = flat ? M * (N / 8) : M * P->per_row;
}

tp_status check_packed(const void* const* q, const void* const* e, int n, bool work) {
  if (!work) return TP_OK;
  TP_TRY(check_ptrs(q, n, true));
  if (e == nullptr) return TP_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (e[i] == nullptr) return TP_ERR_INVALID_ARG;
  return TP_OK;
}

}  // namespace

namespace tpf {

tp_status ckpt_restore(const void* const* q, const void* const* e, void* const* plain, void* const* gelu, int n, int64_t M,
                       int64_t N, cudaStream_t stream) {
  if (M == 0 || N == 0) return TP_OK;
  CkptParams P;
  std::memset(&P, 0, sizeof(P));
  fill_units(&P, M, N);
  for (int i = 0; i < n; ++i) {
    P.q[i] = q[i];
    P.e[i] = e[i];
    P.plain[i] = plain ? plain[i] : nullptr;
    P.gelu[i] = gelu ? gelu[i] : nullptr;
  }
  const dim3 grid(static_cast<unsigned>(cdiv(P.units, kThreads * kUnroll)), static_cast<unsigned>(n));
  return launch_dependent(N % 32 == 0 ? ckpt_restore_kernel<true> : ckpt_restore_kernel<false>, grid, kThreads, 0, stream, P);
}

}  // namespace tpf

extern "C" tp_status tp_ckpt_pack(const void* const* x, void* const* q, void* const* e, int p, int64_t M, int64_t N,
                                  cudaStream_t stream) {
  TP_TRY(check_sizes(p, M, N, 0, 0, TP_BF16));
  const bool work = M > 0 && N > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(x, p, work));
  TP_TRY(check_packed(in(q), in(e), p, work));
  if (!work) return TP_OK;
  RangeList ins, outs;
  add_ranges(&ins, x, p, static_cast<size_t>(M * N) * 2);
  add_ranges(&outs, in(q), p, static_cast<size_t>(M * N));
  add_ranges(&outs, in(e), p, static_cast<size_t>(M * cdiv(N, 32)));
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  CkptParams P;
  std::memset(&P, 0, sizeof(P));
  fill_units(&P, M, N);
  for (int i = 0; i < p; ++i) {
    P.x[i] = x[i];
    P.q[i] = q[i];
    P.e[i] = e[i];
  }
  const dim3 grid(static_cast<unsigned>(cdiv(P.units, kThreads * kUnroll)), static_cast<unsigned>(p));
  return launch_dependent(N % 32 == 0 ? ckpt_pack_kernel<true> : ckpt_pack_kernel<false>, grid, kThreads, 0, stream, P);
}

extern "C" tp_status tp_ckpt_unpack(const void* const* q, const void* const* e, void* const* y, tp_epilogue epi, int p, int64_t M,
                                    int64_t N, cudaStream_t stream) {
  TP_TRY(check_sizes(p, M, N, 0, 0, TP_BF16));
  if (epi != TP_EPI_NONE && epi != TP_EPI_GELU) return TP_ERR_INVALID_ARG;
  const bool work = M > 0 && N > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_packed(q, e, p, work));
  TP_TRY(check_ptrs(in(y), p, work));
  if (!work) return TP_OK;
  RangeList ins, outs;
  add_ranges(&ins, q, p, static_cast<size_t>(M * N));
  add_ranges(&ins, e, p, static_cast<size_t>(M * cdiv(N, 32)));
  add_ranges(&outs, in(y), p, static_cast<size_t>(M * N) * 2);
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  const bool g = epi == TP_EPI_GELU;
  return ckpt_restore(q, e, g ? nullptr : y, g ? y : nullptr, p, M, N, stream);
}
