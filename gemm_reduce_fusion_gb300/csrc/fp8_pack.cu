// Packing of matrices into 8-bit operands, rows and transpose at once, and
// their restoring.
//
// A block of 128 along the contraction shares the smallest power of two 2^k
// with max|x| <= 448 * 2^k; x / 2^k is exact, so that rounding to e4m3 is the
// only one.  (Against a scale of max|x| / 448 this costs up to one bit of the
// block's range and none of its precision above 2^-6 of the largest value.)
//
// fp8_pack_kernel: a thread block takes 128 rows x 128 columns: what it reads
// gives the row operand from registers and, through shared memory, the
// transposed one, so that x is read once for both.  4 x 4096 x 4096 take 64 us
// for both, 0.62 of the copy rate (2 bytes read and 2 written an element), and
// 59 us for the transpose of their GeLU, 0.50 (2 and 1): the instructions of
// both operands' maxima and conversions, and GeLU's two special functions an
// element, bound it.
//
// fp8_pack_rows_kernel: a warp for each 128 columns of a row, where there are
// too few rows for the blocks above to fill the GPU.
#include <cuda_bf16.h>

#include <cstring>

#include "fp8.h"
#include "fp8_device.cuh"
#include "fp8_pack.cuh"
#include "gelu.cuh"
#include "vec_util.cuh"

using namespace tpf;

namespace {

constexpr int kThreads = 256;
constexpr int kPitch = 128 * 2 + 16;  // bytes of a row in shared memory

struct PackParams {
  const __nv_bfloat16* x[8];
  uint8_t *q[8], *e[8], *qt[8], *et[8];
  int64_t rows, cols;          // of a matrix
  int64_t ldq, ldqt;           // bytes of a row of q, qt
  int64_t e_block, et_block;   // bytes of 128 rows of exponents
  int64_t e_mat, et_mat;       // of a matrix
  uint32_t batch, strips;      // matrices a tensor; strips of 128 rows of a matrix
  int32_t tiles, gelu;
  const int32_t *plan_tiles, *slot;  // or null
  const float* weights;              // of the slots, or null
  int32_t gather, k, tile_rows;
};

// The source row of row r of the plan (or of the matrix), null for none.
__device__ __forceinline__ const __nv_bfloat16* source(const PackParams& P, const __nv_bfloat16* x, int64_t r, float& w) {
  w = 1.f;
  if (r >= P.rows) return nullptr;
  if (P.slot == nullptr) return x + r * P.cols;
  const int32_t s = __ldcg(P.slot + r);
  if (s < 0) return nullptr;
  if (P.weights) w = P.weights[s];
  return x + (P.gather ? s / P.k : r) * P.cols;
}

// What becomes of an element before it is packed.
enum Source : int { PLAIN = 0, GELU = 1, WEIGHTED = 2 };

// Two neighbours of a row, as they are packed.
template <int SRC>
__device__ __forceinline__ void pair_of(uint32_t u, float w, float& lo, float& hi) {
  lo = bf_lo(u);
  hi = bf_hi(u);
  if constexpr (SRC == GELU) gelu2_to8(lo, hi);
  if constexpr (SRC == WEIGHTED) lo *= w, hi *= w;
}

template <bool FINITE>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float inv) {
  return FINITE ? fp8_pack4_finite(a, b, c, d, inv) : fp8_pack4(a, b, c, d, inv);
}

// Two columns x 32 rows of the tile, as they were read (PLAIN) or formed, to
// the transposed operand's two rows.
template <bool FINITE, int SRC>
__device__ __forceinline__ void put_columns(const uint32_t* raw, const float* keep, float ilo, float ihi, uint8_t* to, int64_t ld) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t lo4[4], hi4[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = half * 16 + n * 4 + j;
        if (SRC == PLAIN) {
          lo[j] = bf_lo(raw[SRC == PLAIN ? i : 0]);
          hi[j] = bf_hi(raw[SRC == PLAIN ? i : 0]);
        } else {
          lo[j] = keep[SRC == PLAIN ? 0 : 2 * i];
          hi[j] = keep[SRC == PLAIN ? 0 : 2 * i + 1];
        }
      }
      lo4[n] = pack4<FINITE>(lo[0], lo[1], lo[2], lo[3], ilo);
      hi4[n] = pack4<FINITE>(hi[0], hi[1], hi[2], hi[3], ihi);
    }
    *reinterpret_cast<uint4*>(to + half * 16) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
    *reinterpret_cast<uint4*>(to + ld + half * 16) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
  }
}

template <bool Q, bool QT, int SRC>
__global__ void __launch_bounds__(kThreads) fp8_pack_kernel(const __grid_constant__ PackParams P) {
  __shared__ __align__(16) uint8_t tile[QT ? 128 * kPitch : 16];
  __shared__ float2 red[4][64];
  __shared__ float row_w[128], warp_top[8];
  __shared__ int64_t row_at[128];  // element of x at which a row begins, or -1
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t t = blockIdx.z / P.batch, mat = blockIdx.z % P.batch, strip = blockIdx.y, b = blockIdx.x;
  if (P.plan_tiles != nullptr && strip * 128 >= static_cast<uint32_t>(__ldcg(P.plan_tiles) * P.tile_rows)) return;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const __nv_bfloat16* x = P.x[t] + mat * P.rows * P.cols;
  const int64_t r0 = static_cast<int64_t>(strip) * 128;
  const uint32_t sub = lane >> 4, piece = lane & 15;  // row of two, 16 bytes of a row
  const int64_t c = static_cast<int64_t>(b) * 128 + piece * 8;
  if (P.slot != nullptr) {
    if (tid < 128) {
      float w;
      const __nv_bfloat16* src = source(P, x, r0 + tid, w);
      row_at[tid] = src ? src - x : -1;
      row_w[tid] = w;
    }
    __syncthreads();
  }
  uint4 v[8];
  float w[8];
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) {
    const uint32_t r = warp * 16 + i * 2 + sub;
    const int64_t at = P.slot != nullptr ? row_at[r] : r0 + r < P.rows ? (r0 + r) * P.cols : -1;
    w[i] = SRC == WEIGHTED ? row_w[r] : 1.f;
    v[i] = at >= 0 && c < P.cols ? *reinterpret_cast<const uint4*>(x + at + c) : make_uint4(0, 0, 0, 0);
  }
  if (QT) {
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(tile + (warp * 16 + i * 2 + sub) * kPitch + piece * 16) = v[i];
  }
  float all = 0.f;
  if (P.tiles) {
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        pair_of<SRC>(u[j], w[i], lo, hi);
        all = fmaxf(all, fmaxf(finite_abs(lo), finite_abs(hi)));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xFFFFFFFFu, all, o));
    if (lane == 0) warp_top[warp] = all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) all = fmaxf(all, warp_top[i]);
  }
  if (Q) {
    uint8_t* q = P.q[t] + (mat * P.rows + r0) * P.ldq + b * 128 + piece * 8;
    uint8_t* e = P.e[t] + mat * P.e_mat + strip * P.e_block + static_cast<int64_t>(b >> 2) * 512;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = warp * 16 + i * 2 + sub;
      float f[8], top = 0.f;
      bool finite = false;
      pair_of<SRC>(v[i].x, w[i], f[0], f[1]);
      pair_of<SRC>(v[i].y, w[i], f[2], f[3]);
      pair_of<SRC>(v[i].z, w[i], f[4], f[5]);
      pair_of<SRC>(v[i].w, w[i], f[6], f[7]);
      if (SRC == PLAIN && !P.tiles) {
        uint32_t m = max_abs(max_abs(max_abs(max_abs(0, v[i].x), v[i].y), v[i].z), v[i].w);
        m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        finite = m < kInfinite;
        top = __uint_as_float(m << 16);
      }
      const bool warp_finite = SRC == PLAIN && __all_sync(0xFFFFFFFFu, finite);
      if (!warp_finite) {
        top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(f[j]));
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      }
      const uint32_t ex = fp8_exponent(P.tiles ? all : top);
      const float inv = fp8_inverse(ex);
      uint2 o;
      if (warp_finite) o = make_uint2(fp8_pack4_finite(f[0], f[1], f[2], f[3], inv), fp8_pack4_finite(f[4], f[5], f[6], f[7], inv));
      else o = make_uint2(fp8_pack4(f[0], f[1], f[2], f[3], inv), fp8_pack4(f[4], f[5], f[6], f[7], inv));
      if (r0 + r < P.rows) *reinterpret_cast<uint2*>(q + r * P.ldq) = o;
      if (piece == 0) e[fp8_e_at(r, b & 3)] = r0 + r < P.rows ? static_cast<uint8_t>(ex) : 0;
    }
  }
  if (QT) {
    // two columns and a quarter of the rows a thread
    __syncthreads();
    const uint32_t pair = tid & 63, quarter = tid >> 6;
    const uint8_t* from = tile + quarter * 32 * kPitch + pair * 4;
    float tlo = all, thi = all;
    uint32_t raw[SRC == PLAIN ? 32 : 1];
    float keep[SRC == PLAIN ? 1 : 64];
    uint32_t mlo = 0, mhi = 0;  // the largest magnitudes, as integers
    if (SRC == PLAIN) {
      uint32_t m = 0;
#pragma unroll
      for (uint32_t i = 0; i < 32; ++i) {
        raw[SRC == PLAIN ? i : 0] = *reinterpret_cast<const uint32_t*>(from + i * kPitch);
        m = max_abs(m, raw[SRC == PLAIN ? i : 0]);
      }
      mlo = m << 16;
      mhi = m & 0xFFFF0000u;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 32; ++i) {
        float &lo = keep[SRC == PLAIN ? 0 : 2 * i], &hi = keep[SRC == PLAIN ? 0 : 2 * i + 1];
        pair_of<SRC>(*reinterpret_cast<const uint32_t*>(from + i * kPitch), SRC == WEIGHTED ? row_w[quarter * 32 + i] : 1.f, lo, hi);
        mlo = max(mlo, __float_as_uint(fabsf(lo)));
        mhi = max(mhi, __float_as_uint(fabsf(hi)));
      }
    }
    const bool all_finite = !P.tiles && !__syncthreads_or(max(mlo, mhi) >= kInfinite << 16);
    if (!P.tiles) {
      if (!all_finite) {  // an infinity or NaN in the tile: magnitudes of the others
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) {
          lo = fmaxf(lo, finite_abs(SRC == PLAIN ? bf_lo(raw[SRC == PLAIN ? i : 0]) : keep[SRC == PLAIN ? 0 : 2 * i]));
          hi = fmaxf(hi, finite_abs(SRC == PLAIN ? bf_hi(raw[SRC == PLAIN ? i : 0]) : keep[SRC == PLAIN ? 0 : 2 * i + 1]));
        }
        mlo = __float_as_uint(lo);
        mhi = __float_as_uint(hi);
      }
      red[quarter][pair] = make_float2(__uint_as_float(mlo), __uint_as_float(mhi));
      __syncthreads();
      tlo = thi = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 o = red[i][pair];
        tlo = fmaxf(tlo, o.x);
        thi = fmaxf(thi, o.y);
      }
    }
    const uint32_t elo = fp8_exponent(tlo), ehi = fp8_exponent(thi);
    const float ilo = fp8_inverse(elo), ihi = fp8_inverse(ehi);
    const int64_t col = static_cast<int64_t>(b) * 128 + pair * 2;
    if (col < P.cols) {
      uint8_t* to = P.qt[t] + (mat * P.cols + col) * P.ldqt + r0 + quarter * 32;
      if (all_finite) put_columns<true, SRC>(raw, keep, ilo, ihi, to, P.ldqt);
      else put_columns<false, SRC>(raw, keep, ilo, ihi, to, P.ldqt);
    }
    if (quarter == 0) {  // of columns past the matrix too, where no product uses them
      uint8_t* e = P.et[t] + mat * P.et_mat + b * P.et_block + static_cast<int64_t>(strip >> 2) * 512;
      e[fp8_e_at(pair * 2, strip & 3)] = static_cast<uint8_t>(elo);
      e[fp8_e_at(pair * 2 + 1, strip & 3)] = static_cast<uint8_t>(ehi);
    }
  }
}

// A warp for 128 columns of a row.
__global__ void __launch_bounds__(kThreads) fp8_pack_rows_kernel(const __grid_constant__ PackParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t blocks = static_cast<uint32_t>(P.ldq / 128), lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t r = unit / blocks;
  const uint32_t b = static_cast<uint32_t>(unit % blocks), t = blockIdx.y;
  if (r >= P.rows) return;
  const int64_t c = static_cast<int64_t>(b) * 128 + lane * 4;
  const uint2 v = c < P.cols ? *reinterpret_cast<const uint2*>(P.x[t] + r * P.cols + c) : make_uint2(0, 0);
  float f[4] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)}, top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (P.gelu) f[j] = gelu_f(f[j]);
    top = fmaxf(top, finite_abs(f[j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const uint32_t e = fp8_exponent(top);
  *reinterpret_cast<uint32_t*>(P.q[t] + r * P.ldq + b * 128 + lane * 4) = fp8_pack4(f[0], f[1], f[2], f[3], fp8_inverse(e));
  if (lane == 0) P.e[t][r / 128 * P.e_block + (b >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(r % 128), b & 3)] = static_cast<uint8_t>(e);
}

// A warp for 512 columns of a token, which go to the rows of all of its
// slots: read and packed once.  (Gathered by the rows, each of six slots packed
// for itself, 4096 tokens of 4096 took 60 us, so 23 us.)  Rows without a slot are
// not written.
__global__ void __launch_bounds__(kThreads) fp8_pack_tokens_kernel(const __grid_constant__ TokenPack P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t fours = static_cast<uint32_t>(P.e_block / 512), lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), t = unit / fours;
  if (t >= P.tokens) return;
  const uint32_t four = static_cast<uint32_t>(unit % fours);
  const int32_t my_row = static_cast<int32_t>(lane) < P.k ? __ldcg(P.row + t * P.k + lane) : -1;  // k <= 32
  pack_token(P, t, four, my_row, lane);
}

template <int SRC>
tp_status launch_pack(const Fp8Pack& d, dim3 grid, const PackParams& P, cudaStream_t stream) {
  if (d.q && d.qt) return launch_dependent(fp8_pack_kernel<true, true, SRC>, grid, kThreads, 0, stream, P);
  if (d.q) return launch_dependent(fp8_pack_kernel<true, false, SRC>, grid, kThreads, 0, stream, P);
  return launch_dependent(fp8_pack_kernel<false, true, SRC>, grid, kThreads, 0, stream, P);
}

struct UnpackParams {
  const uint8_t *q[8], *e[8];
  __nv_bfloat16* y[8];
  int64_t rows, cols, ldq, e_block, e_mat;
  uint32_t batch;
};

// Eight columns a thread.
__global__ void __launch_bounds__(kThreads) fp8_unpack_kernel(const __grid_constant__ UnpackParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t t = blockIdx.y / P.batch, mat = blockIdx.y % P.batch;
  const uint32_t per_row = static_cast<uint32_t>(P.cols / 8);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, r = unit / per_row;
  if (r >= P.rows) return;
  const uint32_t c = static_cast<uint32_t>(unit % per_row) * 8, b = c / 128;
  const uint2 v = *reinterpret_cast<const uint2*>(P.q[t] + (mat * P.rows + r) * P.ldq + c);
  const uint32_t e = P.e[t][mat * P.e_mat + r / 128 * P.e_block + (b >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(r % 128), b & 3)];
  // 2^(e - 127), which below the normal range is 2^-127; 255 stands for NaN
  const float s = e == 255 ? __uint_as_float(0x7FC00000u) : e ? __uint_as_float(e << 23) : __uint_as_float(0x00400000u);
  float f[8];
  fp8_unpack4(v.x, f);
  fp8_unpack4(v.y, f + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= s;
  *reinterpret_cast<uint4*>(P.y[t] + (mat * P.rows + r) * P.cols + c) = pack8(f);
}

}  // namespace

namespace tpf {

tp_status check_fp8(const tp_fp8* a, int n, bool need) {
  if (!need) return TP_OK;
  if (a == nullptr) return TP_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (a[i].q == nullptr || a[i].e == nullptr) return TP_ERR_INVALID_ARG;
    if (!aligned16(a[i].q) || !aligned16(a[i].e)) return TP_ERR_ALIGNMENT;
  }
  return TP_OK;
}

void add_fp8(RangeList* v, const tp_fp8* a, int n, int64_t rows, int64_t cols, int64_t batch) {
  if (a == nullptr) return;
  for (int i = 0; i < n; ++i) {
    v->push_back({a[i].q, batch * fp8_q_bytes(rows, cols)});
    v->push_back({a[i].e, batch * fp8_e_bytes(rows, cols)});
  }
}

tp_status fp8_pack(const Fp8Pack& d, cudaStream_t stream) {
  if (d.rows <= 0 || d.cols <= 0 || d.batch <= 0) return TP_OK;
  PackParams P;
  std::memset(&P, 0, sizeof(P));
  for (int i = 0; i < d.n; ++i) {
    P.x[i] = static_cast<const __nv_bfloat16*>(d.x[i]);
    if (d.q) P.q[i] = static_cast<uint8_t*>(d.q[i].q), P.e[i] = static_cast<uint8_t*>(d.q[i].e);
    if (d.qt) P.qt[i] = static_cast<uint8_t*>(d.qt[i].q), P.et[i] = static_cast<uint8_t*>(d.qt[i].e);
  }
  P.rows = d.rows;
  P.cols = d.cols;
  P.ldq = fp8_pitch(d.cols);
  P.ldqt = fp8_pitch(d.rows);
  P.e_block = cdiv(d.cols, 512) * 512;
  P.et_block = cdiv(d.rows, 512) * 512;
  P.e_mat = static_cast<int64_t>(fp8_e_bytes(d.rows, d.cols));
  P.et_mat = static_cast<int64_t>(fp8_e_bytes(d.cols, d.rows));
  P.batch = static_cast<uint32_t>(d.batch);
  P.strips = static_cast<uint32_t>(cdiv(d.rows, 128));
  P.tiles = d.tiles;
  P.gelu = d.gelu;
  P.tile_rows = 128;
  if (d.plan) {
    P.plan_tiles = d.plan->tiles;
    P.slot = d.plan->slot;
    P.weights = d.weights;
    P.gather = d.gather;
    P.k = d.plan->k;
    P.tile_rows = static_cast<int32_t>(d.plan->tile_rows);
  }
  // A block of 128 rows for each 128 columns fills the GPU's 152 SMs from some
  // 256 rows on.
  if (d.qt == nullptr && !d.tiles && d.batch == 1 && d.plan == nullptr && d.rows <= 256) {
    const int64_t units = d.rows * (P.ldq / 128);
    if (cdiv(units, kThreads / 32) > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
    return launch_dependent(fp8_pack_rows_kernel, dim3(static_cast<unsigned>(cdiv(units, kThreads / 32)), static_cast<unsigned>(d.n)), kThreads, 0,
                            stream, P);
  }
  if (P.strips > 65535u || d.batch * d.n > 65535) return TP_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid(static_cast<unsigned>(cdiv(d.cols, 128)), P.strips, static_cast<unsigned>(d.batch * d.n));
  if (d.gelu) return launch_pack<GELU>(d, grid, P, stream);
  if (d.weights) return launch_pack<WEIGHTED>(d, grid, P, stream);
  return launch_pack<PLAIN>(d, grid, P, stream);
}

tp_status fp8_pack_tokens(const TokenPack& P, cudaStream_t stream) {
  const int64_t blocks = cdiv(P.tokens * (P.e_block / 512), kThreads / 32);
  if (blocks > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
  return launch_dependent(fp8_pack_tokens_kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, P);
}

}  // namespace tpf

namespace {

// Sizes of `batch` matrices [M, N] a tensor.
tp_status check_batch(int p, int64_t batch, int64_t M, int64_t N) {
  TP_TRY(check_sizes(p, M, N, 0, 0, TP_BF16));
  if (batch < 0) return TP_ERR_INVALID_ARG;
  if (batch * p > 65535 || cdiv(M, 128) > 65535) return TP_ERR_UNSUPPORTED_SHAPE;
  return TP_OK;
}

}  // namespace

extern "C" tp_status tp_fp8_pack(const void* const* x, const tp_fp8* q, const tp_fp8* qt, int tiles, tp_epilogue epi, int p, int64_t batch,
                                 int64_t M, int64_t N, cudaStream_t stream) {
  TP_TRY(check_batch(p, batch, M, N));
  if (epi != TP_EPI_NONE && epi != TP_EPI_GELU) return TP_ERR_INVALID_ARG;
  if (tiles != 0 && tiles != 1) return TP_ERR_INVALID_ARG;
  if (q == nullptr && qt == nullptr) return TP_ERR_INVALID_ARG;
  const bool work = M > 0 && N > 0 && batch > 0;
  TP_TRY(check_ptrs(x, p, work));
  TP_TRY(check_fp8(q, p, work && q != nullptr));
  TP_TRY(check_fp8(qt, p, work && qt != nullptr));
  if (!work) return TP_OK;
  RangeList ins, outs;
  add_ranges(&ins, x, p, static_cast<size_t>(batch * M * N) * 2);
  add_fp8(&outs, q, p, M, N, batch);
  add_fp8(&outs, qt, p, N, M, batch);
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  Fp8Pack d;
  d.x = x;
  d.q = q;
  d.qt = qt;
  d.n = p;
  d.batch = batch;
  d.rows = M;
  d.cols = N;
  d.tiles = tiles != 0;
  d.gelu = epi == TP_EPI_GELU;
  return fp8_pack(d, stream);
}

extern "C" tp_status tp_fp8_unpack(const tp_fp8* q, void* const* y, int p, int64_t batch, int64_t M, int64_t N, cudaStream_t stream) {
  TP_TRY(check_batch(p, batch, M, N));
  const bool work = M > 0 && N > 0 && batch > 0;
  TP_TRY(check_fp8(q, p, work));
  TP_TRY(check_ptrs(const_cast<const void* const*>(y), p, work));
  if (!work) return TP_OK;
  RangeList ins, outs;
  add_fp8(&ins, q, p, M, N, batch);
  add_ranges(&outs, const_cast<const void* const*>(y), p, static_cast<size_t>(batch * M * N) * 2);
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  UnpackParams P;
  std::memset(&P, 0, sizeof(P));
  for (int i = 0; i < p; ++i) {
    P.q[i] = static_cast<const uint8_t*>(q[i].q);
    P.e[i] = static_cast<const uint8_t*>(q[i].e);
    P.y[i] = static_cast<__nv_bfloat16*>(y[i]);
  }
  P.rows = M;
  P.cols = N;
  P.ldq = fp8_pitch(N);
  P.e_block = cdiv(N, 512) * 512;
  P.e_mat = static_cast<int64_t>(fp8_e_bytes(M, N));
  P.batch = static_cast<uint32_t>(batch);
  const int64_t blocks = cdiv(M * (N / 8), kThreads);
  if (blocks > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
  return launch_dependent(fp8_unpack_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(batch * p)), kThreads, 0, stream, P);
}
