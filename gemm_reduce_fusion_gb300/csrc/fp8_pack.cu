// Packing of matrices into 8-bit operands, rows and transpose at once, and
// their restoring.
//
// A block of 128 along the contraction shares the smallest power of two 2^k
// with max|x| <= 448 * 2^k; x / 2^k is exact, so that rounding to e4m3 is the
// only one.  (Against a scale of max|x| / 448 this costs up to one bit of the
// block's range and none of its precision above 2^-6 of the largest value.)
//
// fp8_pack_kernel: a thread block takes 128 rows x 512 columns, 128 x 128 at a
// time: what it reads gives the row operand from registers and, through
// shared memory, the transposed one, so that x is read once for both.  Four
// blocks of columns fill the words of exponents.  Bound by HBM, 2 bytes read
// and 1 or 2 written an element.
//
// fp8_pack_rows_kernel: a warp for each 128 columns of a row, where there are
// too few rows for the blocks above to fill the GPU.
#include <cuda_bf16.h>

#include <cstring>

#include "fp8.h"
#include "fp8_device.cuh"
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

__device__ __forceinline__ float gelu_if(int32_t on, float v) { return on ? gelu_f(v) : v; }

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

template <bool Q, bool QT>
__global__ void __launch_bounds__(kThreads) fp8_pack_kernel(const __grid_constant__ PackParams P) {
  __shared__ __align__(16) uint8_t tile[QT ? 128 * kPitch : 16];
  __shared__ float red[4][128], row_w[128], warp_top[8];
  __shared__ uint32_t words[128];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t t = blockIdx.z / P.batch, mat = blockIdx.z % P.batch, strip = blockIdx.y;
  if (P.plan_tiles != nullptr && strip * 128 >= __ldcg(P.plan_tiles) * P.tile_rows) return;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const __nv_bfloat16* x = P.x[t] + mat * P.rows * P.cols;
  const int64_t r0 = static_cast<int64_t>(strip) * 128;
  const uint32_t sub = lane >> 4, piece = lane & 15;  // row of two, 16 bytes of a row
  const __nv_bfloat16* src[8];
  float w[8];
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) src[i] = source(P, x, r0 + warp * 16 + i * 2 + sub, w[i]);
  if (QT && P.weights && piece == 0) {
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) row_w[warp * 16 + i * 2 + sub] = w[i];
  }
  if (tid < 128) words[tid] = 0;
  const uint32_t blocks = static_cast<uint32_t>((P.cols + 127) / 128);
  for (uint32_t b = blockIdx.x * 4; b < min(blockIdx.x * 4 + 4, blocks); ++b) {
    const int64_t c = static_cast<int64_t>(b) * 128 + piece * 8;
    uint4 v[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
      v[i] = src[i] != nullptr && c < P.cols ? __ldcs(reinterpret_cast<const uint4*>(src[i] + c)) : make_uint4(0, 0, 0, 0);
    __syncthreads();  // the tile before is used up; `words` is clear
    if (QT) {
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(tile + (warp * 16 + i * 2 + sub) * kPitch + piece * 16) = v[i];
    }
    float all = 0.f;
    if (P.tiles) {
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) all = fmaxf(all, finite_abs(gelu_if(P.gelu, f[j])));
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
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t r = warp * 16 + i * 2 + sub;
        float f[8], top = 0.f;
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = gelu_if(P.gelu, f[j]);
          if (P.weights) f[j] *= w[i];
          top = fmaxf(top, finite_abs(f[j]));
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const uint32_t e = fp8_exponent(P.tiles ? all : top);
        const float inv = fp8_inverse(e);
        if (r0 + r < P.rows) {
          *reinterpret_cast<uint2*>(q + r * P.ldq) = make_uint2(fp8_pack4(f[0], f[1], f[2], f[3], inv), fp8_pack4(f[4], f[5], f[6], f[7], inv));
          if (piece == 0) reinterpret_cast<uint8_t*>(words + (r & 31) * 4 + (r >> 5))[b & 3] = static_cast<uint8_t>(e);
        }
      }
    }
    if (QT) {
      // two columns and a quarter of the rows a thread
      __syncthreads();
      const uint32_t pair = tid & 63, quarter = tid >> 6;
      float lo[32], hi[32], tlo = 0.f, thi = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < 32; ++i) {
        const uint32_t r = quarter * 32 + i;
        const uint32_t u = *reinterpret_cast<const uint32_t*>(tile + r * kPitch + pair * 4);
        lo[i] = gelu_if(P.gelu, bf_lo(u));
        hi[i] = gelu_if(P.gelu, bf_hi(u));
        if (P.weights) {
          lo[i] *= row_w[r];
          hi[i] *= row_w[r];
        }
        tlo = fmaxf(tlo, finite_abs(lo[i]));
        thi = fmaxf(thi, finite_abs(hi[i]));
      }
      if (P.tiles) {
        tlo = thi = all;
      } else {
        *reinterpret_cast<float2*>(&red[quarter][pair * 2]) = make_float2(tlo, thi);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tlo = fmaxf(tlo, red[i][pair * 2]);
          thi = fmaxf(thi, red[i][pair * 2 + 1]);
        }
      }
      const uint32_t elo = fp8_exponent(tlo), ehi = fp8_exponent(thi);
      const float ilo = fp8_inverse(elo), ihi = fp8_inverse(ehi);
      const int64_t col = static_cast<int64_t>(b) * 128 + pair * 2;
      if (col < P.cols) {
        uint8_t* to = P.qt[t] + (mat * P.cols + col) * P.ldqt + r0 + quarter * 32;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int o = half * 16;
          *reinterpret_cast<uint4*>(to + o) =
              make_uint4(fp8_pack4(lo[o], lo[o + 1], lo[o + 2], lo[o + 3], ilo), fp8_pack4(lo[o + 4], lo[o + 5], lo[o + 6], lo[o + 7], ilo),
                         fp8_pack4(lo[o + 8], lo[o + 9], lo[o + 10], lo[o + 11], ilo), fp8_pack4(lo[o + 12], lo[o + 13], lo[o + 14], lo[o + 15], ilo));
          *reinterpret_cast<uint4*>(to + P.ldqt + o) =
              make_uint4(fp8_pack4(hi[o], hi[o + 1], hi[o + 2], hi[o + 3], ihi), fp8_pack4(hi[o + 4], hi[o + 5], hi[o + 6], hi[o + 7], ihi),
                         fp8_pack4(hi[o + 8], hi[o + 9], hi[o + 10], hi[o + 11], ihi), fp8_pack4(hi[o + 12], hi[o + 13], hi[o + 14], hi[o + 15], ihi));
        }
      }
      if (quarter == 0) {  // columns past the matrix: exponent 0
        uint8_t* e = P.et[t] + mat * P.et_mat + b * P.et_block + static_cast<int64_t>(strip >> 2) * 512;
        e[fp8_e_at(pair * 2, strip & 3)] = static_cast<uint8_t>(elo);
        e[fp8_e_at(pair * 2 + 1, strip & 3)] = static_cast<uint8_t>(ehi);
      }
    }
  }
  if (Q) {
    __syncthreads();
    if (tid < 128)
      reinterpret_cast<uint32_t*>(P.e[t] + mat * P.e_mat + strip * P.e_block + static_cast<int64_t>(blockIdx.x) * 512)[tid] = words[tid];
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
  if (P.plan_tiles != nullptr && r >= static_cast<int64_t>(__ldcg(P.plan_tiles)) * P.tile_rows) return;
  float w;
  const __nv_bfloat16* src = source(P, P.x[t], r, w);
  if (src == nullptr) return;  // a row of the plan that no token has
  const int64_t c = static_cast<int64_t>(b) * 128 + lane * 4;
  const uint2 v = c < P.cols ? *reinterpret_cast<const uint2*>(src + c) : make_uint2(0, 0);
  float f[4] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)}, top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = gelu_if(P.gelu, f[j]);
    if (P.weights) f[j] *= w;
    top = fmaxf(top, finite_abs(f[j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const uint32_t e = fp8_exponent(top);
  *reinterpret_cast<uint32_t*>(P.q[t] + r * P.ldq + b * 128 + lane * 4) = fp8_pack4(f[0], f[1], f[2], f[3], fp8_inverse(e));
  if (lane == 0) {
    const int64_t block = r / P.tile_rows;
    P.e[t][block * P.e_block + (b >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(r - block * P.tile_rows), b & 3)] = static_cast<uint8_t>(e);
  }
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
  // A block of 128 rows for each 512 columns fills the GPU's 152 SMs from
  // some 256 rows on; a plan of smaller tiles has its own blocks of exponents.
  const bool few = d.qt == nullptr && !d.tiles && d.batch == 1 && (P.tile_rows < 128 || (d.plan == nullptr && d.rows <= 256));
  if (few) {
    const int64_t units = d.rows * (P.ldq / 128);
    if (cdiv(units, kThreads / 32) > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
    return launch_dependent(fp8_pack_rows_kernel, dim3(static_cast<unsigned>(cdiv(units, kThreads / 32)), static_cast<unsigned>(d.n)), kThreads, 0,
                            stream, P);
  }
  if (P.strips > 65535u || d.batch * d.n > 65535) return TP_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid(static_cast<unsigned>(cdiv(d.cols, 512)), P.strips, static_cast<unsigned>(d.batch * d.n));
  if (d.q && d.qt) return launch_dependent(fp8_pack_kernel<true, true>, grid, kThreads, 0, stream, P);
  if (d.q) return launch_dependent(fp8_pack_kernel<true, false>, grid, kThreads, 0, stream, P);
  return launch_dependent(fp8_pack_kernel<false, true>, grid, kThreads, 0, stream, P);
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
