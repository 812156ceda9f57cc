// The 8-bit sharded Linear: plans, launches and the C ABI of the products.
//
// A product runs on 256 x 256 tiles of CTA pairs or on 128 x 128 tiles of
// single CTAs (fp8_gemm.cuh).  With fewer tiles than SMs the contraction is
// split and the parts, kept in the workspace in fp32, are joined in their
// order by fp8_join_kernel, which then has the epilogue.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "fp8.h"
#include "fp8_gemm.cuh"
#include "tensor_map.h"

using namespace tpf;

namespace {

constexpr int kSMs = 152;
constexpr int kJoinThreads = 256;

// A warp for 128 columns of an output's row: the parts' sum and the epilogue.
__global__ void __launch_bounds__(kJoinThreads) fp8_join_kernel(const __grid_constant__ Fp8GemmParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31, blocks = static_cast<uint32_t>((P.cols + 127) / 128);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = unit / blocks;
  const uint32_t b = static_cast<uint32_t>(unit % blocks), g = blockIdx.y;
  if (row >= P.rows) return;
  if (P.mode == FP8_ROWS) {  // whole tiles of 128 rows are contracted over in a backward pass: all their rows are written
    if (row >= static_cast<int64_t>(__ldcg(P.plan_tiles)) * P.tile_rows) return;
    if (P.tile_rows < 128 && __ldcg(P.plan_slot + row) < 0) return;
  }
  const int32_t c = static_cast<int32_t>(b * 128 + lane * 4);
  const bool in = c < P.cols;
  float v[4] = {};
  if (in) {
    const int64_t step = static_cast<int64_t>(P.groups) * P.part_rows * P.cols;
    const float* from = P.part + (static_cast<int64_t>(g) * P.part_rows + row) * P.cols + c;
#pragma unroll 4
    for (int32_t s = 0; s < P.splits; ++s) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(from + s * step));
      v[0] += f.x;
      v[1] += f.y;
      v[2] += f.z;
      v[3] += f.w;
    }
    const int64_t at = row * P.cols + c;
    if (P.bias[g]) {
      const uint2 w = *reinterpret_cast<const uint2*>(P.bias[g] + c);
      v[0] += bf_lo(w.x);
      v[1] += bf_hi(w.x);
      v[2] += bf_lo(w.y);
      v[3] += bf_hi(w.y);
    }
    if (P.epi == TP_EPI_DGELU) {
      const uint2 h = *reinterpret_cast<const uint2*>(P.aux[g] + at);
      times_gelu_prime2(v[0], v[1], bf_lo(h.x), bf_hi(h.x));
      times_gelu_prime2(v[2], v[3], bf_lo(h.y), bf_hi(h.y));
    } else if (P.epi == TP_EPI_GELU) {
      if (P.aux[g]) *reinterpret_cast<uint2*>(P.aux[g] + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      gelu2(v[0], v[1]);
      gelu2(v[2], v[3]);
    }
    if (P.out[g]) *reinterpret_cast<uint2*>(P.out[g] + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
  if (P.zq[g]) {
    float top = fmaxf(fmaxf(finite_abs(v[0]), finite_abs(v[1])), fmaxf(finite_abs(v[2]), finite_abs(v[3])));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const uint32_t e = fp8_exponent(top);
    *reinterpret_cast<uint32_t*>(P.zq[g] + row * P.zq_ld + c) = fp8_pack4(v[0], v[1], v[2], v[3], fp8_inverse(e));
    if (lane == 0) {
      const int64_t block = row / P.tile_rows;
      P.ze[g][block * P.ze_ld + (b >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(row - block * P.tile_rows), b & 3)] = static_cast<uint8_t>(e);
    }
  }
}

// The values [rows, cols] of an operand, boxes of 128 columns x `box` rows.
bool encode_q(CUtensorMap* m, const void* q, int64_t rows, int64_t cols, int64_t box) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t pitch = static_cast<cuuint64_t>(fp8_pitch(cols));
  const cuuint64_t dims[2] = {pitch, static_cast<cuuint64_t>(rows)}, strides[1] = {pitch};
  const cuuint32_t boxes[2] = {128u, static_cast<cuuint32_t>(box)}, estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Its exponents: 512 bytes x (fours of blocks) x `blocks` (128s of rows), boxes of `box` of the last.
bool encode_e(CUtensorMap* m, const void* e, int64_t blocks, int64_t cols, int box) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t fours = static_cast<cuuint64_t>(cdiv(cols, 512));
  const cuuint64_t dims[3] = {128u, fours, static_cast<cuuint64_t>(blocks)}, strides[2] = {512u, fours * 512u};
  const cuuint32_t boxes[3] = {128u, 1u, static_cast<cuuint32_t>(box)}, estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void*>(e), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CTAS, bool QUANT>
tp_status launch_gemm(const Fp8GemmParams& P, int64_t units, cudaStream_t stream) {
  static KernelInfo info;
  using C = Fp8Cfg<CTAS>;
  void (*k)(Fp8GemmParams) = fp8_gemm_kernel<CTAS, QUANT>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  const int64_t clusters = std::min<int64_t>(units, kSMs / CTAS);
  return launch_dependent(k, dim3(static_cast<unsigned>(clusters * CTAS)), static_cast<unsigned>(C::THREADS), static_cast<size_t>(C::SMEM),
                          stream, P, CTAS);
}

}  // namespace

namespace tpf {

Fp8Launch fp8_plan(int32_t mode, int64_t rows, int64_t cols, int64_t depth, int groups, int segs, int64_t row_tiles, int64_t plan_rows) {
  Fp8Launch l;
  l.ctas = 1;
  l.splits = 1;
  const int64_t kb = segs * cdiv(depth, 128);
  const int64_t pairs = groups * cdiv(rows, 256) * cdiv(cols, 256);
  if (mode != FP8_ROWS && rows > 128 && cols > 128 && pairs >= kSMs / 4) l.ctas = 2;
  if (l.ctas == 1 && mode != FP8_CONTRACT) {
    const int64_t tiles = mode == FP8_ROWS ? row_tiles * cdiv(cols, 128) : groups * cdiv(rows, 128) * cdiv(cols, 128);
    if (tiles > 0 && tiles < kSMs) l.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({16, 2 * kSMs / tiles, kb / 4})));
  }
  l.kb_split = std::max<int64_t>(1, cdiv(kb, l.splits));
  l.splits = static_cast<int>(std::max<int64_t>(1, cdiv(kb, l.kb_split)));
  l.part_rows = mode == FP8_ROWS ? plan_rows : rows;
  l.part_bytes = l.splits > 1 ? static_cast<size_t>(l.splits) * groups * l.part_rows * cols * sizeof(float) : 0;
  return l;
}

tp_status fp8_product(const Fp8Product& d, const Fp8Launch& l, float* part, uint32_t* status, cudaStream_t stream) {
  if (d.rows <= 0 || d.cols <= 0) return TP_OK;
  Fp8GemmParams P;
  std::memset(&P, 0, sizeof(P));
  const bool by_rows = d.mode == FP8_ROWS, contract = d.mode == FP8_CONTRACT;
  P.mode = d.mode;
  P.groups = d.groups;
  P.segs = d.segs;
  P.a_by_g = d.na > 1 && d.groups > 1;
  P.a_by_s = d.na > 1 && d.segs > 1;
  P.b_by_g = d.nb > 1 && d.groups > 1;
  P.b_by_s = d.nb > 1 && d.segs > 1;
  P.tile_rows = by_rows ? static_cast<int32_t>(std::min<int64_t>(d.plan->tile_rows, 128))
                        : static_cast<int32_t>(std::min<int64_t>(128, cdiv(d.rows, 16) * 16));
  P.m_tiles = static_cast<int32_t>(cdiv(d.rows, 128 * l.ctas));
  P.n_tiles = static_cast<int32_t>(cdiv(d.cols, 128 * l.ctas));
  P.kb = static_cast<int32_t>(cdiv(d.depth, 128));
  P.splits = l.splits;
  P.kb_split = static_cast<int32_t>(l.kb_split);
  P.rows = static_cast<int32_t>(d.rows);
  P.cols = static_cast<int32_t>(d.cols);
  P.band = 8;
  P.per = d.per;
  P.eb_blocks = static_cast<int32_t>(cdiv(d.cols, 128));
  if (d.plan) {
    P.plan_tiles = d.plan->tiles;
    P.plan_expert = d.plan->expert;
    P.plan_first = d.plan->first;
    P.plan_slot = d.plan->slot;
    P.max_tiles = static_cast<int32_t>(d.plan->max_tiles);
    P.experts = d.plan->E;
    P.kb_tile = static_cast<int32_t>(d.plan->tile_rows / 128);
  }
  P.epi = d.epi;
  const int outs = contract ? d.groups / d.per : by_rows ? 1 : d.groups;
  for (int i = 0; i < outs; ++i) {
    P.out[i] = static_cast<__nv_bfloat16*>(d.out ? d.out[i] : nullptr);
    P.aux[i] = static_cast<__nv_bfloat16*>(d.aux ? d.aux[i] : nullptr);
    P.bias[i] = static_cast<const __nv_bfloat16*>(d.bias ? d.bias[i] : nullptr);
    P.zq[i] = static_cast<uint8_t*>(d.z ? d.z[i].q : nullptr);
    P.ze[i] = static_cast<uint8_t*>(d.z ? d.z[i].e : nullptr);
  }
  P.zq_ld = fp8_pitch(d.cols);
  P.ze_ld = cdiv(d.cols, 512) * 512;
  P.part = part;
  P.part_rows = l.part_rows;
  P.status = status;
  P.timeout_ns = device_timeout_ns();
  P.drop = static_cast<int32_t>(debug_drop());
  if (d.depth > 0) {
    // rows of an operand's matrix, and blocks of its exponents
    const int64_t a_blocks = by_rows ? d.plan->max_tiles * cdiv(d.plan->tile_rows, 128) : cdiv(d.rows, 128);
    const int64_t b_rows = by_rows ? d.per * d.cols : d.cols, b_blocks = by_rows ? d.per * cdiv(d.cols, 128) : cdiv(d.cols, 128);
    for (int i = 0; i < d.na; ++i)
      if (!encode_q(&P.a[i], d.a[i].q, d.rows, d.depth, contract ? 128 : P.tile_rows) || !encode_e(&P.ea[i], d.a[i].e, a_blocks, d.depth, 1))
        return TP_ERR_CUDA;
    for (int i = 0; i < d.nb; ++i)
      if (!encode_q(&P.b[i], d.b[i].q, b_rows, d.depth, 128) || !encode_e(&P.eb[i], d.b[i].e, b_blocks, d.depth, l.ctas)) return TP_ERR_CUDA;
  }
  const int64_t row_tiles = by_rows ? d.plan->max_tiles : P.m_tiles;
  const int64_t units = d.groups * row_tiles * P.n_tiles * P.splits;
  if (units > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
  const bool quant = d.z != nullptr && l.splits == 1;
  if (l.ctas == 2) {
    TP_TRY(quant ? (launch_gemm<2, true>(P, units, stream)) : (launch_gemm<2, false>(P, units, stream)));
  } else {
    TP_TRY(quant ? (launch_gemm<1, true>(P, units, stream)) : (launch_gemm<1, false>(P, units, stream)));
  }
  if (l.splits == 1 || d.keep_parts) return TP_OK;
  const int64_t warps = d.rows * cdiv(d.cols, 128);
  return launch_dependent(fp8_join_kernel, dim3(static_cast<unsigned>(cdiv(warps, kJoinThreads / 32)), static_cast<unsigned>(d.groups)),
                          kJoinThreads, 0, stream, P);
}

size_t fp8_linear_workspace(tp_op op, int p, int64_t M, int64_t N, int64_t K) {
  size_t most = 0;
  // A backward call with one of its products alone may know M or N as its
  // operands hold it, rounded up.
  const bool back = op == TP_OP_COL_BWD_FP8 || op == TP_OP_ROW_BWD_FP8;
  if (back) M = fp8_pitch(M), N = fp8_pitch(N);
  switch (op) {
    case TP_OP_COL_FP8: most = fp8_plan(FP8_DENSE, M, N, K, p, 1).part_bytes; break;
    case TP_OP_ROW_FP8: most = fp8_plan(FP8_DENSE, M, N, K, 1, p).part_bytes; break;
    case TP_OP_COL_BWD_FP8: most = std::max(fp8_plan(FP8_DENSE, M, K, N, 1, p).part_bytes, fp8_plan(FP8_DENSE, K, N, M, p, 1).part_bytes); break;
    default: most = std::max(fp8_plan(FP8_DENSE, M, K, N, p, 1).part_bytes, fp8_plan(FP8_DENSE, K, N, M, p, 1).part_bytes); break;
  }
  return most ? kDataOffset + most : kStatusBytes;
}

}  // namespace tpf

namespace {

const void* const* in(void* const* a) { return const_cast<const void* const*>(a); }

float* parts_of(void* ws) { return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kDataOffset); }

// A bias is read 8 (or 4) columns at a time.
tp_status check_bias(const void* const* bias, int n, bool work) {
  if (bias == nullptr) return TP_OK;
  for (int i = 0; i < n; ++i) TP_TRY(check_ptr(bias[i], bias[i] != nullptr && work));
  return TP_OK;
}

tp_status forward(bool row, const tp_fp8* x, const tp_fp8* w, const void* const* bias, void* const* y, const tp_fp8* z, void* const* preact,
                  tp_epilogue epi, int p, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_sizes(p, M, N, K, 0, TP_BF16));
  if (epi != TP_EPI_NONE && epi != TP_EPI_GELU) return TP_ERR_INVALID_ARG;
  const int nx = row ? p : 1, ny = row ? 1 : p;
  const bool work = M > 0 && N > 0, sum = work && K > 0;
  if ((y == nullptr) == (z == nullptr)) return TP_ERR_INVALID_ARG;
  if (preact != nullptr && epi != TP_EPI_GELU) return TP_ERR_INVALID_ARG;
  TP_TRY(check_fp8(x, nx, sum));
  TP_TRY(check_fp8(w, p, sum));
  TP_TRY(check_ptrs(in(y), ny, work && y != nullptr));
  TP_TRY(check_fp8(z, ny, work && z != nullptr));
  TP_TRY(check_ptrs(in(preact), ny, work && preact != nullptr));
  TP_TRY(check_bias(bias, ny, work));
  TP_TRY(check_ws(ws, ws_bytes, fp8_linear_workspace(row ? TP_OP_ROW_FP8 : TP_OP_COL_FP8, p, M, N, K)));
  if (!work) return TP_OK;
  {
    RangeList ins, outs;
    add_fp8(&ins, x, nx, M, K);
    add_fp8(&ins, w, p, N, K);
    add_ranges(&ins, bias, ny, static_cast<size_t>(N) * 2);
    add_ranges(&outs, in(y), ny, static_cast<size_t>(M * N) * 2);
    add_fp8(&outs, z, ny, M, N);
    add_ranges(&outs, in(preact), ny, static_cast<size_t>(M * N) * 2);
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  Fp8Product d;
  d.a = x;
  d.na = nx;
  d.b = w;
  d.nb = p;
  d.rows = M;
  d.cols = N;
  d.depth = K;
  d.groups = ny;
  d.segs = nx;
  d.epi = epi;
  d.out = y;
  d.z = z;
  d.aux = preact;
  d.bias = bias;
  return fp8_product(d, fp8_plan(FP8_DENSE, M, N, K, d.groups, d.segs), parts_of(ws), static_cast<uint32_t*>(ws), stream);
}

tp_status backward(bool row, const tp_fp8* xt, const tp_fp8* w, const tp_fp8* dy, const tp_fp8* dyt, void* const* dx, void* const* dw,
                   const void* const* preact, int p, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_sizes(p, M, N, K, 0, TP_BF16));
  if (static_cast<int64_t>(p) * N > (int64_t(1) << 31) - 1) return TP_ERR_UNSUPPORTED_SHAPE;
  const int nx = row ? p : 1, ny = row ? 1 : p;
  const bool work = M > 0 && N > 0 && K > 0;
  if (dx == nullptr && dw == nullptr) return TP_ERR_INVALID_ARG;
  TP_TRY(check_fp8(w, p, work && dx != nullptr));
  TP_TRY(check_fp8(dy, ny, work && dx != nullptr));
  TP_TRY(check_ptrs(in(dx), nx, work && dx != nullptr));
  TP_TRY(check_ptrs(preact, nx, work && dx != nullptr && preact != nullptr));
  TP_TRY(check_fp8(xt, nx, work && dw != nullptr));
  TP_TRY(check_fp8(dyt, ny, work && dw != nullptr));
  TP_TRY(check_ptrs(in(dw), p, work && dw != nullptr));
  TP_TRY(check_ws(ws, ws_bytes, fp8_linear_workspace(row ? TP_OP_ROW_BWD_FP8 : TP_OP_COL_BWD_FP8, p, M, N, K)));
  if (!work) return TP_OK;
  {
    RangeList ins, outs;
    if (dx) {
      add_fp8(&ins, w, p, K, N);
      add_fp8(&ins, dy, ny, M, N);
      add_ranges(&ins, preact, nx, static_cast<size_t>(M * K) * 2);
      add_ranges(&outs, in(dx), nx, static_cast<size_t>(M * K) * 2);
    }
    if (dw) {
      add_fp8(&ins, xt, nx, K, M);
      add_fp8(&ins, dyt, ny, N, M);
      add_ranges(&outs, in(dw), p, static_cast<size_t>(K * N) * 2);
    }
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  if (dx) {
    Fp8Product d;
    d.a = dy;
    d.na = ny;
    d.b = w;
    d.nb = p;
    d.rows = M;
    d.cols = K;
    d.depth = N;
    d.groups = nx;
    d.segs = ny;
    d.out = dx;
    d.epi = preact ? TP_EPI_DGELU : TP_EPI_NONE;
    d.aux = const_cast<void* const*>(preact);
    TP_TRY(fp8_product(d, fp8_plan(FP8_DENSE, M, K, N, d.groups, d.segs), parts_of(ws), static_cast<uint32_t*>(ws), stream));
  }
  if (dw) {
    Fp8Product d;
    d.a = xt;
    d.na = nx;
    d.b = dyt;
    d.nb = ny;
    d.rows = K;
    d.cols = N;
    d.depth = M;
    d.groups = p;
    d.out = dw;
    TP_TRY(fp8_product(d, fp8_plan(FP8_DENSE, K, N, M, p, 1), parts_of(ws), static_cast<uint32_t*>(ws), stream));
  }
  return TP_OK;
}

}  // namespace

extern "C" tp_status tp_col_linear_fwd_fp8(const tp_fp8* x, const tp_fp8* w, const void* const* bias, void* const* y, const tp_fp8* z,
                                           void* const* preact, tp_epilogue epi, int p, int64_t M, int64_t N, int64_t K, void* ws,
                                           size_t ws_bytes, cudaStream_t stream) {
  return forward(false, x, w, bias, y, z, preact, epi, p, M, N, K, ws, ws_bytes, stream);
}

extern "C" tp_status tp_row_linear_fwd_fp8(const tp_fp8* x, const tp_fp8* w, const void* bias, void* y, int p, int64_t M, int64_t N, int64_t K,
                                           void* ws, size_t ws_bytes, cudaStream_t stream) {
  return forward(true, x, w, &bias, &y, nullptr, nullptr, TP_EPI_NONE, p, M, N, K, ws, ws_bytes, stream);
}

extern "C" tp_status tp_col_linear_bwd_fp8(const tp_fp8* xt, const tp_fp8* w, const tp_fp8* dy, const tp_fp8* dyt, void* dx, void* const* dw,
                                           int p, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return backward(false, xt, w, dy, dyt, dx ? &dx : nullptr, dw, nullptr, p, M, N, K, ws, ws_bytes, stream);
}

extern "C" tp_status tp_row_linear_bwd_fp8(const tp_fp8* xt, const tp_fp8* w, const tp_fp8* dy, const tp_fp8* dyt, void* const* dx,
                                           void* const* dw, const void* const* preact, int p, int64_t M, int64_t N, int64_t K, void* ws,
                                           size_t ws_bytes, cudaStream_t stream) {
  return backward(true, xt, w, dy, dyt, dx, dw, preact, p, M, N, K, ws, ws_bytes, stream);
}
