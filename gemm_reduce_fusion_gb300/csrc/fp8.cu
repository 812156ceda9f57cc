// The 8-bit sharded Linear: plans, launches and the C ABI of the products.
//
// A product runs on 256 x 256 tiles of CTA pairs or on 128 x 128 tiles of
// single CTAs (fp8_gemm.cuh), these either whole or as runs: all tiles'
// k-blocks laid end to end and cut into as many equal runs as there are SMs,
// with the parts of a tile that several runs share kept in the workspace in
// fp32 and added up, in the order of the runs, by a second kernel.  (The CTA
// that finishes a tile last can do so itself, but waits a microsecond for
// memory some eight times on the way: the row layer of 77 tokens took 16 us
// so, 11 with the second kernel.)
//
// One token, p = 8, 12288 -> 49152 in all: 94 us, HBM at 0.95 of the copy rate.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "fp8.h"
#include "fp8_gemm.cuh"
#include "tensor_map.h"

using namespace tpf;

namespace {

constexpr int kSMs = 152;
// Runs that share a tile, one more at its ends (16384 deep, 4 and 16 tiles: 3
// runs 25.7 and 19.6 us, 6 runs 21.6 and 17.5, 12 runs the same; 32 tiles of
// 8192: 19.6, 19.6, 21.6).
constexpr int64_t kMostParts = 6;
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

// bf16 results: `mats` matrices [rows, cols], boxes of an epilogue warp's 32 x 32.
bool encode_out(CUtensorMap* m, void* out, int64_t mats, int64_t rows, int64_t cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t n = static_cast<cuuint64_t>(cols), r = static_cast<cuuint64_t>(rows);
  const cuuint64_t dims[3] = {n, r, static_cast<cuuint64_t>(mats)}, strides[2] = {n * 2, n * r * 2};
  const cuuint32_t boxes[3] = {32u, 32u, 1u}, estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, out, dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CTAS, bool QUANT, bool TURNED>
tp_status launch_gemm(const Fp8GemmParams& P, int64_t units, cudaStream_t stream) {
  static KernelInfo info;
  using C = Fp8Cfg<CTAS, TURNED>;
  void (*k)(Fp8GemmParams) = fp8_gemm_kernel<CTAS, QUANT, TURNED>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  const int64_t clusters = std::min<int64_t>(units, kSMs / CTAS);
  return launch_dependent(k, dim3(static_cast<unsigned>(clusters * CTAS)), static_cast<unsigned>(C::THREADS), static_cast<size_t>(C::SMEM),
                          stream, P, CTAS);
}
template <int CTAS, bool TURNED>
tp_status launch_gemm(bool quant, const Fp8GemmParams& P, int64_t units, cudaStream_t stream) {
  return quant ? launch_gemm<CTAS, true, TURNED>(P, units, stream) : launch_gemm<CTAS, false, TURNED>(P, units, stream);
}

}  // namespace

namespace tpf {

static int64_t tile_rows_of(int32_t mode, int64_t rows, const Fp8Plan* plan) {
  return mode == FP8_ROWS ? plan->tile_rows : std::min<int64_t>(128, cdiv(rows, 16) * 16);
}

Fp8Launch fp8_plan(int32_t mode, int64_t rows, int64_t cols, int64_t depth, int groups, int segs, const Fp8Plan* plan) {
  Fp8Launch l;
  l.ctas = 1;
  l.runs = 0;
  l.min_run = 1;
  l.part_bytes = 0;
  if (rows <= 0 || cols <= 0) return l;
  const int64_t kb = segs * cdiv(depth, 128);
  const int64_t pairs = groups * cdiv(rows, 256) * cdiv(cols, 256);
  // Fewer pairs leave more SMs idle than a pair's larger tile saves (4096 deep;
  // pairs against single tiles): 20 and 32 pairs 22 against 17.5 us, 40 pairs
  // 21.6 / 25.7, 60 pairs 22.7 / 25.8, 256 pairs 54 / 60.
  if (mode != FP8_ROWS && rows > 128 && cols > 128 && pairs >= kSMs / 4) l.ctas = 2;
  if (mode == FP8_ROWS && cols > 128 && plan->paired) l.ctas = 2;
  if (l.ctas == 2 || mode == FP8_CONTRACT || kb == 0) return l;
  // Whole tiles leave SMs idle in their last wave, runs do not, but the join
  // kernel and the parts (64 KiB at 128 rows, written and read, at each end of
  // a run) take as long as some 48 k-blocks of 0.13 us (whole tiles against
  // runs: 384 tiles 12288 deep 113.8 / 115.8 us; 32 tiles 16384 deep, with the
  // 128 of 4096 before them, 57.5 / 52.4.  128 rows, weights from HBM, tiles x
  // k-blocks, in front the k-blocks that idle SMs would have done: 8, 20 x 8
  // 5.3 / 9.1; 7, 240 x 16 15.4 / 25.3; 30, 160 x 32 25.0 / 30.2; 30, 80 x 64
  // 22.0 / 29.0; 54, 480 x 64 95.5 / 103.6; 56, 20 x 64 18.5 / 16.3; 61, 160 x
  // 64 44.7 / 44.8; 111, 20 x 128 33.2 / 19.3; 121, 160 x 128 86.9 / 74.3.  16
  // rows change sides at the same place.)
  const int64_t tile_rows = tile_rows_of(mode, rows, plan);
  const int64_t tiles = (mode == FP8_ROWS ? plan->max_tiles : groups * cdiv(rows, 128)) * cdiv(cols, 128);
  if (cdiv(tiles, kSMs) * kb <= tiles * kb / kSMs + 48 || tiles * kb > (int64_t(1) << 30)) return l;
  l.min_run = std::max<int64_t>(std::min<int64_t>(4, kb), cdiv(kb, kMostParts));
  l.runs = static_cast<int>(std::min<int64_t>(kSMs, cdiv(tiles * kb, l.min_run)));
  l.part_bytes = static_cast<size_t>(2 * l.runs * tile_rows) * 128 * sizeof(float);
  return l;
}

tp_status fp8_product(const Fp8Product& d, const Fp8Launch& l, void* part, uint32_t* status, cudaStream_t stream) {
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
  P.tile_rows = static_cast<int32_t>(tile_rows_of(d.mode, d.rows, d.plan));
  // (48 rows 15.5 us as N, 17.5 as M; 64 rows 15.5 / 16.5; 96 and 128 the same)
  const bool turned = by_rows || (l.ctas == 1 && P.tile_rows <= 64);
  P.m_tiles = static_cast<int32_t>(cdiv(d.rows, 128 * l.ctas));
  P.n_tiles = static_cast<int32_t>(cdiv(d.cols, 128 * l.ctas));
  P.kb = static_cast<int32_t>(cdiv(d.depth, 128));
  P.stream = l.runs > 0;
  P.runs = l.runs;
  P.min_run = static_cast<int32_t>(l.min_run);
  P.rows = static_cast<int32_t>(d.rows);
  P.cols = static_cast<int32_t>(d.cols);
  P.band = 8;
  P.per = d.per;
  P.eb_blocks = static_cast<int32_t>(cdiv(d.cols, 128));
  if (d.plan) {
    P.plan_tiles = d.plan->tiles;
    P.plan_expert = d.plan->expert;
    P.plan_pairs = d.plan->pairs;
    P.plan_pair = d.plan->pair;
    P.plan_first = d.plan->first;
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
  P.out32 = d.out32;
  P.part = static_cast<float*>(part);
  P.status = status;
  P.timeout_ns = device_timeout_ns();
  P.drop = static_cast<int32_t>(debug_drop());
  if (d.depth > 0) {
    // rows of an operand's matrix, and blocks of its exponents
    const int64_t a_blocks = by_rows ? d.plan->max_tiles : cdiv(d.rows, 128);
    const int64_t b_rows = by_rows ? d.per * d.cols : d.cols, b_blocks = by_rows ? d.per * cdiv(d.cols, 128) : cdiv(d.cols, 128);
    P.fours = static_cast<int32_t>(cdiv(d.depth, 512));
    for (int i = 0; i < d.na; ++i) {
      if (!encode_q(&P.a[i], d.a[i].q, d.rows, d.depth, P.tile_rows)) return TP_ERR_CUDA;
      if (by_rows && l.ctas == 2 && !encode_q(&P.a[1], d.a[0].q, d.rows, d.depth, 32)) return TP_ERR_CUDA;
      P.ea_at[i] = static_cast<const uint8_t*>(d.a[i].e);
      if (l.ctas == 2 && !encode_e(&P.ea[i], d.a[i].e, a_blocks, d.depth, turned ? 2 : 1)) return TP_ERR_CUDA;
    }
    for (int i = 0; i < d.nb; ++i) {
      if (!encode_q(&P.b[i], d.b[i].q, b_rows, d.depth, 128)) return TP_ERR_CUDA;
      P.eb_at[i] = static_cast<const uint8_t*>(d.b[i].e);
      if (l.ctas == 2 && !encode_e(&P.eb[i], d.b[i].e, b_blocks, d.depth, turned ? 1 : 2)) return TP_ERR_CUDA;
    }
  }
  for (int i = 0; i < outs; ++i)
    if (!turned && d.out && !encode_out(&P.out_map[i], d.out[i], contract ? d.per : 1, d.rows, d.cols)) return TP_ERR_CUDA;
  const int64_t tiles = d.groups * (by_rows ? d.plan->max_tiles : P.m_tiles) * P.n_tiles;
  if (tiles > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
  const int64_t ctas = l.runs > 0 ? l.runs : tiles;
  if (l.ctas == 2) return turned ? launch_gemm<2, true>(d.z != nullptr, P, ctas, stream) : launch_gemm<2, false>(d.z != nullptr, P, ctas, stream);
  TP_TRY(turned ? (launch_gemm<1, true>(d.z != nullptr, P, ctas, stream)) : (launch_gemm<1, false>(d.z != nullptr, P, ctas, stream)));
  if (l.runs < 2) return TP_OK;
  return launch_dependent(fp8_join_kernel, dim3(static_cast<unsigned>(l.runs - 1), static_cast<unsigned>(cdiv(P.tile_rows, kJoinThreads / 32))),
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

void* parts_of(void* ws) { return static_cast<uint8_t*>(ws) + kDataOffset; }

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
  // an empty contraction has zeros for its product, and operands without bytes
  const bool for_x = dx != nullptr && M > 0 && K > 0, for_w = dw != nullptr && N > 0 && K > 0;
  if (dx == nullptr && dw == nullptr) return TP_ERR_INVALID_ARG;
  TP_TRY(check_fp8(w, p, for_x && N > 0));
  TP_TRY(check_fp8(dy, ny, for_x && N > 0));
  TP_TRY(check_ptrs(in(dx), nx, for_x));
  TP_TRY(check_ptrs(preact, nx, for_x && preact != nullptr));
  TP_TRY(check_fp8(xt, nx, for_w && M > 0));
  TP_TRY(check_fp8(dyt, ny, for_w && M > 0));
  TP_TRY(check_ptrs(in(dw), p, for_w));
  TP_TRY(check_ws(ws, ws_bytes, fp8_linear_workspace(row ? TP_OP_ROW_BWD_FP8 : TP_OP_COL_BWD_FP8, p, M, N, K)));
  if (!for_x && !for_w) return TP_OK;
  {
    RangeList ins, outs;
    if (for_x) {
      add_fp8(&ins, w, p, K, N);
      add_fp8(&ins, dy, ny, M, N);
      add_ranges(&ins, preact, nx, static_cast<size_t>(M * K) * 2);
      add_ranges(&outs, in(dx), nx, static_cast<size_t>(M * K) * 2);
    }
    if (for_w) {
      add_fp8(&ins, xt, nx, K, M);
      add_fp8(&ins, dyt, ny, N, M);
      add_ranges(&outs, in(dw), p, static_cast<size_t>(K * N) * 2);
    }
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  if (for_x) {
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
  if (for_w) {
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
