// Internal interface of the 8-bit products (fp8.cu) and of the packing
// kernels (fp8_pack.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "host_util.h"

namespace tpf {

inline int64_t fp8_pitch(int64_t cols) { return cdiv(cols, 128) * 128; }
inline size_t fp8_q_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows * fp8_pitch(cols)); }
inline size_t fp8_e_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(cdiv(rows, 128) * cdiv(cols, 512)) * 512; }

// Pointers of n operands of `batch` matrices [rows, cols], as an argument.
tp_status check_fp8(const tp_fp8* a, int n, bool need);
void add_fp8(RangeList* v, const tp_fp8* a, int n, int64_t rows, int64_t cols, int64_t batch = 1);

// The rows that the experts take (experts.cu): tiles of `tile_rows` rows of
// one expert each.
struct Fp8Plan {
  const int32_t* tiles;   // row tiles in use
  const int32_t* pairs;   // pairs of them, for CTA pairs: two tiles of an expert, or its last one
  const int32_t* pair;    // first tile of a pair, and its expert << 9 | rows that it has
  const int32_t* expert;  // expert << 9 | rows of a tile
  const int32_t* first;   // first tile of an expert, E + 1
  const int32_t* slot;    // token * k + choice of a row, or -1
  int64_t max_tiles, tile_rows;
  int E, k;
  bool paired;            // products on CTA pairs
};

// ------------------------------------------------------------------ products

enum Fp8Mode : int32_t {
  FP8_DENSE = 0,     // groups x segments of whole matrices
  FP8_ROWS = 1,      // row tiles of the experts: tile -> expert by the plan
  FP8_CONTRACT = 2,  // a product for each expert, contracted over its rows
};

// D = A B^T over segments of the contraction (see fp8_gemm.cuh).
struct Fp8Product {
  int32_t mode = 0;              // Fp8Mode
  const tp_fp8 *a = nullptr, *b = nullptr;
  int na = 1, nb = 1;            // operands
  int64_t rows = 0, cols = 0;    // of an output (FP8_ROWS: rows of the plan)
  int64_t depth = 0;             // of a segment (FP8_CONTRACT: rows of the plan)
  int groups = 1, segs = 1;
  const Fp8Plan* plan = nullptr;
  int per = 1;                   // experts of a shard
  tp_epilogue epi = TP_EPI_NONE;
  void* const* out = nullptr;
  const tp_fp8* z = nullptr;     // or 8-bit outputs
  void* const* aux = nullptr;    // H, out (GELU) or in (DGELU)
  const void* const* bias = nullptr;
  float* out32 = nullptr;        // FP8_ROWS: or fp32 outputs
};

struct Fp8Launch {
  int ctas;
  int runs;           // runs of k-blocks, 0: whole tiles
  int64_t min_run;    // k-blocks of the shortest
  size_t part_bytes;  // of the parts of shared tiles
};
// How a product is run.
Fp8Launch fp8_plan(int32_t mode, int64_t rows, int64_t cols, int64_t depth, int groups, int segs, const Fp8Plan* plan = nullptr);
tp_status fp8_product(const Fp8Product& d, const Fp8Launch& l, void* part, uint32_t* status, cudaStream_t stream);

// ------------------------------------------------------------------ packing

struct Fp8Pack {
  const void* const* x = nullptr;
  const tp_fp8 *q = nullptr, *qt = nullptr;
  int n = 1;
  int64_t batch = 1, rows = 0, cols = 0;
  bool tiles = false, gelu = false;
  const Fp8Plan* plan = nullptr;   // rows of x[0] by the plan's slots, rows = those of the plan
  const float* weights = nullptr;  // a factor for each slot
  bool gather = true;              // false: x[0] has the plan's rows
};
tp_status fp8_pack(const Fp8Pack& p, cudaStream_t stream);
// Tokens into the rows of their slots (fp8_pack.cuh).
struct TokenPack;
tp_status fp8_pack_tokens(const TokenPack& p, cudaStream_t stream);

size_t fp8_linear_workspace(tp_op op, int p, int64_t M, int64_t N, int64_t K);

}  // namespace tpf
