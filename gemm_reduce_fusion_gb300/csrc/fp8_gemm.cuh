// Persistent tcgen05 GEMM on 8-bit operands with a power of two for each
// block of 128 along the contraction (see tp_fused.h for the operands):
//   D[m, n] = sum_b 2^(ea[m, b] + eb[n, b] - 254) sum_{k in block b} A[m, k] B[n, k].
// The scales are applied by the tensor cores (kind::mxf8f6f4, one scale for
// each row and 32 of the contraction; the four steps of a block use the same
// byte), so that the accumulator stays in tensor memory for the whole
// contraction and the ranks' segments, and no multiplication by a scale is
// left for the epilogue.  An operand's exponents lie in memory as tensor
// memory wants them: 512 bytes hold four blocks of 128 rows, which one copy
// brings to shared memory and one tcgen05.cp to tensor memory every four
// k-blocks; the byte is picked by the instruction descriptor.
//
// CTAS = 1: 128 x 128 tiles of one CTA; CTAS = 2: 256 x 256 tiles of a CTA
// pair, each of which holds 128 rows of A and of B.  A k-block is 128 deep:
// 32 KiB a CTA in both.  A pair moves 64 bytes an SM and cycle from L2 at the
// full MMA rate, a single CTA's tile 128.  TURNED: A's rows are the N of the
// MMAs, B's the M (see there).
//
// Roles: warp 0 loads, warp 1 issues the MMAs, the others (eight; 16 of a
// TURNED pair's CTA) are the epilogue, which overlaps the next tile's MMAs on
// the other accumulator.  With 256 columns the two accumulators share 32
// columns of tensor memory, which the epilogue reads first: 480 of the 512
// columns, the rest for the scales.
//
// Loads and MMAs are issued by whole warps, of which one lane executes them:
// the compiler then keeps their operands in uniform registers (in code of one
// lane each MMA cost its thread some 120 cycles: a k-block 0.28 us, so 0.13).
//
// 4096 x 16384 x 4096 and the like, 0.55 TFLOP, take 163-182 us, 3.0-3.4
// PFLOP/s; without the loads 140-150 us, without the MMAs 115.  With two or
// three k-blocks a tile (the experts' weight gradients) what is left is the
// way from one tile's last MMA to the next tile's first, by the epilogue's
// first read: 58 us of 82 with nothing stored.
//
// Every wait is bounded (device_wait.cuh).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "device_wait.cuh"
#include "fp8.h"
#include "fp8_device.cuh"
#include "gelu.cuh"
#include "vec_util.cuh"

namespace tpf {

struct Fp8GemmParams {
  CUtensorMap a[8], b[8], ea[8], eb[8];  // ea, eb: CTAS = 2; a[1] of FP8_ROWS: a[0]'s in 32 rows at a time
  CUtensorMap out_map[8];                // bf16 results, not TURNED
  const uint8_t *ea_at[8], *eb_at[8];    // CTAS = 1: the exponents themselves
  int32_t fours;                         // of k-blocks, in a block of exponents
  int32_t mode;
  int32_t groups, segs;         // outputs; contraction segments (ranks reduced)
  int32_t a_by_g, a_by_s, b_by_g, b_by_s;
  int32_t m_tiles, n_tiles;     // of a group (FP8_ROWS: m_tiles from the plan)
  int32_t kb;                   // k-blocks of a segment
  int32_t stream;               // runs of k-blocks instead of whole tiles (CTAS = 1)
  int32_t min_run;              // the shortest of them
  int32_t rows, cols;           // of an output (FP8_ROWS: rows not used)
  int32_t tile_rows;            // rows of an A tile that are loaded (CTAS = 1: 16 .. 128)
  int32_t band;                 // m-tiles that go together through the n-tiles
  int32_t per, eb_blocks;       // experts of a shard; 128-row blocks of an expert's B
  const int32_t* plan_tiles;    // FP8_ROWS, FP8_CONTRACT: row tiles in use
  const int32_t* plan_expert;   // FP8_ROWS: expert of a row tile, and how many rows it has (expert_rows)
  const int32_t *plan_pairs, *plan_pair;  // FP8_ROWS, CTAS = 2: pairs of row tiles; of each the first tile, expert and rows
  const int32_t* plan_first;    // FP8_CONTRACT: first row tile of an expert, E + 1
  int32_t max_tiles, experts;   // bounds of what the plan may say
  int32_t kb_tile;              // FP8_CONTRACT: k-blocks of a row tile
  int32_t epi;                  // tp_epilogue
  __nv_bfloat16* out[8];        // bf16 results, or null
  __nv_bfloat16* aux[8];        // GELU: H out, or null; DGELU: H in
  uint8_t* zq[8];               // 8-bit results, or null
  uint8_t* ze[8];
  const __nv_bfloat16* bias[8];
  int64_t zq_ld, ze_ld;         // bytes of a row of zq, of 128 rows of ze
  float* out32;                 // FP8_ROWS: fp32 results instead, or null
  float* part;                  // fp32 sums of the tiles that runs share
  int32_t runs;
  uint32_t* status;
  uint64_t timeout_ns;
  int32_t drop;                 // test hook (TP_DEBUG_DROP_LOAD)
};

// A word of the plan: an expert and the rows, up to 256, that its tile or pair of tiles has.
__device__ __forceinline__ int32_t word_rows(int32_t w) { return min(max(w & 511, 1), 256); }
__device__ __forceinline__ int32_t word_expert(int32_t w) { return w >> 9; }

// Places of a stage: A's k-blocks, of `rows` rows each, then B's.  (With 65 to
// 127 rows the MMA reads 128 from where A begins: what lies behind its rows
// goes into rows of D that are not used.)
template <int CTAS>
struct Fp8Ring {
  uint32_t base, a_bytes, stage_bytes;
  int count;
  __device__ __forceinline__ Fp8Ring(uint32_t base, int32_t rows);
  __device__ __forceinline__ uint32_t a(int stage, int d) const { return base + stage * stage_bytes + d * a_bytes; }
  __device__ __forceinline__ uint32_t b(int stage, int d) const;
  __device__ __forceinline__ uint32_t e(int stage, int d) const;
};

// TURNED: the rows are the N of the MMAs.
template <int CTAS, bool TURNED = false>
struct Fp8Cfg {
  static constexpr int BN = 128 * CTAS;
  // A stage has two k-blocks of A, two of B and their exponents.  (With one,
  // the loads alone of the MLP's launches took 148 us, with two 115: each
  // stage costs its loader some 150 ns beside the copies.)  A pair has three
  // stages; a single CTA's are shorter, and more, where a tile has few rows.
  static constexpr int DEEP = 2;
  static constexpr uint32_t B_BYTES = 128 * 128;  // of a k-block
  static constexpr uint32_t EA_BYTES = 512, EB_BYTES = 512 * CTAS, E_BYTES = EA_BYTES + EB_BYTES;
  static constexpr uint32_t RING = 192 * 1024;
  static constexpr int MAX_STAGES = CTAS == 1 ? 5 : 3;
  static constexpr int EPI_WARPS = TURNED ? 8 * CTAS : 8;
  static constexpr int COLS = BN / 2;  // of an epilogue warp, not TURNED
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr uint32_t STG_BYTES = 2048;  // staging of an epilogue warp, not TURNED
  static constexpr uint32_t E_OFF = RING, STG_OFF = E_OFF + MAX_STAGES * DEEP * E_BYTES, BAR_OFF = STG_OFF + 8 * STG_BYTES;
  static constexpr uint32_t SMEM = 1024 + BAR_OFF + 256;
  // tensor memory: accumulators of BN columns at 0 and ACC1, scales from SF
  // on (A 4 columns, B 4 CTAS), two of them by turns
  static constexpr uint32_t SHARED = CTAS == 1 ? 0 : 32;  // columns of both accumulators
  static constexpr uint32_t ACC1 = BN - SHARED, SF = 480;
  static_assert(ACC1 + BN <= SF, "accumulators before the scales");
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};

template <int CTAS>
__device__ __forceinline__ Fp8Ring<CTAS>::Fp8Ring(uint32_t at, int32_t rows) {
  using C = Fp8Cfg<CTAS>;
  base = at;
  a_bytes = (CTAS == 2 ? 128u : static_cast<uint32_t>(rows)) * 128u;
  stage_bytes = C::DEEP * (a_bytes + C::B_BYTES);
  count = CTAS == 2 ? C::MAX_STAGES : min(static_cast<int>(C::RING / stage_bytes), C::MAX_STAGES);
}
template <int CTAS>
__device__ __forceinline__ uint32_t Fp8Ring<CTAS>::b(int stage, int d) const {
  return base + stage * stage_bytes + Fp8Cfg<CTAS>::DEEP * a_bytes + d * Fp8Cfg<CTAS>::B_BYTES;
}
template <int CTAS>
__device__ __forceinline__ uint32_t Fp8Ring<CTAS>::e(int stage, int d) const {
  return base + Fp8Cfg<CTAS>::E_OFF + (stage * Fp8Cfg<CTAS>::DEEP + d) * Fp8Cfg<CTAS>::E_BYTES;
}

struct Fp8Unit {
  int32_t t;          // tile
  int32_t g, nt;
  int32_t tile;       // row tile (of CTA 0)
  int32_t rows;       // that it has (with few, and CTA 1's)
  int32_t q0, q1;     // k-blocks
  int32_t a_row, ea;  // first row of A's tile (CTA 0), its block of exponents
  int32_t b_row, eb;
  int32_t bi;         // map of B (FP8_ROWS: the expert's shard)
  int64_t out_off;    // FP8_CONTRACT: the expert's place in its shard
};

// What all lanes of a warp have, in a form that the compiler knows to be so.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

template <int CTAS>
__device__ __forceinline__ int32_t fp8_tiles(const Fp8GemmParams& P) {
  if (P.mode == FP8_ROWS) return min(uniform(__ldcg(CTAS == 2 ? P.plan_pairs : P.plan_tiles)), P.max_tiles) * P.n_tiles;
  return P.groups * P.m_tiles * P.n_tiles;
}

// What the plan says about a tile.  It is read a tile ahead: from L2 that
// takes as long as two k-blocks.
struct Fp8Words {
  int32_t a, b;
};
template <int CTAS>
__device__ __forceinline__ Fp8Words fp8_words(const Fp8GemmParams& P, int32_t t) {
  Fp8Words w = {0, 0};
  if (P.mode == FP8_ROWS) {
    const int32_t v = t / P.n_tiles;
    if (CTAS == 2) {
      w.a = __ldcg(P.plan_pair + 2 * v);
      w.b = __ldcg(P.plan_pair + 2 * v + 1);
    } else {
      w.a = v;
      w.b = __ldcg(P.plan_expert + v);
    }
  } else if (P.mode == FP8_CONTRACT) {
    const int32_t g = t / (P.m_tiles * P.n_tiles);
    w.a = __ldcg(P.plan_first + g);
    w.b = __ldcg(P.plan_first + g + 1);
  }
  return w;
}

template <int CTAS>
__device__ __forceinline__ Fp8Unit fp8_unit(const Fp8GemmParams& P, int32_t t, const Fp8Words& words) {
  Fp8Unit u;
  u.t = t;
  int32_t v = t;
  u.out_off = 0;
  u.q0 = 0;
  u.q1 = P.segs * P.kb;
  if (P.mode == FP8_ROWS) {
    // an expert's weights are read by its row tiles one after the other
    u.nt = v % P.n_tiles;
    u.tile = min(max(uniform(words.a), 0), P.max_tiles - 1);
    const int32_t word = uniform(words.b), e = min(max(word_expert(word), 0), P.experts - 1), local = e % P.per;
    u.rows = min(word_rows(word), P.tile_rows * CTAS);
    u.g = 0;
    u.bi = e / P.per;
    u.a_row = u.tile * P.tile_rows;
    u.ea = u.tile;
    u.b_row = local * P.cols + u.nt * Fp8Cfg<CTAS>::BN;
    u.eb = local * P.eb_blocks + u.nt * CTAS;
    return u;
  }
  const int32_t per_group = P.m_tiles * P.n_tiles;
  u.g = v / per_group;
  v -= u.g * per_group;
  const int32_t strip = v / (P.band * P.n_tiles), first = strip * P.band;
  const int32_t tall = min(P.band, P.m_tiles - first);
  v -= first * P.n_tiles;
  u.nt = v / tall;
  u.tile = (first + v % tall) * CTAS;
  u.bi = 0;
  u.a_row = u.tile * 128;
  u.rows = min(P.rows - u.a_row, P.tile_rows * CTAS);
  u.ea = u.tile;
  u.b_row = u.nt * Fp8Cfg<CTAS>::BN;
  u.eb = u.nt * CTAS;
  if (P.mode == FP8_CONTRACT) {
    u.q0 = min(max(uniform(words.a), 0), P.max_tiles) * P.kb_tile;
    u.q1 = min(uniform(words.b), P.max_tiles) * P.kb_tile;
    u.bi = u.g / P.per;  // of the outputs
    u.out_off = static_cast<int64_t>(u.g % P.per) * P.rows * P.cols;
  }
  return u;
}

// What a CTA (or pair) goes through: whole tiles, `stride` apart, or with
// P.stream its run of all tiles' k-blocks laid end to end.
template <int CTAS>
struct Fp8Walk {
  int32_t at, end, stride;  // tiles; or k-blocks, stride 0
  int32_t run, depth;       // k-blocks of a run, of a tile
  Fp8Words words;           // of the next

  __device__ __forceinline__ Fp8Walk(const Fp8GemmParams& P) {
    const int32_t me = static_cast<int32_t>(blockIdx.x) / CTAS, all = static_cast<int32_t>(gridDim.x) / CTAS, tiles = fp8_tiles<CTAS>(P);
    depth = P.segs * P.kb;
    if (CTAS == 1 && P.stream) {
      const int32_t work = tiles * depth;
      run = max((work + P.runs - 1) / P.runs, P.min_run);
      at = min(me * run, work);
      end = min(at + run, work);
      stride = 0;
    } else {
      run = 0;
      at = me;
      end = tiles;
      stride = all;
    }
    if (at < end) words = fp8_words<CTAS>(P, stride ? at : at / depth);
  }
  __device__ __forceinline__ bool next(const Fp8GemmParams& P, Fp8Unit& u) {
    if (at >= end) return false;
    if (CTAS == 1 && stride == 0) {
      const int32_t t = at / depth;
      u = fp8_unit<CTAS>(P, t, words);
      u.q0 = at - t * depth;
      u.q1 = min(depth, u.q0 + end - at);
      at += u.q1 - u.q0;
    } else {
      u = fp8_unit<CTAS>(P, at, words);
      at += stride;
    }
    if (at < end) words = fp8_words<CTAS>(P, stride ? at : at / depth);
    return true;
  }
};

// The maps of k-block q and its place in them.
struct Fp8Block {
  int32_t ai, bi, k;
};
__device__ __forceinline__ Fp8Block fp8_block(const Fp8GemmParams& P, const Fp8Unit& u, int32_t q) {
  Fp8Block b;
  if (P.mode == FP8_DENSE) {
    const int32_t s = P.segs == 1 || P.kb == 0 ? 0 : q / P.kb;  // no k-block: an empty contraction
    b.k = q - s * P.kb;
    b.ai = P.a_by_g * u.g + P.a_by_s * s;
    b.bi = P.b_by_g * u.g + P.b_by_s * s;
  } else {
    b.k = q;
    b.ai = 0;
    b.bi = P.mode == FP8_ROWS ? u.bi : 0;
  }
  return b;
}

// ------------------------------------------------------------------ epilogue

// 32 rows x 64 bytes of the warp's staging buffer, 16-byte pieces swizzled.
__device__ __forceinline__ uint32_t stg_at(uint32_t stg, uint32_t row, uint32_t piece) {
  return stg + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Staging buffer -> memory, eight rows an instruction, 64 bytes each.
// `bytes`: of a row that are the matrix's.
__device__ __forceinline__ void stg_out(uint32_t stg, uint8_t* to, int64_t pitch, int32_t rows, int32_t bytes, uint32_t lane) {
  __syncwarp();
  const uint32_t piece = lane & 3;
  if (static_cast<int32_t>(piece * 16) < bytes) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = i * 8 + (lane >> 2);
      if (static_cast<int32_t>(r) < rows) *reinterpret_cast<uint4*>(to + r * pitch + piece * 16) = ld_shared_v4(stg_at(stg, r, piece));
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void stg_in(uint32_t stg, const uint8_t* from, int64_t pitch, int32_t rows, int32_t bytes, uint32_t lane) {
  const uint32_t piece = lane & 3;
  const bool some = static_cast<int32_t>(piece * 16) < bytes;
  uint4 v[4];
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t r = i * 8 + (lane >> 2);
    v[i] = some && static_cast<int32_t>(r) < rows ? *reinterpret_cast<const uint4*>(from + r * pitch + piece * 16) : make_uint4(0, 0, 0, 0);
  }
  __syncwarp();
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) st_shared_v4(stg_at(stg, i * 8 + (lane >> 2), piece), v[i]);
  __syncwarp();
}

__device__ __forceinline__ void add_bias(float (&v)[32], const __nv_bfloat16* bias, int32_t c, int32_t cols) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    if (c + i < cols) {
      float b[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(bias + c + i)), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i + j] += b[j];
    }
  }
}

__device__ __forceinline__ void stage_bf16(const float (&v)[32], uint32_t stg, uint32_t row) {
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    st_shared_v4(stg_at(stg, row, i),
                 make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]), pack_bf16(v[8 * i + 4], v[8 * i + 5]),
                            pack_bf16(v[8 * i + 6], v[8 * i + 7])));
}

// 32 columns of a warp's of the accumulator.
struct FromTmem {
  uint32_t taddr;
  bool empty;  // no contraction: zeros
  __device__ __forceinline__ void operator()(int j, float (&v)[32]) const {
    if (empty) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
      return;
    }
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + j * 32, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  }
};

// One warp's 32 rows x COLS columns of a finished tile.  `released` is called
// once the columns that both accumulators have are in registers: the 32 that
// drain_bf16 takes first.
struct Fp8Place {
  int32_t row, rows;  // first row in the output, rows of the warp that are the output's
  int32_t col;        // first column
  int32_t o;          // which output
  int64_t off;        // elements before the output's matrix
  int32_t mat;        // and matrices
  int32_t eblock, erow;  // 128 rows of exponents of an 8-bit result, first row in them
};

template <int COLS, typename Released>
__device__ __forceinline__ void drain_bf16(const Fp8GemmParams& P, const Fp8Place& w, const FromTmem& load, bool last_first, uint32_t stg,
                                           uint32_t lane, Released released) {
  const int64_t pitch = static_cast<int64_t>(P.cols) * 2;
  const __nv_bfloat16* bias = P.bias[w.o];
#pragma unroll 1
  for (int part = 0; part < COLS / 32; ++part) {
    const int j = last_first ? (part + COLS / 32 - 1) % (COLS / 32) : part;
    const int32_t c = w.col + j * 32, bytes = min(P.cols - c, 32) * 2;
    const int64_t at = (w.off + static_cast<int64_t>(w.row) * P.cols + c) * 2;
    float v[32];
    load(j, v);
    if (part == 0) released();
    if (bytes <= 0) continue;
    if (bias) add_bias(v, bias, c, P.cols);
    if (lane == 0) bulk_wait_read_all();  // the staging buffer is free
    __syncwarp();
    if (P.epi == TP_EPI_DGELU) {
      stg_in(stg, reinterpret_cast<const uint8_t*>(P.aux[w.o]) + at, pitch, w.rows, bytes, lane);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        float h[8];
        unpack8(ld_shared_v4(stg_at(stg, lane, i)), h);
#pragma unroll
        for (int m = 0; m < 8; m += 2) times_gelu_prime2(v[8 * i + m], v[8 * i + m + 1], h[m], h[m + 1]);
      }
      __syncwarp();
    } else if (P.epi == TP_EPI_GELU) {
      if (P.aux[w.o]) {
        stage_bf16(v, stg, lane);
        stg_out(stg, reinterpret_cast<uint8_t*>(P.aux[w.o]) + at, pitch, w.rows, bytes, lane);
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) gelu2(v[i], v[i + 1]);
    }
    stage_bf16(v, stg, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      store_3d(&P.out_map[w.o], stg, c, w.row, w.mat);
      bulk_commit();
    }
  }
}

// The same with the result in 8 bits.  COLS = 128: a thread has the columns of
// its row that share an exponent; 64: half of them, and `red` (of this warp's
// rows: [2][32], `half` its own) and a barrier with the other half's warp.
template <int COLS, typename Released>
__device__ __forceinline__ void drain_fp8(const Fp8GemmParams& P, const Fp8Place& w, const FromTmem& load, uint32_t stg, uint32_t lane,
                                          float (*red)[32], uint32_t half, uint32_t barrier, Released released) {
  const int64_t pitch = static_cast<int64_t>(P.cols) * 2;
  const __nv_bfloat16* bias = P.bias[w.o];
  float v[COLS / 32][32];
#pragma unroll
  for (int j = 0; j < COLS / 32; ++j) load(j, v[j]);
  released();
  const int32_t block = w.col / 128;
  if (block * 128 >= P.cols) return;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < COLS / 32; ++j) {
    const int32_t c = w.col + j * 32, bytes = min(P.cols - c, 32) * 2;
    const int64_t at = (w.off + static_cast<int64_t>(w.row) * P.cols + c) * 2;
    if (bias) add_bias(v[j], bias, c, P.cols);
    if (P.aux[w.o] && bytes > 0) {
      stage_bf16(v[j], stg, lane);
      stg_out(stg, reinterpret_cast<uint8_t*>(P.aux[w.o]) + at, pitch, w.rows, bytes, lane);
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      if (P.epi == TP_EPI_GELU) gelu2_to8(v[j][i], v[j][i + 1]);
      if (c + (i & ~7) >= P.cols) v[j][i] = v[j][i + 1] = 0.f;  // past the matrix, in eights: zeros
      top = fmaxf(top, fmaxf(finite_abs(v[j][i]), finite_abs(v[j][i + 1])));
    }
  }
  if constexpr (COLS == 64) {
    red[half][lane] = top;
    asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory");
    top = fmaxf(top, red[half ^ 1][lane]);
    asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory");  // read, before the next tile's is written
  }
  const uint32_t e = fp8_exponent(top);
  const float inv = fp8_inverse(e);
#pragma unroll
  for (uint32_t piece = 0; piece < COLS / 64; ++piece) {
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      uint32_t o[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t n = piece * 64 + j * 16 + i * 4;
        o[i] = fp8_pack4(v[n / 32][n % 32], v[n / 32][n % 32 + 1], v[n / 32][n % 32 + 2], v[n / 32][n % 32 + 3], inv);
      }
      st_shared_v4(stg_at(stg, lane, j), make_uint4(o[0], o[1], o[2], o[3]));
    }
    stg_out(stg, P.zq[w.o] + w.row * P.zq_ld + w.col + piece * 64, P.zq_ld, w.rows, 64, lane);
  }
  if (static_cast<int32_t>(lane) < w.rows && (COLS == 128 || half == 0))
    P.ze[w.o][w.eblock * P.ze_ld + (block >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(w.erow) + lane, block & 3)] = static_cast<uint8_t>(e);
}

// fp32 sums of a tile that several runs share: COLS columns of [rows][128].
template <int COLS>
__device__ __forceinline__ void drain_sums(float* to, int32_t rows, const FromTmem& load, uint32_t stg, uint32_t lane) {
#pragma unroll 1
  for (int j = 0; j < COLS / 32; ++j) {
    float v[32];
    load(j, v);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const int n = half * 16 + i * 4;
        st_shared_v4(stg_at(stg, lane, i), make_uint4(__float_as_uint(v[n]), __float_as_uint(v[n + 1]), __float_as_uint(v[n + 2]),
                                                      __float_as_uint(v[n + 3])));
      }
      stg_out(stg, reinterpret_cast<uint8_t*>(to + j * 32 + half * 16), 128 * 4, rows, 64, lane);
    }
  }
}

// ------------------------------------------------------------------ rows as the N of the MMAs
//
// With the rows as N and the columns (the weights' rows) as M a tile costs
// what its rows cost, in steps of 16 (32 of a pair): the tiles of few rows of
// a decode step, and the experts' tiles, of which each expert's last is
// filled by chance.  As M a tile of few rows took 530 cycles a k-block,
// whatever the rows, and an expert's last pair of tiles counted as 256.
//
// A lane of tensor memory has a column then, a column of it a row.  Neighbours
// exchange halves (two bf16, or four bytes of four rows) so that each stores
// four bytes of a row; 32 lanes write 64 or 32 bytes of each.  (Turned in
// shared memory instead, 32 rows at a time with two barriers, 4096 tokens
// through the experts took 513 us, so 501; with eight warps, and lanes that
// exchange, 507.)

template <int THREADS>
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "n"(THREADS)
      : "memory");
  return all != 0;
}

// Two rows of a lane's column -> the column and its neighbour of one of them
// (even lanes the first), and back.
__device__ __forceinline__ uint32_t turn2(uint32_t own, uint32_t odd) {
  const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
  return __byte_perm(own, other, odd ? 0x3276 : 0x5410);
}
// Four rows of a lane's column, a byte each -> four columns of row lane % 4.
__device__ __forceinline__ uint32_t turn4(uint32_t own, uint32_t lane) {
  uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
  own = __byte_perm(own, other, (lane & 1) ? 0x3715 : 0x6240);
  other = __shfl_xor_sync(0xFFFFFFFFu, own, 2);
  return __byte_perm(own, other, (lane & 2) ? 0x3276 : 0x5410);
}

struct Fp8Lane {
  uint32_t lane, quarter;        // 32 columns
  uint32_t part, parts;          // every parts-th chunk of 16 rows
  uint32_t barrier;              // of the four quarters
};

// n <= N of the 16 rows of a chunk, from `first` of the tile on.
template <bool QUANT, int N>
__device__ __forceinline__ void turned_chunk(const Fp8GemmParams& P, const Fp8Place& w, int32_t first, int32_t n, float (&v)[16], float bias,
                                             int32_t col, const Fp8Lane& me, float (*exchange)[16]) {
  const int32_t odd = me.lane & 1;
  const bool in = col < P.cols;
  // of the lane's row of two, its column and the neighbour's
  const int64_t at2 = w.off + (static_cast<int64_t>(w.row) + first + odd) * P.cols + (col & ~1);
  const int64_t two = static_cast<int64_t>(P.cols) * 2;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] += bias;
  if (P.epi == TP_EPI_DGELU) {
    uint32_t h[N / 2];
    const __nv_bfloat16* from = P.aux[w.o] + at2;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) h[j] = in && 2 * j + odd < n ? *reinterpret_cast<const uint32_t*>(from + j * two) : 0u;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const uint32_t f = turn2(h[j], odd);
      times_gelu_prime2(v[2 * j], v[2 * j + 1], bf_lo(f), bf_hi(f));
    }
  } else if (P.epi == TP_EPI_GELU) {
    if (P.aux[w.o]) {
      __nv_bfloat16* to = P.aux[w.o] + at2;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const uint32_t o = turn2(pack_bf16(v[2 * j], v[2 * j + 1]), odd);
        if (in && 2 * j + odd < n) *reinterpret_cast<uint32_t*>(to + j * two) = o;
      }
    }
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      if constexpr (QUANT) gelu2_to8(v[j], v[j + 1]);
      else gelu2(v[j], v[j + 1]);
    }
  }
  if constexpr (!QUANT) {
    if (P.out32) {
      float* to = P.out32 + (static_cast<int64_t>(w.row) + first) * P.cols + col;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (in && j < n) to[static_cast<int64_t>(j) * P.cols] = v[j];
      return;
    }
    __nv_bfloat16* to = P.out[w.o] + at2;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const uint32_t o = turn2(pack_bf16(v[2 * j], v[2 * j + 1]), odd);
      if (in && 2 * j + odd < n) *reinterpret_cast<uint32_t*>(to + j * two) = o;
    }
  } else {
    uint32_t top[N], most = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!in || j >= n) v[j] = 0.f;  // past the matrix: zeros
      top[j] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v[j])));
      most = max(most, top[j]);
    }
    const bool finite = most < 0x7F800000u;
    if (!finite) {
#pragma unroll
      for (int j = 0; j < N; ++j) top[j] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(finite_abs(v[j])));
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) mine = me.lane == j ? top[j] : mine;
    if (me.lane < 16) exchange[me.quarter][me.lane] = __uint_as_float(mine);
    asm volatile("bar.sync %0, 128;" ::"r"(me.barrier) : "memory");
    float all = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) all = fmaxf(all, exchange[j][me.lane & 15]);
    const uint32_t e = fp8_exponent(all);
    const float inv = fp8_inverse(e);
    const int32_t block = w.col / 128;
    if (me.quarter == 0 && static_cast<int32_t>(me.lane) < n)
      P.ze[w.o][(w.eblock + (first >> 7)) * P.ze_ld + (block >> 2) * 512 + fp8_e_at((first & 127) + me.lane, block & 3)] = static_cast<uint8_t>(e);
    uint8_t* to = P.zq[w.o] + (static_cast<int64_t>(w.row) + first + (me.lane & 3)) * P.zq_ld + (col & ~3);
    const int64_t four = P.zq_ld * 4;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      float f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = v[j + m] * __shfl_sync(0xFFFFFFFFu, inv, j + m);
      const uint32_t o = turn4(finite ? fp8_pack4_finite(f[0], f[1], f[2], f[3], 1.f) : fp8_pack4(f[0], f[1], f[2], f[3], 1.f), me.lane);
      if (j + static_cast<int32_t>(me.lane & 3) < n) *reinterpret_cast<uint32_t*>(to + (j / 4) * four) = o;
    }
  }
}

// A finished tile, `rows` rows from w.row on, 128 columns from w.col on.
// sums: fp32 sums [rows][128] instead of results, or null.  red: [2][4][16].
template <bool QUANT, typename Released>
__device__ __forceinline__ void drain_turned(const Fp8GemmParams& P, const Fp8Place& w, int32_t rows, float* sums, uint32_t taddr, bool empty,
                                             bool last_first, const Fp8Lane& me, float (*red)[4][16], uint32_t& turn, Released released) {
  const int32_t part = static_cast<int32_t>(me.part), parts = static_cast<int32_t>(me.parts);
  const int32_t mine = ((rows + 15) / 16 - part + parts - 1) / parts;
  if (mine <= 0 || w.col >= P.cols) {
    released();
    return;
  }
  const int32_t in_tile = static_cast<int32_t>(me.quarter * 32 + me.lane), col = w.col + in_tile;
  const float bias = P.bias[w.o] && col < P.cols ? __bfloat162float(P.bias[w.o][col]) : 0.f;
#pragma unroll 1
  for (int32_t i = 0; i < mine; ++i) {
    const int32_t first = (part + parts * (last_first ? mine - 1 - i : i)) * 16, n = min(rows - first, 16);
    float v[16];
    if (empty) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
    } else {
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + first, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
    }
    if (i == 0) released();
    if (sums) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < n) __stcg(sums + (first + j) * 128 + in_tile, v[j]);
      continue;
    }
    float (*exchange)[16] = red[QUANT ? turn++ & 1 : 0];
    if (n <= 4) turned_chunk<QUANT, 4>(P, w, first, n, v, bias, col, me, exchange);
    else turned_chunk<QUANT, 16>(P, w, first, n, v, bias, col, me, exchange);
  }
}

// ------------------------------------------------------------------ tiles that several runs share (CTAS = 1)
//
// A run has at most two parts, [tile_rows][128] each: of the tile that is not
// finished when it ends (the even one) and of the one that was not when it
// began.  The join kernel adds them up in the order of the runs.

__device__ __forceinline__ float* part_at(const Fp8GemmParams& P, int32_t run, bool begins) {
  return P.part + (static_cast<int64_t>(2 * run + (begins ? 0 : 1)) * P.tile_rows) * 128;
}

constexpr int kJoinThreads = 256;

// blockIdx.x: the end of a run inside a tile, the first in it; a warp has a
// row, a lane four of its columns.
__global__ void __launch_bounds__(kJoinThreads) fp8_join_kernel(const __grid_constant__ Fp8GemmParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  const int32_t i = static_cast<int32_t>(blockIdx.x) + 1;
  const int32_t depth = P.segs * P.kb, work = fp8_tiles<1>(P) * depth, run = max((work + P.runs - 1) / P.runs, P.min_run);
  const int32_t end = i * run, t = end / depth, from = t * depth;
  if (end >= work || end == from || end - run > from) return;
  const int32_t lo = i - 1, hi = (from + depth - 1) / run;
  const Fp8Unit u = fp8_unit<1>(P, t, fp8_words<1>(P, t));
  const int32_t r = static_cast<int32_t>(blockIdx.y) * (kJoinThreads / 32) + static_cast<int32_t>(threadIdx.x >> 5);
  const int64_t row = static_cast<int64_t>(u.tile) * P.tile_rows + r;
  if (r >= u.rows) return;
  const int32_t o = P.mode == FP8_DENSE ? u.g : 0, c = u.nt * 128 + static_cast<int32_t>(lane) * 4;
  float v[4] = {};
#pragma unroll 4
  for (int32_t k = lo; k <= hi; ++k) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(part_at(P, k, k == lo) + r * 128) + lane);
    v[0] += f.x;
    v[1] += f.y;
    v[2] += f.z;
    v[3] += f.w;
  }
  if (c < P.cols) {
    const int64_t at = row * P.cols + c;
    if (P.bias[o]) {
      const uint2 w = *reinterpret_cast<const uint2*>(P.bias[o] + c);
      v[0] += bf_lo(w.x);
      v[1] += bf_hi(w.x);
      v[2] += bf_lo(w.y);
      v[3] += bf_hi(w.y);
    }
    if (P.epi == TP_EPI_DGELU) {
      const uint2 h = *reinterpret_cast<const uint2*>(P.aux[o] + at);
      times_gelu_prime2(v[0], v[1], bf_lo(h.x), bf_hi(h.x));
      times_gelu_prime2(v[2], v[3], bf_lo(h.y), bf_hi(h.y));
    } else if (P.epi == TP_EPI_GELU) {
      if (P.aux[o]) *reinterpret_cast<uint2*>(P.aux[o] + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      gelu2(v[0], v[1]);
      gelu2(v[2], v[3]);
    }
    if (P.out32) *reinterpret_cast<float4*>(P.out32 + at) = make_float4(v[0], v[1], v[2], v[3]);
    else if (P.out[o]) *reinterpret_cast<uint2*>(P.out[o] + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
    v[0] = v[1] = v[2] = v[3] = 0.f;
  }
  if (P.zq[o]) {
    float top = fmaxf(fmaxf(finite_abs(v[0]), finite_abs(v[1])), fmaxf(finite_abs(v[2]), finite_abs(v[3])));
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
    const uint32_t e = fp8_exponent(top);
    *reinterpret_cast<uint32_t*>(P.zq[o] + row * P.zq_ld + c) = fp8_pack4(v[0], v[1], v[2], v[3], fp8_inverse(e));
    if (lane == 0) P.ze[o][u.tile * P.ze_ld + (u.nt >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(r), u.nt & 3)] = static_cast<uint8_t>(e);
  }
}

// ------------------------------------------------------------------ kernel

template <int CTAS, bool QUANT, bool TURNED>
__global__ void __launch_bounds__(Fp8Cfg<CTAS, TURNED>::THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams P) {
  using C = Fp8Cfg<CTAS, TURNED>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  __shared__ float red[CTAS == 1 && QUANT && !TURNED ? 4 : 1][2][32];
  __shared__ float turned[QUANT && TURNED ? 2 * CTAS : 1][2][4][16];
  const Fp8Ring<CTAS> ring(base, P.tile_rows);
  const int STAGES = ring.count;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + C::BAR_OFF);
  const uint32_t bar0 = base + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::MAX_STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * C::MAX_STAGES + b); };
  const uint32_t begun_bar = bar0 + 8u * (2 * C::MAX_STAGES + 2), drain_bar = begun_bar + 16u;
  auto done_bar = [&](uint32_t n) { return begun_bar + 8u * (n & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::MAX_STAGES + 5);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  const uint32_t warp = static_cast<uint32_t>(uniform(static_cast<int32_t>(threadIdx.x >> 5))), lane = threadIdx.x & 31;
  const uint32_t crank = CTAS == 2 ? cluster_ctarank() : 0;
  const bool leader = crank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(tfull_bar(b), 1);
    mbar_init(begun_bar, CTAS * C::EPI_WARPS);
    if (CTAS == 1) mbar_init(done_bar(1), C::EPI_WARPS);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // maps that the first loads need
    if (P.kb > 0) {
      for (int i = 0; i < (P.a_by_s ? P.segs : 1); ++i) tma_prefetch_desc(&P.a[i]);
      tma_prefetch_desc(&P.b[0]);
      if (CTAS == 2) {
        tma_prefetch_desc(&P.ea[0]);
        tma_prefetch_desc(&P.eb[0]);
      }
    }
  }
  if (warp == 1) {
    if (CTAS == 2) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (CTAS == 2) {
    __syncwarp();
    cluster_sync_all();  // both CTAs' barriers exist before any remote signal
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int32_t>(*tmem_slot)));
  griddep_wait();
  griddep_launch_dependents();

  Fp8Walk<CTAS> walk(P);
  Fp8Unit u;
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t role) {
    return wait_bar(bar, parity & 1u, P.timeout_ns, P.status, abort_flag, role);
  };

  // Waits of the loading and the issuing warp: all lanes give up together.
  auto wait_warp = [&](uint32_t bar, uint32_t parity, uint32_t role) { return __all_sync(0xFFFFFFFFu, wait(bar, parity, role)) != 0; };

  if (warp == 0) {
    // -------------------------------------------------------------- loads (both CTAs)
    const uint32_t one = elect_one();
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    int32_t issued = 0;
    bool ok = true;
    while (ok && walk.next(P, u)) {
      // a CTA of a pair holds half of the rows that are the N
      const int32_t a_half = TURNED ? (u.rows + 31) / 32 * 16 : 128;
      const bool whole = CTAS == 1 || !TURNED || a_half > 96;  // else 32 rows at a time: single tiles load half as much
      const uint32_t block_bytes = C::B_BYTES + (whole ? ring.a_bytes : static_cast<uint32_t>((a_half + 31) / 32) * 4096u);
      const int32_t a_row = u.a_row + static_cast<int32_t>(crank) * a_half, b_row = u.b_row + static_cast<int32_t>(crank) * 128;
      Fp8Block b = fp8_block(P, u, u.q0);
      for (int32_t q = u.q0; q < u.q1; q += C::DEEP) {
        const int32_t deep = min(u.q1 - q, C::DEEP);
        if (!wait_warp(empty_bar(stage), phase ^ 1u, 1u)) {
          ok = false;
          break;
        }
        const bool drop = blockIdx.x == 0 && issued++ == P.drop;  // test hook: the consumer's wait runs out
        // bytes of the stage: exponents with its first k-block and the first of every four
        uint32_t bytes = deep * block_bytes;
        const uint32_t fb = CTAS == 2 ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
        Fp8Block at[C::DEEP];
        bool scales[C::DEEP];
#pragma unroll
        for (int d = 0; d < C::DEEP; ++d) {
          at[d] = b;
          scales[d] = d < deep && (q + d == u.q0 || (b.k & 3) == 0);
          bytes += scales[d] ? C::E_BYTES : 0u;
          if (++b.k == P.kb && P.mode == FP8_DENSE) b = fp8_block(P, u, q + d + 1);
        }
        if (!drop) {
          if (leader) expect_bytes(one, full_bar(stage), CTAS * bytes);
#pragma unroll
          for (int d = 0; d < C::DEEP; ++d) {
            if (d >= deep) continue;
            if (whole) {
              load_2d<CTAS>(one, ring.a(stage, d), &P.a[at[d].ai], fb, at[d].k * 128, a_row);
            } else {
              for (int32_t r = 0; r < a_half; r += 32) load_2d<CTAS>(one, ring.a(stage, d) + r * 128, &P.a[1], fb, at[d].k * 128, a_row + r);
            }
            load_2d<CTAS>(one, ring.b(stage, d), &P.b[at[d].bi], fb, at[d].k * 128, b_row);
            if (scales[d]) {
              const uint32_t se = ring.e(stage, d);
              if constexpr (CTAS == 2) {
                // 512 bytes of the M of this CTA, 1024 of the pair's N
                const int32_t my = static_cast<int32_t>(crank);
                load_3d_pair(one, TURNED ? se + C::EA_BYTES : se, &P.ea[at[d].ai], fb, 0, at[d].k >> 2, TURNED ? u.ea : u.ea + my);
                load_3d_pair(one, TURNED ? se : se + C::EA_BYTES, &P.eb[at[d].bi], fb, 0, at[d].k >> 2, TURNED ? u.eb + my : u.eb);
              } else {
                load_512(one, TURNED ? se + C::EA_BYTES : se, P.ea_at[at[d].ai] + (static_cast<int64_t>(u.ea) * P.fours + (at[d].k >> 2)) * 512, fb);
                load_512(one, TURNED ? se : se + C::EA_BYTES, P.eb_at[at[d].bi] + (static_cast<int64_t>(u.eb) * P.fours + (at[d].k >> 2)) * 512, fb);
              }
            }
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every armed stage's last bytes have landed before the CTA goes on
    if (leader)
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) drain_wait(full_bar(s), (armed_parity >> s) & 1u, P.timeout_ns);
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------------------------ MMAs (CTA 0)
      const uint32_t one = elect_one();
      int stage = 0;
      uint32_t phase = 0, n = 0, quads = 0;
      bool ok = true;
      for (; ok && walk.next(P, u); ++n) {
        // CTAS = 2: the epilogue has begun the tile before, so that it is done
        // with the one before that, and with the columns that both accumulators
        // have; CTAS = 1: it is done with the tile before the last
        if (CTAS == 2 ? n > 0 && !wait_warp(begun_bar, n - 1, 2u) : n > 1 && !wait_warp(done_bar(n), (n >> 1) - 1, 2u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + ((n & 1) ? C::ACC1 : 0);
        uint32_t sf = tmem + C::SF;
        const uint32_t n_of = TURNED ? (u.rows + 16 * CTAS - 1) / (16 * CTAS) * (16 * CTAS) : C::BN;
        int32_t k = fp8_block(P, u, u.q0).k;
        for (int32_t q = u.q0; q < u.q1; q += C::DEEP) {
          if (!wait_warp(full_bar(stage), phase, 3u)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int d = 0; d < C::DEEP; ++d) {
            if (q + d >= u.q1) continue;
            if (q + d == u.q0 || (k & 3) == 0) {
              // copies and MMAs of a thread run in the order in which they are issued
              sf = tmem + C::SF + (quads++ & 1) * 16;
              const uint32_t se = ring.e(stage, d);
#pragma unroll
              for (int i = 0; i < 1 + CTAS; ++i) tmem_cp_scales<CTAS>(one, sf + 4 * i, se + 512 * i);
            }
            const uint32_t idesc = make_idesc_mxf8(128 * CTAS, n_of, k & 3);
            const uint64_t ra = make_sw128_desc(ring.a(stage, d), 16, 1024), rb = make_sw128_desc(ring.b(stage, d), 16, 1024);
            const uint64_t ad = TURNED ? rb : ra, bd = TURNED ? ra : rb;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_mxf8<CTAS>(one, d_tmem, ad + 2 * i, bd + 2 * i, idesc, sf, sf + 4, (q + d > u.q0 || i > 0) ? 1u : 0u);
            if (++k == P.kb && P.mode == FP8_DENSE) k = 0;
          }
          commit_to<CTAS>(one, empty_bar(stage), 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit_to<CTAS>(one, tfull_bar(n & 1), 0x3);
      }
      commit_to<CTAS>(one, drain_bar, 0x1);
      drain_wait(drain_bar, 0, P.timeout_ns);
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const uint32_t quarter = warp & 3, part = (warp - 2) >> 2;  // lanes of tensor memory; half of the columns, or some of the rows
    const uint32_t stg = base + C::STG_OFF + (warp - 2) * C::STG_BYTES;
    uint32_t n = 0, turn = 0;
    for (; walk.next(P, u); ++n) {
      bool ok = wait(tfull_bar(n & 1), n >> 1, 4u);
      // the warps that meet at barriers below give up together
      ok = QUANT && (CTAS == 1 || TURNED) ? epilogue_all<32 * C::EPI_WARPS>(ok) : __all_sync(0xFFFFFFFFu, ok) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((quarter * 32) << 16) + ((n & 1) ? C::ACC1 : 0) + part * C::COLS;
      const bool empty = u.q0 >= u.q1;
      auto begun = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CTAS == 2) mbar_arrive_cluster(mapa_shared(begun_bar, 0));
          else mbar_arrive(done_bar(n));
        }
      };
      Fp8Place w;
      w.o = P.mode == FP8_DENSE ? u.g : P.mode == FP8_CONTRACT ? u.bi : 0;
      w.off = u.out_off;
      w.mat = P.mode == FP8_CONTRACT ? u.g % P.per : 0;
      w.col = u.nt * C::BN + static_cast<int32_t>(part) * C::COLS;
      const int32_t tile_row = static_cast<int32_t>(quarter) * 32;
      const int32_t tile = u.tile + static_cast<int32_t>(crank);
      w.row = u.a_row + static_cast<int32_t>(crank) * 128 + tile_row;
      const int32_t all_rows = u.rows - static_cast<int32_t>(crank) * 128;
      w.rows = min(max(all_rows - tile_row, 0), 32);
      w.eblock = tile;
      w.erow = tile_row;
      // The shared columns are the first accumulator's last 32 and the
      // second's first; without them the tile counts as begun at once.
      const bool shared_mine = C::SHARED != 0 && part == ((n & 1) ? 0u : 1u);
      const bool early = CTAS == 2 && !TURNED && (!shared_mine || w.rows == 0);
      if (early) begun();
      auto released = [&] {
        if (CTAS == 2 && !early) begun();
      };
      const FromTmem acc{taddr, empty};
      const bool partial = CTAS == 1 && walk.stride == 0 && u.q1 - u.q0 < walk.depth;
      if constexpr (TURNED) {
        float* sums = partial ? part_at(P, static_cast<int32_t>(blockIdx.x), u.q0 == 0) : nullptr;
        w.row = u.a_row;
        w.eblock = u.tile;
        w.col = u.nt * C::BN + static_cast<int32_t>(crank) * 128;
        // the chunks in the shared columns first
        drain_turned<QUANT>(P, w, u.rows, sums, tmem + ((quarter * 32) << 16) + ((n & 1) ? C::ACC1 : 0), empty, (n & 1) == 0,
                            Fp8Lane{lane, quarter, part, C::EPI_WARPS / 4, 2 + part}, turned[QUANT ? part : 0], turn, released);
      } else if (w.rows > 0) {
        if (partial) {
          float* to = part_at(P, static_cast<int32_t>(blockIdx.x), u.q0 == 0) + tile_row * 128 + part * C::COLS;
          if (lane == 0) bulk_wait_read_all();  // of the tile before
          __syncwarp();
          drain_sums<C::COLS>(to, w.rows, acc, stg, lane);
        } else if constexpr (QUANT) {
          drain_fp8<C::COLS>(P, w, acc, stg, lane, red[CTAS == 1 ? quarter : 0], part, 2 + quarter, released);
        } else {
          drain_bf16<C::COLS>(P, w, acc, (n & 1) == 0, stg, lane, released);
        }
      }
      if (CTAS == 1) begun();
    }
    if (!QUANT && !TURNED && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) {
    __syncwarp();
    if (*abort_flag) {
      // after a timeout, give the peer's copies into this CTA time to land
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000ull) {
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA frees tensor memory or exits while its peer may use it
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (CTAS == 2) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

}  // namespace tpf
