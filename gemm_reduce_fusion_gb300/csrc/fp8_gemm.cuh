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
// full MMA rate, a single CTA's tile 128.
//
// Roles: warp 0 loads, warp 1 issues the MMAs, eight others are the epilogue,
// each with 32 rows and half of the columns, which overlaps the next tile's
// MMAs on the other accumulator.  With 256 columns the two accumulators share 32 columns of
// tensor memory, which the epilogue reads first: 480 of the 512 columns, the
// rest for the scales.
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
  CUtensorMap a[8], b[8], ea[8], eb[8];  // ea, eb: CTAS = 2
  const uint8_t *ea_at[8], *eb_at[8];    // CTAS = 1: the exponents themselves
  int32_t fours;                         // of k-blocks, in a block of exponents
  int32_t mode;
  int32_t groups, segs;         // outputs; contraction segments (ranks reduced)
  int32_t a_by_g, a_by_s, b_by_g, b_by_s;
  int32_t m_tiles, n_tiles;     // of a group (FP8_ROWS: m_tiles from the plan)
  int32_t kb;                   // k-blocks of a segment
  int32_t stream;               // runs of k-blocks instead of whole tiles (CTAS = 1)
  int32_t min_run;              // the shortest of them
  int32_t few;                  // tiles of few rows, the N of the MMAs (CTAS = 1)
  int32_t rows, cols;           // of an output (FP8_ROWS: rows not used)
  int32_t tile_rows;            // rows of an A tile that are loaded (CTAS = 1: 16 .. 128)
  int32_t band;                 // m-tiles that go together through the n-tiles
  int32_t per, eb_blocks;       // experts of a shard; 128-row blocks of an expert's B
  const int32_t* plan_tiles;    // FP8_ROWS, FP8_CONTRACT: row tiles in use
  const int32_t* plan_expert;   // FP8_ROWS: expert of a row tile
  const int32_t *plan_pairs, *plan_pair;  // FP8_ROWS, CTAS = 2: pairs of row tiles; the first, + kSingle if alone
  const int32_t* plan_first;    // FP8_CONTRACT: first row tile of an expert, E + 1
  const int32_t* plan_slot;     // FP8_ROWS: token and choice of a row, or -1
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

constexpr int32_t kSingle = 1 << 30;

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

template <int CTAS>
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
  static constexpr int EPI_WARPS = 8;
  static constexpr int COLS = BN / 2;  // of an epilogue warp
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr uint32_t STG_BYTES = 2048;  // staging of an epilogue warp
  static constexpr uint32_t E_OFF = RING, STG_OFF = E_OFF + MAX_STAGES * DEEP * E_BYTES, BAR_OFF = STG_OFF + EPI_WARPS * STG_BYTES;
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
  bool single;        // FP8_ROWS: CTA 1 has no row tile
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

template <int CTAS>
__device__ __forceinline__ Fp8Unit fp8_unit(const Fp8GemmParams& P, int32_t t) {
  Fp8Unit u;
  u.t = t;
  int32_t v = t;
  u.out_off = 0;
  u.single = false;
  u.q0 = 0;
  u.q1 = P.segs * P.kb;
  if (P.mode == FP8_ROWS) {
    // an expert's weights are read by its row tiles one after the other
    u.tile = v / P.n_tiles;
    u.nt = v % P.n_tiles;
    if (CTAS == 2) {
      const int32_t pair = uniform(__ldcg(P.plan_pair + u.tile));
      u.single = (pair & kSingle) != 0;
      u.tile = min(max(pair & (kSingle - 1), 0), P.max_tiles - 1);
    }
    const int32_t e = min(max(uniform(__ldcg(P.plan_expert + u.tile)), 0), P.experts - 1), local = e % P.per;
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
  u.ea = u.tile;
  u.b_row = u.nt * Fp8Cfg<CTAS>::BN;
  u.eb = u.nt * CTAS;
  if (P.mode == FP8_CONTRACT) {
    u.q0 = min(max(uniform(__ldcg(P.plan_first + u.g)), 0), P.max_tiles) * P.kb_tile;
    u.q1 = min(uniform(__ldcg(P.plan_first + u.g + 1)), P.max_tiles) * P.kb_tile;
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
  }
  __device__ __forceinline__ bool next(const Fp8GemmParams& P, Fp8Unit& u) {
    if (at >= end) return false;
    if (CTAS == 1 && stride == 0) {
      const int32_t t = at / depth;
      u = fp8_unit<CTAS>(P, t);
      u.q0 = at - t * depth;
      u.q1 = min(depth, u.q0 + end - at);
      at += u.q1 - u.q0;
    } else {
      u = fp8_unit<CTAS>(P, at);
      at += stride;
    }
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
    const int32_t s = P.segs == 1 ? 0 : q / P.kb;
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
    stg_out(stg, reinterpret_cast<uint8_t*>(P.out[w.o]) + at, pitch, w.rows, bytes, lane);
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
      if (P.epi == TP_EPI_GELU) gelu2(v[j][i], v[j][i + 1]);
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

// fp32 results: COLS columns from `to` on, of which `cols` are there.
template <int COLS, typename Released>
__device__ __forceinline__ void drain_f32(float* to, int64_t pitch, int32_t cols, int32_t rows, const FromTmem& load, uint32_t stg,
                                          uint32_t lane, Released released) {
#pragma unroll 1
  for (int j = 0; j < COLS / 32; ++j) {
    float v[32];
    load(j, v);
    if (j == COLS / 32 - 1) released();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int32_t c = j * 32 + half * 16;
      if (c >= cols) continue;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const int n = half * 16 + i * 4;
        st_shared_v4(stg_at(stg, lane, i), make_uint4(__float_as_uint(v[n]), __float_as_uint(v[n + 1]), __float_as_uint(v[n + 2]),
                                                      __float_as_uint(v[n + 3])));
      }
      stg_out(stg, reinterpret_cast<uint8_t*>(to + c), pitch * 4, rows, min(cols - c, 16) * 4, lane);
    }
  }
}

// ------------------------------------------------------------------ tiles of few rows (CTAS = 1)
//
// Up to 64 rows are the N of the MMAs and the 128 columns their M: the tensor
// cores then read the weights' 16 KiB of a k-block from shared memory and the
// rows', not 128 rows, half of which or more would be for nothing (a k-block
// took 530 cycles so, whatever the rows; shared memory's bandwidth, which TMA
// needs too, is what bounds it).  A lane of tensor memory has a column then, a
// column of it a row: the epilogue turns 32 rows at a time in shared memory,
// where all 256 threads take a share, G neighbours a row, four columns each at
// a time.

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ uint32_t pass_at(uint32_t buf, uint32_t row, uint32_t piece) { return buf + row * 512 + ((piece ^ (row & 7)) << 4); }

// 16 rows, from `row` of the 32 on, of the warp's 32 columns.
__device__ __forceinline__ void pass_rows(uint32_t taddr, bool empty, uint32_t buf, uint32_t row, uint32_t col) {
  uint32_t v[16];
  if (empty) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0;
  } else {
    tmem_ld_32x32b_x16(taddr, v);
    tmem_wait_ld();
  }
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i)
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(pass_at(buf, row + i, col >> 2) + (col & 3) * 4), "r"(v[i]) : "memory");
}

// part: fp32 sums [rows][128] instead of results, or null.
template <bool QUANT, int G>
__device__ __forceinline__ void drain_few(const Fp8GemmParams& P, const Fp8Place& w, float* part, uint32_t buf, uint32_t t) {
  constexpr int N = 32 / G;
  const uint32_t r = t / G, g = t % G;
  const bool mine = static_cast<int32_t>(r) < w.rows;
  const int64_t at = w.off + (static_cast<int64_t>(w.row) + r) * P.cols + w.col;
  float v[N][4], top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint4 f = ld_shared_v4(pass_at(buf, r, i * G + g));
    v[i][0] = __uint_as_float(f.x), v[i][1] = __uint_as_float(f.y), v[i][2] = __uint_as_float(f.z), v[i][3] = __uint_as_float(f.w);
  }
  if (part) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (mine) __stcg(reinterpret_cast<float4*>(part + r * 128) + i * G + g, make_float4(v[i][0], v[i][1], v[i][2], v[i][3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int32_t c = (i * G + static_cast<int32_t>(g)) * 4;  // of the tile
    const bool in = mine && w.col + c < P.cols;
    if (in) {
      if (P.bias[w.o]) {
        const uint2 b = *reinterpret_cast<const uint2*>(P.bias[w.o] + w.col + c);
        v[i][0] += bf_lo(b.x), v[i][1] += bf_hi(b.x), v[i][2] += bf_lo(b.y), v[i][3] += bf_hi(b.y);
      }
      if (P.epi == TP_EPI_DGELU) {
        const uint2 h = *reinterpret_cast<const uint2*>(P.aux[w.o] + at + c);
        times_gelu_prime2(v[i][0], v[i][1], bf_lo(h.x), bf_hi(h.x));
        times_gelu_prime2(v[i][2], v[i][3], bf_lo(h.y), bf_hi(h.y));
      } else if (P.epi == TP_EPI_GELU) {
        if (P.aux[w.o]) *reinterpret_cast<uint2*>(P.aux[w.o] + at + c) = make_uint2(pack_bf16(v[i][0], v[i][1]), pack_bf16(v[i][2], v[i][3]));
        gelu2(v[i][0], v[i][1]);
        gelu2(v[i][2], v[i][3]);
      }
      if constexpr (!QUANT) {
        if (P.out32) *reinterpret_cast<float4*>(P.out32 + at + c) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        else *reinterpret_cast<uint2*>(P.out[w.o] + at + c) = make_uint2(pack_bf16(v[i][0], v[i][1]), pack_bf16(v[i][2], v[i][3]));
      }
    } else {
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
    }
    if constexpr (QUANT) top = fmaxf(top, fmaxf(fmaxf(finite_abs(v[i][0]), finite_abs(v[i][1])), fmaxf(finite_abs(v[i][2]), finite_abs(v[i][3]))));
  }
  if constexpr (QUANT) {
    if (w.col >= P.cols) return;
#pragma unroll
    for (int o = G / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const uint32_t e = fp8_exponent(top);
    const float inv = fp8_inverse(e);
    if (mine) {
      uint32_t* to = reinterpret_cast<uint32_t*>(P.zq[w.o] + (static_cast<int64_t>(w.row) + r) * P.zq_ld + w.col);
#pragma unroll
      for (int i = 0; i < N; ++i) to[i * G + g] = fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3], inv);
      const int32_t b = w.col / 128;
      if (g == 0)
        P.ze[w.o][w.eblock * P.ze_ld + (b >> 2) * 512 + fp8_e_at(static_cast<uint32_t>(w.erow) + r, b & 3)] = static_cast<uint8_t>(e);
    }
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
  const Fp8Unit u = fp8_unit<1>(P, t);
  const int32_t r = static_cast<int32_t>(blockIdx.y) * (kJoinThreads / 32) + static_cast<int32_t>(threadIdx.x >> 5);
  const int64_t row = static_cast<int64_t>(u.tile) * P.tile_rows + r;
  if (r >= P.tile_rows || (P.mode != FP8_ROWS && row >= P.rows)) return;
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

template <int CTAS, bool QUANT>
__global__ void __launch_bounds__(Fp8Cfg<CTAS>::THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams P) {
  using C = Fp8Cfg<CTAS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  __shared__ float red[CTAS == 1 && QUANT ? 4 : 1][2][32];
  const Fp8Ring<CTAS> ring(base, P.tile_rows);
  const int STAGES = ring.count;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + C::BAR_OFF);
  const uint32_t bar0 = base + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::MAX_STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * C::MAX_STAGES + b); };
  const uint32_t begun_bar = bar0 + 8u * (2 * C::MAX_STAGES + 2), drain_bar = begun_bar + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::MAX_STAGES + 4);
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
    const uint32_t block_bytes = ring.a_bytes + C::B_BYTES;
    while (ok && walk.next(P, u)) {
      const int32_t a_row = u.a_row + static_cast<int32_t>(crank) * 128, b_row = u.b_row + static_cast<int32_t>(crank) * 128;
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
            load_2d<CTAS>(one, ring.a(stage, d), &P.a[at[d].ai], fb, at[d].k * 128, a_row);
            load_2d<CTAS>(one, ring.b(stage, d), &P.b[at[d].bi], fb, at[d].k * 128, b_row);
            if (scales[d]) {
              const uint32_t se = ring.e(stage, d);
              if constexpr (CTAS == 2) {
                load_3d_pair(one, se, &P.ea[at[d].ai], fb, 0, at[d].k >> 2, u.ea + static_cast<int32_t>(crank));
                load_3d_pair(one, se + C::EA_BYTES, &P.eb[at[d].bi], fb, 0, at[d].k >> 2, u.eb);
              } else {
                load_512(one, se, P.ea_at[at[d].ai] + (static_cast<int64_t>(u.ea) * P.fours + (at[d].k >> 2)) * 512, fb);
                load_512(one, se + C::EA_BYTES, P.eb_at[at[d].bi] + (static_cast<int64_t>(u.eb) * P.fours + (at[d].k >> 2)) * 512, fb);
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
        // the epilogue has begun the tile before: it is done with the one
        // before that, and with the columns that both accumulators have
        if (n > 0 && !wait_warp(begun_bar, n - 1, 2u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + ((n & 1) ? C::ACC1 : 0);
        uint32_t sf = tmem + C::SF;
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
            const bool few = CTAS == 1 && P.few;  // the rows are the N
            const uint32_t idesc = few ? make_idesc_mxf8(128, P.tile_rows, k & 3) : make_idesc_mxf8(128 * CTAS, C::BN, k & 3);
            const uint64_t ra = make_sw128_desc(ring.a(stage, d), 16, 1024), rb = make_sw128_desc(ring.b(stage, d), 16, 1024);
            const uint64_t ad = few ? rb : ra, bd = few ? ra : rb;
            const uint32_t sfa = few ? sf + 4 : sf, sfb = few ? sf : sf + 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_mxf8<CTAS>(one, d_tmem, ad + 2 * i, bd + 2 * i, idesc, sfa, sfb, (q + d > u.q0 || i > 0) ? 1u : 0u);
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
    const uint32_t quarter = warp & 3, part = (warp - 2) >> 2;  // lanes of tensor memory, half of the columns
    const uint32_t stg = base + C::STG_OFF + (warp - 2) * C::STG_BYTES;
    uint32_t n = 0;
    for (; walk.next(P, u); ++n) {
      bool ok = wait(tfull_bar(n & 1), n >> 1, 4u);
      // the warps that meet at barriers below give up together
      ok = CTAS == 1 ? epilogue_all(ok) : __all_sync(0xFFFFFFFFu, ok) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((quarter * 32) << 16) + ((n & 1) ? C::ACC1 : 0) + part * C::COLS;
      const bool empty = u.q0 >= u.q1;
      auto begun = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CTAS == 2) mbar_arrive_cluster(mapa_shared(begun_bar, 0));
          else mbar_arrive(begun_bar);
        }
      };
      Fp8Place w;
      w.o = P.mode == FP8_DENSE ? u.g : P.mode == FP8_CONTRACT ? u.bi : 0;
      w.off = u.out_off;
      w.col = u.nt * C::BN + static_cast<int32_t>(part) * C::COLS;
      const int32_t tile_row = static_cast<int32_t>(quarter) * 32;
      const int32_t tile = u.tile + static_cast<int32_t>(crank);
      int32_t all_rows;  // of the tile
      if (P.mode == FP8_ROWS) {
        w.row = tile * P.tile_rows + tile_row;
        all_rows = u.single && crank == 1 ? 0 : P.tile_rows;
      } else {
        w.row = tile * 128 + tile_row;
        all_rows = P.rows - tile * 128;
      }
      w.rows = min(max(all_rows - tile_row, 0), 32);
      w.eblock = tile;
      w.erow = tile_row;
      // The shared columns are the first accumulator's last 32 and the
      // second's first; without them the tile counts as begun at once.
      const bool shared_mine = C::SHARED != 0 && part == ((n & 1) ? 0u : 1u);
      const bool early = !shared_mine || w.rows == 0;
      if (early) begun();
      auto released = [&] {
        if (!early) begun();
      };
      const FromTmem acc{taddr, empty};
      const bool partial = CTAS == 1 && walk.stride == 0 && u.q1 - u.q0 < walk.depth;
      if (CTAS == 1 && P.few) {
        const uint32_t buf = base + C::STG_OFF, t = threadIdx.x - 64;
        float* part32 = partial ? part_at(P, static_cast<int32_t>(blockIdx.x), u.q0 == 0) : nullptr;
        w.row -= tile_row;
        w.col = u.nt * C::BN;
        for (int32_t q = 0; q * 32 < all_rows && q < 4; ++q) {
          if (q * 32 + static_cast<int32_t>(part) * 16 < P.tile_rows)
            pass_rows(tmem + ((quarter * 32) << 16) + ((n & 1) ? C::ACC1 : 0) + q * 32 + part * 16, empty, buf, part * 16, quarter * 32 + lane);
          epilogue_sync();
          w.rows = min(all_rows - q * 32, 32);
          w.erow = q * 32;
          if (P.tile_rows <= 16) drain_few<QUANT, 16>(P, w, part32, buf, t);
          else drain_few<QUANT, 8>(P, w, part32 ? part32 + q * 32 * 128 : nullptr, buf, t);
          w.row += 32;
          epilogue_sync();
        }
      } else if (w.rows > 0) {
        if (partial) {
          float* to = part_at(P, static_cast<int32_t>(blockIdx.x), u.q0 == 0) + tile_row * 128 + part * C::COLS;
          drain_f32<C::COLS>(to, 128, C::COLS, w.rows, acc, stg, lane, [] {});
        } else if constexpr (QUANT) {
          drain_fp8<C::COLS>(P, w, acc, stg, lane, red[CTAS == 1 ? quarter : 0], part, 2 + quarter, released);
        } else if (P.out32) {
          drain_f32<C::COLS>(P.out32 + static_cast<int64_t>(w.row) * P.cols + w.col, P.cols, P.cols - w.col, w.rows, acc, stg, lane, released);
        } else {
          drain_bf16<C::COLS>(P, w, acc, (n & 1) == 0, stg, lane, released);
        }
      }
      tc_fence_before();
    }
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
