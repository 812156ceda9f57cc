// The sharded Linear with 4-bit weights for a few tokens: both forward
// layouts, packing and unpacking.
//
// A weight is (q - 8) * s, q in 0..15, with one bf16 scale s for each column
// and group of G rows.  A product of up to 64 tokens is bound by the bytes of
// the weights (K N (1/2 + 2/G)), so that the kernel streams each of them once
// and has to spend few instructions on it.  The tokens' dot products run on
// mma.sync m16n8k16 with the weights' columns as its 16 rows and the tokens
// as its 8 columns: 8 tokens cost what one does, where the 128-row tiles of
// tcgen05 would need the dequantised weights written to tensor memory or
// shared memory first, which costs more than the product at these sizes.
//
// Layout (32 columns x 64 rows a tile of 1024 bytes): a lane's 16 bytes are
// its A fragments of four mma, so that weights go from memory to registers
// without a shuffle or a transposition.  A word holds the rows 8 t + 4 j ..
// + 3 (of 32) of the columns i and i + 8, in the order that makes
//   ((word >> 4 r) & 0x000F000F) | 0x43004300
// the bf16 pair 128 + q of fragment register r; subtracting 136 leaves q - 8
// exactly.  The scale is applied to the group's fp32 sum (once in G rows
// instead of once a weight), so no product is rounded before it is added.
//
// The work, blocks of 256 columns x stages of 128 rows (of every rank), is
// cut into equal runs of stages, one for each thread block, whatever the
// shapes: a block of columns that several thread blocks share is summed by
// the last of them to finish, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "gelu.cuh"
#include "host_util.h"
#include "vec_util.cuh"
#include "w4.h"

using namespace tpf;

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCols = 32 * kWarps;  // columns of a thread block
constexpr int kStageK = 128;        // rows of a stage
constexpr int kXPitch = kStageK * 2 + 64;  // bytes of a token's row in shared memory (lanes of two tokens hit different banks)
constexpr int kMaxTokens = 64;
constexpr int kSMs = 152;

struct W4Params {
  const void* x[8];
  const void* q[8];
  const void* s[8];
  const __nv_bfloat16* bias[8];
  void* y[8];
  unsigned long long* count;  // [blocks]
  float* part;                // [2 * gridDim.x][kCols * 8 NT]
  unsigned long long epoch;
  uint32_t M, N, K;
  uint32_t ktiles, groups, pairs;  // 64-row tiles, scale groups, 32-column pairs of strips of a shard
  uint32_t nblocks;                // column blocks of a shard
  uint32_t kstages;                // stages of a shard
  uint32_t spb;                    // stages of a column block: row layout p * kstages, column layout kstages
  uint32_t stages;                 // all
  int32_t row, epi, out_f32;
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  const uint32_t n = valid ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// D += A . B, 16 x 8 x 16, bf16 in, fp32 accumulator.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes of one stage in shared memory: weights, scales, tokens.
template <int NT, int GB>
struct StageLayout {
  static constexpr int kScales = 4 / GB;  // scale groups of a stage
  static constexpr int kW = kThreads * 64, kS = kWarps * kScales * 64, kX = NT * 8 * kXPitch;
  static constexpr int kBytes = kW + kS + kX;
};

// NT: tiles of 8 tokens; GB: rows of a scale group / 32.
template <int NT, int GB, int STAGES>
__global__ void __launch_bounds__(kThreads, NT <= 4 ? 2 : 1) w4_linear_kernel(const __grid_constant__ W4Params P) {
  using L = StageLayout<NT, GB>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t is_last;
  const uint32_t base = smem_u32(smem);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t u0 = static_cast<uint32_t>(static_cast<uint64_t>(blockIdx.x) * P.stages / gridDim.x);
  const uint32_t u1 = static_cast<uint32_t>(static_cast<uint64_t>(blockIdx.x + 1) * P.stages / gridDim.x);

  // load cursor: column block, and stage in it as (rank, stage of the rank)
  uint32_t lblock = u0 / P.spb, lrank = (u0 % P.spb) / P.kstages, lk = (u0 % P.spb) % P.kstages, lu = u0;
  auto fetch = [&](uint32_t slot) {
    if (lu < u1) {
      const uint32_t shard = P.row ? lrank : lblock / P.nblocks;
      const uint32_t pair = (P.row ? lblock : lblock % P.nblocks) * kWarps + warp;
      const uint32_t dst = base + slot * L::kBytes;
      if (pair < P.pairs) {
        const uint8_t* q = static_cast<const uint8_t*>(P.q[shard]) +
                           (static_cast<int64_t>(pair) * P.ktiles + lk * (kStageK / 64)) * 1024 + lane * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool ok = lk * 2 + i / 2 < P.ktiles;
          cp_async16_zfill(dst + (warp * 4 + i) * 512 + lane * 16, ok ? q + i * 512 : q, ok);
        }
        if (lane < L::kScales * 4) {
          const uint32_t first = lk * L::kScales;
          const bool ok = first + lane / 4 < P.groups;
          const uint8_t* s = static_cast<const uint8_t*>(P.s[shard]) + (static_cast<int64_t>(pair) * P.groups + first) * 64;
          cp_async16_zfill(dst + L::kW + warp * (L::kScales * 64) + lane * 16, ok ? s + lane * 16 : s, ok);
        }
      }
      const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(P.x[P.row ? lrank : 0]) + lk * kStageK;
      const uint32_t left = P.K - lk * kStageK;  // columns of x from here on
      for (uint32_t c = threadIdx.x; c < P.M * (kStageK / 8); c += kThreads) {
        const uint32_t tok = c / (kStageK / 8), col = c % (kStageK / 8) * 8;
        const bool ok = col < left;
        cp_async16_zfill(dst + L::kW + L::kS + tok * kXPitch + col * 2, x + static_cast<int64_t>(tok) * P.K + (ok ? col : 0), ok);
      }
      ++lu;
      if (++lk == P.kstages) {
        lk = 0;
        if (!P.row || ++lrank == P.spb / P.kstages) {
          lrank = 0;
          ++lblock;
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  float acc[2][NT][4];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][n][i] = 0.f;

  uint32_t block = u0 / P.spb, left = P.spb - u0 % P.spb;  // stages to the end of the column block
  uint32_t slot = 0;
  for (uint32_t u = u0; u < u1; ++u) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();  // stage u is here for everybody, and everybody is done with stage u - 1
    fetch(slot == 0 ? STAGES - 1 : slot - 1);
    const uint32_t src = base + slot * L::kBytes;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    const uint32_t pair = (P.row ? block : block % P.nblocks) * kWarps + warp;
    if (pair < P.pairs) {
      const uint32_t wsrc = src + warp * 2048 + lane * 16, xsrc = src + L::kW + L::kS + g * kXPitch + t * 16;
      const uint32_t ssrc = src + L::kW + warp * (L::kScales * 64) + g * 4;
      float part[2][NT][4];
      uint4 w[2];
#pragma unroll
      for (int b = 0; b < 4; ++b) {  // 32 rows each
        if (b % 2 == 0) {
#pragma unroll
          for (int f = 0; f < 2; ++f) w[f] = ld_shared_v4(wsrc + ((b / 2) * 2 + f) * 512);
        }
        if (b % GB == 0) {
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[f][n][i] = 0.f;
        }
        uint32_t a[2][2][4];
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t word = b % 2 == 0 ? (j == 0 ? w[f].x : w[f].y) : (j == 0 ? w[f].z : w[f].w);
#pragma unroll
            for (int r = 0; r < 4; ++r) a[f][j][r] = sub_bf16x2(((word >> (4 * r)) & 0x000F000Fu) | 0x43004300u, 0x43084308u);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 xv = ld_shared_v4(xsrc + n * (8 * kXPitch) + b * 64);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            mma16816(part[f][n], a[f][0], xv.x, xv.y);
            mma16816(part[f][n], a[f][1], xv.z, xv.w);
          }
        }
        if (b % GB == GB - 1) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            uint32_t sc;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc) : "r"(ssrc + (b / GB) * 64 + f * 32));
            const float s0 = bf_lo(sc), s1 = bf_hi(sc);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[f][n][0] = fmaf(s0, part[f][n][0], acc[f][n][0]);
              acc[f][n][1] = fmaf(s0, part[f][n][1], acc[f][n][1]);
              acc[f][n][2] = fmaf(s1, part[f][n][2], acc[f][n][2]);
              acc[f][n][3] = fmaf(s1, part[f][n][3], acc[f][n][3]);
            }
          }
        }
      }
    }
    if (--left != 0 && u + 1 != u1) continue;

    // the run of this column block ends here
    const uint32_t b0 = block * P.spb, b1 = b0 + P.spb;
    const uint32_t c0 = static_cast<uint32_t>(((static_cast<uint64_t>(b0) + 1) * gridDim.x - 1) / P.stages);
    const uint32_t c1 = static_cast<uint32_t>((static_cast<uint64_t>(b1) * gridDim.x - 1) / P.stages);
    constexpr int kSlab = kThreads * 2 * NT * 4;  // floats of a block's sums, in the threads' own order
    bool write = true;
    if (c0 != c1) {
      // slab 0 of a thread block is for the column block its run begins in,
      // slab 1 for the one it ends in
      auto slab = [&](uint32_t c) {
        const bool begins = static_cast<uint64_t>(c) * P.stages / gridDim.x >= b0;
        return P.part + static_cast<int64_t>(2 * c + (begins ? 0 : 1)) * kSlab;
      };
      // (the run of c begins at or after b0 for all but c0, whose run may
      // have begun in an earlier column block)
      float4* mine = reinterpret_cast<float4*>(slab(blockIdx.x)) + threadIdx.x;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          __stcg(mine + (f * NT + n) * kThreads, make_float4(acc[f][n][0], acc[f][n][1], acc[f][n][2], acc[f][n][3]));
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        // (launch number << 16 | arrivals); a counter left by another launch
        // counts as zero.  Each failed exchange is another block's success.
        unsigned long long* cnt = P.count + block;
        const uint32_t n = c1 - c0 + 1;
        unsigned long long cur = *reinterpret_cast<volatile unsigned long long*>(cnt), next = 0;
        bool done = false;
        for (uint32_t i = 0; i <= n + 4 && !done; ++i) {
          next = (cur >> 16) == P.epoch ? cur + 1 : ((P.epoch << 16) | 1ull);
          const unsigned long long prev = atomicCAS(cnt, cur, next);
          done = prev == cur;
          cur = prev;
        }
        is_last = done && (next & 0xFFFFull) == n;
        if (is_last) atomicExch(cnt, 0ull);
        __threadfence();
      }
      __syncthreads();
      write = is_last != 0;
      if (write) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t c = c0; c <= c1; ++c) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(slab(c)) + threadIdx.x + (f * NT + n) * kThreads);
              v.x += o.x;
              v.y += o.y;
              v.z += o.z;
              v.w += o.w;
            }
            acc[f][n][0] = v.x;
            acc[f][n][1] = v.y;
            acc[f][n][2] = v.z;
            acc[f][n][3] = v.w;
          }
      }
    }
    if (write && pair < P.pairs) {
      const uint32_t shard = P.row ? 0 : block / P.nblocks;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t n = pair * 32 + f * 16 + r * 8 + g;
          if (n < P.N) {
            const float bias = P.bias[shard] ? __bfloat162float(P.bias[shard][n]) : 0.f;
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t tok = k * 8 + 2 * t + i;
                if (tok < P.M) {
                  float v = acc[f][k][2 * r + i] + bias;
                  if (P.epi == TP_EPI_GELU) v = gelu_f(v);
                  const int64_t o = static_cast<int64_t>(tok) * P.N + n;
                  if (P.out_f32) static_cast<float*>(P.y[shard])[o] = v;
                  else static_cast<__nv_bfloat16*>(P.y[shard])[o] = __float2bfloat16_rn(v);
                }
              }
          }
        }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][n][i] = 0.f;
    ++block;
    left = P.spb;
  }
  cp_async_wait<0>();
}

// ----------------------------------------------------------------- packing

struct W4PackParams {
  const __nv_bfloat16* w[8];  // pack: in; unpack: out (written)
  uint8_t* q[8];
  __nv_bfloat16* s[8];
  uint32_t N, K, G, ktiles, groups, pairs;
};

// One thread: the columns n and n + 8 (of 16) over one scale group.
// s = max|w| / 7 rounded to bf16, q = w / s rounded to nearest even, in
// -7..7 (the correctly rounded quotient: two bf16 differ from a half-way
// point by more than the fp32 division's error, or not at all).
__global__ void __launch_bounds__(256) w4_pack_kernel(const __grid_constant__ W4PackParams P) {
  const uint32_t strips = P.pairs * 2, per = strips * 8;
  const uint32_t id = blockIdx.x * 256 + threadIdx.x;
  const uint32_t shard = blockIdx.z, group = blockIdx.y;
  if (id >= per) return;
  const uint32_t strip = id / 8, i = id % 8;
  const uint32_t n0 = strip * 16 + i, n1 = n0 + 8;
  const __nv_bfloat16* w = P.w[shard];
  const uint32_t k0 = group * P.G, k1 = min(k0 + P.G, P.K), kend = min((k0 + P.G + 63) / 64 * 64, P.ktiles * 64);
  auto at = [&](uint32_t k, uint32_t n) {
    return k < k1 && n < P.N ? __bfloat162float(w[static_cast<int64_t>(k) * P.N + n]) : 0.f;
  };
  float m0 = 0.f, m1 = 0.f;
  bool bad0 = false, bad1 = false;
  for (uint32_t k = k0; k < k1; ++k) {
    const float a = fabsf(at(k, n0)), b = fabsf(at(k, n1));
    bad0 |= !(a <= 3.4028235e38f);
    bad1 |= !(b <= 3.4028235e38f);
    m0 = fmaxf(m0, a);
    m1 = fmaxf(m1, b);
  }
  const float nan = __uint_as_float(0x7FC00000u);
  const __nv_bfloat16 s0 = __float2bfloat16_rn(bad0 ? nan : m0 / 7.f), s1 = __float2bfloat16_rn(bad1 ? nan : m1 / 7.f);
  __nv_bfloat16* so = P.s[shard] + (static_cast<int64_t>(strip / 2) * P.groups + group) * 32 + (strip % 2) * 16 + i * 2;
  so[0] = s0;
  so[1] = s1;
  const float f0 = __bfloat162float(s0), f1 = __bfloat162float(s1);
  auto quant = [](float v, float s) -> uint32_t {
    if (!(s > 0.f)) return 8u;
    const float r = rintf(v / s);
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(r, -7.f), 7.f)) + 8);
  };
  // groups of 32 rows share their 64-row tile with the next group; the last
  // group fills up the tile it ends in
  const bool last = group + 1 == P.groups;
  const uint32_t stop = last ? kend : k0 + P.G;
  for (uint32_t k = k0; k < stop; k += 4) {
    uint32_t word = 0;
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d) {
      const uint32_t pos = 4 * (d & 1) + 2 * (d >> 1);
      word |= quant(at(k + d, n0), f0) << (4 * pos);
      word |= quant(at(k + d, n1), f1) << (4 * (pos + 1));
    }
    const uint32_t kk = k % 64, b = kk / 32, t = kk / 8 % 4, j = kk / 4 % 2;
    const int64_t off = (static_cast<int64_t>(strip / 2) * P.ktiles + k / 64) * 1024 + (strip % 2) * 512 + (i * 4 + t) * 16 + (b * 2 + j) * 4;
    *reinterpret_cast<uint32_t*>(P.q[shard] + off) = word;
  }
}

// One block: 128 columns x 64 rows, through shared memory so that the rows
// are written in whole lines.  (q - 8) * s has up to 12 significant bits and
// is rounded to bf16, the type of the products' operands, here.
constexpr int kUnpackPitch = 128 + 8;
__global__ void __launch_bounds__(256) w4_unpack_kernel(const __grid_constant__ W4PackParams P) {
  __shared__ __align__(16) __nv_bfloat16 tile[64 * kUnpackPitch];
  const uint32_t shard = blockIdx.z, kt = blockIdx.y, pair = blockIdx.x * 4 + threadIdx.x / 64;
  const uint32_t f = threadIdx.x / 32 % 2, lane = threadIdx.x % 32, i = lane / 4, t = lane % 4;
  if (pair < P.pairs) {
    const uint4 v = *reinterpret_cast<const uint4*>(P.q[shard] + (static_cast<int64_t>(pair) * P.ktiles + kt) * 1024 + f * 512 + lane * 16);
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
    const uint32_t col = (threadIdx.x / 64) * 32 + f * 16 + i;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t group = min((kt * 64 + b * 32) / P.G, P.groups - 1);
      const __nv_bfloat16* s = P.s[shard] + (static_cast<int64_t>(pair) * P.groups + group) * 32 + f * 16 + i * 2;
      const float s0 = __bfloat162float(s[0]), s1 = __bfloat162float(s[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t pos = 4 * (d & 1) + 2 * (d >> 1), k = b * 32 + t * 8 + j * 4 + d;
          const int q0 = (words[b * 2 + j] >> (4 * pos)) & 15, q1 = (words[b * 2 + j] >> (4 * (pos + 1))) & 15;
          tile[k * kUnpackPitch + col] = __float2bfloat16_rn(static_cast<float>(q0 - 8) * s0);
          tile[k * kUnpackPitch + col + 8] = __float2bfloat16_rn(static_cast<float>(q1 - 8) * s1);
        }
    }
  }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < 64 * 16; c += 256) {
    const uint32_t k = kt * 64 + c / 16, n = blockIdx.x * 128 + c % 16 * 8;
    if (k < P.K && n < P.N)
      *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(P.w[shard]) + static_cast<int64_t>(k) * P.N + n) =
          *reinterpret_cast<const uint4*>(&tile[(c / 16) * kUnpackPitch + c % 16 * 8]);
  }
}

// ----------------------------------------------------------------- host

struct Plan {
  uint32_t ktiles, pairs, nblocks, kstages, spb, stages, grid, nt;
};

int tiles_for(int64_t M) {
  const int n = static_cast<int>(cdiv(M, 8));
  return n <= 2 ? n : n <= 4 ? 4 : n <= 6 ? 6 : 8;
}

bool make_plan(bool row, int p, int64_t M, int64_t N, int64_t K, Plan* out) {
  Plan P;
  P.nt = static_cast<uint32_t>(tiles_for(M));
  P.ktiles = static_cast<uint32_t>(cdiv(K, 64));
  P.pairs = static_cast<uint32_t>(cdiv(N, 32));
  P.nblocks = static_cast<uint32_t>(cdiv(N, kCols));
  P.kstages = static_cast<uint32_t>(cdiv(K, kStageK));
  const int64_t spb = row ? static_cast<int64_t>(p) * P.kstages : P.kstages;
  const int64_t stages = spb * P.nblocks * (row ? 1 : p);
  if (stages > 0x7FFFFFFFll) return false;
  P.spb = static_cast<uint32_t>(spb);
  P.stages = static_cast<uint32_t>(stages);
  P.grid = static_cast<uint32_t>(std::min<int64_t>(stages, static_cast<int64_t>(kSMs) * (P.nt <= 4 ? 2 : 1)));
  *out = P;
  return true;
}

size_t counter_bytes(const Plan& L, bool row, int p) {
  return static_cast<size_t>(cdiv(static_cast<int64_t>(L.nblocks) * (row ? 1 : p) * 8, 256)) * 256;
}

template <int NT, int GB, int STAGES>
tp_status run_w4(const W4Params& P, uint32_t grid, cudaStream_t stream) {
  static KernelInfo info;
  void (*k)(W4Params) = w4_linear_kernel<NT, GB, STAGES>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  return launch_dependent(k, dim3(grid), static_cast<unsigned>(kThreads), static_cast<size_t>(STAGES) * StageLayout<NT, GB>::kBytes,
                          stream, P);
}

template <int NT, int STAGES>
tp_status run_group(const W4Params& P, int G, uint32_t grid, cudaStream_t stream) {
  if (G == 32) return run_w4<NT, 1, STAGES>(P, grid, stream);
  if (G == 64) return run_w4<NT, 2, STAGES>(P, grid, stream);
  return run_w4<NT, 4, STAGES>(P, grid, stream);
}

tp_status check_group(int64_t G) { return G == 32 || G == 64 || G == 128 ? TP_OK : TP_ERR_INVALID_ARG; }

size_t q_bytes(int64_t N, int64_t K) { return static_cast<size_t>(cdiv(N, 32) * cdiv(K, 64)) * 1024; }
size_t s_bytes(int64_t N, int64_t K, int64_t G) { return static_cast<size_t>(cdiv(N, 32) * cdiv(K, G)) * 64; }

tp_status w4_forward(bool row, const void* const* x, const void* const* q, const void* const* s, const void* const* bias,
                     void* const* y, tp_epilogue epi, int p, int64_t M, int64_t N, int64_t K, int64_t G, tp_dtype out_dtype,
                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_sizes(p, M, N, K, 0, out_dtype));
  TP_TRY(check_group(G));
  if (epi != TP_EPI_NONE && epi != TP_EPI_GELU) return TP_ERR_INVALID_ARG;
  if (M > kMaxTokens) return TP_ERR_UNSUPPORTED_SHAPE;
  const int nx = row ? p : 1, ny = row ? 1 : p;
  const bool work = M > 0 && N > 0, sum = work && K > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(x, nx, sum));
  TP_TRY(check_ptrs(q, p, sum));
  TP_TRY(check_ptrs(s, p, sum));
  TP_TRY(check_ptrs(in(y), ny, work));
  if (bias != nullptr && !row) TP_TRY(check_ptrs(bias, ny, work));
  if (bias != nullptr && row) TP_TRY(check_ptr(bias[0], bias[0] != nullptr && work));
  Plan L;
  // an empty contraction still has its epilogue: one stage of zero rows
  if (!make_plan(row, p, M, N, std::max<int64_t>(K, 1), &L)) return TP_ERR_UNSUPPORTED_SHAPE;
  TP_TRY(check_ws(ws, ws_bytes, w4_workspace(row, p, M, N, K)));
  if (!work) return TP_OK;
  {
    std::vector<Range> ins, outs;
    ins.reserve(40);
    outs.reserve(10);
    add_ranges(&ins, x, nx, static_cast<size_t>(M * K) * 2);
    add_ranges(&ins, q, p, q_bytes(N, K));
    add_ranges(&ins, s, p, s_bytes(N, K, G));
    add_ranges(&ins, bias, ny, static_cast<size_t>(N) * 2);
    add_ranges(&outs, in(y), ny, static_cast<size_t>(M * N) * esize(out_dtype));
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  W4Params P;
  std::memset(&P, 0, sizeof(P));
  for (int r = 0; r < p; ++r) {  // with K == 0 every copy is a zero fill, which reads nothing
    P.q[r] = K > 0 ? q[r] : ws;
    P.s[r] = K > 0 ? s[r] : ws;
  }
  for (int r = 0; r < nx; ++r) P.x[r] = K > 0 ? x[r] : ws;
  for (int r = 0; r < ny; ++r) {
    P.y[r] = y[r];
    P.bias[r] = static_cast<const __nv_bfloat16*>(bias ? bias[r] : nullptr);
  }
  P.count = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  P.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes + counter_bytes(L, row, p));
  P.epoch = g_launch_epoch.fetch_add(1) + 1;
  P.M = static_cast<uint32_t>(M);
  P.N = static_cast<uint32_t>(N);
  P.K = static_cast<uint32_t>(K);
  P.ktiles = static_cast<uint32_t>(cdiv(K, 64));
  P.groups = static_cast<uint32_t>(cdiv(K, G));
  P.pairs = L.pairs;
  P.nblocks = L.nblocks;
  P.kstages = L.kstages;
  P.spb = L.spb;
  P.stages = L.stages;
  P.row = row;
  P.epi = epi;
  P.out_f32 = out_dtype == TP_FP32;
  switch (L.nt) {
    case 1: return run_group<1, 4>(P, static_cast<int>(G), L.grid, stream);
    case 2: return run_group<2, 4>(P, static_cast<int>(G), L.grid, stream);
    case 4: return run_group<4, 4>(P, static_cast<int>(G), L.grid, stream);
    case 6: return run_group<6, 5>(P, static_cast<int>(G), L.grid, stream);
    default: return run_group<8, 5>(P, static_cast<int>(G), L.grid, stream);
  }
}

tp_status pack_params(W4PackParams* P, const void* const* w, const void* const* q, const void* const* s, int p, int64_t N, int64_t K,
                      int64_t G) {
  std::memset(P, 0, sizeof(*P));
  for (int r = 0; r < p; ++r) {
    P->w[r] = static_cast<const __nv_bfloat16*>(w[r]);
    P->q[r] = static_cast<uint8_t*>(const_cast<void*>(q[r]));
    P->s[r] = static_cast<__nv_bfloat16*>(const_cast<void*>(s[r]));
  }
  P->N = static_cast<uint32_t>(N);
  P->K = static_cast<uint32_t>(K);
  P->G = static_cast<uint32_t>(G);
  P->ktiles = static_cast<uint32_t>(cdiv(K, 64));
  P->groups = static_cast<uint32_t>(cdiv(K, G));
  P->pairs = static_cast<uint32_t>(cdiv(N, 32));
  if (P->ktiles > 65535u || P->groups > 65535u) return TP_ERR_UNSUPPORTED_SHAPE;
  return TP_OK;
}

}  // namespace

namespace tpf {

size_t w4_workspace(bool row, int p, int64_t M, int64_t N, int64_t K) {
  Plan L;
  if (M <= 0 || N <= 0 || M > kMaxTokens || !make_plan(row, p, M, N, std::max<int64_t>(K, 1), &L)) return kStatusBytes;
  return kStatusBytes + counter_bytes(L, row, p) + static_cast<size_t>(L.grid) * 2 * kThreads * 2 * L.nt * 4 * sizeof(float);
}

}  // namespace tpf

extern "C" tp_status tp_col_linear_fwd_w4(const void* x, const void* const* q, const void* const* s, const void* const* bias,
                                          void* const* y, tp_epilogue epi, int p, int64_t M, int64_t N, int64_t K, int64_t group,
                                          tp_dtype out_dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return w4_forward(false, &x, q, s, bias, y, epi, p, M, N, K, group, out_dtype, ws, ws_bytes, stream);
}

extern "C" tp_status tp_row_linear_fwd_w4(const void* const* x, const void* const* q, const void* const* s, const void* bias,
                                          void* y, int p, int64_t M, int64_t N, int64_t K, int64_t group, tp_dtype out_dtype,
                                          void* ws, size_t ws_bytes, cudaStream_t stream) {
  return w4_forward(true, x, q, s, &bias, &y, TP_EPI_NONE, p, M, N, K, group, out_dtype, ws, ws_bytes, stream);
}

extern "C" tp_status tp_w4_pack(const void* const* w, void* const* q, void* const* s, int p, int64_t N, int64_t K, int64_t group,
                                cudaStream_t stream) {
  TP_TRY(check_sizes(p, 0, N, K, 0, TP_BF16));
  TP_TRY(check_group(group));
  const bool work = N > 0 && K > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(w, p, work));
  TP_TRY(check_ptrs(in(q), p, work));
  TP_TRY(check_ptrs(in(s), p, work));
  if (!work) return TP_OK;
  W4PackParams P;
  TP_TRY(pack_params(&P, w, in(q), in(s), p, N, K, group));
  std::vector<Range> ins, outs;
  add_ranges(&ins, w, p, static_cast<size_t>(N * K) * 2);
  add_ranges(&outs, in(q), p, q_bytes(N, K));
  add_ranges(&outs, in(s), p, s_bytes(N, K, group));
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  w4_pack_kernel<<<dim3(static_cast<unsigned>(cdiv(static_cast<int64_t>(P.pairs) * 16, 256)), P.groups, static_cast<unsigned>(p)), 256, 0,
                   stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

extern "C" tp_status tp_w4_unpack(const void* const* q, const void* const* s, void* const* w, int p, int64_t N, int64_t K,
                                  int64_t group, cudaStream_t stream) {
  TP_TRY(check_sizes(p, 0, N, K, 0, TP_BF16));
  TP_TRY(check_group(group));
  const bool work = N > 0 && K > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(q, p, work));
  TP_TRY(check_ptrs(s, p, work));
  TP_TRY(check_ptrs(in(w), p, work));
  if (!work) return TP_OK;
  W4PackParams P;
  TP_TRY(pack_params(&P, in(w), q, s, p, N, K, group));
  std::vector<Range> ins, outs;
  add_ranges(&ins, q, p, q_bytes(N, K));
  add_ranges(&ins, s, p, s_bytes(N, K, group));
  add_ranges(&outs, in(w), p, static_cast<size_t>(N * K) * 2);
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  w4_unpack_kernel<<<dim3(static_cast<unsigned>(cdiv(N, 128)), P.ktiles, static_cast<unsigned>(p)), 256, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}
