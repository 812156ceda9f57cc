// The sharded Linear with 4-bit weights for a few tokens: both forward
// layouts, packing and unpacking.
//
// A weight is (q - 8) * s, q in 0..15, with one bf16 scale s for each column
// and group of G rows.  A product of up to 64 tokens is bound by the bytes of
// the weights (K N (1/2 + 2/G)), so that the kernel streams each of them once
// and has to spend few instructions on it.  The tokens' dot products run on
// mma.sync m16n8k16 with the weights' columns as its 16 rows and the tokens
// as its 8 columns: 8 tokens cost what one does, and a weight goes from
// memory to its product through registers alone.  More tokens on large
// weights are the work of w4_wide_kernel (w4_wide.cuh), on tcgen05.
//
// Layout (32 columns x 64 rows a tile of 1024 bytes): a lane's 16 bytes are
// its A fragments of four mma, so that weights go from memory to registers
// without a shuffle or a transposition.  A word holds the rows 8 t + 4 j ..
// + 3 (of 32) of the columns i and i + 8, two rows of one column to a
// fragment register.  The bits of a bf16 below 256 are its value in units of
// 2^-133 (subnormals and the first binade), so that a masked nibble is the
// bf16 q * 2^-133 (column i) or 16 q * 2^-133 (column i + 8) as it stands.
// One fused multiply-add of a pair makes it an exact operand:
//   2^127 * (word & 0x000F000F) - 2^-3 = (q - 8) / 64     (column i)
//   2^127 * (word & 0x00F000F0) - 2    = (q - 8) / 4      (column i + 8)
// Five logic instructions and four multiply-adds for eight weights, each at
// half the rate of the others, and the mma (eight cycles of the tensor pipe
// each) bound the kernel beside HBM.  (Masked nibbles as operands as they
// are, against tokens times 2^64 and less 8 sum(x), gain 2 us of 54 at 1
// token, lose 8 at 16, and turn infinite tokens into NaN.)
// The scale is applied to the group's fp32 sum (once in G rows instead of
// once a weight), so no product is rounded before it is added; the power of
// two that is left over comes with the bias.
//
// The work, blocks of columns x stages of rows (of every rank), is cut into
// equal runs of stages, one for each thread block, whatever the shapes.  A
// column block that several runs share is added up by a second kernel, in
// the order of the runs.  (Several shorter runs to a thread block, taken
// from a counter, would even out the SMs' unequal shares of HBM's bandwidth,
// up to 20 %; the sums at their ends cost as much: 66 to 69 us at 1 token,
// 97 to 101 us at 16, p = 8, 12288 -> 49152.)
//
// Measured with scale groups of 128 (of 64 at 16 tokens), both kernels:
//   p = 8, 12288 -> 49152, 1 token    (312 MB)  54 us, 5.8 TB/s
//   p = 8, 49152 -> 12288, 16 tokens  (323 MB)  75 us, 4.3 TB/s
// against 46 and 48 us at the copy rate.  The second kernel takes 5 to 7
// us of it, most of them the latency of its few reads.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "gelu.cuh"
#include "host_util.h"
#include "vec_util.cuh"
#include "w4.h"
#include "w4_device.cuh"
#include "w4_wide.cuh"

using namespace tpf;

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxTokens = 64;
constexpr int kSMs = 152;

// How a thread block is divided for NT tiles of 8 tokens and scale groups of
// 32 GB rows.  A warp owns NS strips of 16 columns (as many as the sums of NT
// tiles leave registers for) and, with few tokens, half of a stage's rows.
// It streams its weights in pieces of 64 rows; a lane fills and empties its
// own part of the PIECES buffers, and refills each for the next stage as soon
// as it has been used.  Only the tokens, shared by all warps, need a barrier,
// one a stage.
template <int NT, int GB>
struct Shape {
  static constexpr int NS = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;
  static constexpr int KH = NT <= 2 ? 2 : 1;               // row halves
  static constexpr int PIECES = NT <= 2 && GB == 1 ? 2 : 4;
  static constexpr int NO = NS / KH;                       // strips a warp finishes
  static constexpr int kStrips = kWarps / KH * NS;         // strips of a block
  static constexpr int kStageK = 64 * PIECES * KH;         // rows of a stage
  static constexpr int kXPitch = kStageK * 2 + 64;         // bytes of a token's row: lanes of two tokens hit different banks
  static constexpr int kGroups = 2 * PIECES / GB;          // scale groups of a warp's stage
  // shared memory: the pieces, then two stages of scales and tokens
  static constexpr int kPiece = kWarps * NS * 512, kS = kWarps * NS * kGroups * 32, kX = NT * 8 * kXPitch;
  static constexpr int kBytes = PIECES * kPiece + 2 * (kS + kX);
  static_assert(NS * kGroups * 2 <= 32, "a lane copies 16 bytes of the warp's scales");
  static_assert(2 * (kBytes + 2048) <= 227 * 1024, "two thread blocks share an SM");
  // token tiles whose sums the row halves exchange at a time, in a stage's buffer
  static constexpr int kSwap = (kS + kX) / (kWarps * NO * 512) < NT ? 1 : NT;
  static_assert(KH == 1 || kSwap * kWarps * NO * 512 <= kS + kX, "the row halves meet in a stage's buffer");
};

// D += A . B, 16 x 8 x 16, bf16 in, fp32 accumulator; the other form starts from zero.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Where run r keeps its sums of a column block that it shares: its first
// slab for the block it begins in, its second for a later one (the block it
// ends in: those between are its own).
template <int NT, int GB>
__device__ __forceinline__ float4* slab_of(const W4Params& P, uint32_t r, uint32_t block) {
  constexpr int kSlab = kThreads * Shape<NT, GB>::NO * NT;
  const bool begins = r * P.run_stages >= block * P.spb;
  return reinterpret_cast<float4*>(P.part) + static_cast<int64_t>(2 * r + (begins ? 0 : 1)) * kSlab;
}

// Epilogue of the four sums that thread `tid` of a thread block has of its
// strip o and token tile n: rows (columns of Y) g and g + 8, tokens 2 t and
// 2 t + 1.
template <int NT, int GB>
__device__ __forceinline__ void write_out(const W4Params& P, uint32_t block, uint32_t tid, uint32_t o, uint32_t n, const float4& v) {
  using S = Shape<NT, GB>;
  const uint32_t warp = tid >> 5, g = (tid & 31) >> 2, t = tid & 3;
  const uint32_t cg = warp % (kWarps / S::KH), kh = warp / (kWarps / S::KH);
  const uint32_t shard = P.row ? 0 : block / P.nblocks;
  const uint32_t strip = (P.row ? block : block % P.nblocks) * S::kStrips + cg * S::NS + kh * S::NO + o;
  const float vals[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t col = strip * 16 + r * 8 + g;
    if (col >= P.N) continue;
    const float bias = P.bias[shard] ? __bfloat162float(P.bias[shard][col]) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t tok = n * 8 + 2 * t + i;
      if (tok >= P.M) continue;
      write_one(P, shard, tok, col, bias, vals[2 * r + i]);
    }
  }
}

// NT: tiles of 8 tokens; GB: rows of a scale group / 32.
template <int NT, int GB>
__global__ void __launch_bounds__(kThreads, 2) w4_linear_kernel(const __grid_constant__ W4Params P) {
  using S = Shape<NT, GB>;
  constexpr int NS = S::NS, KH = S::KH, PIECES = S::PIECES, GROUPS = S::kGroups, NO = S::NO;
  constexpr uint32_t kShared = S::kS + S::kX;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t cg = warp % (kWarps / KH), kh = warp / (kWarps / KH);
  const uint32_t cell = smem_u32(smem) + warp * (NS * 512) + lane * 16;  // this lane's part of piece 0
  const uint32_t shared = smem_u32(smem) + PIECES * S::kPiece;           // scales and tokens, two stages in turn
  griddep_wait();
  griddep_launch_dependents();
  // The run: stages u .. u1 - 1.
  uint32_t u = blockIdx.x * P.run_stages;
  const uint32_t u1 = min(u + P.run_stages, P.stages);

  // The stage to load, one ahead of the one worked on: column block, rank and
  // stage of the rank, and pointers of the thread's own, which move on by a
  // constant until the rank or block ends.
  constexpr int XC = S::kStageK / 8, XT = kThreads / XC;  // 16-byte pieces of a token's stage; tokens of one sweep
  const uint32_t xtok = threadIdx.x / XC, xcol = threadIdx.x % XC * 8;
  const uint32_t sn = lane / (2 * GROUPS), sg = lane / 2 % GROUPS;  // strip and group of this lane's 16 bytes of scales
  uint32_t lu = u, lblock = u / P.spb, lrank = (u % P.spb) / P.kstages, lk = (u % P.spb) % P.kstages;
  const uint8_t *wq = nullptr, *sp = nullptr;
  const __nv_bfloat16* xp = nullptr;
  uint32_t strips = 0;  // of the warp's that exist
  const int64_t pair_bytes = static_cast<int64_t>(P.ktiles) * 1024;
  auto aim = [&] {
    const uint32_t shard = P.row ? lrank : lblock / P.nblocks;
    const uint32_t strip = (P.row ? lblock : lblock % P.nblocks) * S::kStrips + cg * NS;
    strips = min(static_cast<uint32_t>(NS), max(P.pairs * 2, strip) - strip);
    wq = static_cast<const uint8_t*>(P.q[shard]) + (strip / 2) * pair_bytes + (lk * KH + kh) * (PIECES * 1024ll) + strip % 2 * 512 + lane * 16;
    sp = static_cast<const uint8_t*>(P.s[shard]) +
         (static_cast<int64_t>((strip + sn) / 2) * P.groups + (lk * KH + kh) * GROUPS + sg) * 64 + (strip + sn) % 2 * 32 + lane % 2 * 16;
    xp = static_cast<const __nv_bfloat16*>(P.x[P.row ? lrank : 0]) + static_cast<int64_t>(xtok) * P.K + lk * S::kStageK + xcol;
  };
  aim();
  auto fetch_weights = [&](int h) {
    if (lu >= u1) return;
    const uint32_t tile = (lk * KH + kh) * PIECES + h, dst = cell + h * S::kPiece;
    if (strips == NS && tile < P.ktiles) {
#pragma unroll
      for (int n = 0; n < NS; ++n) cp_async16(dst + n * 512, wq + (n / 2) * pair_bytes + (h * 1024 + n % 2 * 512));
    } else {  // past the shard's columns or rows: zero nibbles, which meet zero scales or zero tokens
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const bool ok = static_cast<uint32_t>(n) < strips && tile < P.ktiles;
        cp_async16_zfill(dst + n * 512, ok ? wq + (n / 2) * pair_bytes + (h * 1024 + n % 2 * 512) : static_cast<const uint8_t*>(P.q[0]), ok);
      }
    }
  };
  auto fetch_shared = [&](uint32_t dst) {
    if (lu >= u1) return;
    if (lane < NS * GROUPS * 2) {
      const bool ok = sn < strips && (lk * KH + kh) * GROUPS + sg < P.groups;
      cp_async16_zfill(dst + warp * (NS * GROUPS * 32) + lane * 16, ok ? sp : static_cast<const uint8_t*>(P.s[0]), ok);
    }
    const bool ok = lk * S::kStageK + xcol < P.K;
#pragma unroll
    for (int i = 0; i < (NT * 8 + XT - 1) / XT; ++i)
      if (xtok + i * XT < P.M)
        cp_async16_zfill(dst + S::kS + (xtok + i * XT) * S::kXPitch + xcol * 2,
                         ok ? xp + static_cast<int64_t>(i) * XT * P.K : static_cast<const __nv_bfloat16*>(P.x[0]), ok);
  };
  auto advance = [&] {
    if (++lu >= u1) return;
    wq += KH * PIECES * 1024;
    sp += KH * GROUPS * 64;
    xp += S::kStageK;
    if (++lk == P.kstages) {
      lk = 0;
      if (++lrank * P.kstages == P.spb) {
        lrank = 0;
        ++lblock;
      }
      aim();
    }
  };
  fetch_shared(shared);
#pragma unroll
  for (int h = 0; h < PIECES; ++h) {
    fetch_weights(h);
    cp_async_commit();
  }
  advance();

  float acc[NS][NT][4];
  auto clear = [&] {
#pragma unroll
    for (int f = 0; f < NS; ++f)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][n][i] = 0.f;
  };
  clear();

  uint32_t block = u / P.spb, left = P.spb - u % P.spb;  // stages to the end of the column block
  uint32_t here = shared, ahead = shared + kShared;
  while (u < u1) {
    const uint32_t ssrc = here + warp * (NS * GROUPS * 32) + g * 4;
    const uint32_t xsrc = here + S::kS + g * S::kXPitch + kh * (PIECES * 128) + t * 16;
    float part[NS][NT][4];
#pragma unroll
    for (int h = 0; h < PIECES; ++h) {
      cp_async_wait<PIECES - 1>();
      if (h == 0) {
        __syncthreads();  // this stage's tokens are here, and everybody is done with the last stage's
        fetch_shared(ahead);
      }
      uint4 w[NS];
#pragma unroll
      for (int f = 0; f < NS; ++f) w[f] = ld_shared_v4(cell + h * S::kPiece + f * 512);
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {  // 32 rows each
        const int b = h * 2 + hb;
        uint4 xv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[n] = ld_shared_v4(xsrc + n * (8 * S::kXPitch) + b * 64);
#pragma unroll
        for (int f = 0; f < NS; ++f) {
          uint32_t a[4];
          dequant(hb == 0 ? w[f].x : w[f].z, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (b % GB == 0) mma16816_first(part[f][n], a, xv[n].x, xv[n].y);
            else mma16816(part[f][n], a, xv[n].x, xv[n].y);
          }
          dequant(hb == 0 ? w[f].y : w[f].w, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(part[f][n], a, xv[n].z, xv[n].w);
        }
        if (b % GB == GB - 1) {
#pragma unroll
          for (int f = 0; f < NS; ++f) {
            uint32_t sc;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc) : "r"(ssrc + (f * GROUPS + b / GB) * 32));
            const float s0 = bf_lo(sc), s1 = bf_hi(sc) * kEven;
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
      // the lane's part of this piece is used up: the next stage's goes there
      fetch_weights(h);
      cp_async_commit();
    }
    advance();
    const uint32_t done = here;
    here = ahead;
    ahead = done;
    ++u;
    if (--left != 0 && u != u1) continue;

    // the run of this column block ends here: the row halves first give each
    // other half of their strips, after which a warp finishes NO of them
    if constexpr (KH > 1) {
      float4* swap = reinterpret_cast<float4*>(smem + (done - smem_u32(smem)));  // the stage just used
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += S::kSwap) {
        __syncthreads();
#pragma unroll
        for (int n = n0; n < n0 + S::kSwap; ++n)
#pragma unroll
          for (int o = 0; o < NO; ++o) {
            const float(&v)[4] = kh == 0 ? acc[NO + o][n] : acc[o][n];
            swap[((warp * NO + o) * S::kSwap + n - n0) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
          }
        __syncthreads();
#pragma unroll
        for (int n = n0; n < n0 + S::kSwap; ++n)
#pragma unroll
          for (int o = 0; o < NO; ++o) {
            const float4 v = swap[(((warp ^ (kWarps / 2)) * NO + o) * S::kSwap + n - n0) * 32 + lane];
            float(&d)[4] = kh == 0 ? acc[o][n] : acc[NO + o][n];
            // a sum of two: the same whichever half comes first
            d[0] += v.x;
            d[1] += v.y;
            d[2] += v.z;
            d[3] += v.w;
          }
      }
      if (kh == 1) {
#pragma unroll
        for (int o = 0; o < NO; ++o)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[o][n][i] = acc[NO + o][n][i];
      }
    }
    const Parts parts = parts_of(P, block);
    if (parts.first != parts.last) {
      float4* mine = slab_of<NT, GB>(P, blockIdx.x, block) + threadIdx.x;
#pragma unroll
      for (int o = 0; o < NO; ++o)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n * 8 + 2 * t < P.M)
            __stcg(mine + (o * NT + n) * kThreads, make_float4(acc[o][n][0], acc[o][n][1], acc[o][n][2], acc[o][n][3]));
    } else {
#pragma unroll
      for (int o = 0; o < NO; ++o)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          write_out<NT, GB>(P, block, threadIdx.x, o, n, make_float4(acc[o][n][0], acc[o][n][1], acc[o][n][2], acc[o][n][3]));
    }
    clear();
    ++block;
    left = P.spb;
  }
  cp_async_wait<0>();
}

// Adds up the column blocks that several runs share: blockIdx.x the column
// block, blockIdx.y one of its (strip, token tile) pairs.
template <int NT, int GB>
__global__ void __launch_bounds__(kThreads) w4_join_kernel(const __grid_constant__ W4Params P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t block = blockIdx.x, o = blockIdx.y / NT, n = blockIdx.y % NT;
  if (n * 8 + 2 * (threadIdx.x & 3) >= P.M) return;
  const Parts parts = parts_of(P, block);
  if (parts.first == parts.last) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (uint32_t r = parts.first; r <= parts.last; ++r) {
    const float4 a = __ldcg(slab_of<NT, GB>(P, r, block) + blockIdx.y * kThreads + threadIdx.x);
    v.x += a.x;
    v.y += a.y;
    v.z += a.z;
    v.w += a.w;
  }
  write_out<NT, GB>(P, block, threadIdx.x, o, n, v);
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
  uint32_t ktiles, pairs, nblocks, kstages, spb, stages, runs, run_stages, blocks, nt;
  bool wide;    // w4_wide_kernel
  size_t slab;  // bytes of a thread block's sums of one column block
};

// Token tiles of 8 of w4_linear_kernel.
int tiles_for(int64_t M) {
  const int n = static_cast<int>(cdiv(M, 8));
  return n <= 2 ? n : n <= 4 ? 4 : n <= 6 ? 6 : 8;
}

// Whether w4_wide_kernel takes the call.  It has more to set up and a longer
// way from a weight to its sum, so that it wants more than 16 tokens, eight
// stages for each SM (of 256 columns x 128 rows), and scale groups of 64 rows
// or more, unless there are so many tokens that mma.sync is slower still.
// Measured, w4_linear_kernel against w4_wide_kernel, us:
//   p = 8, 49152 -> 12288, groups of 128: 24 tokens 117 / 105, 48 177 / 117,
//     64 250 / 125; groups of 64: 32 tokens 129 / 125, 64 238 / 162; groups
//     of 32: 32 tokens 140 / 166, 48 199 / 202, 64 246 / 220;
//   p = 4, 4096 -> 16384, groups of 128 (13 stages an SM): 20 tokens 25 / 25,
//     48 33 / 27, 64 41 / 31;
//   p = 2, 4096 -> 12288 (10 stages), groups of 64: 20 and 32 tokens 27 / 25,
//     48 33 / 27, 64 41 / 31; groups of 128: 25 / 23, 31 / 25, 39 / 27;
//   p = 4, 4096 -> 10240 (8.4 stages): 25 / 24, 29 / 26, 35 / 27; 25 / 23,
//     27 / 25, 35 / 25;
//   p = 2, 4096 -> 7680 (6.3 stages): 20 / 22, 26 / 24, 30 / 26; 20 / 22,
//     24 / 24, 30 / 24;
//   p = 4, 4096 -> 6144 (5.1 stages): 20 / 21, 24 / 24, 28 / 26; 20 / 19,
//     24 / 22, 28 / 24;
//   4096 -> 4096, groups of 128 (3 stages): 20 tokens 17 / 15, 64 21 / 23.
// From eight stages on w4_wide_kernel is ahead at every count; below, each
// side is ahead by up to 2 us at 20 to 48 tokens, and w4_wide_kernel by 2 to
// 6 at 64 from five stages on.  At 16 tokens w4_linear_kernel takes 75 in the
// first of these.  It spills 12 to 200 bytes from 17 tokens on.
bool is_wide(int p, int64_t M, int64_t N, int64_t K, int64_t G) {
  return M > 16 && p * cdiv(N, kWideCols) * cdiv(K, kWideRows) >= 8 * kSMs && (G > 32 || M > 48);
}

template <int NT, int GB>
void shape_of(Plan* P, int64_t N, int64_t K) {
  using S = Shape<NT, GB>;
  P->nblocks = static_cast<uint32_t>(cdiv(N, 16 * S::kStrips));
  P->kstages = static_cast<uint32_t>(cdiv(K, S::kStageK));
  P->slab = static_cast<size_t>(kThreads) * S::NO * NT * 4 * sizeof(float);
}

template <int NT>
void shape_of(Plan* P, int64_t N, int64_t K, int64_t G) {
  if (G == 32) shape_of<NT, 1>(P, N, K);
  else if (G == 64) shape_of<NT, 2>(P, N, K);
  else shape_of<NT, 4>(P, N, K);
}

bool make_plan(bool row, int p, int64_t M, int64_t N, int64_t K, int64_t G, Plan* out) {
  Plan P;
  P.wide = is_wide(p, M, N, K, G);
  P.nt = static_cast<uint32_t>(P.wide ? cdiv(M, 16) * 16 : tiles_for(M));
  P.ktiles = static_cast<uint32_t>(cdiv(K, 64));
  P.pairs = static_cast<uint32_t>(cdiv(N, 32));
  switch (P.nt) {
    case 1: shape_of<1>(&P, N, K, G); break;
    case 2: shape_of<2>(&P, N, K, G); break;
    case 4: shape_of<4>(&P, N, K, G); break;
    case 6: shape_of<6>(&P, N, K, G); break;
    case 8: shape_of<8>(&P, N, K, G); break;
    default:  // wide
      P.nblocks = static_cast<uint32_t>(cdiv(N, kWideCols));
      P.kstages = static_cast<uint32_t>(cdiv(K, kWideRows));
      P.slab = static_cast<size_t>(kWideCols) * P.nt * sizeof(float);
      break;
  }
  const int64_t spb = row ? static_cast<int64_t>(p) * P.kstages : P.kstages;
  const int64_t stages = spb * P.nblocks * (row ? 1 : p);
  if (stages > 0x7FFFFFFFll) return false;
  P.spb = static_cast<uint32_t>(spb);
  P.stages = static_cast<uint32_t>(stages);
  P.blocks = static_cast<uint32_t>(P.nblocks * (row ? 1 : p));
  P.run_stages = static_cast<uint32_t>(cdiv(stages, std::min<int64_t>(stages, static_cast<int64_t>(kSMs) * (P.wide ? 1 : 2))));
  P.runs = static_cast<uint32_t>(cdiv(stages, P.run_stages));
  *out = P;
  return true;
}

template <int NT, int GB>
tp_status run_w4(const W4Params& P, const Plan& L, cudaStream_t stream) {
  static KernelInfo info;
  void (*k)(W4Params) = w4_linear_kernel<NT, GB>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  TP_TRY(launch_dependent(k, dim3(L.runs), static_cast<unsigned>(kThreads), static_cast<size_t>(Shape<NT, GB>::kBytes), stream, P));
  if (L.run_stages == L.spb) return TP_OK;  // every column block is one run's
  return launch_dependent(w4_join_kernel<NT, GB>, dim3(L.blocks, NT * Shape<NT, GB>::NO), static_cast<unsigned>(kThreads), 0, stream, P);
}

template <int NB, int GB>
tp_status run_wide(const W4Params& P, const Plan& L, cudaStream_t stream) {
  static KernelInfo info;
  void (*k)(W4Params) = w4_wide_kernel<NB, GB>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  TP_TRY(launch_dependent(k, dim3(L.runs), static_cast<unsigned>(kWideThreads), static_cast<size_t>(WideShape<NB, GB>::kBytes), stream, P));
  if (L.run_stages == L.spb) return TP_OK;
  return launch_dependent(w4_wide_join_kernel<NB>, dim3(L.blocks, static_cast<unsigned>(cdiv(P.M, 4))), static_cast<unsigned>(kWideCols), 0,
                          stream, P);
}

template <int NB>
tp_status run_wide_group(const W4Params& P, int G, const Plan& L, cudaStream_t stream) {
  if (G == 32) return run_wide<NB, 1>(P, L, stream);
  if (G == 64) return run_wide<NB, 2>(P, L, stream);
  return run_wide<NB, 4>(P, L, stream);
}

template <int NT>
tp_status run_group(const W4Params& P, int G, const Plan& L, cudaStream_t stream) {
  if (G == 32) return run_w4<NT, 1>(P, L, stream);
  if (G == 64) return run_w4<NT, 2>(P, L, stream);
  return run_w4<NT, 4>(P, L, stream);
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
  if (!make_plan(row, p, M, N, std::max<int64_t>(K, 1), G, &L)) return TP_ERR_UNSUPPORTED_SHAPE;
  TP_TRY(check_ws(ws, ws_bytes, w4_workspace(row, p, M, N, K)));
  if (!work) return TP_OK;
  {
    RangeList ins, outs;
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
  P.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kDataOffset);
  P.run_stages = L.run_stages;
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
  P.status = static_cast<uint32_t*>(ws);
  P.timeout_ns = device_timeout_ns();
  P.drop = static_cast<int32_t>(debug_drop());
  switch (L.nt) {
    case 1: return run_group<1>(P, static_cast<int>(G), L, stream);
    case 2: return run_group<2>(P, static_cast<int>(G), L, stream);
    case 4: return run_group<4>(P, static_cast<int>(G), L, stream);
    case 6: return run_group<6>(P, static_cast<int>(G), L, stream);
    case 8: return run_group<8>(P, static_cast<int>(G), L, stream);
    case 32: return run_wide_group<32>(P, static_cast<int>(G), L, stream);
    case 48: return run_wide_group<48>(P, static_cast<int>(G), L, stream);
    default: return run_wide_group<64>(P, static_cast<int>(G), L, stream);
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
  size_t most = kStatusBytes;
  if (M <= 0 || N <= 0 || M > kMaxTokens) return most;
  for (int64_t G : {32, 64, 128}) {  // the size does not ask for the group
    Plan L;
    if (make_plan(row, p, M, N, std::max<int64_t>(K, 1), G, &L))
      most = std::max(most, kDataOffset + static_cast<size_t>(L.runs) * 2 * L.slab);
  }
  return most;
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
  RangeList ins, outs;
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
  RangeList ins, outs;
  add_ranges(&ins, q, p, q_bytes(N, K));
  add_ranges(&ins, s, p, s_bytes(N, K, group));
  add_ranges(&outs, in(w), p, static_cast<size_t>(N * K) * 2);
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  w4_unpack_kernel<<<dim3(static_cast<unsigned>(cdiv(N, 128)), P.ktiles, static_cast<unsigned>(p)), 256, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}
