// The 4-bit sharded Linear for more tokens (17 to 64) and large weights, on
// tcgen05, where mma.sync would take longer than the weights' bytes.
//
// A thread block has 256 columns of the weights as two A operands of 128 rows
// and the tokens as the N of tcgen05.mma.  The dequantised weights go to
// tensor memory, from which the MMA takes its A operand, and never through
// shared memory: a lane has its 16 bytes' worth of them in the order in which
// a 16x256b store lays out 16 lanes x 8 words, with the words 2 t and 2 t + 1
// of lane group t = the rows 8 t + 4 j .. + 3 of the weights.  The tokens'
// rows are put in that order as they are copied to shared memory, in pieces
// of 8 bytes.
//
// A scale group's products (q - 8) x are exact; the tensor cores add at most
// 128 of them in fp32.  The sum leaves tensor memory once, is multiplied by
// the scale and added in registers.
//
// Roles: 16 warps dequantise and add up the finished groups of the stage
// before; two threads issue the MMAs, one for each half of the columns (one
// alone, among the busy warps, takes 112 cycles an MMA, which take 45); two
// warps copy tokens.  A stage is 128 rows.  Two buffers of A, two to four of
// D (of a scale group's sums) and rings of weights and tokens keep them apart.
//
// Measured at p = 8, 49152 -> 12288, groups of 128: 105 us for 32 tokens, 125
// for 64 (47 us at the copy rate; the MMAs alone 33): the issue slots (75 %
// used, 62 % of the integer pipe), which the conversion and the scaling of
// the groups' sums share, bound it.
#pragma once
#include "device_wait.cuh"
#include "w4_device.cuh"

namespace tpf {

constexpr int kWideCols = 256, kWideRows = 128;
constexpr int kWideWorkers = 16, kWideIssuers = 2, kWideLoaders = 64;  // warps, warps, threads
constexpr int kWideThreads = 32 * (kWideWorkers + kWideIssuers) + kWideLoaders;

// NB: tokens, in 16s; GB: rows of a scale group / 32.
template <int NB, int GB>
struct WideShape {
  static constexpr int kGroups = 4 / GB;  // of a stage
  static constexpr int RING = 4;          // stages of weights in shared memory
  static constexpr int XRING = 6;         // of tokens: LAG on their way, the rest with the MMAs
  static constexpr int LAG = 3;
  static constexpr int DS = NB <= 16 ? 16 : NB <= 32 ? 32 : 64;  // columns of tensor memory of a D buffer
  static constexpr int DB = 128 / DS < 4 ? 128 / DS : 4;         // D buffers of each half of the columns
  static constexpr uint32_t kA = 256;                            // A buffers after 2 x 128 columns of D
  // shared memory: tokens (1024-byte aligned), weights, scales
  static constexpr int kX = NB * kWideRows * 2, kW = kWideWorkers * 1024, kS = kWideWorkers * kGroups * 64;
  static constexpr int kBytes = XRING * kX + RING * (kW + kS) + 1024;
  static constexpr size_t kSlab = static_cast<size_t>(kWideCols) * NB * sizeof(float);
  static_assert(kBytes + 1024 <= 227 * 1024, "a thread block an SM");
  static_assert(kX % 2048 == 0, "swizzle atoms of 1024 bytes");
};

__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void* src, bool valid) {
  const uint32_t n = valid ? 8u : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulator, 1 CTA;
// executed by a whole warp, issued by one lane of it.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, one;\n\t"
      "elect.sync _|one, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Commit of the MMAs that umma_bf16_ts issued (elect.sync picks the same lane each time).
__device__ __forceinline__ void umma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred one;\n\t"
      "elect.sync _|one, 0xFFFFFFFF;\n\t"
      "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// 16 lanes x 32 columns: registers 4 n .. 4 n + 3 are the words 2 t, 2 t + 1
// of lane g, then of lane g + 8, in the columns 8 n ..
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int NB>
__device__ __forceinline__ float* wide_slab(const W4Params& P, uint32_t r, uint32_t block) {
  const bool begins = r * P.run_stages >= block * P.spb;
  return P.part + static_cast<int64_t>(2 * r + (begins ? 0 : 1)) * (kWideCols * NB);
}

template <int NB, int GB>
__global__ void __launch_bounds__(kWideThreads, 1) w4_wide_kernel(const __grid_constant__ W4Params P) {
  using S = WideShape<NB, GB>;
  constexpr int GROUPS = S::kGroups, RING = S::RING, XRING = S::XRING, LAG = S::LAG, DB = S::DB;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * 4 + 2 * XRING + 4 * DB + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_word;
  volatile int32_t* abort_flag = &abort_word;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  // of each half of the columns: A and D buffers full and empty, MMAs done
  auto a_full = [&](uint32_t half, uint32_t i) { return bar0 + 8 * (half * 2 + i); };
  auto a_empty = [&](uint32_t half, uint32_t i) { return bar0 + 8 * (4 + half * 2 + i); };
  auto d_full = [&](uint32_t half, uint32_t i) { return bar0 + 8 * (8 + half * DB + i); };
  auto d_empty = [&](uint32_t half, uint32_t i) { return bar0 + 8 * (8 + 2 * DB + half * DB + i); };
  auto x_full = [&](uint32_t i) { return bar0 + 8 * (8 + 4 * DB + i); };
  auto x_empty = [&](uint32_t i) { return bar0 + 8 * (8 + 4 * DB + XRING + i); };
  auto drain_bar = [&](uint32_t half) { return bar0 + 8 * (8 + 4 * DB + 2 * XRING + half); };
  const uint32_t xs = (smem_u32(smem) + 1023u) & ~1023u, wsm = xs + XRING * S::kX, ssm = wsm + RING * S::kW;
  if (threadIdx.x == 0) {
    for (uint32_t half = 0; half < 2; ++half) {
      for (uint32_t i = 0; i < 2; ++i) {
        mbar_init(a_full(half, i), kWideWorkers / 2);
        mbar_init(a_empty(half, i), 1);
      }
      for (uint32_t i = 0; i < DB; ++i) {
        mbar_init(d_full(half, i), 1);
        mbar_init(d_empty(half, i), kWideWorkers / 2);
      }
      mbar_init(drain_bar(half), 1);
    }
    for (uint32_t i = 0; i < XRING; ++i) {
      mbar_init(x_full(i), kWideLoaders);
      mbar_init(x_empty(i), kWideIssuers);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  // rows of tokens past M stay zero; the others are written every stage
  for (uint32_t i = threadIdx.x * 16; i < XRING * S::kX; i += kWideThreads * 16)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(xs + i), "r"(0) : "memory");
  fence_proxy_async_smem();
  griddep_wait();
  griddep_launch_dependents();
  if (warp == kWideWorkers) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t role) {
    return wait_bar(bar, parity & 1u, P.timeout_ns, P.status, abort_flag, role);
  };

  const uint32_t u0 = blockIdx.x * P.run_stages, u1 = min(u0 + P.run_stages, P.stages), count = u1 - u0;
  // The stage to load: column block, rank, stage of the rank.  Pointers move
  // on by a constant until the rank or block ends.
  uint32_t lblock = u0 / P.spb, lrank = (u0 % P.spb) / P.kstages, lk = (u0 % P.spb) % P.kstages;
  auto advance = [&] {  // true: to be aimed anew
    if (++lk != P.kstages) return false;
    lk = 0;
    if (++lrank * P.kstages == P.spb) {
      lrank = 0;
      ++lblock;
    }
    return true;
  };

  if (warp < kWideWorkers) {
    // -------------------------------------------------- weights and sums
    // warp: a quarter of a half's lanes of tensor memory, which are its 32
    // columns; `side`: which 64 rows of a stage it dequantises and which half
    // of the tokens it adds up.
    constexpr int TOK = NB / 2;
    const uint32_t quarter = warp & 3, half = warp >> 2 & 1, side = warp >> 3;
    const uint32_t cols = half * 4 + quarter;
    uint32_t loaded = 0;
    bool here = false;  // the shard has these columns
    const uint8_t *wq = nullptr, *sp = nullptr;
    auto aim = [&] {
      const uint32_t shard = P.row ? lrank : lblock / P.nblocks;
      const uint32_t pair = (P.row ? lblock : lblock % P.nblocks) * (kWideCols / 32) + cols;
      here = pair < P.pairs;
      wq = static_cast<const uint8_t*>(P.q[shard]);
      sp = static_cast<const uint8_t*>(P.s[shard]);
      if (here) {
        wq += (static_cast<int64_t>(pair) * P.ktiles + lk * 2 + side) * 1024 + lane * 16;
        sp += (static_cast<int64_t>(pair) * P.groups + lk * GROUPS) * 64 + lane * 16;
      }
    };
    aim();
    const uint32_t wdst = wsm + warp * 1024 + lane * 16, sdst = ssm + warp * (GROUPS * 64) + lane * 16;
    auto fetch = [&] {
      if (loaded < count) {
        const uint32_t slot = loaded % RING;
        const bool some = here && lk * 2 + side < P.ktiles;
#pragma unroll
        for (int f = 0; f < 2; ++f)
          cp_async16_zfill(wdst + slot * S::kW + f * 512, some ? wq + f * 512 : static_cast<const uint8_t*>(P.q[0]), some);
        if (lane < 4 * GROUPS) {
          const bool ok = here && lk * GROUPS + lane / 4 < P.groups;
          cp_async16_zfill(sdst + slot * S::kS, ok ? sp : static_cast<const uint8_t*>(P.s[0]), ok);
        }
        wq += 2048;
        sp += GROUPS * 64;
        ++loaded;
        if (advance() && loaded < count) aim();
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) fetch();

    // The thread's column is its lane of tensor memory: 16 f + 8 r + i of the
    // pair, whose scale stands at 16 f + 2 i + r.
    const uint32_t scale_at = (lane & 16) + 2 * (lane & 7) + (lane >> 3 & 1);
    const float even = (lane & 8) ? kEven : 1.f;
    const uint32_t at = tmem + ((quarter * 32) << 16);
    uint64_t acc[TOK / 2];  // tokens in pairs
    float scale[GROUPS] = {};
#pragma unroll
    for (int i = 0; i < TOK / 2; ++i) acc[i] = 0;
    uint32_t drained = 0;  // D buffers used up
    uint32_t block = u0 / P.spb, left = P.spb - u0 % P.spb;
    bool ok = true;

    // Adds the stage before's groups; writes the sums out where it was the
    // last of its column block or of the run.
    auto drain = [&](bool last) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const uint32_t db = drained % DB;
        ok = __all_sync(0xFFFFFFFFu, wait(d_full(half, db), drained / DB, 4u));
        if (!ok) return;
        tc_fence_after();
        uint32_t d[TOK];
        const uint32_t from = at + half * 128 + db * S::DS + side * TOK;
#pragma unroll
        for (int c = 0; c < TOK; c += 8) tmem_ld_32x32b_x8(from + c, d + c);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < TOK / 2; ++i)
          acc[i] = fma2(pk2(scale[g], scale[g]), pk2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), acc[i]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(half, db));
        ++drained;
      }
      if (--left != 0 && !last) return;
      const Parts parts = parts_of(P, block);
      const uint32_t c = cols * 32 + lane, tok0 = side * TOK;
      float sum[TOK];
#pragma unroll
      for (int i = 0; i < TOK / 2; ++i) {
        upk2(acc[i], sum[2 * i], sum[2 * i + 1]);
        acc[i] = 0;
      }
      if (parts.first != parts.last) {
        float* out = wide_slab<NB>(P, blockIdx.x, block) + tok0 * kWideCols + c;
#pragma unroll
        for (int i = 0; i < TOK; ++i)
          if (tok0 + i < P.M) __stcg(out + i * kWideCols, sum[i]);
      } else {
        const uint32_t shard = P.row ? 0 : block / P.nblocks, col = (P.row ? block : block % P.nblocks) * kWideCols + c;
        if (col < P.N) {
          const float bias = P.bias[shard] ? __bfloat162float(P.bias[shard][col]) : 0.f;
#pragma unroll
          for (int i = 0; i < TOK; ++i)
            if (tok0 + i < P.M) write_one(P, shard, tok0 + i, col, bias, sum[i]);
        }
      }
      ++block;
      left = P.spb;
    };

    for (uint32_t it = 0; it < count && ok; ++it) {
      const uint32_t slot = it % RING, ab = it & 1;
      cp_async_wait<RING - 2>();
      __syncwarp();  // the lanes' scales are there for all
      ok = __all_sync(0xFFFFFFFFu, wait(a_empty(half, ab), (it >> 1) ^ 1u, 2u));
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = wsm + slot * S::kW + warp * 1024 + lane * 16;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint4 v = ld_shared_v4(src + f * 512);
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a[4];
          dequant(words[j], a);
          r[4 * j] = a[0];
          r[4 * j + 1] = a[2];
          r[4 * j + 2] = a[1];
          r[4 * j + 3] = a[3];
        }
        tmem_st_16x256b_x4(at + ((16 * f) << 16) + S::kA + (ab * 2 + half) * 64 + side * 32, r);
      }
      float next[GROUPS];
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        uint16_t b;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(b) : "r"(ssm + slot * S::kS + (warp * GROUPS + g) * 64 + scale_at * 2));
        next[g] = __uint_as_float(static_cast<uint32_t>(b) << 16) * even;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full(half, ab));
      fetch();  // into the slot of the stage before, which all lanes are done with
      if (it > 0) drain(false);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) scale[g] = next[g];
    }
    if (ok) drain(true);
    cp_async_wait<0>();
  } else if (warp < kWideWorkers + kWideIssuers) {
    // -------------------------------------------------- MMAs of a half of the columns
    // (the whole warp goes through this, so that what it computes is uniform
    // and takes few of the issue slots)
    const uint32_t half = __shfl_sync(0xFFFFFFFFu, warp - kWideWorkers, 0);
    const uint32_t base = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    constexpr uint32_t idesc = make_idesc_bf16(128, NB, false, false);
    auto all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity, 3u)) != 0; };
    uint32_t db = 0, dphase = 1, xb = 0, xphase = 0;  // D buffers handed out, token buffers used
    bool ok = true;
    for (uint32_t it = 0; it < count; ++it) {
      const uint32_t ab = it & 1;
      ok = all(x_full(xb), xphase) && all(a_full(half, ab), it >> 1);
      if (!ok) break;
      tc_fence_after();
      const uint64_t b0 = make_sw128_desc(xs + xb * S::kX, 0, 1024);
      const uint32_t a0 = base + S::kA + (ab * 2 + half) * 64;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        ok = all(d_empty(half, db), dphase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d0 = base + half * 128 + db * S::DS;
#pragma unroll
        for (int k = 0; k < 2 * GB; ++k) {
          const int kk = g * 2 * GB + k;  // of the stage's 8 steps of 16 rows
          umma_bf16_ts(d0, a0 + kk * 8, b0 + (((kk >> 2) * (NB * 128) + (kk & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
        }
        umma_commit_elect(d_full(half, db));
        if (++db == DB) {
          db = 0;
          dphase ^= 1u;
        }
      }
      if (!ok) break;
      umma_commit_elect(a_empty(half, ab));
      umma_commit_elect(x_empty(xb));
      if (++xb == XRING) {
        xb = 0;
        xphase ^= 1u;
      }
    }
    // all MMAs are done before tensor memory is freed
    umma_commit_elect(drain_bar(half));
    drain_wait(drain_bar(half), 0, P.timeout_ns);
    __syncwarp();
  } else {
    // -------------------------------------------------- tokens
    // 16 bytes of a token: rows 8 t .. + 7 of 32 (block b of the stage's
    // four), whose halves go to the MMA steps 2 b and 2 b + 1 as their words
    // 2 t and 2 t + 1.
    const uint32_t t = threadIdx.x - 32 * (kWideWorkers + kWideIssuers), piece = t & 15, b = piece >> 2, tt = piece & 3, tok0 = t >> 4;
    constexpr uint32_t SWEEP = kWideLoaders / 16;  // tokens at a time: rows tok0, tok0 + 4 of 8 by turns
    uint32_t put[2][2];  // of a row and half of the 16 bytes: the place in the stage's buffer
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        const uint32_t kk = 2 * b + i, row = tok0 + r * SWEEP;
        put[r][i] = (kk >> 2) * (NB * 128) + row * 128 + ((((kk & 3) * 2 + (tt >> 1)) ^ (row & 7)) << 4) + (tt & 1) * 8;
      }
    const int64_t sweep = static_cast<int64_t>(SWEEP) * P.K;
    const __nv_bfloat16* x = nullptr;  // of the thread's first token
    auto aim = [&] {
      x = static_cast<const __nv_bfloat16*>(P.x[P.row ? lrank : 0]) + static_cast<int64_t>(tok0) * P.K + lk * kWideRows + piece * 8;
    };
    aim();
    auto give = [&](uint32_t it) {
      if (static_cast<int32_t>(it) != P.drop || blockIdx.x != 0) mbar_arrive(x_full(it % XRING));
    };
    for (uint32_t it = 0; it < count; ++it) {
      const uint32_t xb = it % XRING;
      if (!wait(x_empty(xb), (it / XRING) ^ 1u, 1u)) break;
      const bool ok = lk * kWideRows + piece * 8 < P.K;
      const __nv_bfloat16* src = ok ? x : static_cast<const __nv_bfloat16*>(P.x[0]);
      const int64_t step = ok ? sweep : 0;
      const uint32_t to = xs + xb * S::kX;
#pragma unroll
      for (uint32_t j = 0; j < NB / SWEEP; ++j) {
        if (tok0 + j * SWEEP < P.M) {
#pragma unroll
          for (uint32_t i = 0; i < 2; ++i) cp_async8_zfill(to + put[j & 1][i] + (j >> 1) * 1024, src + i * 4, ok);
        }
        src += step;
      }
      cp_async_commit();
      x += kWideRows;
      if (advance()) aim();
      if (it >= LAG) {
        cp_async_wait<LAG>();
        fence_proxy_async_smem();
        give(it - LAG);
      }
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    if (*abort_flag == 0)
      for (uint32_t it = count < LAG ? 0 : count - LAG; it < count; ++it) give(it);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWideWorkers) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the column blocks that several runs share: blockIdx.x the column
// block, blockIdx.y four of its tokens, a thread a column.
template <int NB>
__global__ void __launch_bounds__(kWideCols) w4_wide_join_kernel(const __grid_constant__ W4Params P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t block = blockIdx.x, t0 = blockIdx.y * 4;
  const Parts parts = parts_of(P, block);
  const uint32_t shard = P.row ? 0 : block / P.nblocks, col = (P.row ? block : block % P.nblocks) * kWideCols + threadIdx.x;
  if (parts.first == parts.last || col >= P.N) return;
  float v[4] = {};
#pragma unroll 4
  for (uint32_t r = parts.first; r <= parts.last; ++r) {
    const float* from = wide_slab<NB>(P, r, block) + t0 * kWideCols + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + i < P.M) v[i] += __ldcg(from + i * kWideCols);
  }
  const float bias = P.bias[shard] ? __bfloat162float(P.bias[shard][col]) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + i < P.M) write_one(P, shard, t0 + i, col, bias, v[i]);
}

}  // namespace tpf
