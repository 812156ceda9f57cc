// Routed experts on 8-bit operands, forward and backward:
//   y[t] = sum_j weights[t, j] GeLU(x[t] W1_e) W2_e,  e = experts[t, j]
// The p shards hold E/p experts each; the sum over a token's experts is the
// sum over the ranks.
//
// The slots (t, j) of an expert become rows, in the order of t, in tiles of
// `tile_rows` rows of one expert each (dispatch_kernel).  The products walk
// the tiles in use (fp8_gemm.cuh, FP8_ROWS), or contract over an expert's
// rows (FP8_CONTRACT); how many tiles there are stays on the device.  Rows
// without a slot are packed as zeros where they are contracted over, and are
// otherwise neither written nor read for a token.
//
// The tokens' rows go to those of their slots as they are packed, GeLU and the
// activation's packing of the first product's epilogue, and the weighted sum
// one kernel (combine_kernel), which adds a token's rows in fp32 in the order
// of its choices, so that results do not depend on the order of execution.
//
// Up to some hundred rows an expert the weights' bytes bound a call (48 tokens,
// 6 of 64 experts, 4096 x 2048: 173-177 us, 1.07 GB at 0.9 of the copy rate);
// beyond, the MMAs and their tiles' epilogues by turns (4096 tokens: 443-467
// us, of which the products 174 and 182, 2.3 PFLOP/s, packing 23, the sum 40).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fp8.h"
#include "fp8_pack.cuh"
#include "vec_util.cuh"

using namespace tpf;

namespace {

constexpr int kMaxExperts = TP_ROUTE_MAX_EXPERTS, kMaxK = 32;
constexpr int kDispatchThreads = 1024;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int64_t kMostStrips = 65535;  // of 128 rows, that the backward call packs
constexpr int32_t kFewSlots = 512;  // dispatched and packed by one kernel

// ------------------------------------------------------------------ plan

struct DispatchParams {
  const int32_t* experts;  // [S]
  int32_t *tiles, *pairs, *first, *expert, *pair, *slot, *row;
  int32_t S, E, tile_rows, aligned;
  TokenPack pack;  // of few slots
};

__device__ __forceinline__ int32_t tiles_of(int32_t n, int32_t tile_rows) { return (n + tile_rows - 1) / tile_rows; }

// Four slots' experts, -1 past the last.
__device__ __forceinline__ int4 four_slots(const DispatchParams& P, int32_t i) {
  if (P.aligned && i + 4 <= P.S) return *reinterpret_cast<const int4*>(P.experts + i);
  return make_int4(i < P.S ? P.experts[i] : -1, i + 1 < P.S ? P.experts[i + 1] : -1, i + 2 < P.S ? P.experts[i + 2] : -1,
                   i + 3 < P.S ? P.experts[i + 3] : -1);
}

// Where there are few slots, blocks behind the experts' pack the tokens, a
// warp 512 columns, and find their slots' rows by themselves: a launch less
// before the products (one token 30 us, 32 with two kernels).
__device__ __forceinline__ void pack_few(const DispatchParams& P, int32_t* count) {
  const TokenPack& K = P.pack;
  __shared__ int32_t slots[kFewSlots], first[kMaxExperts], warp_sum[kMaxExperts / 32];
  const int32_t tid = static_cast<int32_t>(threadIdx.x);
  const uint32_t lane = tid & 31, warp = tid >> 5;
  for (int32_t e = tid; e < P.E; e += kDispatchThreads) count[e] = 0;
  __syncthreads();
  if (tid < P.S) {
    const int32_t e = P.experts[tid];
    slots[tid] = e;
    if (e >= 0 && e < P.E) atomicAdd(count + e, 1);
  }
  __syncthreads();
  int32_t n = 0, sum = 0;
  if (tid < kMaxExperts) {
    n = sum = tid < P.E ? tiles_of(count[tid], P.tile_rows) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(kAll, sum, o);
      if (static_cast<int32_t>(lane) >= o) sum += u;
    }
    if (lane == 31) warp_sum[warp] = sum;
  }
  __syncthreads();
  if (tid < kMaxExperts) {
    const int32_t other = lane < kMaxExperts / 32 ? warp_sum[lane] : 0;
    first[tid] = (sum - n + __reduce_add_sync(kAll, lane < warp ? other : 0)) * P.tile_rows;
  }
  __syncthreads();
  const uint32_t fours = static_cast<uint32_t>(K.e_block / 512);
  const int64_t unit = static_cast<int64_t>(blockIdx.x - P.E) * (kDispatchThreads / 32) + warp, t = unit / fours;
  if (t >= K.tokens) return;
  int32_t row = -1;
  for (int32_t j = 0; j < K.k; ++j) {
    const int32_t slot = static_cast<int32_t>(t) * K.k + j, e = slots[slot];
    int32_t before = 0;  // slots of the same expert
    for (int32_t i = static_cast<int32_t>(lane); i < slot; i += 32) before += slots[i] == e;
    before = __reduce_add_sync(kAll, before);
    if (static_cast<int32_t>(lane) == j && e >= 0 && e < P.E) row = first[e] + before;
  }
  pack_token(K, t, static_cast<uint32_t>(unit % fours), row, lane);
}

// A thread block an expert.  Each counts all experts' slots, so that no
// kernel has to run before it, and keeps the first 32768 in registers for the
// second pass, which gives its own their rows, in their order.
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(const __grid_constant__ DispatchParams P) {
  constexpr int kKeep = 8, kRound = kDispatchThreads * 4;
  __shared__ int32_t count[kMaxExperts];
  __shared__ int32_t warp_sum[2][kDispatchThreads / 32], begin, total, pair_begin, pair_total;
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int32_t>(blockIdx.x) >= P.E) {
    pack_few(P, count);
    return;
  }
  const int32_t me = static_cast<int32_t>(blockIdx.x), tid = static_cast<int32_t>(threadIdx.x);
  const uint32_t lane = tid & 31, warp = tid >> 5;
  for (int32_t e = tid; e < P.E; e += kDispatchThreads) count[e] = 0;
  if (tid == 0) begin = total = pair_begin = pair_total = 0;
  int4 keep[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) keep[i] = i * kRound < P.S ? four_slots(P, i * kRound + tid * 4) : make_int4(-1, -1, -1, -1);
  __syncthreads();
  auto add = [&](int32_t e) {
    if (e >= 0 && e < P.E) atomicAdd(count + e, 1);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (i * kRound < P.S) add(keep[i].x), add(keep[i].y), add(keep[i].z), add(keep[i].w);
  for (int32_t base = kKeep * kRound; base < P.S; base += kRound) {
    const int4 v = four_slots(P, base + tid * 4);
    add(v.x), add(v.y), add(v.z), add(v.w);
  }
  __syncthreads();
  // tiles (and pairs) before this expert's, and all of them
  if (tid < kMaxExperts) {
    const int32_t n = tid < P.E ? tiles_of(count[tid], P.tile_rows) : 0, pairs = (n + 1) / 2;
    const int32_t a = __reduce_add_sync(kAll, tid < me ? n : 0), b = __reduce_add_sync(kAll, n),
                  c = __reduce_add_sync(kAll, tid < me ? pairs : 0), d = __reduce_add_sync(kAll, pairs);
    if (lane == 0 && b) {
      atomicAdd(&begin, a);
      atomicAdd(&total, b);
      atomicAdd(&pair_begin, c);
      atomicAdd(&pair_total, d);
    }
  }
  __syncthreads();
  const int32_t mine = tiles_of(count[me], P.tile_rows);
  if (tid == 0) {
    P.first[me] = begin;
    if (me == P.E - 1) {
      P.first[P.E] = total;
      *P.tiles = total;
      *P.pairs = pair_total;
    }
  }
  for (int32_t i = tid; i < mine; i += kDispatchThreads) {
    const int32_t rows = count[me] - i * P.tile_rows;
    P.expert[begin + i] = me << 9 | min(rows, P.tile_rows);
    if ((i & 1) == 0) {
      int32_t* pair = P.pair + 2 * (pair_begin + i / 2);
      pair[0] = begin + i;
      pair[1] = me << 9 | min(rows, 2 * P.tile_rows);
    }
  }
  // the slots, in their order
  int32_t at = begin * P.tile_rows;
  auto place = [&](int32_t base, const int4& v, int round) {
    const int32_t e[4] = {v.x, v.y, v.z, v.w}, i0 = base + tid * 4;
    const int32_t n = (e[0] == me) + (e[1] == me) + (e[2] == me) + (e[3] == me);
    int32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(kAll, sum, o);
      if (static_cast<int32_t>(lane) >= o) sum += u;
    }
    if (lane == 31) warp_sum[round & 1][warp] = sum;
    __syncthreads();
    const int32_t other = lane < kDispatchThreads / 32 ? warp_sum[round & 1][lane] : 0;
    int32_t here = at + sum - n + __reduce_add_sync(kAll, lane < warp ? other : 0);
    at += __reduce_add_sync(kAll, other);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e[j] == me) {
        P.slot[here] = i0 + j;
        P.row[i0 + j] = here++;
      } else if (me == 0 && i0 + j < P.S && (e[j] < 0 || e[j] >= P.E)) {
        P.row[i0 + j] = -1;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (i * kRound < P.S) place(i * kRound, keep[i], i);
  int round = kKeep;
  for (int32_t base = kKeep * kRound; base < P.S; base += kRound, ++round) place(base, four_slots(P, base + tid * 4), round);
  for (int32_t r = at + tid; r < (begin + mine) * P.tile_rows; r += kDispatchThreads) P.slot[r] = -1;
}

// ------------------------------------------------------------------ sums over a token's rows

struct CombineParams {
  const __nv_bfloat16* rows;  // [R, N], or null:
  const float* rows32;        // the same in fp32
  const int32_t* row;         // [T, k]
  const float* weights;       // [T, k] or null (ones)
  __nv_bfloat16* y;           // [T, N]
  int64_t T, N;
  int32_t k;
};

// Eight columns of a token a thread.  Bound by HBM: 4096 tokens of 4096, six
// rows each, 40 us, 0.87 of the copy rate.
__global__ void __launch_bounds__(256, 4) combine_kernel(const __grid_constant__ CombineParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t per_row = P.N / 8, unit = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, t = unit / per_row;
  if (t >= P.T) return;
  const int64_t c = (unit - t * per_row) * 8;
  float sum[8] = {};
  for (int32_t j0 = 0; j0 < P.k; j0 += 8) {  // eight rows on their way at a time
    int32_t r[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = j0 + j < P.k;
      r[j] = in ? P.row[t * P.k + j0 + j] : -1;
      w[j] = in && P.weights ? P.weights[t * P.k + j0 + j] : 1.f;
    }
    if (P.rows) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = r[j] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(P.rows + r[j] * P.N + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r[j] < 0) continue;
        float f[8];
        unpack8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
      }
    } else {
      float4 v[8][2];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4* from = reinterpret_cast<const float4*>(P.rows32 + r[j] * P.N + c);
        v[j][0] = r[j] >= 0 ? __ldcg(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[j][1] = r[j] >= 0 ? __ldcg(from + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r[j] < 0) continue;
        const float f[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w, v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
      }
    }
  }
  *reinterpret_cast<uint4*>(P.y + t * P.N + c) = pack8(sum);
}

struct DotParams {
  const __nv_bfloat16 *rows, *dy;
  const int32_t* row;
  __nv_bfloat16* dweights;
  int64_t S, N;
  int32_t k;
};

// The gradient of a slot's weight: dy[t] . rows[slot's row], a warp a slot
// (7 us for 3692 slots of 2048, of which the launch is a third).
__global__ void __launch_bounds__(256) weight_grad_kernel(const __grid_constant__ DotParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (s >= P.S) return;
  const uint32_t lane = threadIdx.x & 31;
  const int32_t r = P.row[s];
  float sum = 0.f;
  if (r >= 0) {
    const __nv_bfloat16 *a = P.rows + static_cast<int64_t>(r) * P.N, *b = P.dy + s / P.k * P.N;
#pragma unroll 4
    for (int64_t c = lane * 8; c < P.N; c += 256) {
      float u[8], v[8];
      unpack8(*reinterpret_cast<const uint4*>(a + c), u);
      unpack8(*reinterpret_cast<const uint4*>(b + c), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(u[i], v[i], sum);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (lane == 0) P.dweights[s] = __float2bfloat16_rn(sum);
}

// ------------------------------------------------------------------ host

struct Sizes {
  int p;
  int64_t E, T, k, h, f;
  int64_t S, tile_rows, max_tiles, max_pairs, rows;
  bool pairs;  // products on CTA pairs
  size_t plan_bytes;
};

// Rows of a tile.  A training step contracts over whole blocks of 128 rows.
// Without one, a tile's rows past its expert's are read for nothing and a
// second tile of an expert reads its weights again (from L2), so that the
// tile goes by the rows that an expert has on average (16 experts, 2048 x
// 2048; 32, 4096 x 1024; tiles of 16, 32, 64, 128 rows): 4 rows 56, 58, 58, 58
// us and 79, 78, 81, 83; 16 rows 61, 56, 58, 60 and 84, 81, 83, 85; 40 rows 63,
// 60, 56, 56 and 103, 93, 87, 89; 64 rows 72, 66, 62, 60 and 125, 103, 95, 93.
int64_t tile_rows_for(int64_t S, int64_t E, bool train) {
  const int64_t active = std::max<int64_t>(1, std::min(E, S)), mean = S / active;
  if (train) return 128;
  return mean <= 8 ? 16 : mean <= 20 ? 32 : mean <= 48 ? 64 : 128;
}

bool sizes_of(int p, int64_t E, int64_t T, int64_t k, int64_t h, int64_t f, bool train, Sizes* s) {
  s->p = p, s->E = E, s->T = T, s->k = k, s->h = h, s->f = f;
  s->S = T * k;
  s->tile_rows = tile_rows_for(s->S, E, train);
  // every expert that has rows leaves at most a tile less one row empty
  s->max_tiles = (s->S + (s->tile_rows - 1) * std::min(E, s->S)) / s->tile_rows;
  s->max_pairs = (s->max_tiles + std::min(E, s->S) + 1) / 2;
  s->rows = s->max_tiles * s->tile_rows;
  // Pairs of tiles on CTA pairs from 128 rows an expert on (16 experts, 2048 x
  // 2048; 32, 4096 x 1024; pairs against single tiles): 64 rows 63 against 61
  // us and 99 against 93, 128 rows 69 / 71 and 116 / 116, 192 rows 73 / 79 and
  // 132 / 138, 1024 rows 198 / 212 and 444 / 468.
  s->pairs = s->tile_rows == 128 && s->S >= 128 * std::min(E, s->S);
  s->plan_bytes = static_cast<size_t>(cdiv(2 + (E + 1) + s->max_tiles + 2 * s->max_pairs + s->rows + s->S, 64) * 64) * 4;
  return s->rows <= (int64_t(1) << 31) - 129;
}

tp_status check_experts(int p, int64_t E, int64_t T, int64_t k, int64_t h, int64_t f) {
  if (p < 1 || p > kMaxP || E < 1 || T < 0 || k < 1 || h < 1 || f < 1) return TP_ERR_INVALID_ARG;
  if (E % p != 0 || E > kMaxExperts || k > kMaxK) return TP_ERR_UNSUPPORTED_SHAPE;
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (T > lim || T * k > lim / 2 || h > lim || f > lim || E / p * std::max(h, f) > lim) return TP_ERR_UNSUPPORTED_SHAPE;
  if (h % 8 != 0 || f % 8 != 0) return TP_ERR_ALIGNMENT;
  return TP_OK;
}

Fp8Plan bounds_of(const Sizes& s) {
  Fp8Plan plan = {};
  plan.paired = s.pairs;
  plan.max_tiles = s.max_tiles;
  plan.tile_rows = s.tile_rows;
  plan.E = static_cast<int>(s.E);
  plan.k = static_cast<int>(s.k);
  return plan;
}

// The plan's arrays in its memory.
struct PlanArrays {
  int32_t *tiles, *pairs, *first, *expert, *pair, *slot, *row;
};
Fp8Plan plan_at(const Sizes& s, int32_t* at, PlanArrays* a) {
  a->tiles = at;
  a->pairs = at + 1;
  a->first = at + 2;
  a->expert = a->first + s.E + 1;
  a->pair = a->expert + s.max_tiles;
  a->slot = a->pair + 2 * s.max_pairs;
  a->row = a->slot + s.rows;
  Fp8Plan plan = bounds_of(s);
  plan.tiles = a->tiles;
  plan.pairs = a->pairs;
  plan.pair = a->pair;
  plan.first = a->first;
  plan.expert = a->expert;
  plan.slot = a->slot;
  return plan;
}

// Pieces of a workspace, one after the other; without memory, their size.
struct Area {
  uint8_t* base;
  size_t at = kDataOffset;
  explicit Area(void* ws) : base(static_cast<uint8_t*>(ws)) {}
  void* take(size_t bytes) {
    void* p = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return p;
  }
  tp_fp8 fp8(int64_t rows, int64_t cols, int64_t blocks) {
    tp_fp8 o;
    o.q = take(fp8_q_bytes(rows, cols));
    o.e = take(static_cast<size_t>(blocks * cdiv(cols, 512)) * 512);
    return o;
  }
};

struct ForwardArea {
  int32_t* plan;
  tp_fp8 xq, zq;
  void* out;     // the experts' outputs, bf16 or
  float* out32;  // fp32
  void* part;
  Fp8Launch first, second;
};

ForwardArea forward_area(const Sizes& s, bool train, Area* a) {
  ForwardArea f;
  const int64_t blocks = s.max_tiles * cdiv(s.tile_rows, 128);
  const Fp8Plan plan = bounds_of(s);
  f.first = fp8_plan(FP8_ROWS, s.rows, s.f, s.h, 1, 1, &plan);
  f.second = fp8_plan(FP8_ROWS, s.rows, s.h, s.f, 1, 1, &plan);
  f.plan = static_cast<int32_t*>(train ? nullptr : a->take(s.plan_bytes));
  f.xq = a->fp8(s.rows, s.h, blocks);
  f.zq = a->fp8(s.rows, s.f, blocks);
  // Few rows: their bytes do not matter.  Of many, the experts' outputs are bf16
  // until they are added up (half a step each, 2^-8): they are the largest
  // intermediate, and the other two bytes, written and read, are 403 MB more for
  // 4096 tokens of 4096 with six choices, 59 us at the copy rate beside 465.
  const bool fp32 = s.tile_rows < 128;
  f.out = train || fp32 ? nullptr : a->take(static_cast<size_t>(s.rows * s.h) * 2);
  f.out32 = static_cast<float*>(fp32 ? a->take(static_cast<size_t>(s.rows * s.h) * 4) : nullptr);
  const size_t part = std::max(f.first.part_bytes, f.second.part_bytes);
  f.part = part ? a->take(part) : nullptr;
  return f;
}

struct BackwardArea {
  tp_fp8 doq, dot, dhq, dht, xt, zt;
  void *dh, *dxr, *part;
  Fp8Launch first, second;
};

BackwardArea backward_area(const Sizes& s, Area* a) {
  BackwardArea b;
  const int64_t blocks = s.rows / 128;
  const Fp8Plan plan = bounds_of(s);
  b.first = fp8_plan(FP8_ROWS, s.rows, s.f, s.h, 1, 1, &plan);
  b.second = fp8_plan(FP8_ROWS, s.rows, s.h, s.f, 1, 1, &plan);
  b.doq = a->fp8(s.rows, s.h, blocks);
  b.dot = a->fp8(s.h, s.rows, cdiv(s.h, 128));
  b.dhq = a->fp8(s.rows, s.f, blocks);
  b.dht = a->fp8(s.f, s.rows, cdiv(s.f, 128));
  b.xt = a->fp8(s.h, s.rows, cdiv(s.h, 128));
  b.zt = a->fp8(s.f, s.rows, cdiv(s.f, 128));
  b.dh = a->take(static_cast<size_t>(s.rows * s.f) * 2);
  b.dxr = a->take(static_cast<size_t>(s.rows * s.h) * 2);  // bf16 until they are added up, as the forward pass's outputs
  const size_t part = std::max(b.first.part_bytes, b.second.part_bytes);
  b.part = part ? a->take(part) : nullptr;
  return b;
}

tp_status combine(const CombineParams& P, cudaStream_t stream) {
  const int64_t blocks = cdiv(P.T * (P.N / 8), 256);
  if (blocks > 0x7FFFFFFFll) return TP_ERR_UNSUPPORTED_SHAPE;
  return launch_dependent(combine_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, P);
}

const void* const* in(void* const* a) { return const_cast<const void* const*>(a); }

tp_status check_word(const void* p, bool need) {
  if (!need) return TP_OK;
  if (p == nullptr) return TP_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 ? TP_OK : TP_ERR_ALIGNMENT;
}

// Operands of `per` matrices [rows, cols] a shard.
void add_experts(RangeList* v, const tp_fp8* a, int p, int64_t per, int64_t rows, int64_t cols) { add_fp8(v, a, p, rows, cols, per); }

tp_status check_saved(const tp_experts_saved* s, bool work) {
  if (s == nullptr) return TP_ERR_INVALID_ARG;
  TP_TRY(check_ptr(s->plan, work));
  TP_TRY(check_ptr(s->preact, work));
  return check_ptr(s->out, work);
}

void add_saved(RangeList* v, const tp_experts_saved* d, const Sizes& s) {
  v->push_back({d->plan, s.plan_bytes});
  v->push_back({d->preact, static_cast<size_t>(s.rows * s.f) * 2});
  v->push_back({d->out, static_cast<size_t>(s.rows * s.h) * 2});
}

}  // namespace

extern "C" int64_t tp_experts_rows(int64_t E, int64_t T, int64_t k) {
  Sizes s;
  if (check_experts(1, E, T, k, 8, 8) != TP_OK || !sizes_of(1, E, T, k, 8, 8, true, &s)) return 0;
  return s.rows;
}

extern "C" size_t tp_experts_plan_size(int64_t E, int64_t T, int64_t k) {
  Sizes s;
  if (check_experts(1, E, T, k, 8, 8) != TP_OK || !sizes_of(1, E, T, k, 8, 8, true, &s)) return 0;
  return s.plan_bytes;
}

extern "C" size_t tp_experts_workspace_size(int p, int64_t E, int64_t T, int64_t k, int64_t h, int64_t f, int backward) {
  Sizes s;
  if (check_experts(p, E, T, k, h, f) != TP_OK || T == 0) return kStatusBytes;
  size_t most = kStatusBytes;
  for (int train = 0; train < (backward ? 2 : 1); ++train) {
    if (!sizes_of(p, E, T, k, h, f, train != 0, &s)) return kStatusBytes;
    Area a(nullptr);
    forward_area(s, train != 0, &a);
    most = std::max(most, a.at);
    if (train) {
      Area b(nullptr);
      backward_area(s, &b);
      most = std::max(most, b.at);
    }
  }
  return most;
}

extern "C" tp_status tp_experts_fwd_fp8(const void* x, const void* experts, const void* weights, const tp_fp8* w1, const tp_fp8* w2, void* y,
                                        const tp_experts_saved* saved, int p, int64_t E, int64_t T, int64_t k, int64_t h, int64_t f, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_experts(p, E, T, k, h, f));
  const bool work = T > 0, train = saved != nullptr;
  TP_TRY(check_ptr(x, work));
  TP_TRY(check_word(experts, work));
  TP_TRY(check_word(weights, work));
  TP_TRY(check_fp8(w1, p, work));
  TP_TRY(check_fp8(w2, p, work));
  TP_TRY(check_ptr(y, work));
  if (train) TP_TRY(check_saved(saved, work));
  Sizes s;
  if (!sizes_of(p, E, T, k, h, f, train, &s) || (train && s.rows / 128 > kMostStrips)) return TP_ERR_UNSUPPORTED_SHAPE;
  size_t need = kStatusBytes;
  if (work) {
    Area a(nullptr);
    forward_area(s, train, &a);
    need = a.at;
  }
  TP_TRY(check_ws(ws, ws_bytes, need));
  if (!work) return TP_OK;
  const int64_t per = E / p;
  {
    RangeList ins, outs;
    ins.push_back({x, static_cast<size_t>(T * h) * 2});
    ins.push_back({experts, static_cast<size_t>(s.S) * 4});
    ins.push_back({weights, static_cast<size_t>(s.S) * 4});
    add_experts(&ins, w1, p, per, f, h);
    add_experts(&ins, w2, p, per, h, f);
    outs.push_back({y, static_cast<size_t>(T * h) * 2});
    if (train) add_saved(&outs, saved, s);
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  Area area(ws);
  const ForwardArea A = forward_area(s, train, &area);
  PlanArrays at;
  const Fp8Plan plan = plan_at(s, train ? static_cast<int32_t*>(saved->plan) : A.plan, &at);
  DispatchParams D;
  D.experts = static_cast<const int32_t*>(experts);
  D.tiles = at.tiles, D.pairs = at.pairs, D.first = at.first, D.expert = at.expert, D.pair = at.pair, D.slot = at.slot, D.row = at.row;
  D.S = static_cast<int32_t>(s.S);
  D.E = static_cast<int32_t>(E);
  D.tile_rows = static_cast<int32_t>(s.tile_rows);
  D.aligned = aligned16(experts);
  TokenPack& K = D.pack;
  K.row = at.row;
  K.x = static_cast<const __nv_bfloat16*>(x);
  K.q = static_cast<uint8_t*>(A.xq.q);
  K.e = static_cast<uint8_t*>(A.xq.e);
  K.tokens = T;
  K.cols = h;
  K.ldq = fp8_pitch(h);
  K.e_block = cdiv(h, 512) * 512;
  K.k = static_cast<int32_t>(k);
  K.tile_rows = D.tile_rows;
  const bool few = s.S <= kFewSlots;
  const int64_t packs = few ? cdiv(T * (K.e_block / 512), kDispatchThreads / 32) : 0;
  TP_TRY(launch_dependent(dispatch_kernel, dim3(static_cast<unsigned>(E + packs)), kDispatchThreads, 0, stream, D));
  if (!few) TP_TRY(fp8_pack_tokens(K, stream));
  uint32_t* status = static_cast<uint32_t*>(ws);
  void* preact = train ? saved->preact : nullptr;
  void* out = train ? saved->out : A.out;
  Fp8Product g;
  g.mode = FP8_ROWS;
  g.a = &A.xq;
  g.b = w1;
  g.nb = p;
  g.rows = s.rows;
  g.cols = f;
  g.depth = h;
  g.plan = &plan;
  g.per = static_cast<int>(per);
  g.epi = TP_EPI_GELU;
  g.z = &A.zq;
  g.aux = preact ? &preact : nullptr;
  TP_TRY(fp8_product(g, A.first, A.part, status, stream));
  Fp8Product o;
  o.mode = FP8_ROWS;
  o.a = &A.zq;
  o.b = w2;
  o.nb = p;
  o.rows = s.rows;
  o.cols = h;
  o.depth = f;
  o.plan = &plan;
  o.per = static_cast<int>(per);
  o.out = &out;
  o.out32 = A.out32;
  TP_TRY(fp8_product(o, A.second, A.part, status, stream));
  CombineParams C;
  std::memset(&C, 0, sizeof(C));
  C.rows = A.out32 ? nullptr : static_cast<const __nv_bfloat16*>(out);
  C.rows32 = A.out32;
  C.row = at.row;
  C.weights = static_cast<const float*>(weights);
  C.y = static_cast<__nv_bfloat16*>(y);
  C.T = T;
  C.N = h;
  C.k = static_cast<int32_t>(k);
  return combine(C, stream);
}

extern "C" tp_status tp_experts_bwd_fp8(const void* x, const void* weights, const void* dy, const tp_fp8* w1t, const tp_fp8* w2t, void* dx,
                                        void* dweights, void* const* dw1, void* const* dw2, const tp_experts_saved* saved, int p, int64_t E,
                                        int64_t T, int64_t k, int64_t h, int64_t f, void* ws, size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_experts(p, E, T, k, h, f));
  const bool work = T > 0;
  if (dx == nullptr && dweights == nullptr && dw1 == nullptr && dw2 == nullptr) return TP_ERR_INVALID_ARG;
  const bool need_h = dx != nullptr || dw1 != nullptr;  // the gradient of the pre-activations
  TP_TRY(check_ptr(x, work && dw1 != nullptr));
  TP_TRY(check_word(weights, work));
  TP_TRY(check_ptr(dy, work));
  TP_TRY(check_fp8(w1t, p, work && dx != nullptr));
  TP_TRY(check_fp8(w2t, p, work && need_h));
  TP_TRY(check_ptr(dx, work && dx != nullptr));
  if (dweights != nullptr && reinterpret_cast<uintptr_t>(dweights) % 2 != 0) return TP_ERR_ALIGNMENT;
  TP_TRY(check_ptrs(in(dw1), p, dw1 != nullptr));
  TP_TRY(check_ptrs(in(dw2), p, dw2 != nullptr));
  TP_TRY(check_saved(saved, work));
  Sizes s;
  if (!sizes_of(p, E, T, k, h, f, true, &s) || s.rows / 128 > kMostStrips) return TP_ERR_UNSUPPORTED_SHAPE;
  size_t need = kStatusBytes;
  if (work) {
    Area a(nullptr);
    backward_area(s, &a);
    need = a.at;
  }
  TP_TRY(check_ws(ws, ws_bytes, need));
  const int64_t per = E / p;
  const size_t dw_bytes = static_cast<size_t>(per * h * f) * 2;
  {
    RangeList ins, outs;
    if (work) {
      ins.push_back({x, x ? static_cast<size_t>(T * h) * 2 : 0});
      ins.push_back({weights, static_cast<size_t>(s.S) * 4});
      ins.push_back({dy, static_cast<size_t>(T * h) * 2});
      if (dx) add_experts(&ins, w1t, p, per, h, f);
      if (need_h) add_experts(&ins, w2t, p, per, f, h);
      add_saved(&ins, saved, s);
    }
    outs.push_back({dx, dx ? static_cast<size_t>(T * h) * 2 : 0});
    outs.push_back({dweights, dweights ? static_cast<size_t>(s.S) * 2 : 0});
    add_ranges(&outs, in(dw1), p, dw_bytes);
    add_ranges(&outs, in(dw2), p, dw_bytes);
    outs.push_back({ws, ws_bytes});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  if (!work) {  // no token: the weights' gradients are zero
    for (int r = 0; r < p; ++r) {
      if (dw1 && cudaMemsetAsync(dw1[r], 0, dw_bytes, stream) != cudaSuccess) return TP_ERR_CUDA;
      if (dw2 && cudaMemsetAsync(dw2[r], 0, dw_bytes, stream) != cudaSuccess) return TP_ERR_CUDA;
    }
    return TP_OK;
  }
  Area area(ws);
  const BackwardArea A = backward_area(s, &area);
  PlanArrays at;
  const Fp8Plan plan = plan_at(s, static_cast<int32_t*>(saved->plan), &at);
  uint32_t* status = static_cast<uint32_t*>(ws);
  if (dweights) {
    DotParams D;
    D.rows = static_cast<const __nv_bfloat16*>(saved->out);
    D.dy = static_cast<const __nv_bfloat16*>(dy);
    D.row = at.row;
    D.dweights = static_cast<__nv_bfloat16*>(dweights);
    D.S = s.S;
    D.N = h;
    D.k = static_cast<int32_t>(k);
    TP_TRY(launch_dependent(weight_grad_kernel, dim3(static_cast<unsigned>(cdiv(s.S, 8))), 256, 0, stream, D));
  }
  if (!need_h && dw2 == nullptr) return TP_OK;
  // the rows' gradients, weights * dy
  Fp8Pack pack;
  pack.x = &dy;
  pack.q = need_h ? &A.doq : nullptr;
  pack.qt = dw2 ? &A.dot : nullptr;
  pack.rows = s.rows;
  pack.cols = h;
  pack.plan = &plan;
  pack.weights = static_cast<const float*>(weights);
  TP_TRY(fp8_pack(pack, stream));
  void *dh = A.dh, *dxr = A.dxr, *preact = saved->preact;
  if (need_h) {
    Fp8Product g;
    g.mode = FP8_ROWS;
    g.a = &A.doq;
    g.b = w2t;
    g.nb = p;
    g.rows = s.rows;
    g.cols = f;
    g.depth = h;
    g.plan = &plan;
    g.per = static_cast<int>(per);
    g.epi = TP_EPI_DGELU;
    g.out = &dh;
    g.aux = &preact;
    TP_TRY(fp8_product(g, A.first, A.part, status, stream));
    const void* src = dh;
    pack = Fp8Pack();
    pack.x = &src;
    pack.q = dx ? &A.dhq : nullptr;
    pack.qt = dw1 ? &A.dht : nullptr;
    pack.rows = s.rows;
    pack.cols = f;
    pack.plan = &plan;
    pack.gather = false;
    TP_TRY(fp8_pack(pack, stream));
  }
  if (dx) {
    Fp8Product g;
    g.mode = FP8_ROWS;
    g.a = &A.dhq;
    g.b = w1t;
    g.nb = p;
    g.rows = s.rows;
    g.cols = h;
    g.depth = f;
    g.plan = &plan;
    g.per = static_cast<int>(per);
    g.out = &dxr;
    TP_TRY(fp8_product(g, A.second, A.part, status, stream));
    CombineParams C;
    std::memset(&C, 0, sizeof(C));
    C.rows = static_cast<const __nv_bfloat16*>(dxr);
    C.row = at.row;
    C.y = static_cast<__nv_bfloat16*>(dx);
    C.T = T;
    C.N = h;
    C.k = static_cast<int32_t>(k);
    TP_TRY(combine(C, stream));
  }
  auto contract = [&](const tp_fp8* a, const tp_fp8* b, int64_t rows, int64_t cols, void* const* out) {
    Fp8Product g;
    g.mode = FP8_CONTRACT;
    g.a = a;
    g.b = b;
    g.rows = rows;
    g.cols = cols;
    g.depth = s.rows;
    g.groups = static_cast<int>(E);
    g.plan = &plan;
    g.per = static_cast<int>(per);
    g.out = out;
    return fp8_product(g, fp8_plan(FP8_CONTRACT, rows, cols, s.rows, g.groups, 1), nullptr, status, stream);
  };
  if (dw1) {
    pack = Fp8Pack();
    pack.x = &x;
    pack.qt = &A.xt;
    pack.rows = s.rows;
    pack.cols = h;
    pack.plan = &plan;
    TP_TRY(fp8_pack(pack, stream));
    TP_TRY(contract(&A.xt, &A.dht, h, f, dw1));
  }
  if (dw2) {
    const void* src = preact;
    pack = Fp8Pack();
    pack.x = &src;
    pack.qt = &A.zt;
    pack.rows = s.rows;
    pack.cols = f;
    pack.gelu = true;
    pack.plan = &plan;
    pack.gather = false;
    TP_TRY(fp8_pack(pack, stream));
    TP_TRY(contract(&A.zt, &A.dot, f, h, dw2));
  }
  return TP_OK;
}
