// Routing of tokens to experts, forward and backward.
//
//   s = softmax(l) or sigmoid(l);  v = s + bias
//   groups: those with the largest sums of their `group_best` largest v stay
//   experts: the k largest v of them, ties to the lower number
//   weights: scale * s, or scale * s / (sum of the chosen s)
// An expert whose logit is -infinity or NaN is closed.
//
// The choice is the one that exact arithmetic makes.  The scores are formed
// in fp32, within kBand of their values; where two that the choice has to
// tell apart are nearer than that, the warp forms the row's scores again in
// 64 bits and chooses by those (about one row in two hundred of 256 experts
// with a bias; the GPU has few 64-bit units, so that a row takes as long as
// some hundred others).  Without a bias and groups no score is compared at
// all: both functions grow with the logit, and the logits are exact.
//
// A warp has a row, its experts spread over the lanes (expert 32 i + lane in
// register i).  A largest value is found by two reductions over the warp, of
// its bits in an order-preserving form and of the lowest expert that has it.
// Bound by latency: 4 MB of logits of 8192 tokens take 0.7 us at the copy
// rate.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "host_util.h"
#include "vec_util.cuh"

using namespace tpf;

namespace {

constexpr int kMaxExperts = TP_ROUTE_MAX_EXPERTS, kMaxK = 32, kMaxGroups = 32;
constexpr int kWarps = 4;  // of a thread block
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kNone = 0xFFFFFFFFu;
// How near two fp32 scores (with their biases, relative to the larger of 1
// and |v|) may be and still be told apart: the sum over the row has an error
// of PER + 5 roundings of 2^-24, expf, the division and the addition some
// units each, and there are two of them.
constexpr float band_of(int per) { return static_cast<float>(per + 12) * 1.1920929e-7f; }

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* experts;
  float* weights;
  int32_t* counts;
  const float* dweights;
  void* dlogits;
  int64_t T;
  int32_t E, k, groups, tops, best;
  int32_t f32, sigmoid, renorm;
  float scale;
};

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = warp_max(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = warp_max(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The logit of an expert: -infinity for a closed one, else finite.
__device__ __forceinline__ float clean(float l) {
  return l > -INFINITY ? fminf(l, FLT_MAX) + 0.f : -INFINITY;  // one zero
}

template <int PER>
__device__ __forceinline__ void load_row(const RouteParams& P, int64_t row, uint32_t lane, float (&l)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int32_t e = i * 32 + static_cast<int32_t>(lane);
    l[i] = -INFINITY;
    if (e < P.E) {
      const int64_t at = row * P.E + e;
      l[i] = clean(P.f32 ? static_cast<const float*>(P.logits)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(P.logits)[at]));
    }
  }
}

template <typename T>
__device__ __forceinline__ T exp_of(T x) {
  if constexpr (sizeof(T) == 8) return exp(x);
  else return expf(x);
}

// Scores of the row's experts; 0 of closed ones.
template <typename T, int PER>
__device__ __forceinline__ void scores(const RouteParams& P, const float (&l)[PER], T (&s)[PER]) {
  if (P.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = l[i] > -INFINITY ? T(1) / (T(1) + exp_of<T>(-static_cast<T>(l[i]))) : T(0);
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  T sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    // both finite, their difference perhaps not: then its exponential is 0
    s[i] = l[i] > -INFINITY ? exp_of<T>(static_cast<T>(l[i]) - static_cast<T>(top)) : T(0);
    sum += s[i];
  }
  sum = warp_sum(sum);
  const T r = sum > 0 ? T(1) / sum : T(0);
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] *= r;
}

// The chosen experts, in order: choice j in lane j of `mine` (kNone: none).
// False if two values that the choice compares are within `band`.  v is used
// up; it is -infinity where an expert cannot be chosen.
template <typename T, int PER>
__device__ __forceinline__ bool choose(const RouteParams& P, const float (&l)[PER], T (&v)[PER], float band, uint32_t lane, uint32_t& mine) {
  bool clear = true;
  T before = 0;
  float l_before = 0.f, b_before = 0.f;
  mine = kNone;
  const T shut = -INFINITY;
  const int32_t rounds = band > 0.f ? P.k + 1 : P.k;  // the first that is left out has to be told apart too
  for (int32_t j = 0; j < rounds; ++j) {
    T own = shut;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (v[i] > own) {
        own = v[i];
        at = i;
      }
    const auto top = warp_max(ordered(own));
    if (top == ordered(shut)) break;
    const uint32_t who = __reduce_min_sync(kAll, ordered(own) == top ? at * 32 + lane : kNone);
    const T val = __shfl_sync(kAll, own, who & 31);
    if (j < P.k && static_cast<int32_t>(lane) == j) mine = who;
    const int slot = static_cast<int>(who >> 5);
    float lv = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i == slot) {
        lv = l[i];
        if ((who & 31) == lane) v[i] = shut;
      }
    if (band > 0.f) {
      // equal logits and biases are equal exactly
      lv = __shfl_sync(kAll, lv, who & 31);
      const float b = P.bias[who];
      if (j > 0 && before - val <= static_cast<T>(band) * fmaxf(1.f, fabsf(static_cast<float>(val))) && !(lv == l_before && b == b_before))
        clear = false;
      l_before = lv;
      b_before = b;
    }
    before = val;
  }
  return clear;
}

// Closes the experts of groups that are not among the best.
template <typename T, int PER>
__device__ __forceinline__ bool keep_groups(const RouteParams& P, T (&v)[PER], float band, uint32_t lane) {
  const T shut = -INFINITY;
  const int32_t size = P.E / P.groups;
  T score = shut;  // of group `lane`
  for (int32_t g = 0; g < P.groups; ++g) {
    T sum = shut;
    uint32_t taken = kNone;
    for (int32_t b = 0; b < P.best; ++b) {
      T own = shut;
      uint32_t at = kNone;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t e = i * 32 + lane;
        if (static_cast<int32_t>(e) >= g * size && static_cast<int32_t>(e) < (g + 1) * size && e != taken && v[i] > own) {
          own = v[i];
          at = e;
        }
      }
      const auto top = warp_max(ordered(own));
      if (top == ordered(shut)) break;
      taken = __reduce_min_sync(kAll, ordered(own) == top ? at : kNone);
      const T val = __shfl_sync(kAll, own, taken & 31);
      sum = b == 0 ? val : sum + val;
    }
    if (static_cast<int32_t>(lane) == g) score = sum;
  }
  // rank of each group among all
  bool clear = true;
  int32_t rank = 0;
  for (int32_t g = 0; g < P.groups; ++g) {
    const T other = __shfl_sync(kAll, score, g);
    if (other > score || (other == score && g < static_cast<int32_t>(lane))) ++rank;
  }
  const bool in = static_cast<int32_t>(lane) < P.groups && rank < P.tops && score > shut;
  if (band > 0.f && P.tops < P.groups) {
    // the last that stays and the first that goes
    T last = in ? score : static_cast<T>(INFINITY), first = !in && static_cast<int32_t>(lane) < P.groups ? score : shut;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const T a = __shfl_xor_sync(kAll, last, o), b = __shfl_xor_sync(kAll, first, o);
      last = a < last ? a : last;
      first = b > first ? b : first;
    }
    if (first > shut && last - first <= static_cast<T>(2 * band) * fmaxf(1.f, fabsf(static_cast<float>(last)))) clear = false;
  }
  const uint32_t kept = __ballot_sync(kAll, in);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t e = i * 32 + lane;
    if (static_cast<int32_t>(e) < P.E && !(kept >> (e / size) & 1u)) v[i] = shut;
  }
  return clear;
}

template <typename T, int PER>
__device__ __forceinline__ bool select(const RouteParams& P, const float (&l)[PER], const T (&s)[PER], float band, uint32_t lane,
                                       uint32_t& mine) {
  T v[PER];
  const bool by_logit = P.bias == nullptr && (P.groups == 1 || P.best == 1);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int32_t e = i * 32 + static_cast<int32_t>(lane);
    if (by_logit) v[i] = static_cast<T>(l[i]);
    else v[i] = l[i] > -INFINITY ? s[i] + (P.bias && e < P.E ? static_cast<T>(P.bias[e]) : T(0)) : static_cast<T>(-INFINITY);
  }
  bool clear = true;
  if (P.groups > 1) {
    clear = keep_groups<T, PER>(P, v, by_logit ? 0.f : band, lane);
    if (P.bias == nullptr && !by_logit) {  // what is left is told apart by its logits
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (v[i] > static_cast<T>(-INFINITY)) v[i] = static_cast<T>(l[i]);
    }
  }
  return choose<T, PER>(P, l, v, P.bias == nullptr ? 0.f : band, lane, mine) && clear;
}

// The value of expert e, another one for each lane; 0 for none.
template <int PER>
__device__ __forceinline__ float pick(const float (&s)[PER], uint32_t e) {
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float o = __shfl_sync(kAll, s[i], e & 31);
    if (e != kNone && static_cast<uint32_t>(i) == e >> 5) v = o;
  }
  return v;
}

template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_fwd_kernel(const __grid_constant__ RouteParams P) {
  extern __shared__ int32_t hist[];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  if (P.counts) {
    for (int32_t e = threadIdx.x; e < P.E; e += kWarps * 32) hist[e] = 0;
    __syncthreads();
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < P.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[PER], s[PER];
    load_row<PER>(P, row, lane, l);
    scores<float, PER>(P, l, s);
    uint32_t mine;
    if (!select<float, PER>(P, l, s, band_of(PER), lane, mine)) {
      double sd[PER];
      scores<double, PER>(P, l, sd);
      select<double, PER>(P, l, sd, 0.f, lane, mine);
    }
    const float sc = pick<PER>(s, mine);
    const float total = P.renorm ? fmaxf(warp_sum(sc), FLT_MIN) : 1.f;
    if (static_cast<int32_t>(lane) < P.k) {
      P.experts[row * P.k + lane] = mine == kNone ? -1 : static_cast<int32_t>(mine);
      P.weights[row * P.k + lane] = P.scale * (sc / total);
      if (P.counts && mine != kNone) atomicAdd(hist + mine, 1);
    }
  }
  if (P.counts) {
    __syncthreads();
    for (int32_t e = threadIdx.x; e < P.E; e += kWarps * 32) {
      if (gridDim.x == 1) P.counts[e] = hist[e];
      else if (hist[e]) atomicAdd(P.counts + e, hist[e]);  // whole numbers: their sum has no order
    }
  }
}

__global__ void route_clear_kernel(const __grid_constant__ RouteParams P) {
  griddep_wait();
  griddep_launch_dependents();
  for (int32_t e = threadIdx.x; e < P.E; e += blockDim.x) P.counts[e] = 0;
}

template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const __grid_constant__ RouteParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < P.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[PER], s[PER];
    load_row<PER>(P, row, lane, l);
    scores<float, PER>(P, l, s);
    uint32_t mine = kNone;
    float g = 0.f;
    if (static_cast<int32_t>(lane) < P.k) {
      const int32_t e = P.experts[row * P.k + lane];
      if (e >= 0 && e < P.E) {
        mine = static_cast<uint32_t>(e);
        g = P.scale * P.dweights[row * P.k + lane];
      }
    }
    const float sc = pick<PER>(s, mine);
    if (P.renorm) {  // w = s / sum s
      const float total = fmaxf(warp_sum(sc), FLT_MIN);
      const float all = warp_sum(g * sc) / total;
      g = mine == kNone ? 0.f : (g - all) / total;
    }
    // the gradient of each expert's score
    float ds[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) ds[i] = 0.f;
    for (int32_t j = 0; j < P.k; ++j) {
      const uint32_t e = __shfl_sync(kAll, mine, j);
      const float v = __shfl_sync(kAll, g, j);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e == i * 32 + lane) ds[i] += v;
    }
    float dot = 0.f;
    if (!P.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) dot += ds[i] * s[i];
      dot = warp_sum(dot);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int32_t e = i * 32 + static_cast<int32_t>(lane);
      if (e < P.E) {
        float d = s[i] * (ds[i] - dot);
        if (P.sigmoid) {  // s (1 - s) without the difference
          const float t = expf(-fabsf(l[i]));
          d = ds[i] * (t / ((1.f + t) * (1.f + t)));
        }
        const int64_t at = row * P.E + e;
        if (P.f32) static_cast<float*>(P.dlogits)[at] = d;
        else static_cast<__nv_bfloat16*>(P.dlogits)[at] = __float2bfloat16_rn(d);
      }
    }
  }
}

tp_status check(const tp_route_desc* d, int64_t T, int64_t E, int64_t k, tp_dtype dt) {
  if (d == nullptr || T < 0 || E < 1 || k < 1) return TP_ERR_INVALID_ARG;
  if (dt != TP_BF16 && dt != TP_FP32) return TP_ERR_INVALID_ARG;
  if (d->score != TP_ROUTE_SOFTMAX && d->score != TP_ROUTE_SIGMOID) return TP_ERR_INVALID_ARG;
  if (d->groups < 1 || d->top_groups < 1 || d->top_groups > d->groups) return TP_ERR_INVALID_ARG;
  if (d->group_best != 1 && d->group_best != 2) return TP_ERR_INVALID_ARG;
  if ((d->renorm != 0 && d->renorm != 1) || !std::isfinite(d->scale)) return TP_ERR_INVALID_ARG;
  if (k > E) return TP_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMaxK || d->groups > kMaxGroups || E % d->groups != 0) return TP_ERR_UNSUPPORTED_SHAPE;
  if (T > (int64_t(1) << 31) - 1) return TP_ERR_UNSUPPORTED_SHAPE;
  return TP_OK;
}

// Logits have no 16-byte rows to keep: any element's alignment does.
tp_status check_at(const void* p, size_t size, bool need) {
  if (!need) return TP_OK;
  if (p == nullptr) return TP_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % size == 0 ? TP_OK : TP_ERR_ALIGNMENT;
}

void fill(RouteParams* P, const tp_route_desc* d, int64_t T, int64_t E, int64_t k, tp_dtype dt) {
  std::memset(P, 0, sizeof(*P));
  P->T = T;
  P->E = static_cast<int32_t>(E);
  P->k = static_cast<int32_t>(k);
  P->groups = d->groups;
  P->tops = d->top_groups;
  P->best = d->group_best;
  P->f32 = dt == TP_FP32;
  P->sigmoid = d->score == TP_ROUTE_SIGMOID;
  P->renorm = d->renorm;
  P->scale = d->scale;
}

// A row a warp; more than 16 thread blocks an SM take several.
unsigned grid_of(int64_t T) { return static_cast<unsigned>(std::min<int64_t>(cdiv(T, kWarps), 152 * 16)); }

template <int PER>
tp_status run(bool fwd, const RouteParams& P, cudaStream_t stream) {
  return fwd ? launch_dependent(route_fwd_kernel<PER>, dim3(grid_of(P.T)), kWarps * 32, P.counts ? P.E * sizeof(int32_t) : 0, stream, P)
             : launch_dependent(route_bwd_kernel<PER>, dim3(grid_of(P.T)), kWarps * 32, 0, stream, P);
}

tp_status run(bool fwd, const RouteParams& P, cudaStream_t stream) {
  if (P.E <= 64) return run<2>(fwd, P, stream);
  if (P.E <= 128) return run<4>(fwd, P, stream);
  if (P.E <= 256) return run<8>(fwd, P, stream);
  return run<16>(fwd, P, stream);
}

}  // namespace

extern "C" tp_status tp_route_fwd(const void* logits, const void* bias, void* experts, void* weights, void* counts, const tp_route_desc* d,
                                  int64_t T, int64_t E, int64_t k, tp_dtype dtype, cudaStream_t stream) {
  TP_TRY(check(d, T, E, k, dtype));
  const bool work = T > 0;
  TP_TRY(check_at(logits, esize(dtype), work));
  TP_TRY(check_at(bias, 4, bias != nullptr && work));
  TP_TRY(check_at(experts, 4, work));
  TP_TRY(check_at(weights, 4, work));
  TP_TRY(check_at(counts, 4, counts != nullptr));
  {
    RangeList ins, outs;
    ins.push_back({logits, static_cast<size_t>(T * E) * esize(dtype)});
    if (bias) ins.push_back({bias, static_cast<size_t>(E) * 4});
    outs.push_back({experts, static_cast<size_t>(T * k) * 4});
    outs.push_back({weights, static_cast<size_t>(T * k) * 4});
    if (counts) outs.push_back({counts, static_cast<size_t>(E) * 4});
    if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  }
  if (!work && counts == nullptr) return TP_OK;
  DevInfo di;
  TP_TRY(device_info(&di));
  RouteParams P;
  fill(&P, d, T, E, k, dtype);
  P.logits = logits;
  P.bias = static_cast<const float*>(bias);
  P.experts = static_cast<int32_t*>(experts);
  P.weights = static_cast<float*>(weights);
  P.counts = static_cast<int32_t*>(counts);
  // one thread block writes its counts, several add theirs to zeros
  if (counts && (!work || grid_of(T) > 1)) TP_TRY(launch_dependent(route_clear_kernel, dim3(1), 256, 0, stream, P));
  return work ? run(true, P, stream) : TP_OK;
}

extern "C" tp_status tp_route_bwd(const void* logits, const void* experts, const void* dweights, void* dlogits, const tp_route_desc* d,
                                  int64_t T, int64_t E, int64_t k, tp_dtype dtype, cudaStream_t stream) {
  TP_TRY(check(d, T, E, k, dtype));
  const bool work = T > 0;
  TP_TRY(check_at(logits, esize(dtype), work));
  TP_TRY(check_at(experts, 4, work));
  TP_TRY(check_at(dweights, 4, work));
  TP_TRY(check_at(dlogits, esize(dtype), work));
  if (!work) return TP_OK;
  RangeList ins, outs;
  ins.push_back({logits, static_cast<size_t>(T * E) * esize(dtype)});
  ins.push_back({experts, static_cast<size_t>(T * k) * 4});
  ins.push_back({dweights, static_cast<size_t>(T * k) * 4});
  outs.push_back({dlogits, static_cast<size_t>(T * E) * esize(dtype)});
  if (any_overlap(outs, ins)) return TP_ERR_INVALID_ARG;
  DevInfo di;
  TP_TRY(device_info(&di));
  RouteParams P;
  fill(&P, d, T, E, k, dtype);
  P.logits = logits;
  P.experts = static_cast<int32_t*>(const_cast<void*>(experts));
  P.dweights = static_cast<const float*>(dweights);
  P.dlogits = dlogits;
  return run(false, P, stream);
}
