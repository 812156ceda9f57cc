// Routing of tokens to experts, forward and backward.
//
//   s = softmax(l) or sigmoid(l);  v = s + bias
//   groups: those with the largest sums of their `group_best` largest v stay
//   experts: the k largest v of them, ties to the lower number
//   weights: scale * s, or scale * s / (sum of the chosen s)
// An expert whose logit is -infinity or NaN is closed.
//
// The choice is the one that exact arithmetic makes.  The scores are formed
// in fp32, within band_of() of their values; where two that the choice has to
// tell apart are nearer than that, the warp forms the row's scores again as
// pairs of fp32 numbers, to some 2^-45 (in 64-bit arithmetic, for which the GPU
// has few units, such a row took 16 us), and chooses by those.  Without a bias
// and groups no score is compared at all: both functions grow with the logit,
// and the logits are exact.
//
// A warp has a row, lane t the experts PER t .. PER t + PER - 1, so that a row
// is read in vectors, a group of experts is a few neighbouring lanes, and the
// lowest lane with a value has the lowest expert.  A largest value is found by
// one reduction over the warp of its bits in an order-preserving form, and the
// lane that has it looks which expert it is.  Bound by instructions (8192
// tokens, 8 of 256 experts from 4 of 8 groups, with counts and gradient: 24 us,
// where the bytes take 2): each choice is a reduction over the warp and a few
// dependent steps.  One token is the launch.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "host_util.h"
#include "vec_util.cuh"

using namespace tpf;

namespace {

constexpr int kMaxExperts = TP_ROUTE_MAX_EXPERTS, kMaxK = 32, kMaxGroups = 32;
constexpr int kWarps = 4;  // of a thread block
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kNone = 0xFFFFFFFFu;
// How near two fp32 values (relative to the larger of 1 and |v|) may be and
// still be told apart, in units of 2^-23.  Sigmoid: exp and the reciprocal are
// off by one unit of theirs, 1 + exp and the sum with the bias by half: with
// s (1 - s) <= 1/4 that is 2.3 units of a value up to 1, for two of them 4.6.
// Softmax: the sum over the row has PER + 5 additions of positive values.
constexpr float kUlp = 1.1920929e-7f;
__device__ __forceinline__ float band_of(int per, bool sigmoid) { return (sigmoid ? 6 : per + 12) * kUlp; }

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
  int32_t vector;       // a lane's logits are one aligned vector
  int32_t group_lanes;  // lanes of a group, 0: groups do not end between lanes
  float scale;
};

// Order-preserving bits: a larger number for a larger value.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kShut = 0x007FFFFFu;  // ordered(-infinity)

// ------------------------------------------------------------------ pairs of fp32 numbers
//
// hi + lo, |lo| at most half a unit in hi's last place; sums and products by
// Dekker (1971) and Knuth (TAOCP 2, 4.2.2), with the product's error from a
// fused multiply-add.

struct Df {
  float hi, lo;
};
__device__ __forceinline__ Df two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Df quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Df add(Df a, Df b) {
  const Df s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Df u = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
  return quick_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Df mul(Df a, Df b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return quick_sum(p, __fadd_rn(__fmaf_rn(a.hi, b.hi, -p), __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}

// exp(x) for x <= 0, 0 below -80: x = n ln 2 + 4 y, |y| < 0.087, with ln 2 in
// three parts (the first of 16 bits, so that n times it is exact), the series
// of exp(y) up to y^8, and two squarings.
__device__ __forceinline__ Df exp_df(Df x) {
  const float n = rintf(x.hi * 1.44269504f);
  const float r1 = __fmaf_rn(-n, 0x1.62e4p-1f, x.hi);
  const float c2 = 0x1.7f7d1cp-20f, p = __fmul_rn(n, c2), pe = __fmaf_rn(n, c2, -p);
  Df r = add(two_sum(r1, x.lo), Df{-p, -pe});
  r = quick_sum(r.hi, __fadd_rn(r.lo, -n * 0x1.ef357ap-45f));
  const Df y = {0.25f * r.hi, 0.25f * r.lo};
  const float q = fmaf(fmaf(fmaf(y.hi, 1.f / 40320.f, 1.f / 5040.f), y.hi, 1.f / 720.f), y.hi, 1.f / 120.f);
  Df h = add(Df{0x1.555556p-5f, -0x1.555556p-30f}, Df{y.hi * q, 0.f});
  h = add(Df{0x1.555556p-3f, -0x1.555556p-28f}, mul(y, h));
  h = add(Df{0.5f, 0.f}, mul(y, h));
  h = add(Df{1.f, 0.f}, mul(y, h));
  h = add(Df{1.f, 0.f}, mul(y, h));
  h = mul(h, h);
  h = mul(h, h);
  const float two = __uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(n) + 127) << 23);
  return x.hi < -80.f ? Df{0.f, 0.f} : Df{h.hi * two, h.lo * two};
}
__device__ __forceinline__ Df inverse(Df d) {  // of 1 and above
  const float q = __fdiv_rn(1.f, d.hi);
  return quick_sum(q, q * __fmaf_rn(-q, d.lo, __fmaf_rn(-q, d.hi, 1.f)));
}
__device__ __forceinline__ Df shfl(Df v, int lane) { return {__shfl_sync(kAll, v.hi, lane), __shfl_sync(kAll, v.lo, lane)}; }
__device__ __forceinline__ Df shfl_xor(Df v, int o) { return {__shfl_xor_sync(kAll, v.hi, o), __shfl_xor_sync(kAll, v.lo, o)}; }
__device__ __forceinline__ bool greater(Df a, Df b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ bool open(Df v) { return v.hi > -INFINITY; }
__device__ __forceinline__ Df larger(Df a, Df b) { return greater(b, a) ? b : a; }
__device__ __forceinline__ Df smaller(Df a, Df b) { return greater(b, a) ? a : b; }

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float shfl(float v, int lane) { return __shfl_sync(kAll, v, lane); }
__device__ __forceinline__ float shfl_xor(float v, int o) { return __shfl_xor_sync(kAll, v, o); }
__device__ __forceinline__ bool greater(float a, float b) { return a > b; }
__device__ __forceinline__ bool open(float v) { return v > -INFINITY; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }

template <typename T>
__device__ __forceinline__ T of(float v) {
  if constexpr (sizeof(T) == 8) return T{v, 0.f};
  else return v;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = warp_max(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = warp_max(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = add(v, shfl_xor(v, o));
  return v;
}

// The logit of an expert: -infinity for a closed one, else finite.
__device__ __forceinline__ float clean(float l) {
  return l > -INFINITY ? fminf(l, FLT_MAX) + 0.f : -INFINITY;  // one zero
}

// PER neighbours of a row, as one vector where rows and pointer allow it.
template <int PER>
__device__ __forceinline__ void load_row(const RouteParams& P, int64_t row, uint32_t lane, float (&l)[PER]) {
  const int32_t e0 = static_cast<int32_t>(lane) * PER;
  const int64_t at = row * P.E + e0;
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = -INFINITY;
  if (P.vector) {
    if (e0 < P.E) {
      if (P.f32) {
        const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(P.logits) + at);
        if constexpr (PER >= 4) {
#pragma unroll
          for (int i = 0; i < PER / 4; ++i) {
            const float4 f = from[i];
            l[4 * i] = f.x, l[4 * i + 1] = f.y, l[4 * i + 2] = f.z, l[4 * i + 3] = f.w;
          }
        } else {
          const float2 f = *reinterpret_cast<const float2*>(from);
          l[0] = f.x, l[1] = f.y;
        }
      } else {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(P.logits) + at);
        uint32_t w[PER / 2];
        if constexpr (PER >= 8) {
#pragma unroll
          for (int i = 0; i < PER / 8; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(from)[i];
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
          }
        } else if constexpr (PER == 4) {
          const uint2 u = *reinterpret_cast<const uint2*>(from);
          w[0] = u.x, w[1] = u.y;
        } else {
          w[0] = *from;
        }
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) l[2 * i] = bf_lo(w[i]), l[2 * i + 1] = bf_hi(w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < P.E) l[i] = P.f32 ? static_cast<const float*>(P.logits)[at + i] : __bfloat162float(static_cast<const __nv_bfloat16*>(P.logits)[at + i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = clean(l[i]);
}

__device__ __forceinline__ float inverse(float x) { return rcp_approx(x); }  // of 1 .. infinity; 0 for what is below 2^-126

// What a softmax score is formed from: exp(l - top) * r.
struct Norm {
  float top, r;
};

// Scores of the row's experts; 0 of closed ones.
template <int PER>
__device__ __forceinline__ Norm scores(const RouteParams& P, const float (&l)[PER], float (&s)[PER]) {
  if (P.sigmoid) {  // exp(infinity) for a closed one: 0
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = inverse(1.f + expf(-l[i]));
    return {0.f, 1.f};
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = unordered(warp_max(ordered(top)));
  if (top == -INFINITY) top = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = expf(l[i] - top);
    sum += s[i];
  }
  sum = warp_sum(sum);
  const float r = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] *= r;
  return {top, r};
}

__device__ __forceinline__ float logit(const RouteParams& P, int64_t row, uint32_t e) {
  const int64_t at = row * P.E + e;
  return clean(P.f32 ? static_cast<const float*>(P.logits)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(P.logits)[at]));
}

// A lane's experts in falling order of v (ordered values), the lower expert
// first of equal ones: neighbours are exchanged where the second is larger.
template <int PER>
__device__ __forceinline__ void sort(uint32_t (&v)[PER], uint32_t (&at)[PER]) {
#pragma unroll
  for (int n = PER - 1; n > 0; --n)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool less = v[i] < v[i + 1];
      const uint32_t a = v[i], b = v[i + 1], c = at[i], d = at[i + 1];
      v[i] = less ? b : a;
      v[i + 1] = less ? a : b;
      at[i] = less ? d : c;
      at[i + 1] = less ? c : d;
    }
}

// The chosen experts, in order: choice j in lane j of `mine` (kNone: none).
// False if two of the values that the choice compares are within `band`
// (> 0; only with a bias) and do not tie exactly;
// lowest: the last of those.  v: ordered values, kShut or less where an expert cannot be chosen.
template <int PER>
__device__ __forceinline__ bool choose(const RouteParams& P, int64_t row, uint32_t (&v)[PER], float band, uint32_t lane, uint32_t& mine,
                                       float& lowest) {
  bool clear = true;
  mine = kNone;
  uint32_t at[PER], last = kNone;
  float before = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) at[i] = lane * PER + i;
  sort<PER>(v, at);
  const int32_t rounds = band > 0.f ? P.k + 1 : P.k;  // the first that is left out has to be told apart too
  for (int32_t j = 0; j < rounds; ++j) {
    const uint32_t top = warp_max(v[0]);
    if (top <= kShut) break;
    const uint32_t owner = __ffs(__ballot_sync(kAll, v[0] == top)) - 1, who = __shfl_sync(kAll, at[0], owner);
    if (static_cast<int32_t>(lane) == j) mine = who;
    const bool own = lane == owner;
#pragma unroll
    for (int i = 0; i + 1 < PER; ++i) {
      v[i] = own ? v[i + 1] : v[i];
      at[i] = own ? at[i + 1] : at[i];
    }
    if (own) v[PER - 1] = 0;
    if (band > 0.f) {
      const float val = unordered(top);
      if (j > 0 && before - val <= band * fmaxf(1.f, fabsf(val)) && !(P.bias[last] == P.bias[who] && logit(P, row, last) == logit(P, row, who)))
        clear = false;
      before = lowest = val;
      last = who;
    }
  }
  if (static_cast<int32_t>(lane) >= P.k) mine = kNone;
  return clear;
}

// Without a bias, the sum of the scores of a and b (-infinity: none) as
// e^m r, 1/2 <= r <= 2, which holds scores of any size.  Softmax, but for what
// all groups have in common: e^a (1 + e^(b - a)).  Sigmoid: of x it is
// e^min(x, 0) / (1 + e^-|x|).
struct LogSum {
  float m;
  Df r;
};
__device__ __forceinline__ bool open(const LogSum& v) { return v.m > -INFINITY; }
__device__ __forceinline__ LogSum shfl(const LogSum& v, int lane) { return {__shfl_sync(kAll, v.m, lane), shfl(v.r, lane)}; }
__device__ __forceinline__ Df exp_of_difference(float x, float y) {  // e^(x - y), x <= y
  return exp_df(x - y < -100.f ? Df{-100.f, 0.f} : two_sum(x, -y));
}
__device__ __forceinline__ bool greater(const LogSum& x, const LogSum& y) {
  if (!open(x) || !open(y)) return open(x) && !open(y);
  if (x.m >= y.m) return greater(x.r, mul(exp_of_difference(y.m, x.m), y.r));
  return greater(mul(exp_of_difference(x.m, y.m), x.r), y.r);
}
__device__ __noinline__ LogSum log_sum(bool sigmoid, float a, float b) {
  LogSum v = {sigmoid ? fminf(a, 0.f) : a, {1.f, 0.f}};
  if (!open(v)) return v;
  if (sigmoid) v.r = inverse(add(Df{1.f, 0.f}, exp_df(Df{-fminf(fabsf(a), 100.f), 0.f})));
  if (b > -INFINITY) {
    Df w = exp_of_difference(sigmoid ? fminf(b, 0.f) : b, v.m);
    if (sigmoid) w = mul(w, inverse(add(Df{1.f, 0.f}, exp_df(Df{-fminf(fabsf(b), 100.f), 0.f}))));
    v.r = add(v.r, w);
  }
  return v;
}

// Whether a lane's group is among the best; score: the group's, `lanes` lanes
// each.  near: one that is and one that is not are within what their scores may
// be off by, which goes by `size`, the largest magnitude that a group adds up (a
// sum near 1 of 64.5 and -63.5 has the roundings of those): for the half of a
// sum (score_of) half of two values' and the sum's roundings, which half of
// band_of() covers (sigmoid: 2 x 2.3 and 1/2 units, half of 5.1, against 3).
template <typename T>
__device__ __forceinline__ bool among_best(const RouteParams& P, T score, float size, int32_t group, int32_t lanes, float band, bool& near) {
  int32_t rank = 0;
#pragma unroll 1
  for (int32_t g = 0; g < P.groups; ++g) {
    const T other = shfl(score, g * lanes);
    if (greater(other, score) || (!greater(score, other) && g < group)) ++rank;
  }
  near = false;
  if constexpr (std::is_same_v<T, float>) {
    if (band > 0.f && P.tops < P.groups) {
      const bool real = group < P.groups, kept = rank < P.tops;
      const float off = 0.5f * band * fmaxf(1.f, size);
      const float least = unordered(~warp_max(real && kept ? ~ordered(score - off) : 0u)),
                  most = unordered(warp_max(real && !kept ? ordered(score + off) : 0u));
      near = most > -INFINITY && most >= least;
    }
  }
  return group < P.groups && rank < P.tops && open(score);
}

// The larger magnitude of what a group adds up: its largest value a and, where
// there is one, b.
__device__ __forceinline__ float size_of(const RouteParams& P, float a, float b) {
  return fmaxf(open(a) ? fabsf(a) : 0.f, P.best == 2 && open(b) ? fabsf(b) : 0.f);
}
__device__ __forceinline__ float size_of(const RouteParams&, Df, Df) { return 0.f; }  // exact: never near

// What a group is ranked by, with sums as their halves: two values of the type's
// lowest do not overflow, and halves are exact (but for values below 2^-125,
// which fp32 does not decide).
__device__ __forceinline__ float half_of(float v) { return 0.5f * v; }
__device__ __forceinline__ Df half_of(Df v) { return {0.5f * v.hi, 0.5f * v.lo}; }
template <typename S, typename T>
__device__ __forceinline__ S score_of(const RouteParams& P, T a, T b) {
  if constexpr (std::is_same_v<S, LogSum>) return log_sum(P.sigmoid, a, b);
  else return P.best == 1 ? a : open(b) ? add(half_of(a), half_of(b)) : half_of(a);
}

// Closes the experts (v: -infinity) of groups that are not among the best;
// false if that is within `band`.  S: what the groups are ranked by (LogSum: v
// are logits).
template <typename S, typename T, int PER>
__device__ __forceinline__ bool keep_groups(const RouteParams& P, T (&v)[PER], float band, uint32_t lane) {
  const T shut = of<T>(-INFINITY);
  const int32_t size = P.E / P.groups;
  bool near;
  if (P.group_lanes > 0) {  // a group is that many neighbouring lanes, a power of two
    T a = shut, b = shut;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b = larger(b, smaller(a, v[i]));
      a = larger(a, v[i]);
    }
    for (int o = 1; o < P.group_lanes; o <<= 1) {
      const T c = shfl_xor(a, o), d = shfl_xor(b, o);
      b = larger(smaller(a, c), larger(b, d));
      a = larger(a, c);
    }
    const S score = score_of<S>(P, a, b);
    if (!among_best<S>(P, score, size_of(P, a, b), static_cast<int32_t>(lane) / P.group_lanes, P.group_lanes, band, near)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = shut;
    }
    return !near;
  }
  S score = {};  // of group `lane`
  float size_here = 0.f;
  for (int32_t g = 0; g < P.groups; ++g) {
    T a = shut, b = shut;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int32_t e = static_cast<int32_t>(lane) * PER + i;
      if (e >= g * size && e < (g + 1) * size) {
        b = larger(b, smaller(a, v[i]));
        a = larger(a, v[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T c = shfl_xor(a, o), d = shfl_xor(b, o);
      b = larger(smaller(a, c), larger(b, d));
      a = larger(a, c);
    }
    if (static_cast<int32_t>(lane) == g) {
      score = score_of<S>(P, a, b);
      size_here = size_of(P, a, b);
    }
  }
  const uint32_t kept = __ballot_sync(kAll, among_best<S>(P, score, size_here, static_cast<int32_t>(lane), 1, band, near));
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int32_t e = static_cast<int32_t>(lane) * PER + i;
    if (e < P.E && !(kept >> (e / size) & 1u)) v[i] = shut;
  }
  return !near;
}

// The values that the choice goes by, from the scores.
template <typename T, int PER>
__device__ __forceinline__ void values(const RouteParams& P, const float (&l)[PER], const T (&s)[PER], uint32_t lane, T (&v)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int32_t e = static_cast<int32_t>(lane) * PER + i;
    v[i] = l[i] > -INFINITY ? (P.bias ? add(s[i], of<T>(P.bias[e])) : s[i]) : of<T>(-INFINITY);
  }
}

// Sigmoid: t = exp(-|l|), then 1 / (1 + t), or t times that.
__device__ __forceinline__ Df sigmoid_df(float l) {
  const Df t = exp_df(Df{-fminf(fabsf(l), 100.f), 0.f}), u = inverse(add(Df{1.f, 0.f}, t));
  return l >= 0.f ? u : mul(t, u);
}

// The values of the choice as pairs; -infinity where it cannot go.
template <int PER>
__device__ __forceinline__ void exact_values(const RouteParams& P, const float (&l)[PER], uint32_t lane, Df (&v)[PER]) {
  if (P.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = sigmoid_df(l[i]);
  } else {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
    top = unordered(warp_max(ordered(top)));
    if (top == -INFINITY) top = 0.f;
    Df sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = l[i] > -INFINITY ? exp_df(l[i] - top < -100.f ? Df{-100.f, 0.f} : two_sum(l[i], -top)) : Df{0.f, 0.f};
      sum = add(sum, v[i]);
    }
    sum = warp_sum(sum);
    const Df r = sum.hi > 0.f ? inverse(sum) : Df{0.f, 0.f};  // the largest score's exponential is 1
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = mul(v[i], r);
  }
  values<Df, PER>(P, l, v, lane, v);
  if (P.groups > 1) keep_groups<Df, Df, PER>(P, v, 0.f, lane);
}

// The choice by scores as pairs, for rows that need it.
template <int PER>
__device__ __noinline__ uint32_t choose_exactly(const RouteParams& P, int64_t row, uint32_t lane) {
  float l[PER];
  load_row<PER>(P, row, lane, l);
  Df v[PER];
  if (P.bias) {
    exact_values<PER>(P, l, lane, v);
  } else {  // groups by sums of two; what is left is told apart by its logits
    keep_groups<LogSum, float, PER>(P, l, 0.f, lane);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = Df{l[i], 0.f};
  }
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = open(v[i]) ? static_cast<uint64_t>(ordered(v[i].hi)) << 32 | ordered(v[i].lo + 0.f) : 0u;
  uint32_t mine = kNone;
  for (int32_t j = 0; j < P.k; ++j) {
    uint64_t best = 0;
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > best) {
        best = key[i];
        which = i;
      }
    const uint64_t most = warp_max(best);
    if (most == 0) break;
    const uint32_t owner = __ffs(__ballot_sync(kAll, best == most)) - 1;
    const uint32_t who = owner * PER + __shfl_sync(kAll, which, owner);
    if (static_cast<int32_t>(lane) == j) mine = who;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane == owner && static_cast<uint32_t>(i) == which) key[i] = 0;
  }
  return mine;
}

// The same where the groups are clear and a score is its logit's alone: only
// the experts from `least` on, one a lane.  `few`: a warp's memory.  kMany if
// there are more of them than lanes.
struct Few {
  uint32_t e[32];
  float l[32];
};
constexpr uint32_t kMany = 0xFFFFFFFEu;
template <int PER>
__device__ __noinline__ uint32_t choose_among_few(const RouteParams& P, int64_t row, float least, Few* few, uint32_t lane) {
  float l[PER], s[PER], v[PER];
  load_row<PER>(P, row, lane, l);
  scores<PER>(P, l, s);
  values<float, PER>(P, l, s, lane, v);
  if (P.groups > 1) keep_groups<float, float, PER>(P, v, 0.f, lane);
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool in = v[i] >= least;
    const uint32_t mask = __ballot_sync(kAll, in), at = n + __popc(mask & ((1u << lane) - 1));
    if (in && at < 32) {
      few->e[at] = lane * PER + i;
      few->l[at] = l[i];
    }
    n += __popc(mask);
  }
  if (n > 32) return kMany;
  __syncwarp();
  Df mine = {-INFINITY, 0.f};
  uint32_t e = kNone;
  if (lane < n) {
    e = few->e[lane];
    mine = add(sigmoid_df(few->l[lane]), Df{P.bias[e], 0.f});
  }
  uint32_t rank = 0;
  for (uint32_t i = 0; i < n; ++i) {
    const Df other = shfl(mine, i);
    const uint32_t oe = __shfl_sync(kAll, e, i);
    if (greater(other, mine) || (!greater(mine, other) && oe < e)) ++rank;
  }
  __syncwarp();
  if (lane < n) few->e[rank] = e;
  __syncwarp();
  const uint32_t out = lane < n && static_cast<int32_t>(lane) < P.k ? few->e[lane] : kNone;
  __syncwarp();
  return out;
}

// The chosen experts of a row, choice j in lane j, and what their scores are
// formed from.
template <int PER>
__device__ __forceinline__ uint32_t select(const RouteParams& P, int64_t row, Few* few, uint32_t lane, Norm& norm) {
  float l[PER], s[PER];
  load_row<PER>(P, row, lane, l);
  const bool by_logit = P.bias == nullptr && (P.groups == 1 || P.best == 1);  // both scores grow with it
  if (!by_logit || !P.sigmoid) norm = scores<PER>(P, l, s);
  uint32_t key[PER], mine;
  float lowest = 0.f;
  if (by_logit) {
    if (P.groups > 1) keep_groups<float, float, PER>(P, l, 0.f, lane);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = ordered(l[i]);
    choose<PER>(P, row, key, 0.f, lane, mine, lowest);
    return mine;
  }
  const float band = band_of(PER, P.sigmoid);
  float v[PER];
  values<float, PER>(P, l, s, lane, v);
  const bool clear = P.groups == 1 || keep_groups<float, float, PER>(P, v, band, lane);
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = open(v[i]) ? ordered(P.bias ? v[i] : l[i]) : 0u;
  if (clear) {
    if (choose<PER>(P, row, key, P.bias ? band : 0.f, lane, mine, lowest)) return mine;
    if (P.sigmoid) {
      mine = choose_among_few<PER>(P, row, lowest - 2.f * band * fmaxf(1.f, fabsf(lowest)), few, lane);
      if (mine != kMany) return mine;
    }
  }
  return choose_exactly<PER>(P, row, lane);
}

// The value of expert e, another one for each lane; 0 for none.
template <int PER>
__device__ __forceinline__ float pick(const float (&s)[PER], uint32_t e) {
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float o = __shfl_sync(kAll, s[i], (e / PER) & 31);
    if (e != kNone && e % PER == i) v = o;
  }
  return v;
}

template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_fwd_kernel(const __grid_constant__ RouteParams P) {
  __shared__ Few few[kWarps];
  __shared__ int32_t hist[kMaxExperts];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  const bool count = P.counts && gridDim.x == 1;  // of several blocks' rows: route_count_kernel
  if (count) {
    for (int32_t e = threadIdx.x; e < P.E; e += kWarps * 32) hist[e] = 0;
    __syncthreads();
  } else if (P.counts && blockIdx.x == 0) {
    for (int32_t e = threadIdx.x; e < P.E; e += kWarps * 32) P.counts[e] = 0;
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < P.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    Norm norm;
    const uint32_t mine = select<PER>(P, row, few + (threadIdx.x >> 5), lane, norm);
    float sc = 0.f;
    if (mine != kNone) {
      const float l = logit(P, row, mine);
      if (P.sigmoid) {  // below 2^-126 too: their shares of a sum need not be small
        const float t = expf(-fabsf(l)), u = inverse(1.f + t);
        sc = l >= 0.f ? u : t * u;
      } else {
        sc = expf(l - norm.top) * norm.r;
      }
    }
    const float total = P.renorm ? fmaxf(warp_sum(sc), FLT_MIN) : 1.f;
    if (static_cast<int32_t>(lane) < P.k) {
      P.experts[row * P.k + lane] = mine == kNone ? -1 : static_cast<int32_t>(mine);
      P.weights[row * P.k + lane] = P.scale * (sc / total);
      if (count && mine != kNone) atomicAdd(hist + mine, 1);
    }
  }
  if (count) {
    __syncthreads();
    for (int32_t e = threadIdx.x; e < P.E; e += kWarps * 32) P.counts[e] = hist[e];
  }
}

// How often each expert was chosen, where several thread blocks had the rows
// (which left zeros): some thousands of slots a block, so that the atomics on
// the same few counters are few.  Whole numbers: their sum has no order.
constexpr int kCountThreads = 512;
__global__ void __launch_bounds__(kCountThreads) route_count_kernel(const __grid_constant__ RouteParams P) {
  __shared__ int32_t hist[kMaxExperts];
  griddep_wait();
  griddep_launch_dependents();
  for (int32_t e = threadIdx.x; e < P.E; e += kCountThreads) hist[e] = 0;
  __syncthreads();
  const int64_t slots = P.T * P.k;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCountThreads + threadIdx.x; i < slots; i += static_cast<int64_t>(gridDim.x) * kCountThreads) {
    const int32_t e = __ldcg(P.experts + i);
    if (e >= 0) atomicAdd(hist + e, 1);
  }
  __syncthreads();
  for (int32_t e = threadIdx.x; e < P.E; e += kCountThreads)
    if (hist[e]) atomicAdd(P.counts + e, hist[e]);
}

// A lane's choice of a row (kNone: none) and scale * the gradient of its weight.
__device__ __forceinline__ float chosen(const RouteParams& P, int64_t row, uint32_t lane, uint32_t& mine) {
  mine = kNone;
  if (static_cast<int32_t>(lane) >= P.k) return 0.f;
  const int32_t e = P.experts[row * P.k + lane];
  if (e < 0 || e >= P.E) return 0.f;
  mine = static_cast<uint32_t>(e);
  return P.scale * P.dweights[row * P.k + lane];
}

// w = s / sum s depends on the chosen logits alone: the gradient of a logit is
// (ds/dl / total) (g - sum_j w_j g_j), and the bracket sum_j w_j (g - g_j),
// which keeps its digits where one w is nearly 1 and is 0 for a single choice.
// slope, ds/dl, is at most s, so that slope / total is at most 1.  (A total
// below the range is a constant: the weights do not add up to 1 then.)
__device__ __forceinline__ float through_sum(const RouteParams& P, float g, float sc, float slope) {
  const float sum = warp_sum(sc), total = fmaxf(sum, FLT_MIN), w = __fdiv_rn(sc, total);
  float rest = 0.f;
  for (int32_t j = 0; j < P.k; ++j) rest = fmaf(__shfl_sync(kAll, w, j), g - __shfl_sync(kAll, g, j), rest);
  return (sum < FLT_MIN ? g : rest) * __fdiv_rn(slope, total);
}

// A number that comes more than once: its first choice gets the sum of their
// gradients, the others none.
__device__ __forceinline__ void add_repeated(const RouteParams& P, uint32_t lane, float& g, uint32_t& mine) {
  const uint32_t same = __match_any_sync(kAll, mine);
  if (!__any_sync(kAll, mine != kNone && (same & (same - 1)) != 0)) return;
  float sum = 0.f;
  for (int32_t j = 0; j < P.k; ++j) {
    const float v = __shfl_sync(kAll, g, j);
    if (same >> j & 1) sum += v;
  }
  const bool first = mine != kNone && static_cast<int32_t>(lane) == __ffs(same) - 1;
  g = first ? sum : 0.f;
  mine = first ? mine : kNone;
}

// Softmax: the gradient of a chosen logit, s (g - sum_j s_j g_j).  As the scores
// add up to 1 the bracket is g times the others' scores and
// sum_j s_j (g - g_j), which keeps its digits where one score is nearly 1.
// Numbers are there once; in: the lane's experts among them, dot: sum_j s_j g_j.
template <int PER>
__device__ __forceinline__ float through_softmax(const RouteParams& P, const float (&s)[PER], float g, uint32_t mine, uint32_t lane,
                                                 uint32_t& in, float& dot) {
  in = 0;
  for (int32_t j = 0; j < P.k; ++j) {
    const uint32_t e = __shfl_sync(kAll, mine, j);
    if (e / PER == lane) in |= 1u << e % PER;
  }
  float others = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) others += in >> i & 1 ? 0.f : s[i];
  const float sc = pick<PER>(s, mine);
  float rest = g * warp_sum(others);
  dot = warp_sum(sc * g);
  for (int32_t j = 0; j < P.k; ++j) rest = fmaf(__shfl_sync(kAll, sc, j), g - __shfl_sync(kAll, g, j), rest);
  return sc * rest;
}

// Sigmoid: only the chosen logits have a gradient, s (1 - s) without the
// difference, and only they are read; the row is zeros but for them.  (By whole
// rows, as for the softmax, 8192 x 256 took 7.1 us, so 4.5.)
__global__ void __launch_bounds__(kWarps * 32) route_bwd_sigmoid_kernel(const __grid_constant__ RouteParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < P.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t at = row * P.E;
    uint32_t mine;
    float g = chosen(P, row, lane, mine), x = -INFINITY;
    if (mine != kNone) x = P.f32 ? static_cast<const float*>(P.logits)[at + mine] : __bfloat162float(static_cast<const __nv_bfloat16*>(P.logits)[at + mine]);
    if (P.vector) {
      const int32_t n = P.E * (P.f32 ? 4 : 2) / 16;
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(P.dlogits) + at * (P.f32 ? 4 : 2));
      for (int32_t i = static_cast<int32_t>(lane); i < n; i += 32) to[i] = make_uint4(0, 0, 0, 0);
    } else {
      for (int32_t i = static_cast<int32_t>(lane); i < P.E; i += 32) {
        if (P.f32) static_cast<float*>(P.dlogits)[at + i] = 0.f;
        else static_cast<__nv_bfloat16*>(P.dlogits)[at + i] = __float2bfloat16_rn(0.f);
      }
    }
    const float t = expf(-fabsf(x)), u = inverse(1.f + t);
    const bool open = x > -INFINITY;  // and not NaN
    const float sc = open ? (x >= 0.f ? u : t * u) : 0.f, slope = open ? t * u * u : 0.f;
    g = P.renorm ? through_sum(P, g, sc, slope) : g * slope;
    add_repeated(P, lane, g, mine);
    __syncwarp();  // the zeros come first
    if (mine != kNone) {
      if (P.f32) static_cast<float*>(P.dlogits)[at + mine] = g;
      else static_cast<__nv_bfloat16*>(P.dlogits)[at + mine] = __float2bfloat16_rn(g);
    }
  }
}

// Softmax.
template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const __grid_constant__ RouteParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < P.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[PER], s[PER];
    load_row<PER>(P, row, lane, l);
    uint32_t mine;
    float g = chosen(P, row, lane, mine);
    scores<PER>(P, l, s);
    uint32_t in = 0;  // the lane's experts that are chosen
    float dot = 0.f;
    if (P.renorm) {
      const float sc = pick<PER>(s, mine);
      g = through_sum(P, g, sc, sc);
    } else {
      add_repeated(P, lane, g, mine);
      g = through_softmax<PER>(P, s, g, mine, lane, in, dot);
    }
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = 0.f;
    for (int32_t j = 0; j < P.k; ++j) {
      const uint32_t e = __shfl_sync(kAll, mine, j);
      const float v = __shfl_sync(kAll, g, j);
      if (e / PER == lane) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (e % PER == i) d[i] += v;
      }
    }
    if (!P.renorm) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (!(in >> i & 1)) d[i] = -s[i] * dot;
    }
    const int32_t e0 = static_cast<int32_t>(lane) * PER;
    const int64_t at = row * P.E + e0;
    if (P.vector) {
      if (e0 < P.E) {
        uint32_t w[PER];
        const int n = P.f32 ? PER : PER / 2;
#pragma unroll
        for (int i = 0; i < PER; ++i) w[i] = P.f32 ? __float_as_uint(d[i]) : 2 * i < PER ? pack_bf16(d[(2 * i) % PER], d[(2 * i + 1) % PER]) : 0u;
        uint32_t* to = P.f32 ? reinterpret_cast<uint32_t*>(static_cast<float*>(P.dlogits) + at)
                             : reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(P.dlogits) + at);
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          if (PER >= 4 && i + 4 <= n) *reinterpret_cast<uint4*>(to + i) = make_uint4(w[i], w[(i + 1) % PER], w[(i + 2) % PER], w[(i + 3) % PER]);
          else if (i + 2 <= n) *reinterpret_cast<uint2*>(to + i) = make_uint2(w[i], w[(i + 1) % PER]);
          else if (i < n) to[i] = w[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (e0 + i >= P.E) continue;
        if (P.f32) static_cast<float*>(P.dlogits)[at + i] = d[i];
        else static_cast<__nv_bfloat16*>(P.dlogits)[at + i] = __float2bfloat16_rn(d[i]);
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
tp_status run(bool fwd, RouteParams& P, cudaStream_t stream) {
  const size_t size = (P.f32 ? 4 : 2) * PER;
  P.vector = P.E % PER == 0 && reinterpret_cast<uintptr_t>(P.logits) % std::min<size_t>(size, 16) == 0 &&
             reinterpret_cast<uintptr_t>(P.dlogits) % std::min<size_t>(size, 16) == 0;
  const int32_t each = P.E / P.groups, lanes = each / PER;
  P.group_lanes = each % PER == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  return fwd ? launch_dependent(route_fwd_kernel<PER>, dim3(grid_of(P.T)), kWarps * 32, 0, stream, P)
             : launch_dependent(route_bwd_kernel<PER>, dim3(grid_of(P.T)), kWarps * 32, 0, stream, P);
}

tp_status run(bool fwd, RouteParams& P, cudaStream_t stream) {
  if (!fwd && P.sigmoid) {
    P.vector = P.E * (P.f32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(P.dlogits) % 16 == 0;
    return launch_dependent(route_bwd_sigmoid_kernel, dim3(grid_of(P.T)), kWarps * 32, 0, stream, P);
  }
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
  const bool one = work && grid_of(T) == 1;
  if (!work) return launch_dependent(route_fwd_kernel<2>, dim3(1), kWarps * 32, 0, stream, P);  // counts of no row
  TP_TRY(run(true, P, stream));
  if (counts == nullptr || one) return TP_OK;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(cdiv(T * k, 2 * kCountThreads), 152));
  return launch_dependent(route_count_kernel, dim3(blocks), kCountThreads, 0, stream, P);
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
