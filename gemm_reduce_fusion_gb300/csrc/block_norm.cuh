// Kernels of the block boundary: y = x + alpha * gate * N_post(z),
// n = N_pre(y), and their gradients.
//
// Both are bound by HBM: the forward pass moves 8 bytes an element (two
// tensors in, two out, bf16), the backward pass 12.  A row is owned by one
// worker, a warp (rows up to 1024) or a CTA, whose threads hold it in
// registers, so that every tensor is read once and written once whatever the
// statistics need.  Loads run ahead of the arithmetic through a ring in
// shared memory that each thread fills (cp.async) and empties by itself: no
// barrier and no wait between threads guards it.  A thread owns the same
// columns in all its rows, which keeps the backward pass's column sums (the
// gradients of weights, biases and gate) in registers over the whole launch.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "vec_util.cuh"

namespace tpf {

enum NormKind : int32_t { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

struct NormParams {
  // row shards: m = M / p rows each
  const void* x[8];     // fwd: residual stream; bwd: y, the stream after the boundary
  const void* z[8];     // block output, or null
  const void* dn[8];    // bwd: gradient of n, or null
  const void* dy[8];    // bwd: gradient of y from later uses, or null
  void* y[8];           // fwd: y; bwd: dx (nullable)
  void* n[8];           // fwd: n; bwd: dz (nullable)
  const uint4* gate;    // [M / rows_per_gate, h], or null
  const uint4* w_post;
  const uint4* b_post;
  const uint4* w_pre;
  const uint4* b_pre;
  float* part;          // bwd: [4][CTAs][h] column sums of each CTA
  float* gpart;         // bwd: [2][workers][h] gate sums of groups that several workers share
  void* dgate;          // bwd: gate gradient where the kernel writes whole groups
  float alpha, eps, inv_h;
  uint32_t M, m, nvec, rows_per_gate, stages;
  int32_t post, pre;
  int32_t has_z, has_dn, has_dy, out_f32;
};

// Sums over the worker's threads, left in every thread.  `red` is shared
// memory of two buffers of N * 32 floats that take turns: a buffer is written
// again only after the barrier of the reduction in between, which every
// thread passes after its reads.
template <int N, bool WARP>
__device__ __forceinline__ void worker_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if constexpr (!WARP) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float* b = red + turn * (12 * 32);
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? b[i * 32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  }
}

// One vector (8 columns) of a bf16 or fp32 row held as raw registers.
template <bool F32>
struct Raw {
  uint4 a;
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(a, v); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
};
template <>
struct Raw<true> {
  uint4 a, b;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = __uint_as_float(a.x);
    v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z);
    v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x);
    v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z);
    v[7] = __uint_as_float(b.w);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
};

template <bool F32>
__device__ __forceinline__ void store_row(void* row, uint32_t v, const float (&f)[8]) {
  if constexpr (F32) {
    uint4* d = static_cast<uint4*>(row) + 2 * v;
    st_global_cs(d, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    st_global_cs(d + 1,
                 make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  } else {
    st_global_cs(static_cast<uint4*>(row) + v, pack8(f));
  }
}

// Row `r` of a tensor of p shards with m rows each; bytes: of one row.
__device__ __forceinline__ const char* shard_row(const void* const (&t)[8], uint32_t r, uint32_t m, int64_t bytes) {
  const uint32_t s = r / m;
  return static_cast<const char*>(t[s]) + static_cast<int64_t>(r - s * m) * bytes;
}
__device__ __forceinline__ char* shard_row(void* const (&t)[8], uint32_t r, uint32_t m, int64_t bytes) {
  const uint32_t s = r / m;
  return static_cast<char*>(t[s]) + static_cast<int64_t>(r - s * m) * bytes;
}

template <bool WARP>
struct Worker {
  uint32_t T, t, id, count;  // threads, this thread, worker, workers in the grid
  __device__ Worker() {
    T = WARP ? 32u : blockDim.x;
    t = WARP ? (threadIdx.x & 31u) : threadIdx.x;
    id = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    count = WARP ? gridDim.x * (blockDim.x >> 5) : gridDim.x;
  }
};

// ----------------------------------------------------------------- forward

// NV vectors of 8 columns per thread; RES32: the residual stream is fp32.
template <int NV, bool RES32, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_fwd_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2 * 12 * 32];
  griddep_wait();
  griddep_launch_dependents();
  const Worker<WARP> W;
  const uint32_t nvec = P.nvec;
  const int64_t row16 = static_cast<int64_t>(nvec) * 16, rowx = RES32 ? 2 * row16 : row16;
  // slot of vector k, part j (x: 1 or 2, z: 1) of stage s: one 16-byte cell
  // per thread, consecutive threads in consecutive cells
  constexpr int PX = RES32 ? 2 : 1, PARTS = PX + 1;
  const uint32_t cell = smem_u32(ring) + threadIdx.x * 16, step = blockDim.x * 16;
  auto slot = [&](uint32_t s, int k, int j) { return cell + ((s * NV + k) * PARTS + j) * step; };
  auto fetch = [&](uint32_t row, uint32_t s) {
    if (row < P.M) {
      const char* x = shard_row(P.x, row, P.m, rowx);
      const char* z = P.has_z ? shard_row(P.z, row, P.m, row16) : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (v < nvec) {
#pragma unroll
          for (int j = 0; j < PX; ++j) cp_async16(slot(s, k, j), x + (static_cast<int64_t>(v) * PX + j) * 16);
          if (P.has_z) cp_async16(slot(s, k, PX), z + static_cast<int64_t>(v) * 16);
        }
      }
    }
    cp_async_commit();
  };
  // one or two stages: the next row, or the next two, are on their way while
  // a row is worked on
  fetch(W.id, 0);
  if (P.stages == 2) fetch(W.id + W.count, 1);
  uint32_t s = 0;
  int turn = 0;
  for (uint32_t row = W.id; row < P.M; row += W.count) {
    if (P.stages == 2) cp_async_wait<1>();
    else cp_async_wait<0>();
    float y[NV][8];
    float z[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Raw<RES32> rx;
      uint4 rz = make_uint4(0, 0, 0, 0);
      rx.zero();
      if (k * W.T + W.t < nvec) {
        rx.a = ld_shared_v4(slot(s, k, 0));
        if constexpr (RES32) rx.b = ld_shared_v4(slot(s, k, 1));
        if (P.has_z) rz = ld_shared_v4(slot(s, k, PX));
      }
      rx.get(y[k]);
      unpack8(rz, z[k]);
    }
    if (P.has_z) {
      float mu = 0.f, r = 1.f;
      if (P.post == NORM_LAYER) {
        float a[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[0] += z[k][i];
        worker_sum<1, WARP>(a, red, turn);
        mu = a[0] * P.inv_h;
      }
      if (P.post != NORM_NONE) {
        float a[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (k * W.T + W.t < nvec) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float d = z[k][i] - mu;
              a[0] = fmaf(d, d, a[0]);
            }
          }
        worker_sum<1, WARP>(a, red, turn);
        r = 1.f / sqrtf(fmaf(a[0], P.inv_h, P.eps));
      }
      const uint4* gate = P.gate ? P.gate + static_cast<int64_t>(row / P.rows_per_gate) * nvec : nullptr;
      char* yo = shard_row(P.y, row, P.m, rowx);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (v < nvec) {
          float o[8], c[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = (z[k][i] - mu) * r;
          if (P.w_post) {
            unpack8(__ldg(P.w_post + v), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= c[i];
          }
          if (P.b_post) {
            unpack8(__ldg(P.b_post + v), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += c[i];
          }
          if (gate) {
            unpack8(__ldg(gate + v), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= c[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) y[k][i] = fmaf(P.alpha, o[i], y[k][i]);
          store_row<RES32>(yo, v, y[k]);
        }
      }
    }
    if (P.pre != NORM_NONE) {
      float mu = 0.f;
      if (P.pre == NORM_LAYER) {
        float a[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[0] += y[k][i];
        worker_sum<1, WARP>(a, red, turn);
        mu = a[0] * P.inv_h;
      }
      float a[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (k * W.T + W.t < nvec) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float d = y[k][i] - mu;
            a[0] = fmaf(d, d, a[0]);
          }
        }
      worker_sum<1, WARP>(a, red, turn);
      const float r = 1.f / sqrtf(fmaf(a[0], P.inv_h, P.eps));
      char* no = shard_row(P.n, row, P.m, row16);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (v < nvec) {
          float o[8], c[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = (y[k][i] - mu) * r;
          if (P.w_pre) {
            unpack8(__ldg(P.w_pre + v), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= c[i];
          }
          if (P.b_pre) {
            unpack8(__ldg(P.b_pre + v), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += c[i];
          }
          store_row<false>(no, v, o);
        }
      }
    }
    // the values of this stage have been used above, so its cells are free
    fetch(row + P.stages * W.count, s);
    if (P.stages == 2) s ^= 1;
  }
  cp_async_wait<0>();
}

// ----------------------------------------------------------------- backward

// The row's sums after the means (s2 and s7..s11 only with a layer norm; yc,
// zc are centred values, d = dn * w_pre, q = gate * w_post):
//   s0 yc^2  s1 d yc  s2 d  s3 zc^2  s4 q zc dy  s5 q zc d  s6 q zc yc
//   s7 q zc  s8 q dy  s9 q d  s10 q yc  s11 q
// With ry = 1/sqrt(s0/h + eps), m1 = s2/h, m2 = ry s1/h:
//   dx = dy + ry (d - m1 - ry m2 yc),  u = alpha q dx,
//   sum u zhat = alpha rz (s4 + ry (s5 - m1 s7 - ry m2 s6)),
//   sum u      = alpha    (s8 + ry (s9 - m1 s11 - ry m2 s10)),
//   dz = rz (u - mean u - zhat mean(u zhat)):
// the sums of the post norm's gradient are linear in dx, so that both norms
// are served by one reduction (a second one, before it, gives a layer norm
// its means).  The worker owns rows [id M / count, (id + 1) M / count).
//
// GROUPS: the gate has more than one row; its sums are kept apart from the
// weights' and given out whenever the group ends.  With one gate row or none,
// t = alpha dx is summed as A = sum t zhat, B = sum t alone, and the last
// kernel forms dw_post = g A, db_post = g B, dgate = w A + b B.
template <int NV, bool RES32, bool LN, bool GROUPS, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_bwd_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2 * 12 * 32];
  griddep_wait();
  griddep_launch_dependents();
  const Worker<WARP> W;
  const uint32_t nvec = P.nvec, h = nvec * 8;
  const int64_t row16 = static_cast<int64_t>(nvec) * 16, rowx = RES32 ? 2 * row16 : row16;
  constexpr int PX = RES32 ? 2 : 1, PARTS = 2 * PX + 2;  // y, dy, dn, z
  const uint32_t cell = smem_u32(ring) + threadIdx.x * 16, step = blockDim.x * 16;
  auto slot = [&](uint32_t s, int k, int j) { return cell + ((s * NV + k) * PARTS + j) * step; };
  const uint32_t r0 = static_cast<uint32_t>(static_cast<uint64_t>(W.id) * P.M / W.count);
  const uint32_t r1 = static_cast<uint32_t>(static_cast<uint64_t>(W.id + 1) * P.M / W.count);
  auto fetch = [&](uint32_t row, uint32_t s) {
    if (row < r1) {
      const char* y = shard_row(P.x, row, P.m, rowx);
      const char* dy = P.has_dy ? shard_row(P.dy, row, P.m, rowx) : nullptr;
      const char* dn = P.has_dn ? shard_row(P.dn, row, P.m, row16) : nullptr;
      const char* z = P.has_z ? shard_row(P.z, row, P.m, row16) : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int64_t v = k * W.T + W.t;
        if (v < nvec) {
#pragma unroll
          for (int j = 0; j < PX; ++j) {
            if (P.has_dn) cp_async16(slot(s, k, j), y + (v * PX + j) * 16);
            if (P.has_dy) cp_async16(slot(s, k, PX + j), dy + (v * PX + j) * 16);
          }
          if (P.has_dn) cp_async16(slot(s, k, 2 * PX), dn + v * 16);
          if (P.has_z) cp_async16(slot(s, k, 2 * PX + 1), z + v * 16);
        }
      }
    }
    cp_async_commit();
  };
  fetch(r0, 0);
  if (P.stages == 2) fetch(r0 + 1, 1);

  float accA[NV][8] = {}, accC[NV][8] = {};
  float accB[LN ? NV : 1][8] = {}, accD[LN ? NV : 1][8] = {}, accE[GROUPS ? NV : 1][8] = {};
  uint32_t s = 0;
  int turn = 0;
  for (uint32_t row = r0; row < r1; ++row) {
    if (P.stages == 2) cp_async_wait<1>();
    else cp_async_wait<0>();
    Raw<RES32> ry_[NV], rdy[NV];
    uint4 rdn[NV], rz_[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      ry_[k].zero();
      rdy[k].zero();
      rdn[k] = rz_[k] = make_uint4(0, 0, 0, 0);
      if (k * W.T + W.t < nvec) {
        if (P.has_dn) {
          ry_[k].a = ld_shared_v4(slot(s, k, 0));
          if constexpr (RES32) ry_[k].b = ld_shared_v4(slot(s, k, 1));
          rdn[k] = ld_shared_v4(slot(s, k, 2 * PX));
        }
        if (P.has_dy) {
          rdy[k].a = ld_shared_v4(slot(s, k, PX));
          if constexpr (RES32) rdy[k].b = ld_shared_v4(slot(s, k, PX + 1));
        }
        if (P.has_z) rz_[k] = ld_shared_v4(slot(s, k, 2 * PX + 1));
      }
    }
    float mu_y = 0.f, mu_z = 0.f;
    if constexpr (LN) {
      float a[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float y[8], z[8];
        ry_[k].get(y);
        unpack8(rz_[k], z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[0] += y[i];
          a[1] += z[i];
        }
      }
      worker_sum<2, WARP>(a, red, turn);
      if (P.pre == NORM_LAYER) mu_y = a[0] * P.inv_h;
      if (P.post == NORM_LAYER) mu_z = a[1] * P.inv_h;
    }
    const uint32_t group = GROUPS ? row / P.rows_per_gate : 0;
    const uint4* gate = P.gate ? P.gate + static_cast<int64_t>(group) * nvec : nullptr;
    constexpr int NS = LN ? 12 : 6;
    float sum[NS] = {};
    // indices of the six sums of the plain case, and of the others
    constexpr int Y2 = 0, DY = 1, Z2 = 2, QZG = 3, QZD = 4, QZY = 5, D1 = 6, QZ = 7, QG = 8, QD = 9, QY = 10, Q1 = 11;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t v = k * W.T + W.t;
      if (v < nvec) {
        float y[8], z[8], d[8], g[8], q[8], c[8];
        ry_[k].get(y);
        rdy[k].get(g);
        unpack8(rdn[k], d);
        unpack8(rz_[k], z);
        if (P.w_pre) {
          unpack8(__ldg(P.w_pre + v), c);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= c[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = 1.f;
        if (P.w_post) unpack8(__ldg(P.w_post + v), q);
        if (gate) {
          unpack8(__ldg(gate + v), c);
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] *= c[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yc = LN ? y[i] - mu_y : y[i], zc = LN ? z[i] - mu_z : z[i], qz = q[i] * zc;
          sum[Y2] = fmaf(yc, yc, sum[Y2]);
          sum[DY] = fmaf(d[i], yc, sum[DY]);
          sum[Z2] = fmaf(zc, zc, sum[Z2]);
          sum[QZG] = fmaf(qz, g[i], sum[QZG]);
          sum[QZD] = fmaf(qz, d[i], sum[QZD]);
          sum[QZY] = fmaf(qz, yc, sum[QZY]);
          if constexpr (LN) {
            sum[D1] += d[i];
            sum[QZ] += qz;
            sum[QG] = fmaf(q[i], g[i], sum[QG]);
            sum[QD] = fmaf(q[i], d[i], sum[QD]);
            sum[QY] = fmaf(q[i], yc, sum[QY]);
            sum[Q1] += q[i];
          }
        }
      }
    }
    worker_sum<NS, WARP>(sum, red, turn);
    // the raw registers of this row are loaded: its cells are free
    fetch(row + P.stages, s);
    if (P.stages == 2) s ^= 1;

    const float ry = P.has_dn ? 1.f / sqrtf(fmaf(sum[Y2], P.inv_h, P.eps)) : 0.f;
    const float m2 = ry * ry * sum[DY] * P.inv_h;  // times yc
    float m1 = 0.f;
    if constexpr (LN) m1 = P.pre == NORM_LAYER ? sum[D1] * P.inv_h : 0.f;
    float rz = 1.f, u1 = 0.f, u2 = 0.f;
    if (P.post != NORM_NONE) {
      rz = 1.f / sqrtf(fmaf(sum[Z2], P.inv_h, P.eps));
      float t = sum[QZG] + ry * (sum[QZD] - m2 * sum[QZY]);
      if constexpr (LN) {
        t -= ry * m1 * sum[QZ];
        if (P.post == NORM_LAYER)
          u1 = P.alpha * P.inv_h * (sum[QG] + ry * (sum[QD] - m1 * sum[Q1] - m2 * sum[QY]));
      }
      u2 = P.alpha * P.inv_h * rz * t;
    }
    char* dxo = P.y[0] ? shard_row(P.y, row, P.m, rowx) : nullptr;
    char* dzo = P.n[0] ? shard_row(P.n, row, P.m, row16) : nullptr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t v = k * W.T + W.t;
      if (v < nvec) {
        float y[8], dx[8], d[8], c[8];
        ry_[k].get(y);
        rdy[k].get(dx);
        unpack8(rdn[k], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = 1.f;
        if (P.w_pre) unpack8(__ldg(P.w_pre + v), c);
        if (P.has_dn) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float yc = LN ? y[i] - mu_y : y[i];
            accC[k][i] = fmaf(d[i] * ry, yc, accC[k][i]);
            if constexpr (LN) accD[k][i] += d[i];
            dx[i] = fmaf(ry, fmaf(d[i], c[i], -m1) - m2 * yc, dx[i]);
          }
        }
        if (dxo) store_row<RES32>(dxo, v, dx);
        if (P.has_z) {
          float z[8], g[8], w[8];
          unpack8(rz_[k], z);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = g[i] = 1.f;
          if (P.w_post) unpack8(__ldg(P.w_post + v), w);
          if (gate) unpack8(__ldg(gate + v), g);
          if constexpr (GROUPS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = 0.f;
            if (P.b_post) unpack8(__ldg(P.b_post + v), c);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float zh = (LN ? z[i] - mu_z : z[i]) * rz, t = P.alpha * dx[i], tg = t * g[i];
            const float acc = GROUPS ? tg : t;
            accA[k][i] = fmaf(acc, zh, accA[k][i]);
            if constexpr (LN) accB[k][i] += acc;
            if constexpr (GROUPS) accE[k][i] = fmaf(t, fmaf(zh, w[i], c[i]), accE[k][i]);
            z[i] = rz * (fmaf(tg, w[i], -u1) - zh * u2);
          }
          if (dzo) store_row<false>(dzo, v, z);
        }
      }
    }
    if constexpr (GROUPS) {
      if (row + 1 == r1 || (row + 1) / P.rows_per_gate != group) {
        // the group ends here, or goes on in the next worker's rows
        const uint64_t g0 = static_cast<uint64_t>(group) * P.rows_per_gate;
        const bool whole = g0 >= r0 && g0 + P.rows_per_gate <= r1;
        float* gp = P.gpart + (static_cast<int64_t>(g0 > r0 ? 1 : 0) * W.count + W.id) * h;
        if (P.gpart) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            const uint32_t v = k * W.T + W.t;
            if (v < nvec) {
              if (!whole) store_row<true>(gp, v, accE[k]);
              else if (P.out_f32) store_row<true>(static_cast<float*>(P.dgate) + static_cast<int64_t>(group) * h, v, accE[k]);
              else store_row<false>(static_cast<__nv_bfloat16*>(P.dgate) + static_cast<int64_t>(group) * h, v, accE[k]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) accE[k][i] = 0.f;
      }
    }
  }
  cp_async_wait<0>();

  // column sums of the CTA: warps that are workers of their own are added in
  // warp order through shared memory (the ring is no longer in use)
  auto give = [&](float (&acc)[NV][8], int which) {
    float* out = P.part + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * h;
    if constexpr (!WARP) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (v < nvec) store_row<true>(out, v, acc[k]);
      }
    } else {
      float* all = reinterpret_cast<float*>(ring);
      const uint32_t warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * 32 + W.t;
        if (v < nvec) {
#pragma unroll
          for (int i = 0; i < 8; ++i) all[(warp * 8 + i) * (NV * 32) + v] = acc[k][i];
        }
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < h; c += blockDim.x) {
        const uint32_t v = c >> 3, i = c & 7;
        float t = 0.f;
        for (uint32_t w = 0; w < warps; ++w) t += all[(w * 8 + i) * (NV * 32) + v];
        out[c] = t;
      }
    }
  };
  if (P.has_dn && P.part) give(accC, 0);
  if (P.has_z && P.part) give(accA, 1);
  if constexpr (LN) {
    if (P.has_dn && P.part) give(accD, 2);
    if (P.has_z && P.part) give(accB, 3);
  }
}

}  // namespace tpf
