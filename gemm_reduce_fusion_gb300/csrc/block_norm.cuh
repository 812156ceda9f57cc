// Kernels of the block boundary: y = x + alpha * gate * N_post(z),
// n = N_pre(y), and their gradients.
//
// Both are bound by HBM: the forward pass moves 8 bytes an element (two
// tensors in, two out, bf16), the backward pass 12.  At HBM's rate an SM has
// about 43 and 65 issue cycles for an element of each, so that the kernels
// are written for few instructions: fp32 arithmetic on packed pairs, vectors
// that all rows share (weights, a gate per channel) multiplied out once and
// kept as fp32 in shared memory, several vectors of 8 columns a thread to
// spread a row's reductions and addresses over many elements.
//
// A row is owned by one worker, so that every tensor is read once and written
// once whatever the statistics need: a warp (rows up to 1024 columns), a CTA,
// or, in the backward pass above 4096 columns, a cluster of two or four CTAs.
// Rows come through cells in shared memory that each thread fills (cp.async)
// and empties by itself: no barrier and no wait between threads guards them.
// The forward pass takes a row into registers and fetches the next one into
// the same cells; the backward pass has two sets of cells and reads a row from
// them in each pass, which leaves the registers to its column sums (the
// gradients of weights, biases and gate): a thread owns the same columns in
// all its rows, and keeps them over the whole launch.
//
// Spills (ptxas, bytes stored a thread), backward: RMS by clusters of up to
// 192 threads 32 with an fp32 stream, and 128 where something optional is left
// out; layer norms with gate groups 32 to 144.  Forward: 4 and 8 in the bf16
// kernels for rows of up to 512 columns with a gate per channel.
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
  float* part;          // bwd: [4][CTAs or clusters][h] column sums of each
  float* gpart;         // bwd: [2][workers][h] gate sums of groups that several workers share
  void* dgate;          // bwd: gate gradient where the kernel writes whole groups
  float alpha, eps, inv_h;
  uint32_t M, m, nvec, rows_per_gate;
  int32_t post, pre;
  int32_t has_z, has_dn, has_dy, out_f32;
  int32_t coef;         // shared memory holds the fp32 coefficients of w_post (bit 0) and w_pre (bit 1)
};

constexpr int kRed = 12 * 32;  // floats of a reduction's buffer

// Who works on a row: a warp, a CTA, or a cluster of two or four CTAs, which
// share out its columns.
enum WorkerKind : int { BY_WARP = 0, BY_CTA = 1, BY_CLUSTER = 2 };

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// (for threads that wrote nothing the others read)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Sums of N values over a warp's 32 lanes (N <= 16).  Instead of N sums of
// five steps, lanes give away half of their values at each step while they
// have more than one: 8 values take 9 shuffles, not 40.  Value i ends up in
// the lanes with holds<N>(lane) == i.
template <int N>
__device__ __forceinline__ constexpr int padded() {
  return N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : 16;
}
template <int N>
__device__ __forceinline__ int holds(int lane) {
  int i = 0, o = 16;
#pragma unroll
  for (int n = padded<N>(); n > 1; n /= 2, o /= 2) i = 2 * i + ((lane & o) != 0);
  return i;
}
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int lane) {
  constexpr int P = padded<N>();
  float a[P];
#pragma unroll
  for (int i = 0; i < P; ++i) a[i] = i < N ? v[i] : 0.f;
  int o = 16;
#pragma unroll
  for (int n = P; n > 1; n /= 2, o /= 2) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? a[i + n / 2] : a[i], give = up ? a[i] : a[i + n / 2];
      a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1)
    if (k <= o) a[0] += __shfl_xor_sync(0xFFFFFFFFu, a[0], k);
  return a[0];
}
// Value i of warp_sums' result, in every lane.
template <int N>
__device__ __forceinline__ float warp_value(float s, int i) {
  int lane = 0, o = 16;
#pragma unroll
  for (int n = padded<N>() / 2; n > 0; n /= 2, o /= 2) lane |= (i & n) ? o : 0;
  return __shfl_sync(0xFFFFFFFFu, s, lane);
}

// Sums over the threads of a warp or CTA, left in every thread.  `red` is
// shared memory of two buffers of kRed floats that take turns: a buffer is
// written again only after the barrier of the reduction in between, which
// every thread passes after its reads.
template <int N, int KIND>
__device__ __forceinline__ void worker_sum(float (&v)[N], float* red, int& turn) {
  const int lane = threadIdx.x & 31;
  float s = warp_sums<N>(v, lane);
  if constexpr (KIND != BY_WARP) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, i = holds<N>(lane);
    float* b = red + turn * kRed;
    turn ^= 1;
    // one lane for each value: the first that holds it
    if (i < N && (lane & (32 / padded<N>() - 1)) == 0) b[i * 32 + warp] = s;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < warps ? b[k * 32 + lane] : 0.f;
    s = warp_sums<N>(v, lane);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_value<N>(s, k);
}

// Shared memory of worker_totals.
struct Totals {
  float part[kRed];     // the warps' sums
  float4 peers[2][12];  // the (up to four) CTAs' sums, by turns
  float4 out[2];        // what is made of the totals
};

// Sums over the worker's threads, which one warp of the CTA turns into a few
// numbers for all: make(total, out) gets a function that gives total i (in
// all lanes) and writes up to 8 floats from lane 0.  The other warps do not
// spend instructions on it.  A cluster's CTAs exchange their sums, so that
// all add them in the same order.
template <int N, int KIND, typename Make>
__device__ __forceinline__ void worker_totals(float (&v)[N], Totals& t, int& turn, float (&got)[8], Make make) {
  const int lane = threadIdx.x & 31;
  float s = warp_sums<N>(v, lane);
  if constexpr (KIND == BY_WARP) {
    auto total = [&](int i) { return warp_value<N>(s, i); };
    make(total, got);
  } else {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, i = holds<N>(lane);
    const bool first = i < N && (lane & (32 / padded<N>() - 1)) == 0;
    if (first) t.part[i * 32 + warp] = s;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = lane < warps ? t.part[k * 32 + lane] : 0.f;
      s = warp_sums<N>(v, lane);
      if constexpr (KIND == BY_CLUSTER) {
        const uint32_t size = cluster_size();
        if (first) {
          const uint32_t at = smem_u32(&t.peers[turn][i]) + cluster_ctarank() * 4;
          for (uint32_t c = 0; c < size; ++c) st_cluster_f32(mapa_shared(at, c), s);
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (first) {
          const float4 p = t.peers[turn][i];
          s = size == 2 ? p.x + p.y : (p.x + p.y) + (p.z + p.w);
        }
        turn ^= 1;
      }
      auto total = [&](int k) { return warp_value<N>(s, k); };
      float o[8];
      make(total, o);
      if (lane == 0) {
        t.out[0] = make_float4(o[0], o[1], o[2], o[3]);
        t.out[1] = make_float4(o[4], o[5], o[6], o[7]);
      }
    } else if constexpr (KIND == BY_CLUSTER) {
      cluster_arrive_relaxed();
      cluster_wait();
    }
    __syncthreads();
    const float4 a = t.out[0], b = t.out[1];
    got[0] = a.x;
    got[1] = a.y;
    got[2] = a.z;
    got[3] = a.w;
    got[4] = b.x;
    got[5] = b.y;
    got[6] = b.z;
    got[7] = b.w;
  }
}

// Eight columns as four packed fp32 pairs.
struct Vec {
  uint64_t p[4];
};

__device__ __forceinline__ uint64_t both(float v) { return pk2(v, v); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  upk2(v, a, b);
  return a + b;
}

__device__ __forceinline__ Vec widen(const uint4& w) {
  Vec v;
  v.p[0] = pk2(bf_lo(w.x), bf_hi(w.x));
  v.p[1] = pk2(bf_lo(w.y), bf_hi(w.y));
  v.p[2] = pk2(bf_lo(w.z), bf_hi(w.z));
  v.p[3] = pk2(bf_lo(w.w), bf_hi(w.w));
  return v;
}
__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; }
__device__ __forceinline__ Vec wide(const uint4& a, const uint4& b) {
  Vec v;
  v.p[0] = pair64(a.x, a.y);
  v.p[1] = pair64(a.z, a.w);
  v.p[2] = pair64(b.x, b.y);
  v.p[3] = pair64(b.z, b.w);
  return v;
}

// One vector of a bf16 or fp32 row as raw registers.
template <bool F32>
struct Raw {
  uint4 a;
  __device__ __forceinline__ Vec get() const { return widen(a); }
  __device__ __forceinline__ void load(uint32_t cell, uint32_t) { a = ld_shared_v4(cell); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
};
template <>
struct Raw<true> {
  uint4 a, b;
  __device__ __forceinline__ Vec get() const { return wide(a, b); }
  __device__ __forceinline__ void load(uint32_t cell, uint32_t step) {
    a = ld_shared_v4(cell);
    b = ld_shared_v4(cell + step);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
};

template <bool F32>
__device__ __forceinline__ void store_row(void* row, uint32_t v, const Vec& f) {
  if constexpr (F32) {
    uint4* d = static_cast<uint4*>(row) + 2 * v;
    st_global_cs(d, make_uint4(static_cast<uint32_t>(f.p[0]), static_cast<uint32_t>(f.p[0] >> 32), static_cast<uint32_t>(f.p[1]),
                               static_cast<uint32_t>(f.p[1] >> 32)));
    st_global_cs(d + 1, make_uint4(static_cast<uint32_t>(f.p[2]), static_cast<uint32_t>(f.p[2] >> 32), static_cast<uint32_t>(f.p[3]),
                                   static_cast<uint32_t>(f.p[3] >> 32)));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      upk2(f.p[i], lo, hi);
      w[i] = pack_bf16(lo, hi);
    }
    st_global_cs(static_cast<uint4*>(row) + v, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// fp32 vector in two cells of a thread, `step` apart.
__device__ __forceinline__ void put_cells(uint32_t cell, uint32_t step, const Vec& f) {
  st_shared_v4(cell, make_uint4(static_cast<uint32_t>(f.p[0]), static_cast<uint32_t>(f.p[0] >> 32), static_cast<uint32_t>(f.p[1]),
                                static_cast<uint32_t>(f.p[1] >> 32)));
  st_shared_v4(cell + step, make_uint4(static_cast<uint32_t>(f.p[2]), static_cast<uint32_t>(f.p[2] >> 32),
                                       static_cast<uint32_t>(f.p[3]), static_cast<uint32_t>(f.p[3] >> 32)));
}
__device__ __forceinline__ Vec get_cells(uint32_t cell, uint32_t step) { return wide(ld_shared_v4(cell), ld_shared_v4(cell + step)); }

// Clears the row cells of a thread's vectors past the row's end.  Nothing is
// copied there, so that sums run over all vectors without asking; only a
// layer norm, which subtracts a mean, and stores do ask.
template <int NV, int PARTS>
__device__ __forceinline__ void clear_cells(uint32_t cell, uint32_t step, uint32_t T, uint32_t t, uint32_t nvec) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (k * T + t >= nvec) {
#pragma unroll
      for (int j = 0; j < PARTS; ++j) st_shared_v4(cell + (k * PARTS + j) * step, make_uint4(0, 0, 0, 0));
    }
}

// Row `r` of a tensor of p shards with m rows each; bytes: of one row.
__device__ __forceinline__ const char* shard_row(const void* const (&t)[8], uint32_t s, uint32_t r, int64_t bytes) {
  return static_cast<const char*>(t[s]) + static_cast<int64_t>(r) * bytes;
}
__device__ __forceinline__ char* shard_row(void* const (&t)[8], uint32_t s, uint32_t r, int64_t bytes) {
  return static_cast<char*>(t[s]) + static_cast<int64_t>(r) * bytes;
}

template <int KIND>
struct Worker {
  uint32_t T, t, id, count;  // threads (of the CTA, or warp), this thread, worker, workers in the grid
  uint32_t v0, nvec;         // this CTA's columns, in vectors
  __device__ explicit Worker(uint32_t all) {
    T = KIND == BY_WARP ? 32u : blockDim.x;
    t = KIND == BY_WARP ? (threadIdx.x & 31u) : threadIdx.x;
    id = KIND == BY_WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : KIND == BY_CLUSTER ? blockIdx.x / cluster_size() : blockIdx.x;
    count = KIND == BY_WARP ? gridDim.x * (blockDim.x >> 5) : KIND == BY_CLUSTER ? gridDim.x / cluster_size() : gridDim.x;
    v0 = 0;
    nvec = all;
    if constexpr (KIND == BY_CLUSTER) {
      const uint32_t part = (all + cluster_size() - 1) / cluster_size();
      v0 = min(cluster_ctarank() * part, all - 1);
      nvec = min(part, all - min(cluster_ctarank() * part, all));
    }
  }
};

// The fp32 coefficients that all rows share, in cells of the thread's own
// after the row cells: alpha * w_post * gate row 0 (forward) or w_post * gate
// row 0 (backward), and w_pre.  What does not fit is formed again each time.
// GATE: the gate has several rows and is not part of the coefficient.
template <int NV, bool GATE, bool FULL = false>  // FULL: both are in shared memory
struct Coefs {
  uint32_t post, pre, step;  // cells of vector 0
  uint32_t v0, nvec;
  float scale;

  // v: of the CTA's vectors.  Past the last one make_post gives zeros, so that
  // the zeros of z there stay zeros whatever the last weights are (times an
  // infinity they would be NaN in the row's sums); make_pre gives the last one.
  __device__ __forceinline__ Vec make_post(const NormParams& P, uint32_t v) const {
    const bool past = v >= nvec;
    v = v0 + min(v, max(nvec, 1u) - 1);
    Vec c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.p[i] = both(scale);
    if (P.w_post) {
      const Vec w = widen(__ldg(P.w_post + v));
#pragma unroll
      for (int i = 0; i < 4; ++i) c.p[i] = mul2(c.p[i], w.p[i]);
    }
    if (!GATE && P.gate) {
      const Vec g = widen(__ldg(P.gate + v));
#pragma unroll
      for (int i = 0; i < 4; ++i) c.p[i] = mul2(c.p[i], g.p[i]);
    }
    if (past) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c.p[i] = 0;
    }
    return c;
  }
  __device__ __forceinline__ Vec make_pre(const NormParams& P, uint32_t v) const {
    if (P.w_pre) return widen(__ldg(P.w_pre + v0 + min(v, max(nvec, 1u) - 1)));
    Vec c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.p[i] = both(1.f);
    return c;
  }
  template <int KIND>
  __device__ __forceinline__ void init(const NormParams& P, uint32_t base, float s, const Worker<KIND>& W) {
    step = blockDim.x * 16;
    v0 = W.v0;
    nvec = W.nvec;
    post = base;
    pre = base + (P.coef & 1 ? 2 * NV * step : 0);
    scale = s;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t v = k * W.T + W.t;
      if (P.coef & 1) put_cells(post + 2 * k * step, step, make_post(P, v));
      if (P.coef & 2) put_cells(pre + 2 * k * step, step, make_pre(P, v));
    }
  }
  __device__ __forceinline__ Vec get_post(const NormParams& P, int k, uint32_t v) const {
    return FULL || (P.coef & 1) ? get_cells(post + 2 * k * step, step) : make_post(P, v);
  }
  __device__ __forceinline__ Vec get_pre(const NormParams& P, int k, uint32_t v) const {
    return FULL || (P.coef & 2) ? get_cells(pre + 2 * k * step, step) : make_pre(P, v);
  }
};

// ----------------------------------------------------------------- forward

// NV vectors of 8 columns per thread; RES32: the residual stream is fp32;
// LN: one of the norms is a layer norm; GATE: the gate has several rows,
// streamed like the other inputs.  Measured, RMS norms and a gate per channel,
// bf16: 8192 x 8192 (537 MB) 93 us, 5.8 TB/s, against 79 us at the copy rate;
// HBM bounds it, with 40 % of the issue slots in use.
template <int NV, bool RES32, bool LN, bool GATE, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_fwd_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2 * kRed];
  griddep_wait();
  griddep_launch_dependents();
  const Worker<KIND> W(P.nvec);
  const uint32_t nvec = P.nvec;
  const int64_t row16 = static_cast<int64_t>(nvec) * 16, rowx = RES32 ? 2 * row16 : row16;
  // cell of vector k, part j (x: 1 or 2, z, gate): 16 bytes a thread,
  // consecutive threads in consecutive cells
  constexpr int PX = RES32 ? 2 : 1, PARTS = PX + 1 + (GATE ? 1 : 0);
  const uint32_t cell = smem_u32(ring) + threadIdx.x * 16, step = blockDim.x * 16;
  auto slot = [&](int k, int j) { return cell + (k * PARTS + j) * step; };
  uint32_t fs = 0, fr = W.id;  // shard and row in it of the next fetch
  auto fetch = [&](uint32_t row) {
    if (row < P.M) {
      while (fr >= P.m) {
        fr -= P.m;
        ++fs;
      }
      const char* x = shard_row(P.x, fs, fr, rowx) + W.t * (PX * 16);
      const char* z = P.has_z ? shard_row(P.z, fs, fr, row16) + W.t * 16 : nullptr;
      const uint4* g = GATE ? P.gate + static_cast<int64_t>(row / P.rows_per_gate) * nvec + W.t : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k * W.T + W.t < nvec) {
#pragma unroll
          for (int j = 0; j < PX; ++j) cp_async16(slot(k, j), x + (k * W.T * PX + j) * 16);
          if (P.has_z) cp_async16(slot(k, PX), z + k * W.T * 16);
          if (GATE) cp_async16(slot(k, PX + 1), g + k * W.T);
        }
      }
    }
    fr += W.count;
    cp_async_commit();
  };
  fetch(W.id);
  clear_cells<NV, PARTS>(cell, step, W.T, W.t, nvec);
  Coefs<NV, GATE> coefs;
  coefs.init(P, cell + NV * PARTS * step, P.alpha, W);
  uint32_t os = 0, orow = W.id;  // shard and row in it of the outputs
  int turn = 0;
  for (uint32_t row = W.id; row < P.M; row += W.count, orow += W.count) {
    while (orow >= P.m) {
      orow -= P.m;
      ++os;
    }
    cp_async_wait<0>();
    Vec y[NV], z[NV];
    uint4 gr[GATE ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Raw<RES32> rx;
      rx.load(slot(k, 0), step);
      y[k] = rx.get();
      z[k] = widen(P.has_z ? ld_shared_v4(slot(k, PX)) : make_uint4(0, 0, 0, 0));
      if constexpr (GATE) gr[k] = ld_shared_v4(slot(k, PX + 1));
    }
    // the cells are in registers: a thread's shared loads are done before
    // copies that it starts later arrive
    fetch(row + W.count);
    if (P.has_z) {
      float r = 1.f;
      if (LN && P.post == NORM_LAYER) {
        uint64_t s = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) s = add2(s, z[k].p[i]);
        float a[1] = {sum2(s)};
        worker_sum<1, KIND>(a, red, turn);
        const uint64_t mu = both(-a[0] * P.inv_h);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[k].p[i] = add2(z[k].p[i], mu);
      }
      if (P.post != NORM_NONE) {
        uint64_t s = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (!LN || k * W.T + W.t < nvec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fma2(z[k].p[i], z[k].p[i], s);
          }
        float a[1] = {sum2(s)};
        worker_sum<1, KIND>(a, red, turn);
        r = rsqrtf(fmaf(a[0], P.inv_h, P.eps));
      }
      const uint64_t r2 = both(r);
      char* yo = shard_row(P.y, os, orow, rowx);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        const Vec c = coefs.get_post(P, k, v);
        if constexpr (!LN && !GATE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[k].p[i] = fma2(z[k].p[i], mul2(c.p[i], r2), y[k].p[i]);
        } else {
          Vec o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o.p[i] = mul2(z[k].p[i], mul2(c.p[i], r2));
          if (LN && P.b_post) {  // alpha * gate * b
            const uint32_t at = min(v, nvec - 1);
            const Vec b = widen(__ldg(P.b_post + at));
            Vec g;
#pragma unroll
            for (int i = 0; i < 4; ++i) g.p[i] = both(P.alpha);
            if (!GATE && P.gate) {
              const Vec gv = widen(__ldg(P.gate + at));
#pragma unroll
              for (int i = 0; i < 4; ++i) g.p[i] = mul2(g.p[i], gv.p[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o.p[i] = fma2(g.p[i], b.p[i], o.p[i]);
          }
          if constexpr (GATE) {
            const Vec g = widen(gr[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[k].p[i] = fma2(o.p[i], g.p[i], y[k].p[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[k].p[i] = add2(o.p[i], y[k].p[i]);
          }
          // (a layer norm leaves something in the vectors past the row's end)
          if (LN && v >= nvec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[k].p[i] = 0;
          }
        }
        if (v < nvec) store_row<RES32>(yo, v, y[k]);
      }
    }
    if (P.pre != NORM_NONE) {
      if (LN && P.pre == NORM_LAYER) {
        uint64_t s = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) s = add2(s, y[k].p[i]);
        float a[1] = {sum2(s)};
        worker_sum<1, KIND>(a, red, turn);
        const uint64_t mu = both(-a[0] * P.inv_h);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[k].p[i] = add2(y[k].p[i], mu);
      }
      uint64_t s = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (!LN || k * W.T + W.t < nvec) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fma2(y[k].p[i], y[k].p[i], s);
        }
      float a[1] = {sum2(s)};
      worker_sum<1, KIND>(a, red, turn);
      const uint64_t r2 = both(rsqrtf(fmaf(a[0], P.inv_h, P.eps)));
      char* no = shard_row(P.n, os, orow, row16);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        const Vec w = coefs.get_pre(P, k, v);
        Vec o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = mul2(mul2(y[k].p[i], r2), w.p[i]);
        if (LN && P.b_pre) {
          const Vec b = widen(__ldg(P.b_pre + min(v, nvec - 1)));
#pragma unroll
          for (int i = 0; i < 4; ++i) o.p[i] = add2(o.p[i], b.p[i]);
        }
        if (v < nvec) store_row<false>(no, v, o);
      }
    }
  }
  cp_async_wait<0>();
}

// ----------------------------------------------------------------- backward

// Thread blocks per SM that the registers of a backward kernel are meant for;
// a layer norm's or a gate's further column sums take the room of one.
constexpr int bwd_blocks(int nv, int threads, bool more) {
  const int n = nv > 2 ? 1 : threads <= 128 ? 4 : threads <= 192 ? 3 : 2;
  return n > 1 && more ? n - 1 : n;
}

// The row's sums after the means (s6..s11 only with a layer norm; yc, zc are
// centred values, d = dn * w_pre, q = gate * w_post):
//   s0 yc^2  s1 d yc  s2 zc^2  s3 q zc dy  s4 q zc d  s5 q zc yc
//   s6 d  s7 q zc  s8 q dy  s9 q d  s10 q yc  s11 q
// With ry = 1/sqrt(s0/h + eps), m1 = s6/h, m2 = ry^2 s1/h:
//   dx = dy + ry (d - m1 - m2 yc),  u = alpha q dx,
//   sum u zhat = alpha rz (s3 + ry (s4 - m1 s7 - m2 s5)),
//   sum u      = alpha    (s8 + ry (s9 - m1 s11 - m2 s10)),
//   dz = rz (u - mean u - zhat mean(u zhat)):
// the sums of the post norm's gradient are linear in dx, so that both norms
// are served by one reduction (a second one, before it, gives a layer norm
// its means).  The worker owns rows [id M / count, (id + 1) M / count).
//
// GATE: the gate has more than one row; its sums are kept apart from the
// weights' and given out whenever a group ends.  With one gate row or none,
// A = sum dx zhat and B = sum dx are kept, and the last kernel forms
// dw_post = alpha g A, db_post = alpha g B, dgate = alpha (w A + b B).
//
// FULL: every input and both dx and dz are there, and the coefficients are in
// shared memory, as in a training step; a row's overhead then has no
// branches for them.
template <int NV, bool RES32, bool LN, bool GATE, int KIND, int MAXT, bool FULL>
__global__ void __launch_bounds__(MAXT, bwd_blocks(NV, MAXT, LN || GATE)) block_norm_bwd_kernel(const __grid_constant__ NormParams P) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ Totals totals;
  const bool has_dn = FULL || P.has_dn, has_dy = FULL || P.has_dy, has_z = FULL || P.has_z;
  griddep_wait();
  griddep_launch_dependents();
  const Worker<KIND> W(P.nvec);
  if constexpr (KIND == BY_CLUSTER) cluster_sync_all();  // all are there before one writes to another
  const uint32_t nvec = W.nvec, h = P.nvec * 8;
  const int64_t row16 = static_cast<int64_t>(P.nvec) * 16, rowx = RES32 ? 2 * row16 : row16;
  constexpr int PX = RES32 ? 2 : 1, PARTS = 2 * PX + 2 + (GATE ? 1 : 0);  // y, dy, dn, z, gate
  const uint32_t cell = smem_u32(ring) + threadIdx.x * 16, step = blockDim.x * 16;
  constexpr int STAGE = NV * PARTS;  // cells of a row; two rows take turns
  uint32_t here = cell, next = cell + STAGE * step;
  auto slot = [&](uint32_t at, int k, int j) { return at + (k * PARTS + j) * step; };
  const uint32_t r0 = static_cast<uint32_t>(static_cast<uint64_t>(W.id) * P.M / W.count);
  const uint32_t r1 = static_cast<uint32_t>(static_cast<uint64_t>(W.id + 1) * P.M / W.count);
  // The next row to fetch: shard, row in it, and pointers to the thread's
  // first vector, which move on by a row until the shard ends.
  uint32_t fs = r0 / P.m, fr = r0 % P.m;
  const char *py = nullptr, *pdy = nullptr, *pdn = nullptr, *pz = nullptr;
  auto aim = [&] {
    const uint32_t at = W.v0 + W.t;
    if (has_dn) py = shard_row(P.x, fs, fr, rowx) + at * (PX * 16);
    if (has_dy) pdy = shard_row(P.dy, fs, fr, rowx) + at * (PX * 16);
    if (has_dn) pdn = shard_row(P.dn, fs, fr, row16) + at * 16;
    if (has_z) pz = shard_row(P.z, fs, fr, row16) + at * 16;
  };
  if (r0 < r1) aim();
  uint32_t os = fs, orow = fr;  // shard and row in it of the outputs
  char *dxo = nullptr, *dzo = nullptr;
  const bool give_dx = FULL || P.y[0] != nullptr, give_dz = FULL || P.n[0] != nullptr;
  auto aim_out = [&] {
    if (give_dx) dxo = shard_row(P.y, os, orow, rowx) + W.v0 * (PX * 16);
    if (give_dz) dzo = shard_row(P.n, os, orow, row16) + W.v0 * 16;
  };
  if (r0 < r1) aim_out();
  auto fetch = [&](uint32_t row, uint32_t at) {
    if (row < r1) {
      const uint4* g = GATE ? P.gate + static_cast<int64_t>(row / P.rows_per_gate) * P.nvec + W.v0 + W.t : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k * W.T + W.t < nvec) {
          const uint32_t o = k * W.T * 16;
#pragma unroll
          for (int j = 0; j < PX; ++j) {
            if (has_dn) cp_async16(slot(at, k, j), py + o * PX + j * 16);
            if (has_dy) cp_async16(slot(at, k, PX + j), pdy + o * PX + j * 16);
          }
          if (has_dn) cp_async16(slot(at, k, 2 * PX), pdn + o);
          if (has_z) cp_async16(slot(at, k, 2 * PX + 1), pz + o);
          if (GATE) cp_async16(slot(at, k, 2 * PX + 2), g + k * W.T);
        }
      }
      py += rowx;
      pdy += rowx;
      pdn += row16;
      pz += row16;
      if (++fr == P.m) {
        fr = 0;
        ++fs;
        if (row + 1 < r1) aim();
      }
    }
    cp_async_commit();
  };
  fetch(r0, here);
  clear_cells<NV, PARTS>(here, step, W.T, W.t, nvec);
  clear_cells<NV, PARTS>(next, step, W.T, W.t, nvec);
  Coefs<NV, GATE, FULL> coefs;
  coefs.init(P, cell + 2 * STAGE * step, 1.f, W);

  Vec accA[NV] = {}, accC[NV] = {};
  Vec accB[LN ? NV : 1] = {}, accD[LN ? NV : 1] = {}, accE[GATE ? NV : 1] = {};
  int turn = 0;
  for (uint32_t row = r0; row < r1; ++row) {
    // the next row goes where the last one was, which this thread is done
    // with; this row is read from its cells in each pass, which leaves the
    // registers to the column sums
    fetch(row + 1, next);
    cp_async_wait<1>();
    auto load_y = [&](int k) {
      Raw<RES32> r;
      r.zero();
      if (has_dn) r.load(slot(here, k, 0), step);
      return r.get();
    };
    auto load_dy = [&](int k) {
      Raw<RES32> r;
      r.zero();
      if (has_dy) r.load(slot(here, k, PX), step);
      return r.get();
    };
    auto load_dn = [&](int k) { return widen(has_dn ? ld_shared_v4(slot(here, k, 2 * PX)) : make_uint4(0, 0, 0, 0)); };
    auto load_z = [&](int k) { return widen(has_z ? ld_shared_v4(slot(here, k, 2 * PX + 1)) : make_uint4(0, 0, 0, 0)); };
    auto load_g = [&](int k) { return widen(ld_shared_v4(slot(here, k, 2 * PX + 2))); };
    uint64_t mu_y = 0, mu_z = 0;  // minus the means
    if constexpr (LN) {
      uint64_t a0 = 0, a1 = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const Vec y = load_y(k), z = load_z(k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a0 = add2(a0, y.p[i]);
          a1 = add2(a1, z.p[i]);
        }
      }
      float a[2] = {sum2(a0), sum2(a1)}, got[8];
      worker_totals<2, KIND>(a, totals, turn, got, [&](auto total, float(&o)[8]) {
        const float y = total(0), z = total(1);
        o[0] = P.pre == NORM_LAYER ? -y * P.inv_h : 0.f;
        o[1] = P.post == NORM_LAYER ? -z * P.inv_h : 0.f;
        o[2] = o[3] = o[4] = o[5] = o[6] = o[7] = 0.f;
      });
      mu_y = both(got[0]);
      mu_z = both(got[1]);
    }
    constexpr int NS = LN ? 12 : 6;
    constexpr int Y2 = 0, DY = 1, Z2 = 2, QZG = 3, QZD = 4, QZY = 5, D1 = 6, QZ = 7, QG = 8, QD = 9, QY = 10, Q1 = 11;
    uint64_t acc[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) acc[i] = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (!LN || v < nvec) {
          const Vec y = load_y(k), g = load_dy(k), z = load_z(k), wp = coefs.get_pre(P, k, v);
          Vec d = load_dn(k), q = coefs.get_post(P, k, v);
          if constexpr (GATE) {
            const Vec gv = load_g(k);
#pragma unroll
            for (int i = 0; i < 4; ++i) q.p[i] = mul2(q.p[i], gv.p[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t yc = LN ? add2(y.p[i], mu_y) : y.p[i], zc = LN ? add2(z.p[i], mu_z) : z.p[i];
            const uint64_t dd = mul2(d.p[i], wp.p[i]), qz = mul2(q.p[i], zc);
            acc[Y2] = fma2(yc, yc, acc[Y2]);
            acc[DY] = fma2(dd, yc, acc[DY]);
            acc[Z2] = fma2(zc, zc, acc[Z2]);
            acc[QZG] = fma2(qz, g.p[i], acc[QZG]);
            acc[QZD] = fma2(qz, dd, acc[QZD]);
            acc[QZY] = fma2(qz, yc, acc[QZY]);
            if constexpr (LN) {
              acc[D1] = add2(acc[D1], dd);
              acc[QZ] = add2(acc[QZ], qz);
              acc[QG] = fma2(q.p[i], g.p[i], acc[QG]);
              acc[QD] = fma2(q.p[i], dd, acc[QD]);
              acc[QY] = fma2(q.p[i], yc, acc[QY]);
              acc[Q1] = add2(acc[Q1], q.p[i]);
            }
          }
        }
      }
    float sum[NS], got[8];
#pragma unroll
    for (int i = 0; i < NS; ++i) sum[i] = sum2(acc[i]);
    worker_totals<NS, KIND>(sum, totals, turn, got, [&](auto total, float(&o)[8]) {
      const float ry = has_dn ? rsqrtf(fmaf(total(Y2), P.inv_h, P.eps)) : 0.f;
      const float m2 = ry * ry * total(DY) * P.inv_h;  // times yc
      float m1 = 0.f;
      if constexpr (LN) m1 = P.pre == NORM_LAYER ? total(D1) * P.inv_h : 0.f;
      float rz = 1.f, u1 = 0.f, u2 = 0.f;
      if (P.post != NORM_NONE) {
        rz = rsqrtf(fmaf(total(Z2), P.inv_h, P.eps));
        float t = total(QZG) + ry * (total(QZD) - m2 * total(QZY));
        if constexpr (LN) {
          t -= ry * m1 * total(QZ);
          if (P.post == NORM_LAYER) u1 = P.alpha * P.inv_h * (total(QG) + ry * (total(QD) - m1 * total(Q1) - m2 * total(QY)));
        }
        u2 = P.alpha * P.inv_h * rz * t;
      }
      o[0] = ry;
      o[1] = -ry * m2;
      o[2] = rz;
      o[3] = P.alpha * rz;
      o[4] = -rz * u2;
      o[5] = -ry * m1;
      o[6] = -rz * u1;
      o[7] = 0.f;
    });
    const uint64_t ry2 = both(got[0]), ym = both(got[1]), rz2 = both(got[2]), arz = both(got[3]), zm = both(got[4]);
    const uint64_t off_d = both(got[5]), off_z = both(got[6]);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        const bool in = v < nvec;
        if (!LN || in) {
          Vec dx = load_dy(k);
          if (has_dn) {
            const Vec y = load_y(k), d = load_dn(k), wp = coefs.get_pre(P, k, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t yc = LN ? add2(y.p[i], mu_y) : y.p[i];
              accC[k].p[i] = fma2(mul2(d.p[i], ry2), yc, accC[k].p[i]);
              uint64_t t = fma2(ym, yc, dx.p[i]);
              if constexpr (LN) {
                accD[k].p[i] = add2(accD[k].p[i], d.p[i]);
                t = add2(t, off_d);
              }
              dx.p[i] = fma2(mul2(d.p[i], wp.p[i]), ry2, t);
            }
          }
          if (give_dx && in) store_row<RES32>(dxo, v, dx);
          if (has_z) {
            Vec z = load_z(k);
            const Vec q = coefs.get_post(P, k, v);
            if constexpr (GATE) {
              const Vec g = load_g(k);
              Vec b;
#pragma unroll
              for (int i = 0; i < 4; ++i) b.p[i] = 0;
              if (LN && P.b_post) b = widen(__ldg(P.b_post + W.v0 + v));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint64_t zh = mul2(LN ? add2(z.p[i], mu_z) : z.p[i], rz2), t = mul2(dx.p[i], g.p[i]);
                accA[k].p[i] = fma2(t, zh, accA[k].p[i]);
                if constexpr (LN) accB[k].p[i] = add2(accB[k].p[i], t);
                accE[k].p[i] = fma2(dx.p[i], fma2(zh, q.p[i], b.p[i]), accE[k].p[i]);
                uint64_t o = mul2(mul2(t, arz), q.p[i]);
                if constexpr (LN) o = add2(o, off_z);
                z.p[i] = fma2(zh, zm, o);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint64_t zh = mul2(LN ? add2(z.p[i], mu_z) : z.p[i], rz2);
                accA[k].p[i] = fma2(dx.p[i], zh, accA[k].p[i]);
                if constexpr (LN) accB[k].p[i] = add2(accB[k].p[i], dx.p[i]);
                uint64_t o = mul2(mul2(dx.p[i], arz), q.p[i]);
                if constexpr (LN) o = add2(o, off_z);
                z.p[i] = fma2(zh, zm, o);
              }
            }
            if (give_dz && in) store_row<false>(dzo, v, z);
          }
        }
      }
    const uint32_t done = here;
    here = next;
    next = done;
    dxo += rowx;
    dzo += row16;
    if (++orow == P.m) {
      orow = 0;
      ++os;
      if (row + 1 < r1) aim_out();
    }
    if constexpr (GATE) {
      const uint32_t group = row / P.rows_per_gate;
      if (row + 1 == r1 || (row + 1) / P.rows_per_gate != group) {
        // the group ends here, or goes on in the next worker's rows
        const uint64_t g0 = static_cast<uint64_t>(group) * P.rows_per_gate;
        const bool whole = g0 >= r0 && g0 + P.rows_per_gate <= r1;
        if (P.gpart) {
          float* gp = P.gpart + (static_cast<int64_t>(g0 > r0 ? 1 : 0) * W.count + W.id) * h;
          const uint64_t a = both(P.alpha);
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            const uint32_t v = k * W.T + W.t;
            if (v < nvec) {
              Vec e;
#pragma unroll
              for (int i = 0; i < 4; ++i) e.p[i] = mul2(accE[k].p[i], a);
              if (!whole) store_row<true>(gp, W.v0 + v, e);
              else if (P.out_f32) store_row<true>(static_cast<float*>(P.dgate) + static_cast<int64_t>(group) * h, W.v0 + v, e);
              else store_row<false>(static_cast<__nv_bfloat16*>(P.dgate) + static_cast<int64_t>(group) * h, W.v0 + v, e);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) accE[k].p[i] = 0;
      }
    }
  }
  cp_async_wait<0>();

  // column sums of the CTA (of a cluster: of its part): warps that are workers of their own are added in
  // warp order through shared memory (the row cells are no longer in use)
  auto give = [&](Vec (&acc)[NV], int which) {
    const uint32_t ctas = KIND == BY_CLUSTER ? W.count : gridDim.x, cta = KIND == BY_CLUSTER ? W.id : blockIdx.x;
    float* out = P.part + (static_cast<int64_t>(which) * ctas + cta) * h;
    if constexpr (KIND != BY_WARP) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t v = k * W.T + W.t;
        if (v < nvec) store_row<true>(out, W.v0 + v, acc[k]);
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
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            upk2(acc[k].p[i], lo, hi);
            all[(warp * 8 + 2 * i) * (NV * 32) + v] = lo;
            all[(warp * 8 + 2 * i + 1) * (NV * 32) + v] = hi;
          }
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
  if (has_dn && P.part) give(accC, 0);
  if (has_z && P.part) give(accA, 1);
  if constexpr (LN) {
    if (has_dn && P.part) give(accD, 2);
    if (has_z && P.part) give(accB, 3);
  }
}

}  // namespace tpf
