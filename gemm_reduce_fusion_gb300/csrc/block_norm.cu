// C ABI of the block boundary (norms, gate, residual) and its gradients:
// argument checks and launches of the kernels in block_norm.cuh.
#include "block_norm.cuh"

#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>

#include "block_norm.h"
#include "host_util.h"

using namespace tpf;

namespace {

struct NormGradParams {
  const float* part;    // [4][ctas][h]: C, A, D, B
  const float* gpart;   // [2][workers][h]
  const __nv_bfloat16 *gate, *w_post, *b_post;  // gate: its only row, or null
  void *dw_pre, *db_pre, *dw_post, *db_post, *dgate;
  float alpha;
  uint32_t h, ctas, workers, M, rows_per_gate, groups;  // groups: gate rows
  int32_t out_f32;
};

__device__ __forceinline__ void put_grad(void* out, int64_t i, float v, int f32) {
  if (out == nullptr) return;
  if (f32) static_cast<float*>(out)[i] = v;
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// Adds the CTAs' column sums in a fixed order: 32 columns a block, 16 lanes
// of partial sums a column, joined in lane order; eight loads of a lane are
// in flight together, since the latency of these few reads is all there is
// to it.  blockIdx.y: 0 C (dw_pre), 1 A (dw_post, and the gate's only row),
// 2 D (db_pre), 3 B (db_post), 4 + g gate row g where several workers hold
// parts of it.
constexpr int kGradLanes = 16;

// at[i * pitch] for i, i + lanes, ... below n, in this order.
__device__ __forceinline__ float strided_sum(const float* at, uint32_t i, uint32_t n, uint32_t pitch) {
  float t = 0.f;
  for (; i < n; i += 8 * kGradLanes) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j * kGradLanes < n ? __ldcg(at + static_cast<int64_t>(i + j * kGradLanes) * pitch) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += v[j];
  }
  return t;
}

__global__ void __launch_bounds__(32 * kGradLanes) block_norm_grad_kernel(const __grid_constant__ NormGradParams P) {
  __shared__ float sh[2][kGradLanes][33];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t col = threadIdx.x & 31, lane = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  const bool in = c < P.h;
  const int64_t plane = static_cast<int64_t>(P.ctas) * P.h;
  auto join = [&](int k) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kGradLanes; ++i) t += sh[k][i][col];
    return t;
  };
  if (blockIdx.y < 4) {
    const uint32_t y = blockIdx.y;
    const bool one = y == 1 && P.dgate != nullptr && P.groups == 1, both = one && P.b_post != nullptr;
    void* out = y == 0 ? P.dw_pre : y == 1 ? P.dw_post : y == 2 ? P.db_pre : P.db_post;
    if (P.part == nullptr || (out == nullptr && !one)) return;
    const float* at = P.part + y * plane + c;
    sh[0][lane][col] = in ? strided_sum(at, lane, P.ctas, P.h) : 0.f;
    sh[1][lane][col] = in && both ? strided_sum(at + 2 * plane, lane, P.ctas, P.h) : 0.f;  // B beside A
    __syncthreads();
    if (lane != 0 || !in) return;
    const bool post = y == 1 || y == 3;
    const float s = join(0) * (post ? P.alpha : 1.f), g = post && P.groups == 1 ? __bfloat162float(P.gate[c]) : 1.f;
    put_grad(out, c, g * s, P.out_f32);
    if (one) {
      const float w = P.w_post ? __bfloat162float(P.w_post[c]) : 1.f, b = both ? __bfloat162float(P.b_post[c]) * P.alpha : 0.f;
      put_grad(P.dgate, c, fmaf(w, s, b * join(1)), P.out_f32);
    }
    return;
  }
  for (uint32_t g = blockIdx.y - 4; g < P.groups; g += gridDim.y - 4) {
    // workers w with rows [w M / W, (w + 1) M / W) that meet the group's rows
    const uint64_t g0 = static_cast<uint64_t>(g) * P.rows_per_gate, g1 = g0 + P.rows_per_gate;
    const uint32_t w0 = static_cast<uint32_t>(((g0 + 1) * P.workers - 1) / P.M);
    const uint32_t w1 = static_cast<uint32_t>((g1 * P.workers - 1) / P.M);
    if (w0 == w1) continue;  // written whole by its worker
    // the first worker holds the group in its second plane unless its rows
    // begin with it; the others' rows begin inside the group
    const bool starts = static_cast<uint64_t>(w0) * P.M / P.workers >= g0;
    const int64_t gplane = static_cast<int64_t>(P.workers) * P.h;
    float t = 0.f;
    if (in) {
      if (lane == 0) t = __ldcg(P.gpart + (starts ? 0 : gplane) + static_cast<int64_t>(w0) * P.h + c);
      t += strided_sum(P.gpart + c, w0 + (lane == 0 ? kGradLanes : lane), w1 + 1, P.h);
    }
    sh[0][lane][col] = t;
    __syncthreads();
    if (lane == 0 && in) put_grad(P.dgate, static_cast<int64_t>(g) * P.h + c, join(0), P.out_f32);
    __syncthreads();
  }
}

// ----------------------------------------------------------------- host

// How a row of nvec 8-column vectors is spread over threads.
struct Shape {
  int kind;     // WorkerKind
  int nv;       // vectors per thread
  int threads;  // of the CTA
};

// Rows of up to 1024 columns go to a warp, which needs no barrier for its
// sums; longer ones to a CTA with nv vectors a thread.
Shape shape_for(int64_t nvec, int nv) {
  if (nvec <= 64) return {BY_WARP, 2, 256};
  if (nvec <= 128) return {BY_WARP, 4, 256};
  return {BY_CTA, nv, static_cast<int>(cdiv(cdiv(nvec, nv), 32) * 32)};
}

constexpr int kSMs = 152;
constexpr size_t kSmemMost = 220 * 1024;  // dynamic shared memory of a CTA, beside the reduction buffers

using Kernel = void (*)(NormParams);

// Which coefficients (32 bytes a thread and vector) find room beside the row
// cells in `room` bytes.
int coefs_for(size_t cells, size_t one, size_t room, bool post, bool pre) {
  int c = 0;
  if (post && cells + one <= room) {
    c |= 1;
    cells += one;
  }
  if (pre && cells + one <= room) c |= 2;
  return c;
}
size_t coef_bytes(int c, size_t one) { return one * ((c & 1) + (c >> 1)); }

template <int NV, bool RES32, bool LN, bool GATE, int KIND, int MAXT>
tp_status run_fwd(const NormParams& P0, const Shape& sh, const DevInfo& di, cudaStream_t stream) {
  static KernelInfo info;
  Kernel k = block_norm_fwd_kernel<NV, RES32, LN, GATE, KIND, MAXT>;
  int regs = 0;
  TP_TRY(kernel_regs(reinterpret_cast<const void*>(k), &info, &regs));
  NormParams P = P0;
  const size_t one = static_cast<size_t>(sh.threads) * NV * 32;
  const size_t cells = static_cast<size_t>(sh.threads) * NV * ((RES32 ? 2 : 1) + 1 + (GATE ? 1 : 0)) * 16;
  P.coef = coefs_for(cells, one, kSmemMost, P.has_z, P.pre != NORM_NONE);
  const size_t smem = cells + coef_bytes(P.coef, one);
  const int per_sm = blocks_per_sm(sh.threads, regs, smem + 2 * kRed * sizeof(float));
  const int workers = KIND == BY_WARP ? sh.threads / 32 : 1;
  const int64_t grid = std::min<int64_t>(cdiv(P.M, workers), static_cast<int64_t>(di.sms) * per_sm);
  return launch_dependent(k, dim3(static_cast<unsigned>(grid)), static_cast<unsigned>(sh.threads), smem, stream, P);
}

template <bool RES32, bool LN, bool GATE>
tp_status pick_fwd(const NormParams& P, const DevInfo& di, cudaStream_t stream) {
  const Shape sh = shape_for(P.nvec, 4);
  if (sh.kind == BY_WARP) {
    return sh.nv == 2 ? run_fwd<2, RES32, LN, GATE, BY_WARP, 256>(P, sh, di, stream)
                      : run_fwd<4, RES32, LN, GATE, BY_WARP, 256>(P, sh, di, stream);
  }
  return run_fwd<4, RES32, LN, GATE, BY_CTA, 512>(P, sh, di, stream);
}

template <bool RES32>
tp_status dispatch_fwd(const NormParams& P, bool gate, const DevInfo& di, cudaStream_t stream) {
  const bool ln = P.post == NORM_LAYER || P.pre == NORM_LAYER;
  if (ln) return gate ? pick_fwd<RES32, true, true>(P, di, stream) : pick_fwd<RES32, true, false>(P, di, stream);
  return gate ? pick_fwd<RES32, false, true>(P, di, stream) : pick_fwd<RES32, false, false>(P, di, stream);
}

// CTAs of a cluster that share a row, in the backward pass: as many as keep
// the row at two vectors a thread of 256, whose column sums leave room in
// registers for two or three CTAs on an SM: the rows under way hide each
// other's reductions.  Measured at 12288 columns and 2048 rows, bf16 (302 MB,
// 45 us at the copy rate): one CTA a row with four vectors a thread, whose
// column sums spill, 91 us for both kernels; clusters of four, 73 us.  What is
// left over is the latency of a row's two barriers, with half of HBM's rate
// and 43 % of the issue slots in use.  (One vector a thread, tried at 1160
// columns: 31 us against 33, for twice the kernels.)
int bwd_cluster(int64_t nvec) { return nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4; }

// Every worker gets a row at least, since the owner of a row is found by
// dividing the rows evenly among the workers.
Shape bwd_shape(int64_t nvec, int64_t M) {
  const int c = bwd_cluster(nvec);
  if (c > 1) return {BY_CLUSTER, 2, static_cast<int>(cdiv(cdiv(cdiv(nvec, c), 2), 32) * 32)};
  Shape s = shape_for(nvec, 2);
  if (s.kind == BY_WARP) s.threads = static_cast<int>(32 * std::max<int64_t>(1, std::min<int64_t>(M, s.threads / 32)));
  return s;
}

int64_t bwd_workers(const Shape& sh) { return sh.kind == BY_WARP ? sh.threads / 32 : 1; }

// CTAs, or clusters of them, of a backward launch at most: the workspace is
// made for these; what the kernel's registers allow may be fewer.  Every CTA
// leaves its column sums, so that each gets a few rows where there are
// enough for all SMs.
int64_t bwd_ctas(const Shape& sh, int64_t nvec, int64_t M) {
  const int64_t rows = M / bwd_workers(sh), sms = kSMs / bwd_cluster(nvec);
  const int64_t most = sms * (sh.threads <= 128 ? 6 : sh.threads <= 192 ? 4 : 3);
  return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(rows, most), std::max<int64_t>(sms, rows / 3)));
}

tp_status check_norm(const tp_block_norm_desc* d, bool has_z, int64_t M, bool need_pre) {
  if (d == nullptr) return TP_ERR_INVALID_ARG;
  for (tp_norm k : {d->post, d->pre})
    if (k != TP_NORM_NONE && k != TP_NORM_RMS && k != TP_NORM_LAYER) return TP_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha)) return TP_ERR_INVALID_ARG;
  if (!has_z && (d->post != TP_NORM_NONE || d->gate != nullptr)) return TP_ERR_INVALID_ARG;
  if (need_pre != (d->pre != TP_NORM_NONE)) return TP_ERR_INVALID_ARG;
  if (d->post == TP_NORM_NONE && d->w_post != nullptr) return TP_ERR_INVALID_ARG;
  if (d->pre == TP_NORM_NONE && d->w_pre != nullptr) return TP_ERR_INVALID_ARG;
  if (d->post != TP_NORM_LAYER && d->b_post != nullptr) return TP_ERR_INVALID_ARG;
  if (d->pre != TP_NORM_LAYER && d->b_pre != nullptr) return TP_ERR_INVALID_ARG;
  for (const void* v : {d->w_post, d->b_post, d->w_pre, d->b_pre, d->gate})
    if (!aligned16(v)) return TP_ERR_ALIGNMENT;
  if (d->gate != nullptr) {
    if (d->gate_rows < 1) return TP_ERR_INVALID_ARG;
    if (M % d->gate_rows != 0) return TP_ERR_UNSUPPORTED_SHAPE;
  }
  return TP_OK;
}

tp_status check_extent(int p, int64_t M, int64_t h, tp_dtype res) {
  TP_TRY(check_sizes(p, M, h, 0, 0, res));
  if (h > TP_BLOCK_NORM_MAX_H || M % p != 0) return TP_ERR_UNSUPPORTED_SHAPE;
  return TP_OK;
}

void fill(NormParams* P, const tp_block_norm_desc* d, int p, int64_t M, int64_t h) {
  std::memset(P, 0, sizeof(*P));
  P->gate = static_cast<const uint4*>(d->gate);
  P->w_post = static_cast<const uint4*>(d->w_post);
  P->b_post = static_cast<const uint4*>(d->b_post);
  P->w_pre = static_cast<const uint4*>(d->w_pre);
  P->b_pre = static_cast<const uint4*>(d->b_pre);
  P->alpha = d->alpha;
  P->eps = d->eps;
  P->inv_h = 1.f / static_cast<float>(h);
  P->M = static_cast<uint32_t>(M);
  P->m = static_cast<uint32_t>(M / p);
  P->nvec = static_cast<uint32_t>(h / 8);
  P->rows_per_gate = static_cast<uint32_t>(d->gate != nullptr ? M / d->gate_rows : M);
  P->post = d->post;
  P->pre = d->pre;
}

// Ranges of the descriptor's vectors, which are inputs.
void add_desc(RangeList* in, const tp_block_norm_desc* d, int64_t h) {
  for (const void* v : {d->w_post, d->b_post, d->w_pre, d->b_pre}) in->push_back({v, v ? static_cast<size_t>(h) * 2 : 0});
  in->push_back({d->gate, d->gate ? static_cast<size_t>(d->gate_rows * h) * 2 : 0});
}

// Refuses overlaps, save that the shard out[s] may be the input shard same[s]
// itself, of `bytes` bytes: a row of it is written only after the same thread
// block has read it.  Other shards' rows, and the other inputs (`ins`), are
// read by blocks that do not wait for one another.
bool clash(const RangeList& outs, const RangeList& ins, const void* const* out, const void* const* same, int p,
           size_t bytes) {
  if (any_overlap(outs, ins)) return true;
  for (int s = 0; s < p && same != nullptr; ++s)
    for (const Range& o : outs) {
      const bool itself = out != nullptr && out[s] == same[s] && o.p == out[s];  // (outputs do not overlap)
      if (!itself && overlap(o, {same[s], bytes})) return true;
    }
  return false;
}

}  // namespace

namespace tpf {

tp_status resident_clusters(const void* kernel, int cluster, int threads, size_t smem, int* out) {
  static std::mutex lock;
  static std::map<std::tuple<int, const void*, int, int, size_t>, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const auto key = std::make_tuple(dev, kernel, cluster, threads, smem);
  std::lock_guard<std::mutex> hold(lock);
  const auto at = known.find(key);
  if (at != known.end()) {
    *out = at->second;
    return TP_OK;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return TP_ERR_CUDA;
  known[key] = n;
  *out = n;
  return TP_OK;
}

size_t block_norm_bwd_workspace(int64_t M, int64_t h) {
  const Shape sh = bwd_shape(cdiv(h, 8), M);
  const int64_t ctas = bwd_ctas(sh, cdiv(h, 8), M), workers = ctas * bwd_workers(sh);
  return kDataOffset + static_cast<size_t>(4 * ctas + 2 * workers) * h * sizeof(float);
}

}  // namespace tpf

extern "C" tp_status tp_block_norm_fwd(const void* const* x, const void* const* z, void* const* y, void* const* n,
                                       const tp_block_norm_desc* d, int p, int64_t M, int64_t h, tp_dtype res_dtype,
                                       cudaStream_t stream) {
  TP_TRY(check_extent(p, M, h, res_dtype));
  TP_TRY(check_norm(d, z != nullptr, M, n != nullptr));
  if ((z != nullptr) != (y != nullptr) || (z == nullptr && n == nullptr)) return TP_ERR_INVALID_ARG;
  const bool work = M > 0 && h > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(x, p, work));
  TP_TRY(check_ptrs(z, p, work && z != nullptr));
  TP_TRY(check_ptrs(in(y), p, work && y != nullptr));
  TP_TRY(check_ptrs(in(n), p, work && n != nullptr));
  if (!work) return TP_OK;
  {
    const size_t one = static_cast<size_t>(M / p * h);
    RangeList ins, outs;
    add_ranges(&ins, z, p, one * 2);
    add_desc(&ins, d, h);
    add_ranges(&outs, in(y), p, one * esize(res_dtype));
    add_ranges(&outs, in(n), p, one * 2);
    if (clash(outs, ins, in(y), x, p, one * esize(res_dtype))) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  NormParams P;
  fill(&P, d, p, M, h);
  P.has_z = z != nullptr;
  for (int s = 0; s < p; ++s) {
    P.x[s] = x[s];
    P.z[s] = z ? z[s] : nullptr;
    P.y[s] = y ? y[s] : nullptr;
    P.n[s] = n ? n[s] : nullptr;
  }
  const bool gate = d->gate != nullptr && d->gate_rows > 1;
  return res_dtype == TP_FP32 ? dispatch_fwd<true>(P, gate, di, stream) : dispatch_fwd<false>(P, gate, di, stream);
}

extern "C" tp_status tp_block_norm_bwd(const void* const* z, const void* const* y, const void* const* dn, const void* const* dy,
                                       void* const* dx, void* const* dz, const tp_block_norm_desc* d,
                                       const tp_block_norm_grads* grads, int p, int64_t M, int64_t h, tp_dtype res_dtype,
                                       tp_dtype out_dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  TP_TRY(check_extent(p, M, h, res_dtype));
  if (out_dtype != TP_BF16 && out_dtype != TP_FP32) return TP_ERR_INVALID_ARG;
  TP_TRY(check_norm(d, z != nullptr, M, dn != nullptr));
  const tp_block_norm_grads none = {};
  const tp_block_norm_grads g = grads != nullptr ? *grads : none;
  if (dn == nullptr && dy == nullptr) return TP_ERR_INVALID_ARG;
  if (dx == nullptr && dz == nullptr && !g.dw_post && !g.db_post && !g.dw_pre && !g.db_pre && !g.dgate) return TP_ERR_INVALID_ARG;
  if (z == nullptr && dz != nullptr) return TP_ERR_INVALID_ARG;
  // a gradient is asked for of a vector that the forward pass can have had
  // (a bias, and a weight of ones, need not be given for it)
  if ((g.dw_post && d->post == TP_NORM_NONE) || (g.db_post && d->post != TP_NORM_LAYER) ||
      (g.dw_pre && d->pre == TP_NORM_NONE) || (g.db_pre && d->pre != TP_NORM_LAYER) || (g.dgate && !d->gate))
    return TP_ERR_INVALID_ARG;
  for (const void* v : {g.dw_post, g.db_post, g.dw_pre, g.db_pre, g.dgate})
    if (!aligned16(v)) return TP_ERR_ALIGNMENT;
  const bool rows = M > 0 && h > 0;
  const auto in = [](void* const* a) { return const_cast<const void* const*>(a); };
  TP_TRY(check_ptrs(y, p, rows && dn != nullptr));
  TP_TRY(check_ptrs(z, p, rows && z != nullptr));
  TP_TRY(check_ptrs(dn, p, rows && dn != nullptr));
  TP_TRY(check_ptrs(dy, p, rows && dy != nullptr));
  TP_TRY(check_ptrs(in(dx), p, rows && dx != nullptr));
  TP_TRY(check_ptrs(in(dz), p, rows && dz != nullptr));
  TP_TRY(check_ws(ws, ws_bytes, block_norm_bwd_workspace(M, h)));
  if (h == 0) return TP_OK;
  {
    const size_t one = static_cast<size_t>(M / p * h), r = esize(res_dtype), o = esize(out_dtype);
    RangeList ins, outs;
    add_ranges(&ins, z, p, one * 2);
    if (dn != nullptr) add_ranges(&ins, y, p, one * r);
    add_ranges(&ins, dn, p, one * 2);
    add_desc(&ins, d, h);
    add_ranges(&outs, in(dx), p, one * r);
    add_ranges(&outs, in(dz), p, one * 2);
    for (void* v : {g.dw_post, g.db_post, g.dw_pre, g.db_pre}) outs.push_back({v, v ? static_cast<size_t>(h) * o : 0});
    outs.push_back({g.dgate, g.dgate ? static_cast<size_t>(d->gate_rows * h) * o : 0});
    outs.push_back({ws, ws_bytes});
    if (clash(outs, ins, in(dx), dy, p, one * r)) return TP_ERR_INVALID_ARG;
  }
  DevInfo di;
  TP_TRY(device_info(&di));
  if (M == 0) {  // sums over no rows
    for (void* v : {g.dw_post, g.db_post, g.dw_pre, g.db_pre})
      if (v != nullptr && cudaMemsetAsync(v, 0, static_cast<size_t>(h) * esize(out_dtype), stream) != cudaSuccess)
        return TP_ERR_CUDA;
    if (g.dgate != nullptr &&
        cudaMemsetAsync(g.dgate, 0, static_cast<size_t>(d->gate_rows * h) * esize(out_dtype), stream) != cudaSuccess)
      return TP_ERR_CUDA;
    return TP_OK;
  }
  NormParams P;
  fill(&P, d, p, M, h);
  P.has_z = z != nullptr;
  P.has_dn = dn != nullptr;
  P.has_dy = dy != nullptr;
  P.out_f32 = out_dtype == TP_FP32;
  for (int s = 0; s < p; ++s) {
    P.x[s] = dn ? y[s] : nullptr;
    P.z[s] = z ? z[s] : nullptr;
    P.dn[s] = dn ? dn[s] : nullptr;
    P.dy[s] = dy ? dy[s] : nullptr;
    P.y[s] = dx ? dx[s] : nullptr;
    P.n[s] = dz ? dz[s] : nullptr;
  }
  const Shape sh = bwd_shape(P.nvec, M);
  const bool groups = d->gate != nullptr && d->gate_rows > 1;
  const bool ln = d->post == TP_NORM_LAYER || d->pre == TP_NORM_LAYER;
  const int64_t ctas = bwd_ctas(sh, P.nvec, M);
  float* area = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kDataOffset);
  const bool sums = g.dw_post || g.db_post || g.dw_pre || g.db_pre || (g.dgate && !groups);
  P.part = sums ? area : nullptr;
  P.gpart = g.dgate && groups ? area + 4 * ctas * h : nullptr;
  P.dgate = g.dgate;
  const size_t one = static_cast<size_t>(sh.threads) * sh.nv * 32;
  const size_t cells = static_cast<size_t>(2 * sh.threads) * sh.nv * (2 * (res_dtype == TP_FP32 ? 2 : 1) + 2 + (groups ? 1 : 0)) * 16;
  P.coef = coefs_for(cells, one, kSmemMost / bwd_blocks(sh.nv, sh.threads, groups || ln), P.has_z, P.has_dn);
  NormBwdLaunch L = {sh.kind, sh.nv, sh.threads, sh.kind == BY_CLUSTER ? bwd_cluster(P.nvec) : 1, static_cast<int>(ctas), cells + coef_bytes(P.coef, one), groups,
                     P.has_dn && P.has_dy && P.has_z && P.coef == 3 && dx != nullptr && dz != nullptr};
  if (res_dtype == TP_FP32) TP_TRY(ln ? block_norm_bwd_run_f32_ln(P, L, stream) : block_norm_bwd_run_f32_rms(P, L, stream));
  else TP_TRY(ln ? block_norm_bwd_run_bf16_ln(P, L, stream) : block_norm_bwd_run_bf16_rms(P, L, stream));
  // gate rows that one worker holds whole are written already: with a row
  // per token that is all of them
  const bool joins = P.gpart != nullptr && P.rows_per_gate > 1;
  if (!sums && !joins) return TP_OK;
  NormGradParams G;
  std::memset(&G, 0, sizeof(G));
  G.part = P.part;
  G.gpart = P.gpart;
  G.gate = static_cast<const __nv_bfloat16*>(groups ? nullptr : d->gate);
  G.w_post = static_cast<const __nv_bfloat16*>(d->w_post);
  G.b_post = static_cast<const __nv_bfloat16*>(d->b_post);
  G.alpha = d->alpha;
  G.dw_pre = g.dw_pre;
  G.db_pre = g.db_pre;
  G.dw_post = g.dw_post;
  G.db_post = g.db_post;
  G.dgate = groups && !joins ? nullptr : g.dgate;
  G.h = static_cast<uint32_t>(h);
  G.ctas = static_cast<uint32_t>(L.ctas);
  G.workers = static_cast<uint32_t>(L.ctas * bwd_workers(sh));
  G.M = static_cast<uint32_t>(M);
  G.rows_per_gate = P.rows_per_gate;
  G.groups = static_cast<uint32_t>(d->gate != nullptr ? d->gate_rows : 0);
  G.out_f32 = P.out_f32;
  const unsigned ny = 4u + (joins ? static_cast<unsigned>(std::min<int64_t>(d->gate_rows, 64)) : 0u);
  return launch_dependent(block_norm_grad_kernel, dim3(static_cast<unsigned>(cdiv(h, 32)), ny), 32u * kGradLanes, 0, stream, G);
}
