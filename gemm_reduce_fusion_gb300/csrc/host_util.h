// Host-side helpers shared by the translation units of the C ABI: the device
// query, argument checks and small arithmetic.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <vector>

#include "../../include/tp_fused.h"

namespace tpf {

constexpr int kMaxP = 8;
constexpr size_t kStatusBytes = 256;     // workspace head: status word, padded
// Behind it the counters of a sliced last wave (tp_fused.cu), at most.  What
// the calls around the sharded Linear keep in a workspace begins after them.
constexpr size_t kSliceCounterBytes = 9728;
constexpr size_t kDataOffset = kStatusBytes + kSliceCounterBytes;

// Limit of a kernel's wait on an mbarrier (tp_fused.cu).
uint64_t device_timeout_ns();
// Stage that a kernel is told never to hand over, or -1 (TP_DEBUG_DROP_LOAD).
int64_t debug_drop();

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t esize(tp_dtype d) { return d == TP_FP32 ? 4 : 2; }

struct DevInfo {
  int sms = 0;
  bool ok = false;
};

// The calling thread's current device, with that device's primary context
// made current on the thread.  A thread that has not yet made a CUDA call of
// its own (an autograd worker thread, a user's thread) may have no current
// context, and tensor-map encoding and launches from it then fail;
// cudaSetDevice binds the primary context.
inline tp_status bind_device(int* dev) {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) return TP_ERR_CUDA;
  if (cudaSetDevice(d) != cudaSuccess) return TP_ERR_CUDA;
  *dev = d;
  return TP_OK;
}

inline tp_status device_info(DevInfo* out) {
  int dev = 0;
  if (bind_device(&dev) != TP_OK) return TP_ERR_CUDA;
  // SM count of each device seen (0: not yet queried; -1: not an sm_103 device)
  static std::atomic<int> sm_count[64] = {};
  if (dev >= 0 && dev < 64) {
    const int c = sm_count[dev].load(std::memory_order_relaxed);
    if (c > 0) {
      out->sms = c;
      out->ok = true;
      return TP_OK;
    }
    if (c < 0) return TP_ERR_ARCH;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return TP_ERR_CUDA;
  if (major != 10 || minor != 3) {
    if (dev >= 0 && dev < 64) sm_count[dev].store(-1, std::memory_order_relaxed);
    return TP_ERR_ARCH;
  }
  if (dev >= 0 && dev < 64 && sms > 0) sm_count[dev].store(sms, std::memory_order_relaxed);
  out->sms = sms;
  out->ok = true;
  return TP_OK;
}

// ------------------------------------------------------------------ validation

struct Range {
  const void* p;
  size_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// A call's ranges without a heap allocation (calls that serve single tokens
// take a few microseconds): at most 8 shards of a few tensors each.  A list
// that was given more overlaps everything.
class RangeList {
 public:
  void push_back(const Range& r) {
    if (r.bytes == 0) return;
    if (n_ < kMost) r_[n_++] = r;
    else full_ = true;
  }
  bool full() const { return full_; }
  size_t size() const { return n_; }
  const Range& operator[](size_t i) const { return r_[i]; }
  const Range* begin() const { return r_; }
  const Range* end() const { return r_ + n_; }

 private:
  static constexpr size_t kMost = 64;
  size_t n_ = 0;
  bool full_ = false;
  Range r_[kMost];
};

inline bool holds_all(const RangeList& r) { return !r.full(); }
inline bool holds_all(const std::vector<Range>&) { return true; }

template <typename Outs, typename Ins>
bool any_overlap(const Outs& outs, const Ins& ins) {
  if (!holds_all(outs) || !holds_all(ins)) return true;
  for (size_t i = 0; i < outs.size(); ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return true;
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

inline tp_status check_sizes(int p, int64_t M, int64_t N, int64_t K, int64_t chunk_m, tp_dtype dt) {
  if (p < 1 || p > kMaxP) return TP_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || chunk_m < 0) return TP_ERR_INVALID_ARG;
  if (dt != TP_BF16 && dt != TP_FP32) return TP_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (M > lim || N > lim || K > lim || static_cast<int64_t>(p) * K > lim) return TP_ERR_UNSUPPORTED_SHAPE;
  if (N % 8 != 0 || K % 8 != 0) return TP_ERR_ALIGNMENT;
  return TP_OK;
}

inline tp_status check_ptrs(const void* const* a, int n, bool need) {
  if (!need) return TP_OK;
  if (a == nullptr) return TP_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (a[i] == nullptr) return TP_ERR_INVALID_ARG;
    if (!aligned16(a[i])) return TP_ERR_ALIGNMENT;
  }
  return TP_OK;
}

inline tp_status check_ptr(const void* a, bool need) {
  if (!need) return TP_OK;
  if (a == nullptr) return TP_ERR_INVALID_ARG;
  return aligned16(a) ? TP_OK : TP_ERR_ALIGNMENT;
}

inline tp_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return TP_ERR_INVALID_ARG;
  if (!aligned16(ws)) return TP_ERR_ALIGNMENT;
  if (ws_bytes < need) return TP_ERR_WORKSPACE_TOO_SMALL;
  return TP_OK;
}

#define TP_TRY(expr)                     \
  do {                                   \
    tp_status _st = (expr);              \
    if (_st != TP_OK) return _st;        \
  } while (0)

template <typename List>
void add_ranges(List* v, const void* const* a, int n, size_t bytes) {
  if (a == nullptr) return;
  for (int i = 0; i < n; ++i)
    if (a[i] != nullptr) v->push_back({a[i], bytes});
}

// Launches `k` as a programmatic dependent of the stream's previous kernel:
// its blocks may be scheduled while that one drains, and wait
// (griddepcontrol.wait) for its completion before they touch memory.
template <typename Params>
inline tp_status launch_dependent(void (*k)(Params), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                                  const Params& params, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, params) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

// What a kernel can use of an SM, read once per device and kernel: `cache`
// is the kernel's own.  Also raises its shared-memory limit.
struct KernelInfo {
  std::atomic<int> regs[64] = {};
};
inline tp_status kernel_regs(const void* k, KernelInfo* cache, int* regs) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  int r = dev < 64 ? cache->regs[dev].load(std::memory_order_acquire) : 0;
  if (r == 0) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, k) != cudaSuccess) return TP_ERR_CUDA;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - static_cast<int>(a.sharedSizeBytes)) != cudaSuccess)
      return TP_ERR_CUDA;
    r = a.numRegs;
    if (dev < 64) cache->regs[dev].store(r, std::memory_order_release);
  }
  *regs = r;
  return TP_OK;
}

// Blocks of `threads` threads, `regs` registers a thread and `smem` bytes
// that fit on an SM at a time (registers are given out in units of 8 a
// thread, shared memory with 1 KiB a block on top).
inline int blocks_per_sm(int threads, int regs, size_t smem) {
  const int by_regs = 65536 / (((regs + 7) / 8 * 8) * threads);
  const int by_smem = static_cast<int>((228 * 1024) / (smem + 1024));
  int n = by_regs < by_smem ? by_regs : by_smem;
  if (n > 2048 / threads) n = 2048 / threads;
  return n < 1 ? 1 : n;
}

}  // namespace tpf
