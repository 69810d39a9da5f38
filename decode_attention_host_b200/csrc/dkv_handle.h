// dkv_handle.h -- what the entry points share: the handle, the caller's device
// guard, the CUDA error path, the pool pointer checks and the merge launch.
#pragma once

#include <cuda_runtime.h>

#include <string>
#include <vector>

#include "dkv.h"
#include "dkv_error.h"
#include "dkv_kernels.cuh"

namespace dkv {

inline int cuda_fail(cudaError_t e, const char* what) {
  return set_error(DKV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

#define DKV_CUDA(call)                                       \
  do {                                                       \
    cudaError_t e_ = (call);                                 \
    if (e_ != cudaSuccess) return dkv::cuda_fail(e_, #call); \
  } while (0)

// Restores the caller's current device on scope exit.
struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess) ok = prev == dev || cudaSetDevice(dev) == cudaSuccess;
    if (prev == dev) prev = -1;   // nothing to restore
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// work counters of a handle (see dkv_handle::work)
constexpr int kWorkWindow = 4;
constexpr int kWorkTables = 6;
constexpr int kWorkWords = 8;

using SplitFn = void (*)(dim3, size_t, cudaStream_t, const SplitParams&, const TileMaps&);
using SplitKernelPtr = const void*;

struct SplitEntry {
  SplitFn fn;
  SplitKernelPtr ptr;
};

// The merge, optionally as a programmatic dependent launch of the split kernel
// just before it on the stream: its grid is set up while that kernel drains
// and its first instruction waits for that kernel's results.
using MergeFn = cudaError_t (*)(int, cudaStream_t, const MergeParams&, bool);
template <int D>
cudaError_t launch_merge(int rows, cudaStream_t s, const MergeParams& p, bool dependent) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(rows);
  cfg.blockDim = dim3(32 * merge_warps(p.nslots, D));
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, p);
}

}  // namespace dkv

struct dkv_handle {
  dkv_config cfg{};
  int G = 0;
  int sm_count = 0;
  int beside_host = 0;        // HBM-kernel CTAs that fit on an SM beside a host-kernel CTA (0 or 1)
  int units_target = 0;       // warps of the widest split launch (one resident wave: 2 CTAs per SM)
  size_t part_rows = 0;
  float qscale = 0.f;
  int host_ctas = 0;           // the configuration's count; 0: chosen per call
  float* part_o = nullptr;
  float* part_lse = nullptr;
  int32_t* status = nullptr;
  int32_t* work = nullptr;    // [kWorkWords]: work counters of the host-side, device-side and windowed split
                              // launches (2 each), CTAs finished of the table launch; zero between launches
  int2* lists = nullptr;      // [max_batch][max_blocks_per_seq]: per-pool block lists of a mixed call
  int2* counts = nullptr;     // [max_batch]
  double* inv_freq = nullptr; // [D/2] frequencies, then [D/2] uint64 turns per position (2^-64 turns)
  cudaStream_t aux = nullptr;
  cudaEvent_t ev_fork = nullptr;
  cudaEvent_t ev_join = nullptr;
  // dev: cp.async; dev_tma: tensor copies
  dkv::SplitEntry host_kernel{}, dev_kernel{}, dev_tma_kernel{}, multi_kernel{};
  dkv::SplitEntry window_kernel{};
  int window_ctas = 0;         // CTAs of the windowed kernel that one wave holds
  // tensor maps of the last device pool and staging pool the HBM kernel read
  struct PoolMaps {
    const void* k = nullptr;
    const void* v = nullptr;
    long long rows = -1;
    dkv::TileMaps maps{};
  } dev_maps, stage_maps, host_maps;
  dkv::MergeFn merge = nullptr;
  const void* ok_host[2] = {nullptr, nullptr};
  const void* ok_dev[4] = {nullptr, nullptr, nullptr, nullptr};
  int last_launches = 0;
  // per-kernel event pairs while profiling: [kernel][call] -> (start, stop)
  int prof_capacity = 0;
  int prof_used[3] = {0, 0, 0};
  std::vector<cudaEvent_t> prof_events[3];
};

namespace dkv {

inline int check_host_pool(dkv_handle* h, const void* p, int which) {
  if (h->ok_host[which] == p) return DKV_OK;
  cudaPointerAttributes a{};
  cudaError_t e = cudaPointerGetAttributes(&a, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(DKV_ERR_INVALID_ARG, "host pool pointer is not known to CUDA (use dkv_host_pool_alloc)");
  }
  if (a.type != cudaMemoryTypeHost || a.devicePointer == nullptr || a.devicePointer != p)
    return set_error(DKV_ERR_INVALID_ARG, "host pool must be mapped pinned host memory passed by its device alias");
  h->ok_host[which] = p;
  return DKV_OK;
}

inline int check_dev_pool(dkv_handle* h, const void* p, int which) {
  if (h->ok_dev[which] == p) return DKV_OK;
  cudaPointerAttributes a{};
  cudaError_t e = cudaPointerGetAttributes(&a, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(DKV_ERR_INVALID_ARG, "device pool pointer is not known to CUDA");
  }
  if (!((a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) && a.device == h->cfg.device))
    return set_error(DKV_ERR_INVALID_ARG, "device pool must be device memory of the handle's GPU");
  h->ok_dev[which] = p;
  return DKV_OK;
}

// Whether dkv_debug_stall_copy is armed on this thread; disarms it.
bool take_stall_copy();

// Picks and prepares the kernels of the serving entry points for h (dkv_serve.cu);
// the caller has made h's device current.
cudaError_t prepare_serving(dkv_handle* h);

}  // namespace dkv
