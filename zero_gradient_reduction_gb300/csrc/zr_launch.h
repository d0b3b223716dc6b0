// Host-side helpers around a kernel launch.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "zr_internal.h"

namespace zr {

constexpr int kSmemMost = 227 * 1024;  // dynamic shared memory that one block may have

inline bool dtype_ok(zr_dtype d) { return d == ZR_F16 || d == ZR_BF16 || d == ZR_F32; }

inline zr_status launch_status(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  return ZR_OK;
}

// Lets a kernel use more dynamic shared memory than a launch gives by itself. That is an
// attribute of the kernel on a device: it is set at the first call on each device.
class SmemAllowance {
 public:
  zr_status allow(const char* what, const void* kernel, int bytes) {
    if (bytes <= 48 * 1024) return ZR_OK;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e == cudaSuccess && (done_.load(std::memory_order_relaxed) & bit)) return ZR_OK;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    done_.fetch_or(bit, std::memory_order_relaxed);
    return ZR_OK;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// A launch of blocks, or clusters of them. `early`: it may begin while the launch before it in the stream
// still runs, where that one lets it; the kernel waits for that one's end before it reads or writes
// what another may write or read. That hides the 1 us of a launch in a chain of short ones.
template <class Kernel, class... Args>
cudaError_t launch(Kernel kernel, int64_t blocks, int threads, int smem, int cluster, bool early, cudaStream_t s,
                   const Args&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (early) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  c.attrs = at;
  c.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// Streaming multiprocessors of the current device (0 and a recorded error on failure).
inline int sm_count(const char* what) {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (n = known[dev & 63].load(std::memory_order_relaxed))) return n;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    fail(ZR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return 0;
  }
  known[dev & 63].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace zr
