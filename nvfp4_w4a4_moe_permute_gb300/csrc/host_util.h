// Host-side helpers shared by the entry points of the minite library.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace minite {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Streaming multiprocessors of the current device (queried once per device).
int num_sms();

// Budget of the GEMM's bounded pipeline waits, in nanoseconds.
uint64_t wait_budget_ns();

// The driver's tensor map encoder (looked up once), null when there is none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Token-chunk size of the permutation for top-k = k (pairs per chunk <= 512).
inline int permute_chunk_tokens(int k) {
  int ct = 512 / (k > 0 ? k : 1);
  return ct < 1 ? 1 : ct;
}

// Allow `kernel` dynamic shared memory of `bytes`, once on each device (the
// attribute belongs to one): `devices` is the call site's own, a bit a device.
inline cudaError_t allow_smem(std::atomic<uint64_t>& devices, const void* kernel, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (devices.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) devices.fetch_or(bit);
  return e;
}
template <typename... KArgs>
inline cudaError_t allow_smem(std::atomic<uint64_t>& devices, void (*kernel)(KArgs...), size_t bytes) {
  return allow_smem(devices, reinterpret_cast<const void*>(kernel), bytes);
}

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel on the stream finishes; it must call pdl_wait() before
// touching global memory (every kernel launched this way does).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Clusters of two CTAs of `kernel` that can be resident at once on the current
// device (queried once per device and Tag; kernels of one type share a type, so
// a tag names one kernel and launch shape).
template <int Tag, typename Kernel>
inline int resident_pairs(Kernel kernel, int threads, size_t smem) {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int v = cache[dev].load();
  if (v > 0) return v;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(num_sms() / 2));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return 0;
  if (n > num_sms() / 2) n = num_sms() / 2;
  cache[dev].store(n);
  return n;
}

// Launch `pairs` clusters of two CTAs with programmatic stream serialization.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pair_pdl(void (*kernel)(KArgs...), int pairs, int threads, size_t smem,
                                   cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace minite
