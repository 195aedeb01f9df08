// decode_internal.cuh -- shared by the translation units of the decode-step
// operators (kv_cache.cu, attn_decode.cu, sample.cu).
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/moe_route.h"

namespace moe {

// bytes of one cached element
__host__ __device__ constexpr int kv_esize(int kv_dtype) {
  return kv_dtype == MOE_KV_F32 ? 4 : kv_dtype == MOE_KV_BF16 ? 2 : 1;
}

// whether n vectors of dim elements, a stride apart, leave room for each other
constexpr bool apart(int n, long long stride, int dim) { return n < 2 || stride >= dim; }

// what head_dim is a multiple of
constexpr int kv_dim_step(int kv_dtype) { return kv_dtype == MOE_KV_E4M3 ? 16 : 8; }

// MOE_OK if the cache descriptor meets the header's requirements
int kv_cache_ok(const moe_kv_cache_t* c);

// SMs of the current device, asked once per device; 0 on an error
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Allow `kern` up to `bytes` of dynamic shared memory on the current device,
// asking the runtime once per device (a microsecond a call otherwise).
// `done`: the caller's static, a bit per device, for one kernel and its
// largest size.
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch `kern` in clusters of `cluster` CTAs (1: none) such that it may
// overlap its predecessor's tail in the stream; the kernel calls pdl_wait()
// before it touches anything the predecessor writes or reads.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, int cluster,
                                  size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace moe
