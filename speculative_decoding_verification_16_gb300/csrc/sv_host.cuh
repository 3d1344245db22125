// sv_host.cuh -- host helpers of the serving operators (include/spec_verify_serve.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "spec_verify_serve.h"

namespace sv {
namespace serve {

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A device pointer that may be NULL but, if given, is aligned.
inline bool null_or_aligned(const void* p, size_t a) { return p == nullptr || aligned_to(p, a); }

// Division of 0 <= n < 2^31 by a fixed d: n / d = (mulhi(n, mul) + n) >> shift with
// mul = 2^32 (2^shift - d) / d + 1, 2^shift >= d (Granlund and Montgomery 1994).
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv by(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t{1} << s) < d) ++s;
    return FastDiv{static_cast<uint32_t>((((uint64_t{1} << s) - d) << 32) / d + 1), s};
  }
  __device__ __forceinline__ int of(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

struct Device {
  int sms = 0;
  int max_smem = 0;
};

// The current device's SM count and opt-in shared memory, read once a device.
int device(Device* out);

// Raises the kernel's dynamic shared memory limit to the device's maximum,
// once per kernel and device; kernels that stay below 48 KB need no call.
int allow_smem(const void* kernel, int max_smem);

// One launch.  cluster > 1: in clusters of that many CTAs.  dependent: as a
// programmatic dependent of the previous launch on the stream (the kernel
// waits in grid_dep_wait before it reads what that one writes).
template <typename K, typename... A>
int launch(K kernel, dim3 grid, int threads, int smem, int cluster, bool dependent,
           cudaStream_t stream, const A&... args) {
  if (smem > 48 * 1024) {
    Device d;
    int rc = device(&d);
    if (rc == SV_OK) rc = allow_smem(reinterpret_cast<const void*>(kernel), d.max_smem);
    if (rc != SV_OK) return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(n);
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace serve
}  // namespace sv
