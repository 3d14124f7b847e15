// abi_common.h -- host checks shared by the exported C entry points (abi.cu, abi_serving.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "devcache.h"
#include "trellis.h"

namespace trellis {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device must be compute capability 10.3 (the library holds
// sm_103a code only).  Cached per device.
inline int device_ok() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
    cudaGetLastError();
    return TRELLIS_EDEVICE;
  }
  static PerDevice<int> ok_of;
  const auto probe = [dev] {
    int major = 0, minor = 0;
    const bool ok = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
                    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) == cudaSuccess &&
                    major == 10 && minor == 3;
    if (!ok) cudaGetLastError();
    return ok ? TRELLIS_OK : TRELLIS_EDEVICE;
  };
  return dev < kMaxDevices ? ok_of.get(dev, probe, TRELLIS_EDEVICE) : probe();
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ECUDA; }

}  // namespace trellis
