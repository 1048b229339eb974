// api_util.h - helpers the ABI files share: device allocation, alignment and
// the device a handle is bound to.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>

#include "dyra.h"
#include "internal.h"

namespace dyra {

inline size_t elem_size(dyra_dtype_t t) { return t == DYRA_F32 ? 4 : 2; }

inline bool fail_alloc_for_test() {
  const char* e = std::getenv("DYRA_TEST_FAIL_ALLOC");
  return e != nullptr && e[0] == '1';
}

inline int dev_alloc(void** p, size_t bytes) {
  if (fail_alloc_for_test()) return DYRA_ERR_ALLOC;
  if (cudaMalloc(p, bytes) != cudaSuccess) {
    cudaGetLastError();
    *p = nullptr;
    return DYRA_ERR_ALLOC;
  }
  return DYRA_OK;
}

inline void dev_free(void*& p) {
  if (p) cudaFree(p);
  p = nullptr;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Run on the handle's device, restoring the caller's device afterwards.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      ok = false;
      return;
    }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

// The current device's attributes (each a lookup of microseconds, where the
// whole property structure takes milliseconds); DYRA_ERR_UNSUPPORTED unless it
// is a B200.
inline int current_device_info(DeviceInfo* info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DYRA_ERR_CUDA;
  }
  int v[6];
  const cudaDeviceAttr attr[6] = {
      cudaDevAttrMultiProcessorCount,       cudaDevAttrMaxSharedMemoryPerBlockOptin,
      cudaDevAttrMaxSharedMemoryPerMultiprocessor, cudaDevAttrReservedSharedMemoryPerBlock,
      cudaDevAttrComputeCapabilityMajor,    cudaDevAttrComputeCapabilityMinor};
  for (int i = 0; i < 6; ++i)
    if (cudaDeviceGetAttribute(&v[i], attr[i], dev) != cudaSuccess) {
      cudaGetLastError();
      return DYRA_ERR_CUDA;
    }
  if (v[4] != 10 || v[5] != 0) return DYRA_ERR_UNSUPPORTED;
  info->device = dev;
  info->sm_count = v[0];
  info->max_smem_optin = v[1];
  info->smem_per_sm = v[2];
  info->smem_reserved = v[3];
  info->cc_major = v[4];
  info->cc_minor = v[5];
  return DYRA_OK;
}

}  // namespace dyra
