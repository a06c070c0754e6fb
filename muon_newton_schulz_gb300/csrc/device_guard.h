// Makes a device current for the length of a scope.
#pragma once

#include <cuda_runtime.h>

namespace muon {

struct DeviceGuard {
  int old = -1;
  bool changed = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&old) == cudaSuccess && old != dev) changed = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (changed) cudaSetDevice(old);
  }
};

}  // namespace muon
