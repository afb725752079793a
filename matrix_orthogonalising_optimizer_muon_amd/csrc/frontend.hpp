// Host helpers shared by the C-ABI front ends (api.cpp, train_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

struct muon_ctx;

namespace muon {

#define MUON_HIP(call)                       \
  do {                                       \
    if ((call) != hipSuccess) return MUON_ERR_HIP; \
  } while (0)
int ctx_device(const muon_ctx* ctx);  // -1: host-only
int ctx_cus(const muon_ctx* ctx);
struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    ok = hipGetDevice(&prev) == hipSuccess && (prev == dev || hipSetDevice(dev) == hipSuccess);
    if (prev == dev) prev = -1;  // nothing to restore
  }
  ~DeviceGuard() {
    if (prev >= 0) (void)hipSetDevice(prev);
  }
};

}  // namespace muon
