// Residual RMS norm: requests and the layout rules that host code and kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wbmm {

constexpr int kNormWaveLen = 64 * 3 * 8;    // longest row (inner = 1) that a wave's registers hold

struct NormRequest {
  int64_t outer, len, inner;      // the norm runs over len, for every (outer, inner)
  int bf16, fmt;
  float eps;
  const void* x;                  // forward: x; backward: s, the sum that was normed
  const void* res;                // forward: the residual, or null; backward: ds, or null
  const float* w;                 // [len] or null (ones)
  const void* dy;
  void* s;                        // forward: x + res, or null
  void* y;                        // forward: y; backward: dx, or null
  uint8_t* codes;                 // of y, or null
  uint8_t* scales;
  float* dw;                      // backward: [len] or null
  void* ws;
};

size_t norm_backward_workspace(int64_t outer, int64_t len, int64_t inner);
hipError_t launch_norm_forward(const NormRequest& r, hipStream_t st);
hipError_t launch_norm_backward(const NormRequest& r, hipStream_t st);

}  // namespace wbmm
