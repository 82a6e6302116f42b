// 8-bit activation checkpoints, device side: the formats and their decoding.
//
// A tensor of n elements is kept as n code bytes and ceil(n / 32) scale bytes, one per group of 32
// elements in memory order:
//   value = q(code) * 2^(byte - 127),   byte 255: NaN,
// with q(code) the int8 value or the OCP e4m3 value. The scale is a power of two, so scaling is
// exact both ways: the only rounding of a checkpoint is the code's (half a step of the group's
// largest value's grid), a decoded value has at most 8 significant bits, and it is exact in bf16.
#pragma once

#include "wbmm_device.hpp"

namespace wbmm {

constexpr int kCkptGroup = 32;
enum CkptFmt { kFmtInt8 = 0, kFmtE4M3 = 1 };

// 2^(byte - 127) as fp32, NaN for byte 255. Byte 0 is a subnormal number.
__device__ __forceinline__ float ckpt_factor(uint32_t byte) {
  uint32_t b = byte << 23;
  b = byte == 0 ? 0x00400000u : b;
  b = byte == 255 ? 0x7fc00000u : b;
  return __uint_as_float(b);
}

// The four codes of a dword as fp32 values, unscaled.
__device__ __forceinline__ void ckpt_decode4(uint32_t w, int fmt, float (&v)[4]) {
  if (fmt == kFmtInt8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(w >> (8 * j));
  } else {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
  }
}
__device__ __forceinline__ float ckpt_decode1(uint32_t code, int fmt) {
  return fmt == kFmtInt8 ? (float)(int8_t)code : __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

}  // namespace wbmm
