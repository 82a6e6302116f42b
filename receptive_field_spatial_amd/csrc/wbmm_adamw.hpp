// AdamW over many tensors: the request, and the table that a plan is.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wbmm {

constexpr int64_t kAdamChunk = 4096;   // elements of a workgroup, within one tensor

// Bits of AdamEntry::flags.
enum { kAdamG16 = 1, kAdam8 = 2, kAdamWide = 4 };

// A plan: an AdamHead, `count` entries, then one uint32 per chunk, the chunk's tensor.
struct AdamHead {
  uint64_t magic, count, chunks, pad;
};
struct AdamEntry {
  float* p;
  const void* g;
  void* m;             // fp32, or codes
  void* v;             // fp32: the second moment; codes: of its root
  uint8_t* ms;         // scales of the codes
  uint8_t* vs;
  uint16_t* copy;
  int64_t n;
  double decay;        // weight decay
  uint32_t first;      // chunk
  uint32_t flags;
};
constexpr uint64_t kAdamMagic = 0x3157414d4d425731ull;

struct AdamRequest {
  const void* table;
  uint32_t chunks, count;
  double lr, beta1, beta2, eps;
  int64_t step;
  const int32_t* step_dev;
  const float* lr_factor;
  const float* grad_factor;
  uint64_t seed;
};

hipError_t launch_adamw(const AdamRequest& r, hipStream_t st);

}  // namespace wbmm
