// One AdamW step over all tensors of a plan, in one launch.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// States in 8 bits are m and r = sqrt(v), each as e4m3 codes with a power-of-two scale per 32
// elements (the checkpoints' format). The root halves v's range in octaves: a group holds roots down
// to 2^-17 of its largest, elements whose gradients differ by five orders of magnitude. Codes are
// rounded up or down at random, to the value itself on average: at b2 = 0.999 a step moves r by up
// to 0.05 %, a sixtieth of half a step of the codes, and rounding to the nearest would hold r
// where it is for ever. A root above zero keeps at least the least code, or its element's next step
// would be divided by eps. The step itself is taken with m and v as computed, before they are rounded.
//
// Random words: Philox 4x32 with 7 rounds (Salmon et al., "Parallel random numbers: as easy as 1,
// 2, 3", 2011), counter (index / 4, tensor, step), key the seed; word index % 4 gives an element its
// 16 bits for m (low) and for r (high). The same seed and step give the same result.
//
// Bound by memory: 28 bytes an element with fp32 states and gradients, 16.1 with 8-bit ones. A
// workgroup takes 4096 elements of one tensor, a thread twice 8 neighbouring ones; four lanes hold a
// group of 32. Measured: 52.5 M parameters with fp32 states 262 us (5.6 TB/s, part of it from the
// last-level cache), with 8-bit ones, bf16 gradients and a bf16 copy 172 (4.9 TB/s); 0.44 M 6.2 us.
// Sums, products and quotients are rounded one by one (no fused multiply-add), so that
// a result does not depend on how the compiler pairs them: a code may hang on a last bit.
#pragma clang fp contract(off)
#include "wbmm_adamw.hpp"
#include "wbmm_ckpt.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

constexpr int kE = 8;                                        // elements of a lane's piece
constexpr int kTile = kThreads * kE;                         // of a workgroup's
static_assert(kAdamChunk % kTile == 0 && kTile % kCkptGroup == 0, "whole pieces and groups");

struct AdamArgs {
  const unsigned char* table;
  const int32_t* step_dev;
  const float* lr_factor;
  const float* grad_factor;
  double lr, beta1, beta2;
  float b1, c1, b2, c2, eps;
  float k1, k2;            // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), without step_dev and lr_factor
  uint32_t step, chunks, count;
  uint32_t key0, key1;
};

struct Scalars {
  float k1, k2, keep, gf;
  uint32_t step;
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ k0, n2 = (uint32_t)(a >> 32) ^ c[3] ^ k1;
    c[0] = n0;
    c[1] = (uint32_t)b;
    c[2] = n2;
    c[3] = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// A scaled value (at most 448) on the grid of its binade, u in [0, 1) deciding between the two
// neighbours; the result is an e4m3 value exactly.
__device__ __forceinline__ float dither(float q, float u, bool keep) {
  const float mag = fabsf(q);
  int b = (int)(__float_as_uint(mag) >> 23) - 127;
  b = (b < -6 ? -6 : b) - 3;
  float n = floorf(ldexpf(mag, -b) + u);
  if (keep) n = mag > 0.f && n < 1.f ? 1.f : n;
  return copysignf(ldexpf(n, b), q);
}

// Codes and scale byte of a lane's 8 values, its quad's group of 32.
__device__ __forceinline__ uint2 encode8(const float (&x)[kE], const uint32_t (&u)[kE], int shift,
                                         bool keep, int& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  m = ckpt_quad_max(m);
  const bool bad = m >= 0x7f800000u;
  byte = ckpt_scale_byte(bad ? 0 : m, kFmtE4M3);
  const float inv = ckpt_inverse(byte);
  float lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float ul = (float)((u[j] >> shift) & 0xffffu) * 0x1p-16f;
    const float uh = (float)((u[4 + j] >> shift) & 0xffffu) * 0x1p-16f;
    lo[j] = bad ? 0.f : dither(x[j] * inv, ul, keep);
    hi[j] = bad ? 0.f : dither(x[4 + j] * inv, uh, keep);
  }
  byte = bad ? 255 : byte;
  return make_uint2(ckpt_encode4(lo, kFmtE4M3), ckpt_encode4(hi, kFmtE4M3));
}

__device__ __forceinline__ void decode8(uint2 c, uint32_t byte, float (&v)[kE]) {
  const float f = ckpt_factor(byte);
  float lo[4], hi[4];
  ckpt_decode4(c.x, kFmtE4M3, lo);
  ckpt_decode4(c.y, kFmtE4M3, hi);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = lo[j] * f, v[4 + j] = hi[j] * f;
}

struct Piece {
  float p[kE], g[kE], m[kE], v[kE];
  uint2 mc, vc;
  uint32_t ms, vs;
};

template <bool WIDE>
__device__ __forceinline__ void load_f8(const float* p, int64_t e, int64_t n, float (&v)[kE]) {
  if (WIDE) {
    const v4f a = *(const v4f*)(p + e), b = *(const v4f*)(p + e + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  } else {
#pragma unroll
    for (int j = 0; j < kE; ++j) v[j] = e + j < n ? p[e + j] : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_f8(float* p, int64_t e, int64_t n, const float (&v)[kE]) {
  if (WIDE) {
    *(v4f*)(p + e) = v4f{v[0], v[1], v[2], v[3]};
    *(v4f*)(p + e + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < kE; ++j)
      if (e + j < n) p[e + j] = v[j];
  }
}
template <bool WIDE>
__device__ __forceinline__ uint2 load_c8(const uint8_t* p, int64_t e, int64_t n) {
  if (WIDE) return *(const uint2*)(p + e);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < kE; ++j)
    if (e + j < n) w[j / 4] |= (uint32_t)p[e + j] << (8 * (j % 4));
  return make_uint2(w[0], w[1]);
}
template <bool WIDE>
__device__ __forceinline__ void store_c8(uint8_t* p, int64_t e, int64_t n, uint2 c) {
  if (WIDE) {
    *(uint2*)(p + e) = c;
  } else {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int j = 0; j < kE; ++j)
      if (e + j < n) p[e + j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
  }
}

template <bool WIDE>
__device__ __forceinline__ void load_piece(const AdamEntry& t, int64_t e, Piece& q) {
  load_f8<WIDE>(t.p, e, t.n, q.p);
  if (t.flags & kAdamG16) {
    const uint16_t* g = (const uint16_t*)t.g;
    if (WIDE) {
      const u32x4 a = *(const u32x4*)(g + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q.g[2 * j] = __uint_as_float(a[j] << 16);
        q.g[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j) q.g[j] = e + j < t.n ? bf2f(g[e + j]) : 0.f;
    }
  } else {
    load_f8<WIDE>((const float*)t.g, e, t.n, q.g);
  }
  if (t.flags & kAdam8) {
    q.mc = load_c8<WIDE>((const uint8_t*)t.m, e, t.n);
    q.vc = load_c8<WIDE>((const uint8_t*)t.v, e, t.n);
    q.ms = e < t.n ? t.ms[e / kCkptGroup] : 0;
    q.vs = e < t.n ? t.vs[e / kCkptGroup] : 0;
  } else {
    load_f8<WIDE>((const float*)t.m, e, t.n, q.m);
    load_f8<WIDE>((const float*)t.v, e, t.n, q.v);
  }
}

template <bool WIDE>
__device__ __forceinline__ void store_piece(const AdamEntry& t, int64_t e, const Piece& q) {
  store_f8<WIDE>(t.p, e, t.n, q.p);
  if (t.copy) {
    if (WIDE) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = (uint32_t)f2bf(q.p[2 * j]) | ((uint32_t)f2bf(q.p[2 * j + 1]) << 16);
      *(u32x4*)(t.copy + e) = o;
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (e + j < t.n) t.copy[e + j] = f2bf(q.p[j]);
    }
  }
  if (t.flags & kAdam8) {
    store_c8<WIDE>((uint8_t*)t.m, e, t.n, q.mc);
    store_c8<WIDE>((uint8_t*)t.v, e, t.n, q.vc);
    if ((threadIdx.x & 3) == 0) {
      t.ms[e / kCkptGroup] = (uint8_t)q.ms;
      t.vs[e / kCkptGroup] = (uint8_t)q.vs;
    }
  } else {
    store_f8<WIDE>((float*)t.m, e, t.n, q.m);
    store_f8<WIDE>((float*)t.v, e, t.n, q.v);
  }
}

// All lanes of a quad take part (codes need their group's largest value), also those past the end.
__device__ __forceinline__ void step_piece(const AdamArgs& a, const AdamEntry& t, uint32_t tensor,
                                           const Scalars& s, int64_t e, Piece& q) {
  const bool small = (t.flags & kAdam8) != 0;
  if (small) {
    decode8(q.mc, q.ms, q.m);
    decode8(q.vc, q.vs, q.v);
#pragma unroll
    for (int j = 0; j < kE; ++j) q.v[j] *= q.v[j];
  }
  float root[kE];
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    const float g = q.g[j] * s.gf;
    q.m[j] = a.b1 * q.m[j] + a.c1 * g;
    q.v[j] = a.b2 * q.v[j] + a.c2 * (g * g);
    root[j] = __builtin_sqrtf(q.v[j]);
    const float den = root[j] * s.k2 + a.eps;
    q.p[j] = q.p[j] * s.keep - s.k1 * q.m[j] / den;
  }
  if (!small) return;
  uint32_t u[kE];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t i = (uint64_t)e / 4 + h;
    uint32_t c[4] = {(uint32_t)i, (uint32_t)(i >> 32), tensor, s.step};
    philox(c, a.key0, a.key1);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[4 * h + j] = c[j];
  }
  // what lies past the end does not count for its group, whatever stands there
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    if (e + j >= t.n) q.m[j] = root[j] = 0.f;
  }
  int mb, vb;
  q.mc = encode8(q.m, u, 0, false, mb);
  q.vc = encode8(root, u, 16, true, vb);
  q.ms = (uint32_t)mb;
  q.vs = (uint32_t)vb;
}

__global__ void __launch_bounds__(kThreads) k_adamw(AdamArgs a) {
  const AdamHead* head = (const AdamHead*)a.table;
  const AdamEntry* entries = (const AdamEntry*)(a.table + sizeof(AdamHead));
  if (head->magic != kAdamMagic || head->chunks != a.chunks || head->count != a.count) return;
  const uint32_t tensor = ((const uint32_t*)(entries + a.count))[blockIdx.x];
  const AdamEntry t = entries[tensor];
  const int64_t e0 = (int64_t)(blockIdx.x - t.first) * kAdamChunk + threadIdx.x * kE;

  Scalars s;
  s.k1 = a.k1;
  s.k2 = a.k2;
  s.step = a.step;
  double lr = a.lr;
  if (a.lr_factor) lr *= (double)*a.lr_factor;
  if (a.step_dev) {
    const int32_t n = *a.step_dev;
    s.step = (uint32_t)n;
    s.k1 = (float)(lr / (1.0 - pow(a.beta1, (double)n)));
    s.k2 = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)n)));
  } else if (a.lr_factor) {
    s.k1 = (float)(lr / (1.0 - pow(a.beta1, (double)s.step)));
  }
  s.keep = (float)(1.0 - lr * t.decay);
  s.gf = a.grad_factor ? *a.grad_factor : 1.f;

  constexpr int kPieces = (int)(kAdamChunk / kTile);
  const bool wide = (t.flags & kAdamWide) != 0;
  Piece q[kPieces];
  if (wide && (int64_t)(blockIdx.x - t.first + 1) * kAdamChunk <= t.n) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) load_piece<true>(t, e0 + k * kTile, q[k]);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      step_piece(a, t, tensor, s, e0 + k * kTile, q[k]);
      store_piece<true>(t, e0 + k * kTile, q[k]);
    }
  } else {   // a tensor's end, or one whose addresses allow no 16-byte accesses
#pragma unroll 1
    for (int k = 0; k < kPieces; ++k) {
      const int64_t e = e0 + k * kTile;
      const bool whole = wide && e + kE <= t.n;
      if (whole) load_piece<true>(t, e, q[0]);
      else load_piece<false>(t, e, q[0]);
      step_piece(a, t, tensor, s, e, q[0]);
      if (whole) store_piece<true>(t, e, q[0]);
      else if (e < t.n) store_piece<false>(t, e, q[0]);
    }
  }
}

}  // namespace

hipError_t launch_adamw(const AdamRequest& r, hipStream_t st) {
  AdamArgs a{};
  a.table = (const unsigned char*)r.table;
  a.step_dev = r.step_dev;
  a.lr_factor = r.lr_factor;
  a.grad_factor = r.grad_factor;
  a.lr = r.lr;
  a.beta1 = r.beta1;
  a.beta2 = r.beta2;
  a.b1 = (float)r.beta1;
  a.c1 = (float)(1.0 - r.beta1);
  a.b2 = (float)r.beta2;
  a.c2 = (float)(1.0 - r.beta2);
  a.eps = (float)r.eps;
  if (!r.step_dev) {
    a.k1 = (float)(r.lr / (1.0 - pow(r.beta1, (double)r.step)));
    a.k2 = (float)(1.0 / sqrt(1.0 - pow(r.beta2, (double)r.step)));
  }
  a.step = (uint32_t)r.step;
  a.chunks = r.chunks;
  a.count = r.count;
  a.key0 = (uint32_t)r.seed;
  a.key1 = (uint32_t)(r.seed >> 32);
  k_adamw<<<dim3(r.chunks), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace wbmm
