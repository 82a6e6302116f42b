// 8-bit activation checkpoints: pack (map -> codes and scales), unpack, and the layer backward
// that takes x and z as checkpoints.
//
// Pack. For a group of 32 elements with largest magnitude amax, the scale exponent is the least
// integer e >= -126 with amax <= top 2^e (top = 127 for int8, 448 for e4m3), and the code of x is
// x 2^-e rounded to the nearest code value, ties to even. e follows from the bits of amax alone:
// with amax = 1.m 2^k, top 2^e >= amax is e >= k - 6 for int8 while 1.m <= 127/64, and
// e >= k - 8 for e4m3 while 1.m <= 1.75, one more otherwise. Magnitudes compare as unsigned
// integers, so infinities and NaN end up as the largest amax: such a group gets byte 255 and
// reads back as NaN, a bad activation stays visible.
//
// Both directions are bound by memory: one lane takes 8 elements (16 or 32 bytes in, 8 out), four
// lanes a group, whose maximum takes two quad moves; each lane has two such pieces in flight.
// Measured (kernel alone; a large copy reaches 5.05 to 5.18 TB/s): 64 x 192 x 28 x 28 fp32 packed to
// int8 in 9.0 us and unpacked in 11.6 us (5.4 and 4.2 TB/s, partly out of the last-level cache); 128 x
// 96 x 56 x 56 bf16 to e4m3 and back 20.0 and 18.8 us (5.8 and 6.2 TB/s).
#include "wbmm_ckpt.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

constexpr int kE = 8;          // elements per lane and piece
constexpr int kPieces = 2;     // pieces per lane, kThreads * kE apart

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* __restrict__ p, size_t e, size_t n, float (&v)[kE]) {
  if (VEC && e + kE <= n) {
    if constexpr (sizeof(T) == 4) {
      const v4f a = *(const v4f*)(p + e), b = *(const v4f*)(p + e + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
      const u32x4 a = *(const u32x4*)(p + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kE; ++j) v[j] = e + j < n ? load_f32<T>(p, e + j) : 0.f;
  }
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f2bf(v); }

__device__ __forceinline__ uint32_t quad_max(uint32_t x) {  // over the lane's group of four lanes
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xf, 0xf, true);
  x = x > a ? x : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xf, 0xf, true);
  return x > b ? x : b;
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(const T* __restrict__ x, size_t n,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  const size_t e0 = ((size_t)blockIdx.x * kPieces * kThreads + threadIdx.x) * kE;
  float v[kPieces][kE];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) load8<T, VEC>(x, e0 + (size_t)q * kThreads * kE, n, v[q]);
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const size_t e = e0 + (size_t)q * kThreads * kE;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const uint32_t b = __float_as_uint(v[q][j]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    m = quad_max(m);
    const bool bad = m >= 0x7f800000u;
    const uint32_t over = FMT == kFmtInt8 ? 0x7e0000u : 0x600000u;
    int byte = (int)(m >> 23) - (FMT == kFmtInt8 ? 6 : 8) + ((m & 0x7fffffu) > over ? 1 : 0);
    byte = byte < 1 ? 1 : byte;
    const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = bad ? 0.f : v[q][4 * h + j] * inv;
      if constexpr (FMT == kFmtInt8) {
        w[h] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[h] |= ((uint32_t)(int)rintf(s[j]) & 0xffu) << (8 * j);
      } else {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
        w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], p, true);
      }
    }
    if (VEC && e + kE <= n) {
      *(uint2*)(codes + e) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (e + j < n) codes[e + j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
    if ((threadIdx.x & 3) == 0 && e < n) scales[e / kCkptGroup] = (uint8_t)(bad ? 255 : byte);
  }
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          size_t n, T* __restrict__ x) {
  const size_t e0 = ((size_t)blockIdx.x * kPieces * kThreads + threadIdx.x) * kE;
  uint32_t w[kPieces][2], sc[kPieces];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const size_t e = e0 + (size_t)q * kThreads * kE;
    sc[q] = e < n ? scales[e / kCkptGroup] : 0;
    if (VEC && e + kE <= n) {
      const uint2 c = *(const uint2*)(codes + e);
      w[q][0] = c.x;
      w[q][1] = c.y;
    } else {
      w[q][0] = w[q][1] = 0;
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (e + j < n) w[q][j / 4] |= (uint32_t)codes[e + j] << (8 * (j % 4));
    }
  }
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const size_t e = e0 + (size_t)q * kThreads * kE;
    const float f = ckpt_factor(sc[q]);
    float v[kE];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4];
      ckpt_decode4(w[q][h], FMT, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j] = t[j] * f;
    }
    if (VEC && e + kE <= n) {
      if constexpr (sizeof(T) == 4) {
        *(v4f*)(x + e) = v4f{v[0], v[1], v[2], v[3]};
        *(v4f*)(x + e + 4) = v4f{v[4], v[5], v[6], v[7]};
      } else {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = (uint32_t)f2bf(v[2 * j]) | ((uint32_t)f2bf(v[2 * j + 1]) << 16);
        *(u32x4*)(x + e) = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (e + j < n) store1(x + e + j, v[j]);
    }
  }
}

template <bool TO_BF16>
__global__ void __launch_bounds__(kThreads) k_cast(const void* __restrict__ src,
                                                   void* __restrict__ dst, size_t n) {
  const size_t step = (size_t)gridDim.x * kThreads;
  for (size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x; e < n; e += step) {
    if constexpr (TO_BF16)
      ((uint16_t*)dst)[e] = f2bf(((const float*)src)[e]);
    else
      ((float*)dst)[e] = bf2f(((const uint16_t*)src)[e]);
  }
}

dim3 piece_grid(size_t n) {
  const size_t per = (size_t)kThreads * kE * kPieces;
  return dim3((unsigned)((n + per - 1) / per));
}

template <typename T, bool VEC>
hipError_t pack_t(const void* x, size_t n, int fmt, uint8_t* codes, uint8_t* scales,
                  hipStream_t st) {
  if (fmt == kFmtInt8)
    k_ckpt_pack<T, kFmtInt8, VEC><<<piece_grid(n), kThreads, 0, st>>>((const T*)x, n, codes, scales);
  else
    k_ckpt_pack<T, kFmtE4M3, VEC><<<piece_grid(n), kThreads, 0, st>>>((const T*)x, n, codes, scales);
  return hipGetLastError();
}
template <typename T, bool VEC>
hipError_t unpack_t(const uint8_t* codes, const uint8_t* scales, size_t n, int fmt, void* x,
                    hipStream_t st) {
  if (fmt == kFmtInt8)
    k_ckpt_unpack<T, kFmtInt8, VEC><<<piece_grid(n), kThreads, 0, st>>>(codes, scales, n, (T*)x);
  else
    k_ckpt_unpack<T, kFmtE4M3, VEC><<<piece_grid(n), kThreads, 0, st>>>(codes, scales, n, (T*)x);
  return hipGetLastError();
}

hipError_t launch_cast(const void* src, void* dst, size_t n, bool to_bf16, hipStream_t st) {
  size_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 8192) blocks = 8192;
  if (to_bf16)
    k_cast<true><<<dim3((unsigned)blocks), kThreads, 0, st>>>(src, dst, n);
  else
    k_cast<false><<<dim3((unsigned)blocks), kThreads, 0, st>>>(src, dst, n);
  return hipGetLastError();
}

bool vec_ok(const void* x, const uint8_t* codes) {
  return ((uintptr_t)x % 16) == 0 && ((uintptr_t)codes % 8) == 0;
}

}  // namespace

hipError_t launch_ckpt_pack(const void* x, size_t n, int bf16, int fmt, uint8_t* codes,
                            uint8_t* scales, hipStream_t st) {
  const bool v = vec_ok(x, codes);
  if (bf16)
    return v ? pack_t<uint16_t, true>(x, n, fmt, codes, scales, st)
             : pack_t<uint16_t, false>(x, n, fmt, codes, scales, st);
  return v ? pack_t<float, true>(x, n, fmt, codes, scales, st)
           : pack_t<float, false>(x, n, fmt, codes, scales, st);
}

hipError_t launch_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, size_t n, int bf16,
                              int fmt, void* x, hipStream_t st) {
  const bool v = vec_ok(x, codes);
  if (bf16)
    return v ? unpack_t<uint16_t, true>(codes, scales, n, fmt, x, st)
             : unpack_t<uint16_t, false>(codes, scales, n, fmt, x, st);
  return v ? unpack_t<float, true>(codes, scales, n, fmt, x, st)
           : unpack_t<float, false>(codes, scales, n, fmt, x, st);
}

// ---------------------------------------------------------------------------- backward
// w = 14 on whole images: the fused kernel of wbmm_ckptbwd.hip; other maps, layouts and windows from 2
// to 16: the one of wbmm_ckptany.hip. Windows of 1 and above 16, and images of which 33 pass 2^32
// bytes: the checkpoints are decoded into fp32 maps in the workspace and the fp32 backward runs on
// them; bf16 dy and T are widened exactly and dx is rounded to bf16 once at the end. The workspace is
// then larger than what the checkpoints save (64 x 192 x 28 x 28, w = 28, with the mix: 184 MiB fp32, 260
// bf16, for 110 and 91 on plain maps; 856 and 889 us, 830 and 530 there).
namespace {

bool fast_call(const BwdCkptRequest& r) {
  const size_t es = r.bf16 ? 2 : 4;
  return fast_ckpt_shape(r.C, r.H, r.W, r.w, r.layout) && (uintptr_t)r.dy % (4 * es) == 0 &&
         (uintptr_t)r.dx % (2 * es) == 0 && (uintptr_t)r.xc % 4 == 0 && (uintptr_t)r.zc % 4 == 0;
}

size_t al256(size_t v) { return (v + 255) / 256 * 256; }

struct CkptWs {
  size_t x, z, dy, T, dx, inner, total;
};
BwdRequest fp32_request(const BwdCkptRequest& r) {
  static const float dummy = 0.f;
  BwdRequest q{};
  q.B = r.B; q.C = r.C; q.H = r.H; q.W = r.W; q.w = r.w; q.layout = r.layout;
  q.x = q.dy = &dummy;
  q.T = &dummy;
  q.mixw = r.mixw;
  q.zsaved = r.mixw ? &dummy : nullptr;
  return q;
}
CkptWs ckpt_ws(const BwdCkptRequest& r) {
  const size_t map = (size_t)r.B * r.C * r.H * r.W * 4;
  const size_t tab = (size_t)r.C * (2 * r.w - 1) * (2 * r.w - 1) * 4;
  CkptWs w{};
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += al256(n);
    return at;
  };
  w.x = take(map);
  w.z = take(r.mixw ? map : 0);
  w.dy = take(r.bf16 ? map : 0);
  w.T = take(r.bf16 ? tab : 0);
  w.dx = take(r.bf16 ? map : 0);
  w.inner = o;
  w.total = o + al256(backward_workspace(fp32_request(r)));
  return w;
}

}  // namespace

bool backward_ckpt_plan_ok(const BwdCkptRequest& r) {
  return any_ckpt_shape(r.B, r.C, r.H, r.W, r.w) || backward_plan_ok(fp32_request(r));
}

size_t backward_ckpt_workspace(const BwdCkptRequest& r) {
  if (fast_call(r)) return fast_ckpt_workspace(r);
  return any_ckpt_shape(r.B, r.C, r.H, r.W, r.w) ? any_ckpt_workspace(r) : ckpt_ws(r).total;
}

hipError_t launch_backward_ckpt(const BwdCkptRequest& r, hipStream_t st) {
  if (fast_call(r)) return launch_backward_ckpt_fast(r, st);
  if (any_ckpt_shape(r.B, r.C, r.H, r.W, r.w)) return launch_backward_ckpt_any(r, st);
  const CkptWs w = ckpt_ws(r);
  const size_t n = (size_t)r.B * r.C * r.H * r.W;
  unsigned char* ws = (unsigned char*)r.ws;
  BwdRequest q = fp32_request(r);
  hipError_t e = hipSuccess;
  q.x = (const float*)(ws + w.x);
  const bool wantW = r.mixw && r.dmixw;
  if (r.dT) e = launch_ckpt_unpack(r.xc, r.xs, n, 0, r.fmt, ws + w.x, st);
  if (e == hipSuccess && r.mixw) {
    q.zsaved = (const float*)(ws + w.z);
    if (wantW) e = launch_ckpt_unpack(r.zc, r.zs, n, 0, r.fmt, ws + w.z, st);
  }
  q.dy = (const float*)r.dy;
  q.T = (const float*)r.T;
  q.dx = (float*)r.dx;
  q.dT = r.dT;
  q.dmixw = wantW ? r.dmixw : nullptr;
  if (r.bf16) {
    const size_t tab = (size_t)r.C * (2 * r.w - 1) * (2 * r.w - 1);
    if (e == hipSuccess) e = launch_cast(r.dy, ws + w.dy, n, false, st);
    if (e == hipSuccess) e = launch_cast(r.T, ws + w.T, tab, false, st);
    q.dy = (const float*)(ws + w.dy);
    q.T = (const float*)(ws + w.T);
    q.dx = r.dx ? (float*)(ws + w.dx) : nullptr;
  }
  if (e != hipSuccess) return e;
  q.ws = ws + w.inner;
  q.ws_bytes = w.total - w.inner;
  e = launch_backward(q, st);
  if (e == hipSuccess && r.bf16 && r.dx) e = launch_cast(ws + w.dx, r.dx, n, true, st);
  return e;
}

}  // namespace wbmm
