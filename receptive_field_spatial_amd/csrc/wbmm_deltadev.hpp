// Gated delta rule, device pieces shared by the forward and backward kernels (see wbmm_delta.hpp for
// the formulas and operand layouts).
#pragma once

#include "wbmm_delta.hpp"
#include "wbmm_device.hpp"

namespace wbmm {

template <int P>
struct Frag {
  u32x4 p[P];
};
template <int P>
struct Half {                  // the four terms of one 16: half a frag
  uint2 p[P];
};

template <int P>
__device__ __forceinline__ Half<P> split4(float a, float b, float c, float d) {
  uint32_t lo[P], hi[P];
  split2<P>(a, b, lo);
  split2<P>(c, d, hi);
  Half<P> h;
#pragma unroll
  for (int i = 0; i < P; ++i) h.p[i] = make_uint2(lo[i], hi[i]);
  return h;
}
template <int P>
__device__ __forceinline__ Frag<P> join(const Half<P>& a, const Half<P>& b) {
  Frag<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) f.p[i] = u32x4{a.p[i].x, a.p[i].y, b.p[i].x, b.p[i].y};
  return f;
}
template <int P>
__device__ __forceinline__ Frag<P> split8(const float (&v)[8]) {
  return join<P>(split4<P>(v[0], v[1], v[2], v[3]), split4<P>(v[4], v[5], v[6], v[7]));
}

// acc + A B over 32 terms: the products of parts i, j with i + j below the larger number of parts.
template <int PA, int PB>
__device__ __forceinline__ v4f mma(const Frag<PA>& a, const Frag<PB>& b, v4f acc) {
  constexpr int M = PA > PB ? PA : PB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i)
      if (s - i >= 0 && s - i < PB) acc = mfma_bf16(a.p[i], b.p[s - i], acc);
  return acc;
}
template <int P, int N>
__device__ __forceinline__ Frag<P> lead(const Frag<N>& f) {   // the P leading parts
  Frag<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.p[i] = f.p[i];
  return r;
}

// Frags in LDS: part p of frag f at base + (f * P + p) * 1024, lane's 16 bytes, half h 8 of them.
template <int P>
__device__ __forceinline__ Frag<P> lds_frag(const unsigned char* base, int f, int lane) {
  Frag<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.p[i] = *(const u32x4*)(base + (f * P + i) * 1024 + lane * 16);
  return r;
}
template <int P>
__device__ __forceinline__ void lds_half(unsigned char* base, int f, int lane, int half,
                                         const Half<P>& h) {
#pragma unroll
  for (int i = 0; i < P; ++i) *(uint2*)(base + (f * P + i) * 1024 + lane * 16 + half * 8) = h.p[i];
}

// The steps of one sequence: step t < n takes position t, or n - 1 - t when reversed.
struct DeltaSeq {
  int n, reverse;
  __device__ __forceinline__ bool live(int t) const { return t < n; }
  __device__ __forceinline__ int pos(int t) const {   // of a step past the end: some position
    return t < n ? (reverse ? n - 1 - t : t) : 0;
  }
};
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs& a, int b) {
  DeltaSeq s;
  s.n = a.L;
  if (a.lens) {
    const int n = a.lens[b];
    s.n = n < 0 ? 0 : n > a.L ? a.L : n;
  }
  s.reverse = a.reverse;
  return s;
}

// Four neighbouring entries i .. i + 3 of a row of `len`; 0 past its end and in a row that is not
// live, whatever stands there.
template <bool VEC>
__device__ __forceinline__ Half<1> load4(const uint16_t* row, int i, int len, bool live) {
  uint2 u;
  if (VEC) {
    const bool in = live && i < len;
    u = *(const uint2*)(row + (i < len ? i : 0));
    u.x = in ? u.x : 0;
    u.y = in ? u.y : 0;
  } else {
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = row[i + j < len ? i + j : 0];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = live && i + j < len ? e[j] : 0;
    u = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
  }
  Half<1> h;
  h.p[0] = u;
  return h;
}
template <bool VEC>
__device__ __forceinline__ v4f load4(const float* row, int i, int len, bool live) {
  v4f u;
  if (VEC) {
    const bool in = live && i < len;
    u = *(const v4f*)(row + (i < len ? i : 0));
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = in ? u[j] : 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = row[i + j < len ? i + j : 0];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = live && i + j < len ? u[j] : 0.f;
  }
  return u;
}
__device__ __forceinline__ Half<1> to_half(Half<1> h) { return h; }
__device__ __forceinline__ Half<3> to_half(v4f v) { return split4<3>(v[0], v[1], v[2], v[3]); }

// Types of a tensor's elements: parts of an input, parts of what only reaches an output, raw quads.
template <typename T>
struct DeltaType;
template <>
struct DeltaType<uint16_t> {
  static constexpr int PI = 1, PO = 2;
  using Quad = Half<1>;
};
template <>
struct DeltaType<float> {
  static constexpr int PI = 3, PO = 3;
  using Quad = v4f;
};

// A 4 x 4 block, rows r[0..3] of four entries, as its four columns of four.
__device__ __forceinline__ void transpose4(const Half<1> (&r)[4], Half<1> (&c)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;   // the upper or lower halves of two words
    const uint32_t a = j < 2 ? r[0].p[0].x : r[0].p[0].y, b = j < 2 ? r[1].p[0].x : r[1].p[0].y;
    const uint32_t d = j < 2 ? r[2].p[0].x : r[2].p[0].y, e = j < 2 ? r[3].p[0].x : r[3].p[0].y;
    c[j].p[0] = make_uint2(__builtin_amdgcn_perm(b, a, sel), __builtin_amdgcn_perm(e, d, sel));
  }
}
__device__ __forceinline__ void transpose4(const v4f (&r)[4], Half<3> (&c)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = split4<3>(r[0][j], r[1][j], r[2][j], r[3][j]);
}

__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Tile (i, j), j <= i, of T or P: 16 rows of 16 floats.
__device__ __forceinline__ constexpr int tri(int i, int j) { return (i * (i + 1) / 2 + j) * 256; }

// A operand of row tile i over terms 32 s ..: rows of a lower triangular matrix.
__device__ __forceinline__ void tri_rows(const float* m, int i, int s, int lane, float (&v)[8]) {
  const int at = (lane & 15) * 16 + (lane >> 4) * 4;
  const v4f x = *(const v4f*)(m + tri(i, 2 * s) + at);
  v4f y = v4f{0.f, 0.f, 0.f, 0.f};
  if (2 * s + 1 <= i) y = *(const v4f*)(m + tri(i, 2 * s + 1) + at);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = x[j], v[4 + j] = y[j];
}
// The same of its transpose: row tile j, terms 32 s .. (2 s + 1 >= j).
__device__ __forceinline__ void tri_cols(const float* m, int j, int s, int lane, float (&v)[8]) {
  const int at = (lane >> 4) * 64 + (lane & 15);
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = 0.f;
  if (2 * s >= j) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = m[tri(2 * s, j) + at + 16 * r];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) v[4 + r] = m[tri(2 * s + 1, j) + at + 16 * r];
}

}  // namespace wbmm
