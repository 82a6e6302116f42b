// Gated delta rule, device pieces shared by the forward and backward kernels (see wbmm_delta.hpp for
// the formulas and operand layouts).
#pragma once

#include "wbmm_delta.hpp"
#include "wbmm_device.hpp"

#include <type_traits>

namespace wbmm {

template <int P>
struct Frag {
  u32x4 p[P];
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <int P>
struct Half {                  // the four terms of one 16: half a frag
  u32x2 p[P];
};

template <int P>
__device__ __forceinline__ Half<P> split4(float a, float b, float c, float d) {
  Half<P> h;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t lo = pk_bf16(a, b), hi = pk_bf16(c, d);
    h.p[i] = u32x2{lo, hi};
    if (i + 1 < P) {
      a -= __uint_as_float(lo << 16);
      b -= __uint_as_float(lo & 0xffff0000u);
      c -= __uint_as_float(hi << 16);
      d -= __uint_as_float(hi & 0xffff0000u);
    }
  }
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

// A matrix of the first launch as an operand in memory: in its three parts, or (M = 2, bf16 tensors) as its 8 fp32
// entries, whose size is two parts' and whose three parts are the reader's to form.
template <int M>
__device__ __forceinline__ Frag<M> packed(const float (&v)[8]) {
  if constexpr (M == 3) return split8<3>(v);
  Frag<M> f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f.p[i] = __builtin_bit_cast(u32x4, v4f{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]});
  return f;
}
__device__ __forceinline__ Frag<3> parts(const Frag<3>& f) { return f; }
__device__ __forceinline__ Frag<3> parts(const Frag<2>& f) {
  const v4f a = __builtin_bit_cast(v4f, f.p[0]), b = __builtin_bit_cast(v4f, f.p[1]);
  return join<3>(split4<3>(a[0], a[1], a[2], a[3]), split4<3>(b[0], b[1], b[2], b[3]));
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
// A B for three parts each, in two chains of three products (a product waits twice as long for the one
// before it in its chain as the matrix core takes).
__device__ __forceinline__ v4f mma_short(const Frag<3>& a, const Frag<3>& b) {
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  v4f lo = mfma_bf16(a.p[0], b.p[2], zero), hi = mfma_bf16(a.p[0], b.p[1], zero);
  lo = mfma_bf16(a.p[1], b.p[1], lo);
  hi = mfma_bf16(a.p[1], b.p[0], hi);
  lo = mfma_bf16(a.p[2], b.p[0], lo);
  hi = mfma_bf16(a.p[0], b.p[0], hi);
  return hi + lo;
}

// Frags in LDS: part p of frag f at base + (f * P + p) * 1024, a lane's 16 bytes in slot(lane), half h 8 of
// them. Operands are read by lane in any case without bank conflicts; writes of transposed blocks run
// over rows 4 apart and over lane groups, which the slot's low bits spread over the banks (without: 55 % of
// the walk's LDS cycles were conflicts).
__device__ __forceinline__ int slot(int lane) { return lane ^ ((lane >> 4) & 3); }
template <int P>
__device__ __forceinline__ Frag<P> lds_frag(const unsigned char* base, int f, int lane) {
  Frag<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.p[i] = *(const u32x4*)(base + (f * P + i) * 1024 + slot(lane) * 16);
  return r;
}
template <int P>
__device__ __forceinline__ void lds_half(unsigned char* base, int f, int lane, int half,
                                         const Half<P>& h) {
#pragma unroll
  for (int i = 0; i < P; ++i) *(u32x2*)(base + (f * P + i) * 1024 + slot(lane) * 16 + half * 8) = h.p[i];
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

// Which head and which columns of dv a workgroup walks. Workgroups go to the 8 XCDs in turn: a head's column tiles are
// 8 apart, so that they run on one XCD at one time and share what they read in its L2 (with the tiles of a head
// a grid's length apart, 512 heads of 64 over 784 steps took 203 us forward and 293 backward, so 137 and 218). The
// grid's second dimension keeps a launch below 2^32 threads in the first.
constexpr int kDeltaOctets = 1 << 15;     // of heads, in a row of the grid
struct DeltaWalkAt {
  int bh, tile;
};
__device__ __forceinline__ DeltaWalkAt delta_walk_at(int tiles) {
  const int g = (int)(blockIdx.x >> 3), b = g / tiles;
  return {8 * (b + kDeltaOctets * (int)blockIdx.y) + (int)(blockIdx.x & 7), g - b * tiles};
}
inline dim3 delta_walk_grid(const DeltaArgs& a, int tiles) {
  const int octets = (a.B * a.H + 7) / 8, row = octets < kDeltaOctets ? octets : kDeltaOctets;
  return dim3((uint32_t)row * 8 * tiles, (octets + row - 1) / row);
}

// Types of a tensor's elements: parts of an input, how P and the gradients' T are kept (see packed), a quad of
// entries, and a quad as it is loaded (nothing is done to it before it is used: the loads of a chunk are
// in flight while the chunk before it is computed).
struct Raw16 {
  uint32_t e[4];
};
template <typename T, bool VEC>
struct DeltaType;
template <bool VEC>
struct DeltaType<uint16_t, VEC> {
  static constexpr int PI = 1, PM = 2;
  using Quad = Half<1>;
  using Raw = typename std::conditional<VEC, u32x2, Raw16>::type;
};
template <bool VEC>
struct DeltaType<float, VEC> {
  static constexpr int PI = 3, PM = 3;
  using Quad = v4f;
  using Raw = v4f;
};

// Buffers: loads at offsets from kNowhere on read 0, stores there are dropped. So what lies past the
// end of a sequence or a row is zero whatever memory holds, without a branch or a select. An offset
// counts from the lowest position of a chunk: at most 64 rows of 2^24 bytes.
constexpr uint32_t kNowhere = 0x7fffff00u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t delta_buf(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)kNowhere,
                                           0x00020000);
}
template <typename T>
__device__ __forceinline__ T buf_load(__amdgpu_buffer_rsrc_t r, uint32_t off);
template <>
__device__ __forceinline__ uint16_t buf_load<uint16_t>(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}
template <>
__device__ __forceinline__ float buf_load<float>(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}
template <>
__device__ __forceinline__ u32x2 buf_load<u32x2>(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
}
template <>
__device__ __forceinline__ v4f buf_load<v4f>(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, uint32_t off, float v, float) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, (int)off, 0, 0);
}
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, uint32_t off, float v, uint16_t) {
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, (int)off, 0, 0);
}
__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(uint16_t v) { return bf2f(v); }

// One entry as it is loaded, in a register of its own.
template <typename T>
__device__ __forceinline__ uint32_t raw1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if constexpr (sizeof(T) == 2) return buf_load<uint16_t>(r, off);
  return __float_as_uint(buf_load<float>(r, off));
}
template <typename T>
__device__ __forceinline__ float wide1(uint32_t v) {
  return __uint_as_float(sizeof(T) == 2 ? v << 16 : v);
}

// Entries i .. i + 3 of a row of `len` at `off` (kNowhere: a row of zeros). VEC: len is a multiple of 4.
template <typename T, bool VEC>
__device__ __forceinline__ typename DeltaType<T, VEC>::Raw raw4(__amdgpu_buffer_rsrc_t r, uint32_t off,
                                                                int i, int len) {
  typename DeltaType<T, VEC>::Raw u;
  if constexpr (VEC) {
    u = buf_load<typename DeltaType<T, VEC>::Raw>(r, i < len ? off + i * sizeof(T) : kNowhere);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const T x = buf_load<T>(r, i + j < len ? off + (i + j) * sizeof(T) : kNowhere);
      if constexpr (sizeof(T) == 2) u.e[j] = x;
      else u[j] = x;
    }
  }
  return u;
}
__device__ __forceinline__ Half<1> quad(u32x2 u) {
  Half<1> h;
  h.p[0] = u;
  return h;
}
__device__ __forceinline__ Half<1> quad(const Raw16& u) {
  return quad(u32x2{u.e[0] | (u.e[1] << 16), u.e[2] | (u.e[3] << 16)});
}
__device__ __forceinline__ v4f quad(const v4f& u) { return u; }
__device__ __forceinline__ Half<1> to_half(const Half<1>& h) { return h; }
__device__ __forceinline__ Half<3> to_half(const v4f& v) { return split4<3>(v[0], v[1], v[2], v[3]); }
template <int P, typename R>
__device__ __forceinline__ Frag<P> operand(const R& a, const R& b) {
  return join<P>(to_half(quad(a)), to_half(quad(b)));
}

// Eight neighbouring entries. VEC: len is a multiple of 8.
template <typename T, bool VEC>
struct Raw8 {
  typename DeltaType<T, VEC>::Raw a, b;
};
template <>
struct Raw8<uint16_t, true> {
  u32x4 a;
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T, VEC> raw8(__amdgpu_buffer_rsrc_t r, uint32_t off, int i, int len) {
  Raw8<T, VEC> u;
  if constexpr (sizeof(T) == 2 && VEC) {
    u.a = __builtin_bit_cast(u32x4, buf_load<v4f>(r, i < len ? off + i * sizeof(T) : kNowhere));
  } else {
    u.a = raw4<T, VEC>(r, off, i, len);
    u.b = raw4<T, VEC>(r, off, i + 4, len);
  }
  return u;
}
// Its two quads in parts.
template <int P>
__device__ __forceinline__ void halves(const Raw8<uint16_t, true>& u, Half<P>& lo, Half<P>& hi) {
  lo.p[0] = u32x2{u.a[0], u.a[1]};
  hi.p[0] = u32x2{u.a[2], u.a[3]};
}
template <int P, typename R>
__device__ __forceinline__ void halves(const R& u, Half<P>& lo, Half<P>& hi) {
  lo = to_half(quad(u.a));
  hi = to_half(quad(u.b));
}

// Rows of one chunk of a sequence, as offsets from its lowest position.
struct DeltaRows {
  int cnt, reverse;      // live steps
  __device__ __forceinline__ bool live(int m) const { return m < cnt; }
  __device__ __forceinline__ uint32_t off(int m, uint32_t stride) const {
    return m < cnt ? (uint32_t)(reverse ? cnt - 1 - m : m) * stride : kNowhere;
  }
};
__device__ __forceinline__ DeltaRows delta_rows(const DeltaSeq& s, int c) {
  const int left = s.n - c * kDeltaChunk;
  return {left < kDeltaChunk ? left : kDeltaChunk, s.reverse};
}
// Lowest position of chunk c, counted over the batch.
__device__ __forceinline__ size_t delta_low(const DeltaArgs& a, const DeltaSeq& s, int b, int c) {
  const int t0 = c * kDeltaChunk, left = s.n - t0;
  const int cnt = left < kDeltaChunk ? left : kDeltaChunk;
  return (size_t)b * a.L + (s.reverse ? s.n - t0 - cnt : t0);
}

// A 4 x 4 block, rows r[0..3] of four entries, as its four columns of four, part by part.
template <int P>
__device__ __forceinline__ void transpose4(const Half<P> (&r)[4], Half<P> (&c)[4]) {
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;   // upper or lower halves of two words
      c[j].p[p] = u32x2{__builtin_amdgcn_perm(r[1].p[p][j >> 1], r[0].p[p][j >> 1], sel),
                        __builtin_amdgcn_perm(r[3].p[p][j >> 1], r[2].p[p][j >> 1], sel)};
    }
}

// Operands of the rows of a 64 x DK matrix in LDS. Rows as terms lie along DK (row tile i, terms 32 s ..)
// at (i KS + s), in the order of the walk: slot j of lane group q is entry 32 s + 8 q + j, so that a lane's 8
// are neighbours. A state's row tile t then has entry 32 (t / 2) + 8 q + 4 (t % 2) + r in row 4 q + r.
__device__ __forceinline__ int walk_entry(int tile, int m) {   // of row m of a state's tile
  return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3);
}
// 4 rows (steps 4 tg ..) of 8 entries (8 dg ..): as rows ...
template <int P, int KS>
__device__ __forceinline__ void lds_rows(unsigned char* to, int tg, int dg, const Half<P> (&lo)[4],
                                         const Half<P> (&hi)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Frag<P> f = join<P>(lo[j], hi[j]);
    unsigned char* at = to + ((tg >> 2) * KS + (dg >> 2)) * P * 1024 +
                        slot((dg & 3) * 16 + 4 * (tg & 3) + j) * 16;
#pragma unroll
    for (int p = 0; p < P; ++p) *(u32x4*)(at + p * 1024) = f.p[p];
  }
}
// ... and transposed, as operands of the state's row tiles over the steps, two frags a tile.
template <int P>
constexpr int kTileBytes = 2 * P * 1024;
template <int P>
__device__ __forceinline__ void lds_cols(unsigned char* to, int tg, int dg, const Half<P> (&lo)[4],
                                         const Half<P> (&hi)[4]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    Half<P> c[4];
    transpose4(e ? hi : lo, c);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      lds_half<P>(to + (2 * (dg >> 2) + e) * kTileBytes<P>, tg >> 3,
                  (tg & 3) * 16 + 4 * (dg & 3) + j, (tg >> 2) & 1, c[j]);
  }
}

__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Frags of a lower triangular 64 x 64 matrix M in memory, 6 of them, as A operands: row tile i over
// terms 32 s .. (2 s <= i), and of its transpose row tile j over terms 32 s .. (2 s + 1 >= j).
__device__ __forceinline__ constexpr int tri_frag(int i, int s) { return s == 0 ? i : 2 + i; }
__device__ __forceinline__ constexpr int trit_frag(int j, int s) { return j < 2 ? 2 * j + s : 2 + j; }
template <int P>
__device__ __forceinline__ Frag<P> mem_frag(const unsigned char* base, int f, int lane) {
  Frag<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i)
    r.p[i] = *(const u32x4*)(base + (uint32_t)((f * P + i) * 1024 + lane * 16));
  return r;
}

// Calls f with the next of the three widths of a key that kernels are made for, and with VEC.
template <typename F>
inline void with_dk(int dk, bool vec, F f) {
  auto go = [&](auto d) {
    if (vec) f(d, std::true_type());
    else f(d, std::false_type());
  };
  if (dk <= 32) go(std::integral_constant<int, 32>());
  else if (dk <= 64) go(std::integral_constant<int, 64>());
  else go(std::integral_constant<int, 128>());
}

}  // namespace wbmm
