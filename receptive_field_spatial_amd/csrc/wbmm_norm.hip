// RMS norm over one axis with the residual's addition in front, and its gradients.
//
// Tensors are dense (outer, len, inner), normed over len for every (outer, inner):
//   t = x + res,   y = t rstd w,   rstd = rsqrt(mean t^2 + eps).
// The sum is formed in fp32 and normed as it is; what is stored of it (s) and of y is rounded once.
// With a checkpoint, its codes are those of the y that is stored. Backward, from the stored s:
//   h = s rstd,   dx = ds + rstd (w dy - h mean(w dy h)),   dw = sum over (outer, inner) of dy h.
//
// Everything is bound by memory, so each element is read once and kept in registers while its
// column's sums are formed. Two layouts:
//   rows    (inner = 1): a row belongs to LPR lanes (4 to 64, or the 256 of a workgroup) that hold K
//           pieces of 8 elements each; several rows per wave where rows are short. Rows whose length or
//           address does not allow 16-byte accesses go element by element, 64 lanes side by side.
//   columns (inner > 1): a lane holds one position (the bf16 forward: two neighbours) and a wave every NW-th entry of len
//           there; the waves' sums meet in LDS.
// Longer axes than the registers hold are read twice, the second time from a cache.
//
// Measured: forward bf16 with codes, 50176 rows of 192, 17.5 us (87 MB, 5.0 TB/s); backward fp32, 128 x 96 x
// 3136, 110 to 113 us (617 MB, 5.5 TB/s, part of it from the last-level cache) and 4.4 for dw's partials; single rows 2 us, a
// launch's own time. Far from that: columns of more than 256 entries (forward 512), read twice, 128 x 384 x 196 bf16
// forward 27 us, backward 54 (77 MB each); few columns, 8 x 768 x 49 bf16 35 and 44 us on 7 workgroups; rows of more than
// 6144, 2000 of 8192 bf16 42 and 194 us (131 MB each).
//
// dw: fp64 sums of fp32 products, then partials of a workgroup, added in a fixed order by a second launch.
#include "wbmm_ckpt.hpp"
#include "wbmm_launch.hpp"
#include "wbmm_norm.hpp"

namespace wbmm {

namespace {

constexpr int kP = 8;              // elements of a row piece
// Workgroups of a backward with dw: two per CU (50176 rows of 192 bf16: 20.9 us; one 24.5, four 23.7).
constexpr int kDwGroups = 512;
// Values of each tensor that a lane of the column kernels keeps (the forward keeps one tensor, the
// backward three): what 16 waves of a workgroup have registers for.
constexpr int kColFwd = 32, kColBwd = 16;

struct NormArgs {
  const void* x;
  const void* res;
  const float* w;
  const void* dy;
  void* s;
  void* y;
  uint8_t* codes;
  uint8_t* scales;
  double* part;                    // [workgroups][len]
  float eps;
  double inv64;                    // 1 / len
  int fmt;
  uint32_t len, rows;              // rows = outer * inner
  uint32_t tiles;
  FastDiv inner;
};

__device__ __forceinline__ void widen8(const float* p, float (&v)[kP]) {
  const v4f a = *(const v4f*)p, b = *(const v4f*)(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
}
__device__ __forceinline__ void widen8(const uint16_t* p, float (&v)[kP]) {
  const u32x4 a = *(const u32x4*)p;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(a[j] << 16);
    v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf_bits(float v) {   // to nearest even
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
// What a value reads back as once it is stored.
template <typename T> __device__ __forceinline__ float stored(float v);
template <> __device__ __forceinline__ float stored<float>(float v) { return v; }
template <> __device__ __forceinline__ float stored<uint16_t>(float v) {
  return (float)(__bf16)v;
}
__device__ __forceinline__ void narrow8(float* p, const float (&v)[kP]) {
  *(v4f*)p = v4f{v[0], v[1], v[2], v[3]};
  *(v4f*)(p + 4) = v4f{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void narrow8(uint16_t* p, const float (&v)[kP]) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = bf_bits(v[2 * j]) | (bf_bits(v[2 * j + 1]) << 16);
  *(u32x4*)p = o;
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)bf_bits(v); }

// Sum over the LPR lanes of a row, in every one of them. LPR = 256: the workgroup's, through sm
// (4 of them, another set for each call between two barriers).
template <int LPR, typename S>
__device__ __forceinline__ S row_sum(S v, S* sm) {
#pragma unroll
  for (int d = 1; d < (LPR < 64 ? LPR : 64); d *= 2) v += __shfl_xor(v, d);
  if (LPR == 256) {
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (sm[0] + sm[1]) + (sm[2] + sm[3]);
  }
  return v;
}

// rstd, and y from it. Sums are fp64 (squares of fp32 numbers can neither overflow nor vanish there). A code of 8 bits, and a bf16 y, hang on y's last bit where y lies between two of
// them, so y is formed to that bit: sum and products in fp64, y = t (rstd w) with one rounding, right also where rstd or
// rstd w is past fp32's range or w is infinite.
__device__ __forceinline__ double rstd_of(double sum, const NormArgs& a) {
  const double m = fma(sum, a.inv64, (double)a.eps), r = __builtin_amdgcn_rsq(m);
  // a Newton step; infinities, zeros and NaN are left as they are
  const double f = fma(r * 0.5, fma(-m * r, r, 1.0), r);
  return __builtin_isfinite(f) && r > 0.0 ? f : r;
}
__device__ __forceinline__ float y_of(float t, double rstd, float w) {
  return (float)((double)t * (rstd * (double)w));
}
// Backward: h, and dx without ds from g = w dy, h and m = mean(w dy h).
__device__ __forceinline__ float h_of(float t, double rstd) { return (float)((double)t * rstd); }
__device__ __forceinline__ float dx_of(float g, float h, float m, double rstd) {
  return (float)(rstd * (double)fmaf(-m, h, g));
}

// ---------------------------------------------------------------------------- rows
// VEC: pieces of 8 neighbouring elements, piece li + LPR k of a row (len a multiple of 8). Otherwise
// a "piece" is 8 elements that lie LPR apart: element li + LPR (8 k + j).
template <typename T, int LPR, int K, bool VEC>
struct RowPieces {
  int li;
  uint32_t len;
  __device__ __forceinline__ bool has(int k) const { return (li + LPR * k) * kP < len; }
  __device__ __forceinline__ uint32_t el(int k, int j) const {
    return VEC ? (uint32_t)(li + LPR * k) * kP + j : li + LPR * (uint32_t)(kP * k + j);
  }
  __device__ __forceinline__ void load(const T* row, int k, float (&v)[kP]) const {
    // past the end: some element of the row again, taken as 0 (no branch between the loads)
    if (VEC) {
      widen8(row + (has(k) ? (li + LPR * k) * kP : 0), v);
#pragma unroll
      for (int j = 0; j < kP; ++j) v[j] = has(k) ? v[j] : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < kP; ++j) v[j] = load_f32<T>(row, el(k, j) < len ? el(k, j) : 0);
#pragma unroll
      for (int j = 0; j < kP; ++j) v[j] = el(k, j) < len ? v[j] : 0.f;
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&v)[K][kP]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!w) {
#pragma unroll
        for (int j = 0; j < kP; ++j) v[k][j] = 1.f;
      } else if (VEC) {
        widen8(w + (has(k) ? (li + LPR * k) * kP : 0), v[k]);
      } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) v[k][j] = w[el(k, j) < len ? el(k, j) : 0];
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int k, const float (&v)[kP]) const {
    if (VEC) {
      if (has(k)) narrow8(row + (li + LPR * k) * kP, v);
    } else {
#pragma unroll
      for (int j = 0; j < kP; ++j)
        if (el(k, j) < len) put(row + el(k, j), v[j]);
    }
  }
};

template <typename T, int LPR, int K, bool VEC>
__global__ void __launch_bounds__(kThreads) k_norm_rows(NormArgs a) {
  constexpr int RPW = kThreads / LPR;   // rows of a workgroup
  __shared__ double sm[4];
  const RowPieces<T, LPR, K, VEC> pc{(int)(threadIdx.x % LPR), a.len};
  const uint32_t row = blockIdx.x * RPW + threadIdx.x / LPR;
  const bool live = row < a.rows;
  const size_t base = (size_t)(live ? row : 0) * a.len;
  float t[K][kP], r[K][kP];
#pragma unroll
  for (int k = 0; k < K; ++k) pc.load((const T*)a.x + base, k, t[k]);
  if (a.res) {
#pragma unroll
    for (int k = 0; k < K; ++k) pc.load((const T*)a.res + base, k, r[k]);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < kP; ++j) t[k][j] += r[k][j];
  }
  float w[K][kP];
  pc.weights(a.w, w);
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < kP; ++j) sum = fma((double)t[k][j], (double)t[k][j], sum);
  const double rstd = rstd_of(row_sum<LPR>(sum, sm), a);
  if (!live) return;   // no barrier and no exchange across rows from here on
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (a.s) pc.store((T*)a.s + base, k, t[k]);
    float y[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) y[j] = y_of(t[k][j], rstd, w[k][j]);
    pc.store((T*)a.y + base, k, y);
    if (VEC && a.codes) {   // len a multiple of 32: a group is a quad's, in or out together
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        y[j] = stored<T>(y[j]);
        const uint32_t b = __float_as_uint(y[j]) & 0x7fffffffu;
        m = b > m ? b : m;
      }
      m = ckpt_quad_max(m);
      const bool bad = m >= 0x7f800000u;
      const int byte = ckpt_scale_byte(bad ? 0 : m, a.fmt);
      const float inv = ckpt_inverse(byte);
      float lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = bad ? 0.f : y[j] * inv;
        hi[j] = bad ? 0.f : y[4 + j] * inv;
      }
      if (pc.has(k)) {
        const size_t e = base + (size_t)pc.el(k, 0);
        *(uint2*)(a.codes + e) = make_uint2(ckpt_encode4(lo, a.fmt), ckpt_encode4(hi, a.fmt));
        if ((threadIdx.x & 3) == 0) a.scales[e / kCkptGroup] = (uint8_t)(bad ? 255 : byte);
      }
    }
  }
}

// Rows longer than the registers: the workgroup reads a row twice.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_rows_long(NormArgs a) {
  __shared__ double sm[4];
  const size_t base = (size_t)blockIdx.x * a.len;
  const T *x = (const T*)a.x + base, *res = a.res ? (const T*)a.res + base : nullptr;
  double sum = 0.0;
  for (uint32_t e = threadIdx.x; e < a.len; e += kThreads) {
    const float t = load_f32<T>(x, e) + (res ? load_f32<T>(res, e) : 0.f);
    sum = fma((double)t, (double)t, sum);
  }
  const double rstd = rstd_of(row_sum<256>(sum, sm), a);
  for (uint32_t e = threadIdx.x; e < a.len; e += kThreads) {
    const float t = load_f32<T>(x, e) + (res ? load_f32<T>(res, e) : 0.f);
    if (a.s) put((T*)a.s + base + e, t);
    put((T*)a.y + base + e, y_of(t, rstd, a.w ? a.w[e] : 1.f));
  }
}

// Backward. A workgroup takes every gridDim.x-th set of rows and keeps dw's sums of its lanes'
// elements in registers.
template <typename T, int LPR, int K, bool VEC, bool DW>
__global__ void __launch_bounds__(kThreads) k_norm_rows_bwd(NormArgs a) {
  constexpr int RPW = kThreads / LPR;
  __shared__ double sm[2][2][4];
  __shared__ double red[DW && LPR < 256 ? kThreads * kP : 1];
  const RowPieces<T, LPR, K, VEC> pc{(int)(threadIdx.x % LPR), a.len};
  float w[K][kP];
  double dw[K][kP];
  pc.weights(a.w, w);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < kP; ++j) dw[k][j] = 0.0;
  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, turn ^= 1) {
    const uint32_t row = tile * RPW + threadIdx.x / LPR;
    const bool live = row < a.rows;
    const size_t base = (size_t)(live ? row : 0) * a.len;
    float t[K][kP], g[K][kP], r[K][kP];
#pragma unroll
    for (int k = 0; k < K; ++k) pc.load((const T*)a.x + base, k, t[k]);
#pragma unroll
    for (int k = 0; k < K; ++k) pc.load((const T*)a.dy + base, k, g[k]);
    if (a.res && a.y)
#pragma unroll
      for (int k = 0; k < K; ++k) pc.load((const T*)a.res + base, k, r[k]);
    double sq = 0.0, dot = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        sq = fma((double)t[k][j], (double)t[k][j], sq);
        dot = fma((double)t[k][j], (double)(g[k][j] * w[k][j]), dot);
      }
    // two turns use different words: a wave still reads the last turn's while another writes
    sq = row_sum<LPR>(sq, sm[turn][0]);
    dot = row_sum<LPR>(dot, sm[turn][1]);
    const double rstd = rstd_of(sq, a);
    const float mean = (float)(dot * rstd * a.inv64);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < kP; ++j) t[k][j] = h_of(t[k][j], rstd);
      if (DW && live)
#pragma unroll
        for (int j = 0; j < kP; ++j) dw[k][j] += (double)(g[k][j] * t[k][j]);
      if (a.y && live) {
        float d[kP];
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          d[j] = dx_of(g[k][j] * w[k][j], t[k][j], mean, rstd);
          if (a.res) d[j] += r[k][j];
        }
        pc.store((T*)a.y + base, k, d);
      }
    }
  }
  if (!DW) return;
  double* part = a.part + (size_t)blockIdx.x * a.len;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (LPR == 256) {
#pragma unroll
      for (int j = 0; j < kP; ++j)
        if (pc.el(k, j) < a.len) part[pc.el(k, j)] = dw[k][j];
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kP; ++j) red[j * kThreads + threadIdx.x] = dw[k][j];
      __syncthreads();
      // element (lane l of a row, j): the RPW row groups' sums in order
      for (int i = threadIdx.x; i < LPR * kP; i += kThreads) {
        const int l = i % LPR, j = i / LPR;
        const uint32_t e = VEC ? (uint32_t)(l + LPR * k) * kP + j : l + LPR * (uint32_t)(kP * k + j);
        double s = 0;
        for (int q = 0; q < RPW; ++q) s += red[j * kThreads + q * LPR + l];
        if (e < a.len) part[e] = s;
      }
    }
  }
}

// Rows longer than the registers; dw's sums are kept in fp64 in the workgroup's partial.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_rows_long_bwd(NormArgs a) {
  __shared__ double sm[2][2][4];
  double* part = a.part ? a.part + (size_t)blockIdx.x * a.len : nullptr;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)row * a.len;
    const T *x = (const T*)a.x + base, *dy = (const T*)a.dy + base;
    const T* res = a.res ? (const T*)a.res + base : nullptr;
    double sq = 0.0, dot = 0.0;
    for (uint32_t e = threadIdx.x; e < a.len; e += kThreads) {
      const float t = load_f32<T>(x, e), g = load_f32<T>(dy, e) * (a.w ? a.w[e] : 1.f);
      sq = fma((double)t, (double)t, sq);
      dot = fma((double)t, (double)g, dot);
    }
    sq = row_sum<256>(sq, sm[turn][0]);
    dot = row_sum<256>(dot, sm[turn][1]);
    const double rstd = rstd_of(sq, a);
    const float mean = (float)(dot * rstd * a.inv64);
    for (uint32_t e = threadIdx.x; e < a.len; e += kThreads) {
      const float h = h_of(load_f32<T>(x, e), rstd), g = load_f32<T>(dy, e);
      if (part) {   // this thread's own elements in every row
        const double add = (double)(g * h);
        part[e] = row == blockIdx.x ? add : part[e] + add;
      }
      if (a.y) {
        const float d = dx_of(g * (a.w ? a.w[e] : 1.f), h, mean, rstd);
        put((T*)a.y + base + e, res ? d + load_f32<T>(res, e) : d);
      }
    }
  }
}

// ---------------------------------------------------------------------------- columns
// A lane's VW positions: one, or two of bf16.
template <typename T, int VW>
__device__ __forceinline__ void load_n(const T* p, float (&v)[VW]) {
  if constexpr (VW == 1) {
    v[0] = load_f32<T>(p, 0);
  } else {
    const uint32_t a = *(const uint32_t*)p;
    v[0] = __uint_as_float(a << 16);
    v[1] = __uint_as_float(a & 0xffff0000u);
  }
}
template <typename T, int VW>
__device__ __forceinline__ void store_n(T* p, const float (&v)[VW]) {
  if constexpr (VW == 1) put(p, v[0]);
  else *(uint32_t*)p = bf_bits(v[0]) | (bf_bits(v[1]) << 16);
}

// Sum over the workgroup's waves of each lane's VW values, in every wave; sm: NW * 64 * VW of them.
template <int VW, typename S>
__device__ __forceinline__ void wave_join(S (&v)[VW], S* sm, int NW) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < VW; ++j) sm[(wv * VW + j) * 64 + lane] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < VW; ++j) v[j] = 0;
  for (int q = 0; q < NW; ++q)
#pragma unroll
    for (int j = 0; j < VW; ++j) v[j] += sm[(q * VW + j) * 64 + lane];
}

// Where a lane's VW positions lie (VW divides inner: they share an outer index).
struct ColAt {
  size_t base;       // of entry 0 of the axis
  uint32_t stride;   // between entries
  bool live;
};
template <int VW>
__device__ __forceinline__ ColAt col_at(const NormArgs& a, uint32_t tile) {
  const uint32_t p = (tile * 64 + (threadIdx.x & 63)) * VW;
  ColAt c;
  c.live = p < a.rows;
  uint32_t o, i;
  fdivmod(c.live ? p : 0, a.inner, o, i);
  c.stride = a.inner.d;
  c.base = (size_t)o * a.len * a.inner.d + i;
  return c;
}

// A wave's entries of the axis in turn: wv, wv + NW, ...; past the end the last one again, so that
// the loads need no branches between them.
template <int N>
struct ColWalk {
  size_t at, step;
  uint32_t e, nw, len;
  __device__ __forceinline__ ColWalk(const NormArgs& a, const ColAt& c, int wv, int NW)
      : step((size_t)c.stride * NW), e(wv), nw(NW), len(a.len) {
    if (e >= len) e = 0;   // a wave without entries
    at = c.base + (size_t)e * c.stride;
  }
  __device__ __forceinline__ size_t next() {
    const size_t now = at;
    e += nw;
    at += e < len ? step : 0;
    return now;
  }
};
template <int N>
__device__ __forceinline__ void col_weights(const NormArgs& a, int wv, int NW, float (&w)[N]) {
  if (a.w) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t e = wv + NW * k;
      w[k] = a.w[e < a.len ? e : 0];
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = 1.f;
  }
}

// The checkpoint of VW neighbouring y, groups of 32 / VW lanes (inner a multiple of 32).
template <typename T, int VW>
__device__ __forceinline__ void col_codes(const NormArgs& a, size_t at, float (&y)[VW], bool live) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < VW; ++j) {
    y[j] = stored<T>(y[j]);
    const uint32_t b = live ? __float_as_uint(y[j]) & 0x7fffffffu : 0u;
    m = b > m ? b : m;
  }
#pragma unroll
  for (int d = 1; d < 32 / VW; d *= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
    m = o > m ? o : m;
  }
  const bool bad = m >= 0x7f800000u;
  const int byte = ckpt_scale_byte(bad ? 0 : m, a.fmt);
  const float inv = ckpt_inverse(byte);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < VW; ++j) s[j] = bad ? 0.f : y[j] * inv;
  const uint32_t w = ckpt_encode4(s, a.fmt);
  if (!live) return;
  if constexpr (VW == 2) *(uint16_t*)(a.codes + at) = (uint16_t)w;
  if constexpr (VW == 1) a.codes[at] = (uint8_t)w;
  if ((threadIdx.x & (32 / VW - 1)) == 0) a.scales[at / kCkptGroup] = (uint8_t)(bad ? 255 : byte);
}

// N: entries of the axis per wave that are kept in registers; 0: any number, read twice.
template <typename T, int VW, int N>
__global__ void __launch_bounds__(1024) k_norm_cols(NormArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  double* const sm = (double*)lds;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), NW = blockDim.x >> 6;
  const ColAt c = col_at<VW>(a, blockIdx.x);
  const T* x = (const T*)a.x + c.base;
  const T* res = a.res ? (const T*)a.res + c.base : nullptr;
  double sq[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) sq[j] = 0.0;
  auto sum_at = [&](uint32_t e, float (&t)[VW]) {
    load_n<T, VW>(x + (size_t)e * c.stride, t);
    if (res) {
      float r[VW];
      load_n<T, VW>(res + (size_t)e * c.stride, r);
#pragma unroll
      for (int j = 0; j < VW; ++j) t[j] += r[j];
    }
  };
  auto finish = [&](uint32_t e, const float (&t)[VW], const double (&rstd)[VW], float w) {
    const size_t at = c.base + (size_t)e * c.stride;
    float y[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) y[j] = y_of(t[j], rstd[j], w);
    if (c.live) {
      if (a.s) store_n<T, VW>((T*)a.s + at, t);
      store_n<T, VW>((T*)a.y + at, y);
    }
    if (a.codes) col_codes<T, VW>(a, at, y, c.live);
  };
  if constexpr (N > 0) {
    float t[N][VW], w[N];
    ColWalk<N> at(a, c, wv, NW);
#pragma unroll
    for (int k = 0; k < N; ++k) load_n<T, VW>((const T*)a.x + at.next(), t[k]);
    if (a.res) {
      ColWalk<N> at2(a, c, wv, NW);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float r[VW];
        load_n<T, VW>((const T*)a.res + at2.next(), r);
#pragma unroll
        for (int j = 0; j < VW; ++j) t[k][j] += r[j];
      }
    }
    col_weights<N>(a, wv, NW, w);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (wv + NW * k < (int)a.len)
#pragma unroll
        for (int j = 0; j < VW; ++j) sq[j] = fma((double)t[k][j], (double)t[k][j], sq[j]);
    wave_join<VW>(sq, sm, NW);
    double rstd[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) rstd[j] = rstd_of(sq[j], a);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t e = wv + NW * k;
      if (e < a.len) finish(e, t[k], rstd, w[k]);
    }
  } else {
    for (uint32_t e = wv; e < a.len; e += NW) {
      float t[VW];
      sum_at(e, t);
#pragma unroll
      for (int j = 0; j < VW; ++j) sq[j] = fma((double)t[j], (double)t[j], sq[j]);
    }
    wave_join<VW>(sq, sm, NW);
    double rstd[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) rstd[j] = rstd_of(sq[j], a);
    for (uint32_t e = wv; e < a.len; e += NW) {
      float t[VW];
      sum_at(e, t);
      finish(e, t, rstd, a.w ? a.w[e] : 1.f);
    }
  }
}

// Backward: a workgroup takes every gridDim.x-th tile. N > 0: dw's sums of the lane's positions
// stay in registers and are added across the wave at the end. N = 0: the wave adds them per tile into
// its workgroup's partial.
template <typename T, int N, bool DW>
__global__ void __launch_bounds__(1024) k_norm_cols_bwd(NormArgs a) {
  constexpr int VW = 1;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  double* const sm = (double*)lds;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), NW = blockDim.x >> 6;
  const int lane = threadIdx.x & 63;
  constexpr int M = N > 0 ? N : 1;
  double dw[M];
#pragma unroll
  for (int k = 0; k < M; ++k) dw[k] = 0.0;
  double* part = DW ? a.part + (size_t)blockIdx.x * a.len : nullptr;
  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, turn ^= 1) {
    const ColAt c = col_at<VW>(a, tile);
    const T *x = (const T*)a.x + c.base, *dy = (const T*)a.dy + c.base;
    const T* res = a.res ? (const T*)a.res + c.base : nullptr;
    double sq[VW], dot[VW], rstd[VW];
    float mean[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) sq[j] = dot[j] = 0.0;
    auto join = [&] {
      double* at = sm + turn * NW * 2 * VW * 64;
      double both[2 * VW];
#pragma unroll
      for (int j = 0; j < VW; ++j) both[j] = sq[j], both[VW + j] = dot[j];
      wave_join<2 * VW>(both, at, NW);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        rstd[j] = rstd_of(both[j], a);
        mean[j] = (float)(both[VW + j] * rstd[j] * a.inv64);
      }
    };
    auto finish = [&](uint32_t e, const float (&h)[VW], const float (&g)[VW],
                      const float (&r)[VW], float w) {
      if (!a.y || !c.live) return;
      float d[VW];
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        d[j] = dx_of(g[j] * w, h[j], mean[j], rstd[j]);
        if (res) d[j] += r[j];
      }
      store_n<T, VW>((T*)a.y + c.base + (size_t)e * c.stride, d);
    };
    auto to_h = [&](float (&t)[VW]) {
#pragma unroll
      for (int j = 0; j < VW; ++j) t[j] = h_of(t[j], rstd[j]);
    };
    auto dw_of = [&](const float (&h)[VW], const float (&g)[VW]) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < VW; ++j) s = fmaf(g[j], h[j], s);
      return c.live ? s : 0.f;
    };
    if constexpr (N > 0) {
      float t[N][VW], g[N][VW], r[N][VW], w[N];
      ColWalk<N> at(a, c, wv, NW);
      const bool add = res && a.y;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const size_t o = at.next();
        load_n<T, VW>((const T*)a.x + o, t[k]);
        load_n<T, VW>((const T*)a.dy + o, g[k]);
      }
      ColWalk<N> at2(a, c, wv, NW);
      if (add)
#pragma unroll
        for (int k = 0; k < N; ++k) load_n<T, VW>((const T*)a.res + at2.next(), r[k]);
      col_weights<N>(a, wv, NW, w);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (wv + NW * k < (int)a.len)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            sq[j] = fma((double)t[k][j], (double)t[k][j], sq[j]);
            dot[j] = fma((double)t[k][j], (double)(g[k][j] * w[k]), dot[j]);
          }
      join();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t e = wv + NW * k;
        if (e < a.len) {
          to_h(t[k]);
          if (DW) dw[k] += (double)dw_of(t[k], g[k]);
          finish(e, t[k], g[k], r[k], w[k]);
        }
      }
    } else {
      for (uint32_t e = wv; e < a.len; e += NW) {
        float t[VW], g[VW];
        load_n<T, VW>(x + (size_t)e * c.stride, t);
        load_n<T, VW>(dy + (size_t)e * c.stride, g);
        const float w = a.w ? a.w[e] : 1.f;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          sq[j] = fma((double)t[j], (double)t[j], sq[j]);
          dot[j] = fma((double)t[j], (double)(g[j] * w), dot[j]);
        }
      }
      join();
      for (uint32_t e = wv; e < a.len; e += NW) {
        float t[VW], g[VW];
        load_n<T, VW>(x + (size_t)e * c.stride, t);
        load_n<T, VW>(dy + (size_t)e * c.stride, g);
        to_h(t);
        if (DW) {
          const double s = wave_sum_f64_last((double)dw_of(t, g));
          if (lane == 63) part[e] = tile == blockIdx.x ? s : part[e] + s;
        }
        float r[VW];
        if (res && a.y) load_n<T, VW>(res + (size_t)e * c.stride, r);
        finish(e, t, g, r, a.w ? a.w[e] : 1.f);
      }
    }
  }
  if constexpr (N > 0 && DW) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t e = wv + NW * k;
      const double s = wave_sum_f64_last(dw[k]);
      if (lane == 63 && e < a.len) part[e] = s;
    }
  }
}

// dw[e] = the workgroups' partials in a fixed order: 16 entries of dw by 64 strands, strand q the
// workgroups q, q + 64, ...; four strands of a wave meet by lane moves, the waves in LDS.
__global__ void __launch_bounds__(1024) k_norm_dw(const double* __restrict__ part, int groups,
                                                  uint32_t len, float* __restrict__ dw) {
  __shared__ double sm[16][16];
  const int l = threadIdx.x & 15, wv = threadIdx.x >> 6;
  const uint32_t e = blockIdx.x * 16 + l;
  double s = 0;
  if (e < len) {
#pragma unroll 8
    for (int g = threadIdx.x >> 4; g < groups; g += 64) s += part[(size_t)g * len + e];
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if ((threadIdx.x & 63) < 16) sm[wv][l] = s;
  __syncthreads();
  if (threadIdx.x < 16 && e < len) {
    s = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) s += sm[q][l];
    dw[e] = (float)s;
  }
}

// ---------------------------------------------------------------------------- host
FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.pad_ = 0;
  f.m = d <= 1 ? 0 : ~0ull / d + 1;
  return f;
}

bool al(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// Rows: 16-byte accesses of everything.
bool rows_vec(const NormRequest& r) {
  return r.len % kP == 0 && al(r.x, 16) && al(r.res, 16) && al(r.dy, 16) && al(r.s, 16) &&
         al(r.y, 16) && al(r.w, 16);
}

// Lanes of a row and pieces per lane: a piece each as long as a wave's lanes suffice, idle ones or not. Against
// the fewest idle lanes (50176 rows of bf16, 192 entries: 8 lanes x 3 pieces): 19.1 us for 20.9 backward, 8 rows
// 4.7 for 6.6; 264 entries, half of whose lanes idle: 8.5 for 7.5 forward. A workgroup's 256 lanes only
// where a wave's 3 pieces end: 20000 rows of 768 in 16.4 us with 64 x 2, 22.4 with 256 x 1. More than 3 pieces
// would not leave a backward (three tensors and dw in fp64, 40 registers a piece) two
// workgroups per SIMD.
struct RowShape { int lpr, k; };
RowShape row_shape(int64_t len) {
  const int64_t pieces = (len + kP - 1) / kP;
  for (int lpr : {4, 8, 16, 32})
    if (lpr >= pieces) return {lpr, 1};
  for (int lpr : {64, 256})
    for (int k = 1; k <= 3; ++k)
      if ((int64_t)lpr * k >= pieces) return {lpr, k};
  return {0, 0};
}

// Columns: positions per lane, waves, entries per wave. 4 bytes a lane: 32 x 192 x 784 bf16 forward 9.0 us,
// with 2 bytes 10.7; 16 bytes (fp32) are slower, 128 x 96 x 3136 94 for 90 us forward and 131 for 119
// backward, 4 x 192 x 784 8.4 for 5.9. The backward with three tensors to keep takes one position: bf16
// 128 x 96 x 3136 68.8 us, two 71.5.
struct ColShape { int vw, nw, n; };
ColShape col_shape(const NormRequest& r, bool backward) {
  const bool two = !backward && r.bf16 && r.inner % 2 == 0 && al(r.x, 4) && al(r.res, 4) && al(r.s, 4) &&
                   al(r.y, 4) && al(r.codes, 2);
  const int cap = backward ? kColBwd : kColFwd;
  for (int vw = two ? 2 : 1; vw >= 1; --vw)
    for (int nw : {4, 8, 16})
      for (int n : {4, 6, 8, 12, 16, 24, 32})
        if ((int64_t)nw * n >= r.len && n * vw <= cap) return {vw, nw, n};
  return {1, 16, 0};
}

NormArgs args_of(const NormRequest& r) {
  NormArgs a{};
  a.x = r.x; a.res = r.res; a.w = r.w; a.dy = r.dy; a.s = r.s; a.y = r.y;
  a.codes = r.codes; a.scales = r.scales; a.part = (double*)r.ws;
  a.eps = r.eps; a.inv64 = 1.0 / (double)r.len; a.fmt = r.fmt;
  a.len = (uint32_t)r.len; a.rows = (uint32_t)(r.outer * r.inner);
  a.inner = fast_div((uint32_t)r.inner);
  return a;
}

uint32_t cdiv(int64_t a, int64_t b) { return (uint32_t)((a + b - 1) / b); }

template <typename T, int LPR, int K>
void rows_fwd(const NormArgs& a, bool vec, hipStream_t st) {
  const dim3 grid(cdiv(a.rows, kThreads / LPR));
  if (vec)
    k_norm_rows<T, LPR, K, true><<<grid, kThreads, 0, st>>>(a);
  else
    k_norm_rows<T, LPR, K, false><<<grid, kThreads, 0, st>>>(a);
}
template <typename T, int LPR, int K>
void rows_bwd(NormArgs a, bool vec, bool dw, hipStream_t st, int& groups) {
  a.tiles = cdiv(a.rows, kThreads / LPR);
  groups = dw && a.tiles > (uint32_t)kDwGroups ? kDwGroups : (int)a.tiles;
  const dim3 grid(groups);
  if (vec && dw) k_norm_rows_bwd<T, LPR, K, true, true><<<grid, kThreads, 0, st>>>(a);
  else if (vec) k_norm_rows_bwd<T, LPR, K, true, false><<<grid, kThreads, 0, st>>>(a);
  else if (dw) k_norm_rows_bwd<T, LPR, K, false, true><<<grid, kThreads, 0, st>>>(a);
  else k_norm_rows_bwd<T, LPR, K, false, false><<<grid, kThreads, 0, st>>>(a);
}

// Calls f with the shape as compile-time constants.
template <typename F>
void with_rows(RowShape s, F f) {
  using One = std::integral_constant<int, 1>;
  auto ks = [&](auto lpr) {
    if (s.k == 1) f(lpr, One());
    else if (s.k == 2) f(lpr, std::integral_constant<int, 2>());
    else f(lpr, std::integral_constant<int, 3>());
  };
  if (s.lpr == 4) f(std::integral_constant<int, 4>(), One());
  else if (s.lpr == 8) f(std::integral_constant<int, 8>(), One());
  else if (s.lpr == 16) f(std::integral_constant<int, 16>(), One());
  else if (s.lpr == 32) f(std::integral_constant<int, 32>(), One());
  else if (s.lpr == 64) ks(std::integral_constant<int, 64>());
  else ks(std::integral_constant<int, 256>());
}
template <typename F>
void with_cols(ColShape s, F f) {
  auto ns = [&](auto vw) {
    if (s.n == 4) f(vw, std::integral_constant<int, 4>());
    else if (s.n == 6) f(vw, std::integral_constant<int, 6>());
    else if (s.n == 8) f(vw, std::integral_constant<int, 8>());
    else if (s.n == 12) f(vw, std::integral_constant<int, 12>());
    else if (s.n == 16) f(vw, std::integral_constant<int, 16>());
    else if (s.n == 24) f(vw, std::integral_constant<int, 24>());
    else if (s.n == 32) f(vw, std::integral_constant<int, 32>());
    else f(vw, std::integral_constant<int, 0>());
  };
  if (s.vw == 2) ns(std::integral_constant<int, 2>());
  else ns(std::integral_constant<int, 1>());
}

template <typename T>
bool forward_t(const NormRequest& r, hipStream_t st) {   // whether the codes were written
  NormArgs a = args_of(r);
  if (r.inner == 1) {
    const bool vec = rows_vec(r);
    const bool pack = r.codes && vec && r.len % kCkptGroup == 0 && al(r.codes, 8);
    if (!pack) a.codes = nullptr;
    const RowShape s = row_shape(r.len);
    if (s.lpr == 0) {
      a.codes = nullptr;
      k_norm_rows_long<T><<<dim3(a.rows), kThreads, 0, st>>>(a);
    } else {
      with_rows(s, [&](auto lpr, auto k) {
        rows_fwd<T, decltype(lpr)::value, decltype(k)::value>(a, vec, st);
      });
    }
    return a.codes != nullptr;
  }
  const ColShape s = col_shape(r, false);
  if (r.inner % kCkptGroup != 0) a.codes = nullptr;
  a.tiles = cdiv(a.rows, 64 * s.vw);
  with_cols(s, [&](auto vw, auto n) {
    constexpr int VW = decltype(vw)::value, N = decltype(n)::value;
    if constexpr (N * VW <= kColFwd && (VW == 1 || (sizeof(T) == 2 && N > 0)))
      k_norm_cols<T, VW, N><<<dim3(a.tiles), 64 * s.nw, s.nw * 64 * VW * 8, st>>>(a);
  });
  return a.codes != nullptr;
}

template <typename T>
void backward_t(const NormRequest& r, hipStream_t st) {
  NormArgs a = args_of(r);
  const bool dw = r.dw != nullptr;
  if (!dw) a.part = nullptr;
  int groups = 0;
  if (r.inner == 1) {
    const RowShape s = row_shape(r.len);
    if (s.lpr == 0) {
      groups = a.rows > (uint32_t)kDwGroups ? kDwGroups : (int)a.rows;
      k_norm_rows_long_bwd<T><<<dim3(dw ? groups : a.rows), kThreads, 0, st>>>(a);
    } else {
      const bool vec = rows_vec(r);
      with_rows(s, [&](auto lpr, auto k) {
        rows_bwd<T, decltype(lpr)::value, decltype(k)::value>(a, vec, dw, st, groups);
      });
    }
  } else {
    const ColShape s = col_shape(r, true);
    a.tiles = cdiv(a.rows, 64 * s.vw);
    groups = dw && a.tiles > (uint32_t)kDwGroups ? kDwGroups : (int)a.tiles;
    with_cols(s, [&](auto vw, auto n) {
      constexpr int VW = decltype(vw)::value, N = decltype(n)::value;
      const size_t lds = (size_t)2 * s.nw * 2 * VW * 64 * 8;
      if constexpr (N <= kColBwd && VW == 1) {
        if (dw)
          k_norm_cols_bwd<T, N, true><<<dim3(groups), 64 * s.nw, lds, st>>>(a);
        else
          k_norm_cols_bwd<T, N, false><<<dim3(groups), 64 * s.nw, lds, st>>>(a);
      }
    });
  }
  if (dw)
    k_norm_dw<<<dim3(cdiv(a.len, 16)), 1024, 0, st>>>((const double*)r.ws, groups, a.len, r.dw);
}

}  // namespace

// A partial of dw per workgroup: at most kDwGroups, and no more than there are positions.
size_t norm_backward_workspace(int64_t outer, int64_t len, int64_t inner) {
  const int64_t rows = outer * inner;
  return (size_t)(rows < kDwGroups ? rows : kDwGroups) * (size_t)len * 8;
}

hipError_t launch_norm_forward(const NormRequest& r, hipStream_t st) {
  const bool packed = r.bf16 ? forward_t<uint16_t>(r, st) : forward_t<float>(r, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !r.codes || packed) return e;
  // groups of 32 that run across rows or columns: from the y just written
  return launch_ckpt_pack(r.y, (size_t)r.outer * r.len * r.inner, r.bf16, r.fmt, r.codes, r.scales,
                          st);
}

hipError_t launch_norm_backward(const NormRequest& r, hipStream_t st) {
  if (r.bf16)
    backward_t<uint16_t>(r, st);
  else
    backward_t<float>(r, st);
  return hipGetLastError();
}

}  // namespace wbmm
