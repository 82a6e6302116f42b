// Device pieces of the layer backward from 8-bit checkpoints, shared by the whole-image kernel
// (wbmm_ckptbwd.hip) and the one for any map (wbmm_ckptany.hip), on the bf16 matrix cores at fp32
// accuracy.
//
// An fp32 number is the exact sum of three bf16 numbers (hi, mid, lo: each the rounding of what the
// ones before it leave), a product of two bf16 numbers is exact in fp32, and the matrix cores take
// bf16 at 16 times their fp32 rate (1131 against 154 TFLOP/s in a large library product). So:
//   dT: x comes from a checkpoint and is exact in bf16, G (the mix adjoint of dy) takes its three
//       parts: 3 products, nothing lost;
//   dX, fp32: T and G in three parts each, the 6 largest products (of the others two are up to 2^-25
//       of the term, one 2^-34): 6/16 of the fp32 matrix time;
//   dX, bf16: T is exact, G in two parts (2^-17 of G, before dx's rounding to 2^-8); where G is dy it is
//       exact in one (the any-map kernel's second part is zero there).
//
// A workgroup of 8 waves takes a unit of 32 windows of one channel. dX: K runs over padded window
// rows (two rows of 16 slots per MFMA), an output tile is one window row (16 slots). Then the block of
// M^T between output row y and rows 2s, 2s + 1 depends on y - 2s only: a wave reads each A operand
// once per difference and uses it for every pair (y, s) that shares it, instead of once per pair,
// which would keep LDS busier than the matrix cores. Padding slots and rows are zero in both
// operands.
#pragma once

#include "wbmm_ckpt.hpp"
#include "wbmm_fast.hpp"

namespace wbmm {

constexpr int kWins = 32;                 // windows of a unit
constexpr int kWaves = 8, kT = 64 * kWaves;

// Sizes that follow from the window.
template <int W>
struct CkWin {
  static constexpr int D = W * W, L1 = 2 * W - 1, L = L1 * L1;
  static constexpr int PAIRS = (W + 1) / 2;               // pairs of rows
  static constexpr int PADB = W % 2;                      // a zero block for the row past an odd W
  static constexpr int BLK = (L1 + PADB) * 256;           // bf16 entries of one part of the blocks
  static constexpr int HALF = (W + 1) / 2;
  static constexpr int TILE = 2 * W * 2 * HALF;           // floats of a row-pair tile with its zeros
  // rows of quarter q of the output rows
  static constexpr int ny(int q) { return W / 4 + (q < W % 4 ? 1 : 0); }
  static constexpr int y0(int q) { return q * (W / 4) + (q < W % 4 ? q : W % 4); }
};

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}
// The NS leading bf16 parts of a pair of fp32 numbers, packed.
template <int NS>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&p)[NS]) {
#pragma unroll
  for (int q = 0; q < NS; ++q) {
    p[q] = pk_bf16(a, b);
    if (q + 1 < NS) {
      a -= __uint_as_float(p[q] << 16);
      b -= __uint_as_float(p[q] & 0xffff0000u);
    }
  }
}

// Sums over the lane's row of 16 lanes, left in its last lane.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum_f32_last(float x) {
  x += dpp_f32<0x111>(x);
  x += dpp_f32<0x112>(x);
  x += dpp_f32<0x114>(x);
  x += dpp_f32<0x118>(x);
  return x;
}


// Blocks of M^T: part q, difference d = y_i - y_j + W - 1 (after a zero block for odd W), entry
// [x_i][x_j] = T[-(y_i - y_j)][x_j - x_i] for x_j < W, 0 for the padding slots.
template <int W, int NT>
__device__ __forceinline__ void table_blocks(const float* Tf, uint32_t* blk, int tid) {
  typedef CkWin<W> C;
  const int xi = (tid & 127) >> 3, xj = 2 * (tid & 7);
  const int c = xj - xi + W - 1;             // column of the table
  const bool in0 = xj < W && c >= 0 && c < C::L1, in1 = xj + 1 < W && c + 1 >= 0 && c + 1 < C::L1;
  for (int d = (tid >> 7) - C::PADB; d < C::L1; d += kT / 128) {
    const float* row = Tf + (C::L1 - 1 - (d < 0 ? 0 : d)) * C::L1;
    const float a = in0 && d >= 0 ? row[c] : 0.f, b = in1 && d >= 0 ? row[c + 1] : 0.f;
    uint32_t p[NT];
    split2<NT>(a, b, p);
#pragma unroll
    for (int q = 0; q < NT; ++q) blk[q * (C::BLK / 2) + (d + C::PADB) * 128 + (tid & 127)] = p[q];
  }
}

// dX of a lane's window (16 windows a wave) for the NY window rows from Y0 on, K in runs of 4 pairs of
// rows to keep the registers of 4 waves per SIMD. gw: the window's G, rows IW floats apart (even).
// acc[y]: row Y0 + y, slots 4 (lane / 16) + 0..3 of window lane % 16.
template <int W, bool F32, int NG, int Y0, int NY, int IW>
__device__ __forceinline__ void dx_rows(const float* gw, const uint16_t* blk, int lane,
                                        v4f (&acc)[NY]) {
  typedef CkWin<W> C;
  constexpr int NT = F32 ? 3 : 1;
  const int kg = lane >> 4;
  const bool odd = kg & 1, second = kg >> 1;
#pragma unroll
  for (int y = 0; y < NY; ++y) acc[y] = v4f{0.f, 0.f, 0.f, 0.f};
  const float* g = gw + (kg >> 1) * IW + 8 * (kg & 1);
  const uint16_t* ab = blk + (W - 1 + C::PADB - (kg >> 1)) * 256 + (lane & 15) * 16 + 8 * (kg & 1);
#pragma unroll
  for (int s0 = 0; s0 < C::PAIRS; s0 += 4) {
    const int ns = C::PAIRS - s0 < 4 ? C::PAIRS - s0 : 4;
    // a run's B operands are formed here, not ahead of the quarters' branches together with the
    // other run's (the registers would not hold them)
    if constexpr (NG > 2) asm volatile("" ::: "memory");
    u32x4 Bf[4][NG];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= ns) continue;
      const bool cutoff = W % 2 == 1 && s0 + s == C::PAIRS - 1;   // the second row is past the window
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f2 v = *(const f2*)(g + 2 * (s0 + s) * IW + 2 * j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // slots past the window's row
          if (2 * j + e >= W) v[e] = 0.f;
          else if (8 + 2 * j + e >= W) v[e] = odd ? 0.f : v[e];
          if (cutoff) v[e] = second ? 0.f : v[e];
        }
        uint32_t p[NG];
        split2<NG>(v[0], v[1], p);
#pragma unroll
        for (int q = 0; q < NG; ++q) Bf[s][q][j] = p[q];
      }
    }
    // differences d = y - 2 (s0 + s)
#pragma unroll
    for (int dd = 0; dd < NY + 6; ++dd) {
      const int d = Y0 - 2 * (s0 + ns - 1) + dd;
      if (d > Y0 + NY - 1 - 2 * s0) continue;
      u32x4 A[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) A[q] = *(const u32x4*)(ab + q * C::BLK + d * 256);
      // smallest terms first
#pragma unroll
      for (int qt = NT - 1; qt >= 0; --qt)
#pragma unroll
        for (int qg = NG - 1; qg >= 0; --qg) {
          if (qt + qg > 2) continue;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int y = d + 2 * (s0 + s) - Y0;
            if (s >= ns || y < 0 || y >= NY) continue;
            acc[y] = mfma_bf16(A[qt], Bf[s][qg], acc[y]);
          }
        }
    }
  }
}

// Place of pixel p's eight windows 8g .. 8g + 7 in a [pixel][window] operand (elements): the groups
// of a pixel are swapped round by the pixel, so that 8 neighbour pixels' groups cover all banks.
__device__ __forceinline__ int slot_of(int p, int g) { return p * kWins + 8 * (g ^ ((p >> 1) & 3)); }

// Row offsets dy ordered 0, +1, -1, +2, ... and dealt to the 8 waves in a snake (w = 14: 24 to 26 of
// the 196 row pairs each).
template <int W, int Q, int J>
struct Row8 {
  static constexpr int T = 8 * J + ((J & 1) ? 7 - Q : Q);
  static constexpr bool valid = T < 2 * W - 1;
  static constexpr int dy = T == 0 ? 0 : ((T & 1) ? (T + 1) / 2 : -(T / 2));
};

// Row pairs of wave Q: acc_j[x1][x2] = sum over y1 - y2 = dy_j and the 32 windows of G[y1][x1]
// x[y2][x2] (one MFMA per pair and part of G). ops: NS parts of G, x after the third, each
// [pixel][window]. The leading parts' products have a chain of their own: every step rounds to the
// chain's size, and one chain for all parts left 1.0e-4 in sums of size 500.
template <int W, int Q, int NS>
__device__ __forceinline__ void dt_rows(const uint16_t* ops, int lane, v4f (&acc)[4]) {
  constexpr int PIX = kWins * W * W;
  const int x = (lane & 15) < W ? lane & 15 : W - 1, kg = lane >> 4;
  constexpr int NC = NS > 1 ? 2 : 1;
  v4f ch[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) ch[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  u32x4 X[W];
#pragma unroll
  for (int y = 0; y < W; ++y) X[y] = *(const u32x4*)(ops + 3 * PIX + slot_of(y * W + x, kg));
#pragma unroll
  for (int y1 = 0; y1 < W; ++y1) {
    u32x4 A[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) A[q] = *(const u32x4*)(ops + q * PIX + slot_of(y1 * W + x, kg));
#pragma unroll
    for (int q = NS - 1; q >= 0; --q) {
      const int i = q > 0 ? NC - 1 : 0;
#define WBMM_CK_STEP(J)                                                            \
  if constexpr (Row8<W, Q, J>::valid) {                                            \
    const int y2 = y1 - Row8<W, Q, J>::dy;                                         \
    if (y2 >= 0 && y2 < W)                                                         \
      ch[i][J] = mfma_bf16(A[q], X[y2 < 0 ? 0 : (y2 < W ? y2 : 0)], ch[i][J]);     \
  }
      WBMM_CK_STEP(0) WBMM_CK_STEP(1) WBMM_CK_STEP(2) WBMM_CK_STEP(3)
#undef WBMM_CK_STEP
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = NC > 1 ? ch[0][j] + ch[NC - 1][j] : ch[0][j];
}

// Diagonal sums of the wave's tiles into (ADD: onto) the workgroup's fp64 partial: pT[dy][dx] = sum
// over x1 - x2 = dx of acc[x1][x2]. Entry (x1, x2) lies at W - 1 + (2W - 1) x1 + x2 among zeros, so
// diagonal dx is every 2W-th float from W - 1 - dx on, whatever its length: lane (half, dx) adds half
// the rows of it.
template <int W, int Q>
__device__ __forceinline__ void dt_partial(float* scr, const v4f (&acc)[4], double* pT, int lane,
                                           bool add) {
  typedef CkWin<W> C;
  constexpr int NV = C::TILE;   // float4 of the four tiles
#pragma unroll
  for (int k = 0; k < (NV + 63) / 64; ++k)
    if (k * 64 + lane < NV) *(v4f*)(scr + 4 * (k * 64 + lane)) = v4f{0.f, 0.f, 0.f, 0.f};
  wave_sync_lds();
  const int x2 = lane & 15, g = lane >> 4;
  if (x2 < W) {
    float* p = scr + W - 1 + C::L1 * 4 * g + x2;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (12 + r < W || 4 * g + r < W) p[j * C::TILE + C::L1 * r] = acc[j][r];
  }
  wave_sync_lds();
  const int dd = lane & 31, dc = dd < C::L1 ? dd : C::L1 - 1;
  const float* q = scr + 2 * (W - 1) - dc + (lane >> 5) * C::HALF * 2 * W;
#define WBMM_CK_SUM(J)                                                             \
  if constexpr (Row8<W, Q, J>::valid) {                                            \
    double s = 0.0;                                                                \
    _Pragma("unroll") for (int k = 0; k < C::HALF; ++k) s += (double)q[J * C::TILE + 2 * W * k]; \
    s += __shfl_down(s, 32, 64);                                                   \
    if (lane < C::L1) {                                                            \
      double* o = pT + (Row8<W, Q, J>::dy + W - 1) * C::L1 + lane;                 \
      *o = add ? *o + s : s;                                                       \
    }                                                                              \
  }
  WBMM_CK_SUM(0) WBMM_CK_SUM(1) WBMM_CK_SUM(2) WBMM_CK_SUM(3)
#undef WBMM_CK_SUM
}

}  // namespace wbmm
