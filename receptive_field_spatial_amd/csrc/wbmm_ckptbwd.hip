// The layer backward from 8-bit checkpoints for w = 14 on whole NCHW images of 14, 28 or 56 pixels
// a side (table input; fp32, or bf16 dy, T and dx), on the bf16 matrix cores at fp32 accuracy.
//
// An fp32 number is the exact sum of three bf16 numbers (hi, mid, lo: each the rounding of what the
// ones before it leave), a product of two bf16 numbers is exact in fp32, and the matrix cores take
// bf16 at 16 times their fp32 rate (1131 against 154 TFLOP/s in a large library product). So:
//   dT: x comes from a checkpoint and is exact in bf16, G (the mix adjoint of dy) takes its three
//       parts: 3 products, nothing lost;
//   dX, fp32: T and G in three parts each, the 6 products that reach 2^-24 (what is left out is
//       below 2^-26 of each term): 6/16 of the fp32 matrix time;
//   dX, bf16: T is exact, G in two parts (2^-17 before one rounding to 2^-9); 1 part without mix.
//
// One workgroup of 8 waves takes a unit of 32 windows (whole images) of one channel through
//   dy, z, x loaded in 16-byte pieces, x kept in registers as codes | mix adjoint and dWmix sums by
//   column strips, dy -> G in LDS as fp32 planes | table blocks | dX | G and x transposed to
//   [pixel][window] | dT by row pairs | fp64 partial of the unit.
// Every phase's LDS lies in the same 54 KB beside G's 25 KB, so two workgroups (4 waves per SIMD)
// share a CU and one's loads and vector work run beside the other's matrix work. Partials are summed
// in a fixed order by k_bwd_reduce.
//
// dX: K runs over padded window rows (two rows of 16 slots per MFMA), an output tile is one window
// row (16 slots, 14 used). Then the block of M^T between output row y and rows 2s, 2s + 1 depends on
// y - 2s only: a wave reads each A operand once per difference and uses it for every pair (y, s)
// that shares it, instead of once per pair, which would keep LDS busier than the matrix cores. Slots
// 14 and 15 are zero in both operands' K.
#include "wbmm_ckpt.hpp"
#include "wbmm_fast.hpp"

namespace wbmm {

namespace {

struct CkptBwdArgs {
  int B, C, groups;            // units per channel
  const uint8_t* xc;
  const uint8_t* xs;
  const uint8_t* zc;
  const uint8_t* zs;
  const void* T;
  const void* dy;
  const float* mixw;
  void* dx;
  double* partT;
  double* partW;
  int fmt, want_dT, want_dW;
};

constexpr int kW = 14, kD = kW * kW, kL1 = 2 * kW - 1, kL = kL1 * kL1;
constexpr int kWins = 32;                 // windows of a unit
constexpr int kPix = kWins * kD;          // its pixels
constexpr int kPieces = kPix / 4;         // 4-element pieces (a piece lies in one image and group)
constexpr int kWaves = 8, kT = 64 * kWaves;
constexpr int kIter = (kPieces + kT - 1) / kT;
constexpr int kTile = 14 * 28;            // floats of a row-pair tile with its zeros
constexpr int kBlk = kL1 * 256;           // bf16 entries of one part of the table blocks

// LDS (bytes): G | U | X, with U the table blocks (dX), dy and z (mix), or the start of the
// [pixel][window] operands (dT), which run on into X; X holds T as fp32, then x as bf16.
constexpr int kOffU = kPix * 4;
constexpr int kOffX = kOffU + 3 * kBlk * 2;
constexpr int kOffR = kOffX + kPix * 2;
constexpr int kLds = kOffR + kWaves * 9 * 4;
static_assert(lds_fits(kLds, 2), "two workgroups per CU");
static_assert(kPix * 6 <= 3 * kBlk * 2, "dy and z fit in U");
static_assert(kOffU + 4 * kPix * 2 <= kOffR, "the four operands of dT fit in U and X");
static_assert(kWaves * 4 * kTile * 4 <= 4 * kPix * 2, "the partial's tiles fit there too");
static_assert(kL * 4 <= kPix * 2, "T fits in X");

template <int IH>
struct Img {
  static constexpr int IW = IH, PLANE = IH * IH, NWX = IH / kW, NWIN = NWX * NWX;
  static constexpr int IMGS = kWins / NWIN;
  // offset of window n's origin in the unit's planes
  __device__ static constexpr int win(int n) {
    return (n / NWIN) * PLANE + ((n % NWIN) / NWX) * kW * IW + (n % NWX) * kW;
  }
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

// Sum over the wave's lanes, left in lane 63 (as wave_sum_f64_last).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_f32(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROW_MASK, 0xf, true));
}
__device__ __forceinline__ float wave_sum_f32_last(float x) {
  x += dpp_f32<0x111, 0xf>(x);
  x += dpp_f32<0x112, 0xf>(x);
  x += dpp_f32<0x114, 0xf>(x);
  x += dpp_f32<0x118, 0xf>(x);
  x += dpp_f32<0x142, 0xa>(x);
  x += dpp_f32<0x143, 0xc>(x);
  return x;
}

// Four codes of a checkpoint, decoded, as two packed bf16 pairs (exact).
__device__ __forceinline__ uint2 decode_piece(uint32_t w, uint32_t scale, int fmt) {
  float v[4];
  ckpt_decode4(w, fmt, v);
  const float f = ckpt_factor(scale);
  return make_uint2(pk_bf16(v[0] * f, v[1] * f), pk_bf16(v[2] * f, v[3] * f));
}

// G = mix adjoint of dy and the wave's dWmix sums. A lane walks a strip of 14 rows of one image
// column with a 3 x 3 window of dy, its neighbour columns on the neighbour lanes; 56 lanes hold
// whole image rows (four images of 14, two strips of 28, one of 56).
template <int IH, bool WANTW>
__device__ __forceinline__ void mix_adjoint(const float* D, const uint16_t* Z, float* G,
                                            const float* __restrict__ w9, float* red, int wave,
                                            int lane) {
  typedef Img<IH> I;
  constexpr int SH = 14, RB = 7;
  float wr[9], dw[9];
#pragma unroll
  for (int q = 0; q < 9; ++q) wr[q] = w9[8 - q], dw[q] = 0.f;
  const bool active = lane < 56;
  const int l = active ? lane : 0, strip = wave * (56 / IH) + l / IH, v = l % IH;
  const int img = strip / (IH / SH), h0 = strip % (IH / SH) * SH;
  const int col = img * I::PLANE + v;
  const bool hasL = v > 0, hasR = v + 1 < I::IW;
  auto expand = [&](float c, float (&w)[3]) {
    const float a = lane_left(c), b = lane_right(c);
    w[0] = hasL ? a : 0.f;
    w[1] = c;
    w[2] = hasR ? b : 0.f;
  };
  float w[3][3];
  {
    const float t = D[col + (h0 > 0 ? h0 - 1 : 0) * I::IW];
    expand(h0 > 0 ? t : 0.f, w[0]);
    expand(D[col + h0 * I::IW], w[1]);
  }
#pragma unroll
  for (int hb = 0; hb < SH; hb += RB) {
    float nx[RB], z[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int h = h0 + hb + j;
      if (hb + j + 1 < SH) {
        nx[j] = D[col + (h + 1) * I::IW];
      } else {   // the row below the strip
        const float t = D[col + (h + 1 < IH ? h + 1 : h) * I::IW];
        nx[j] = h + 1 < IH ? t : 0.f;
      }
      if constexpr (WANTW) z[j] = bf2f(Z[col + h * I::IW]);
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      expand(nx[j], w[2]);
      float g = 0.f;
#pragma unroll
      for (int q = 0; q < 9; ++q) g = fmaf(wr[q], w[q / 3][q % 3], g);
      if (active) G[col + (h0 + hb + j) * I::IW] = g;
      if constexpr (WANTW) {
#pragma unroll
        for (int q = 0; q < 9; ++q) dw[q] = fmaf(z[j], w[2 - q / 3][2 - q % 3], dw[q]);
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        w[0][t] = w[1][t];
        w[1][t] = w[2][t];
      }
    }
  }
  if constexpr (WANTW) {
#pragma unroll
    for (int q = 0; q < 9; ++q) {
      const float s = wave_sum_f32_last(active ? dw[q] : 0.f);
      if (lane == 63) red[wave * 9 + q] = s;
    }
  }
}

// Blocks of M^T: part q, difference d = y_i - y_j + 13, entry [x_i][x_j] = T[-(y_i - y_j)][x_j - x_i]
// for x_j < 14, 0 for the padding slots.
template <int NT>
__device__ __forceinline__ void table_blocks(const float* Tf, uint32_t* blk, int tid) {
  const int xi = (tid & 127) >> 3, xj = 2 * (tid & 7);
  const int c = xj - xi + kW - 1;            // column of the table, -2 .. 27
  const bool in0 = xj < kW && c >= 0 && c < kL1, in1 = xj < kW && c + 1 >= 0 && c + 1 < kL1;
  for (int d = tid >> 7; d < kL1; d += kT / 128) {
    const float* row = Tf + (kL1 - 1 - d) * kL1;
    const float a = in0 ? row[c] : 0.f, b = in1 ? row[c + 1] : 0.f;
    uint32_t p[NT];
    split2<NT>(a, b, p);
#pragma unroll
    for (int q = 0; q < NT; ++q) blk[q * (kBlk / 2) + d * 128 + (tid & 127)] = p[q];
  }
}

// dX of 16 windows and the NY window rows from Y0 on, K in two runs (4 and 3 pairs of rows) to keep
// the registers of 4 waves per SIMD.
template <int IH, bool F32, int NG, int Y0, int NY>
__device__ __forceinline__ void dx_rows(const CkptBwdArgs& a, const float* G, const uint16_t* blk,
                                        size_t base, int cp, int nimg, int wu, int lane) {
  typedef Img<IH> I;
  constexpr int NT = F32 ? 3 : 1;
  const int n = wu * 16 + (lane & 15), kg = lane >> 4;
  const bool odd = kg & 1;
  v4f acc[NY];
#pragma unroll
  for (int y = 0; y < NY; ++y) acc[y] = v4f{0.f, 0.f, 0.f, 0.f};
  const float* g = G + I::win(n) + (kg >> 1) * I::IW + 8 * (kg & 1);
  const uint16_t* ab = blk + (kW - 1 - (kg >> 1)) * 256 + (lane & 15) * 16 + 8 * (kg & 1);
#pragma unroll
  for (int s0 = 0; s0 < 7; s0 += 4) {
    const int ns = s0 == 0 ? 4 : 3;
    u32x4 Bf[4][NG];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= ns) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f2 v = *(const f2*)(g + 2 * (s0 + s) * I::IW + 2 * j);
        if (j == 3) {   // slots 14 and 15
          v[0] = odd ? 0.f : v[0];
          v[1] = odd ? 0.f : v[1];
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
      for (int q = 0; q < NT; ++q) A[q] = *(const u32x4*)(ab + q * kBlk + d * 256);
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
  const int im = n / I::NWIN;
  if (im >= nimg) return;
  const size_t o = base + (size_t)(im * cp) + (I::win(n) - im * I::PLANE) + 4 * kg;
#pragma unroll
  for (int y = 0; y < NY; ++y) {
    const size_t at = o + (Y0 + y) * I::IW;
    if constexpr (F32) {
      float* p = (float*)a.dx + at;
      *(f2*)p = f2{acc[y][0], acc[y][1]};
      if (kg < 3) *(f2*)(p + 2) = f2{acc[y][2], acc[y][3]};
    } else {
      uint16_t* p = (uint16_t*)a.dx + at;
      *(uint32_t*)p = pk_bf16(acc[y][0], acc[y][1]);
      if (kg < 3) *(uint32_t*)(p + 2) = pk_bf16(acc[y][2], acc[y][3]);
    }
  }
}

// Place of pixel p's eight windows 8g .. 8g + 7 in a [pixel][window] operand (elements): the groups
// of a pixel are swapped round by the pixel, so that 8 neighbour pixels' groups cover all banks.
__device__ __forceinline__ int slot_of(int p, int g) { return p * kWins + 8 * (g ^ ((p >> 1) & 3)); }

// Row offsets dy ordered 0, +1, -1, +2, ... and dealt to the 8 waves in a snake: 24 to 26 of the 196
// row pairs each.
template <int Q, int J>
struct Row8 {
  static constexpr int T = 8 * J + ((J & 1) ? 7 - Q : Q);
  static constexpr bool valid = T < kL1;
  static constexpr int dy = T == 0 ? 0 : ((T & 1) ? (T + 1) / 2 : -(T / 2));
};

// Row pairs of wave Q: acc_j[x1][x2] = sum over y1 - y2 = dy_j and the 32 windows of G[y1][x1]
// x[y2][x2] (one MFMA per pair and part of G). The leading parts' products have a chain of their
// own: every step rounds to the chain's size, and one chain for all parts left 1.0e-4 in sums of
// size 500.
template <int Q, int NS>
__device__ __forceinline__ void dt_rows(const uint16_t* ops, int lane, v4f (&acc)[4]) {
  const int x = (lane & 15) < kW ? lane & 15 : kW - 1, kg = lane >> 4;
  constexpr int NC = NS > 1 ? 2 : 1;
  v4f ch[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) ch[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  u32x4 X[kW];
#pragma unroll
  for (int y = 0; y < kW; ++y) X[y] = *(const u32x4*)(ops + 3 * kPix + slot_of(y * kW + x, kg));
#pragma unroll
  for (int y1 = 0; y1 < kW; ++y1) {
    u32x4 A[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) A[q] = *(const u32x4*)(ops + q * kPix + slot_of(y1 * kW + x, kg));
#pragma unroll
    for (int q = NS - 1; q >= 0; --q) {
      const int i = q > 0 ? NC - 1 : 0;
#define WBMM_CK_STEP(J)                                                            \
  if constexpr (Row8<Q, J>::valid) {                                               \
    const int y2 = y1 - Row8<Q, J>::dy;                                            \
    if (y2 >= 0 && y2 < kW)                                                        \
      ch[i][J] = mfma_bf16(A[q], X[y2 < 0 ? 0 : (y2 < kW ? y2 : 0)], ch[i][J]);    \
  }
      WBMM_CK_STEP(0) WBMM_CK_STEP(1) WBMM_CK_STEP(2) WBMM_CK_STEP(3)
#undef WBMM_CK_STEP
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = NC > 1 ? ch[0][j] + ch[NC - 1][j] : ch[0][j];
}

// Diagonal sums of the wave's tiles into the unit's fp64 partial: pT[dy][dx] = sum over
// x1 - x2 = dx of acc[x1][x2]. Entry (x1, x2) lies at 13 + 27 x1 + x2 among zeros, so diagonal dx is
// every 28th float from 13 - dx on, whatever its length: lane (half, dx) adds seven rows of it.
template <int Q>
__device__ __forceinline__ void dt_partial(float* scr, const v4f (&acc)[4], double* pT, int lane) {
  constexpr int NV = 4 * kTile / 4;   // float4 of the four tiles
#pragma unroll
  for (int k = 0; k < (NV + 63) / 64; ++k)
    if (k * 64 + lane < NV) *(v4f*)(scr + 4 * (k * 64 + lane)) = v4f{0.f, 0.f, 0.f, 0.f};
  wave_sync_lds();
  const int x2 = lane & 15, g = lane >> 4;
  if (x2 < kW) {
    float* p = scr + 13 + 27 * 4 * g + x2;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < 2 || g < 3) p[j * kTile + 27 * r] = acc[j][r];
  }
  wave_sync_lds();
  const int dd = lane & 31, dc = dd < kL1 ? dd : kL1 - 1;
  const float* q = scr + 26 - dc + (lane >> 5) * 7 * 28;
#define WBMM_CK_SUM(J)                                                             \
  if constexpr (Row8<Q, J>::valid) {                                               \
    double s = 0.0;                                                                \
    _Pragma("unroll") for (int k = 0; k < 7; ++k) s += (double)q[J * kTile + 28 * k]; \
    const double o = __shfl_down(s, 32, 64);                                       \
    if (lane < kL1) pT[(Row8<Q, J>::dy + kW - 1) * kL1 + lane] = s + o;            \
  }
  WBMM_CK_SUM(0) WBMM_CK_SUM(1) WBMM_CK_SUM(2) WBMM_CK_SUM(3)
#undef WBMM_CK_SUM
}

template <int IH, bool F32, bool MIX>
__global__ void __launch_bounds__(kT) __attribute__((amdgpu_waves_per_eu(4, 4)))
k_bwd_ckpt(CkptBwdArgs a) {
  typedef Img<IH> I;
  constexpr int NT = F32 ? 3 : 1;                       // parts of T
  constexpr int NS = F32 || MIX ? 3 : 1;                // parts of G in dT
  constexpr int NG = F32 ? 3 : (MIX ? 2 : 1);           // parts of G in dX
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_c[];
  float* G = (float*)smem_c;
  unsigned char* U = smem_c + kOffU;
  float* Tf = (float*)(smem_c + kOffX);
  float* red = (float*)(smem_c + kOffR);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x / a.groups, img0 = (blockIdx.x % a.groups) * I::IMGS;
  const int cp = a.C * I::PLANE;
  const size_t base = ((size_t)img0 * a.C + c) * I::PLANE;
  const int nimg = a.B - img0 < I::IMGS ? a.B - img0 : I::IMGS;
  const bool wantW = MIX && a.want_dW;

  // ---- loads: T, dy, z, x in flight together
  constexpr int TQ = (kL + kT - 1) / kT;
  float tv[TQ];
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int q = tid + j * kT, qc = q < kL ? q : kL - 1;
    tv[j] = F32 ? ((const float*)a.T)[(size_t)c * kL + qc]
                : bf2f(((const uint16_t*)a.T)[(size_t)c * kL + qc]);
  }
  typedef uint32_t raw_t __attribute__((ext_vector_type(F32 ? 4 : 2)));
  raw_t dv[kIter];
  uint32_t xw[kIter], xsc[kIter], zw[kIter], zsc[kIter];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = 4 * (tid + it * kT), im = e / I::PLANE;
    // pieces past the unit's images read its first ones and count as zeros below
    const bool in = im < nimg;
    const size_t o = base + (in ? (size_t)(im * cp) + (e - im * I::PLANE) : 0);
    dv[it] = F32 ? *(const raw_t*)((const float*)a.dy + o) : *(const raw_t*)((const uint16_t*)a.dy + o);
    if (wantW) {
      zw[it] = *(const uint32_t*)(a.zc + o);
      zsc[it] = a.zs[o / kCkptGroup];
    }
    if (a.want_dT) {
      xw[it] = *(const uint32_t*)(a.xc + o);
      xsc[it] = a.xs[o / kCkptGroup];
    }
    if (!in) {
#pragma unroll
      for (int j = 0; j < (F32 ? 4 : 2); ++j) dv[it][j] = 0;
      zw[it] = xw[it] = 0;
      zsc[it] = xsc[it] = 127;
    }
  }
#pragma unroll
  for (int j = 0; j < TQ; ++j)
    if (tid + j * kT < kL) Tf[tid + j * kT] = tv[j];
  float* D = MIX ? (float*)U : G;
  uint16_t* Z = (uint16_t*)(U + kPix * 4);
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = 4 * (tid + it * kT);
    if (e >= kPix) continue;
    v4f v;
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(dv[it][j]);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[2 * j] = __uint_as_float(dv[it][j] << 16);
        v[2 * j + 1] = __uint_as_float(dv[it][j] & 0xffff0000u);
      }
    }
    *(v4f*)(D + e) = v;
    if (wantW) *(uint2*)(Z + e) = decode_piece(zw[it], zsc[it], a.fmt);
  }
  __syncthreads();
  if constexpr (MIX) {
    if (wantW)
      mix_adjoint<IH, true>(D, Z, G, a.mixw + c * 9, red, wave, lane);
    else
      mix_adjoint<IH, false>(D, Z, G, a.mixw + c * 9, red, wave, lane);
    __syncthreads();
    if (wantW && tid < 9) {
      double s = 0.0;
      for (int w = 0; w < kWaves; ++w) s += (double)red[w * 9 + tid];
      a.partW[(size_t)blockIdx.x * 9 + tid] = s;
    }
  }

  // ---- dX
  if (a.dx) {
    table_blocks<NT>(Tf, (uint32_t*)U, tid);
    __syncthreads();
    const uint16_t* blk = (const uint16_t*)U;
    switch (wave >> 1) {   // 4, 4, 3 and 3 rows
      case 0: dx_rows<IH, F32, NG, 0, 4>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      case 1: dx_rows<IH, F32, NG, 4, 4>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      case 2: dx_rows<IH, F32, NG, 8, 3>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      default: dx_rows<IH, F32, NG, 11, 3>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
    }
  }
  if (!a.want_dT) return;

  // ---- dT: x to LDS as bf16 planes (over T), then both operands to [pixel][window]
  __syncthreads();
  uint16_t* xl = (uint16_t*)(smem_c + kOffX);
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = 4 * (tid + it * kT);
    if (e < kPix) *(uint2*)(xl + e) = decode_piece(xw[it], xsc[it], a.fmt);
  }
  __syncthreads();
  uint16_t* ops = (uint16_t*)U;
  constexpr int TI = (kD * 4 + kT - 1) / kT;
  u32x4 xt[TI];
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int t = tid + i * kT, tt = t < kD * 4 ? t : 0, g = tt / kD, p = tt % kD;
    const int o = I::win(8 * g) + (p / kW) * I::IW + p % kW;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xt[i][j] = (uint32_t)xl[o + I::win(2 * j)] | ((uint32_t)xl[o + I::win(2 * j + 1)] << 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int t = tid + i * kT, tt = t < kD * 4 ? t : 0, g = tt / kD, p = tt % kD;
    const int o = I::win(8 * g) + (p / kW) * I::IW + p % kW;
    u32x4 part[NS];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t q2[NS];
      split2<NS>(G[o + I::win(2 * j)], G[o + I::win(2 * j + 1)], q2);
#pragma unroll
      for (int q = 0; q < NS; ++q) part[q][j] = q2[q];
    }
    if (t < kD * 4) {
      const int at = slot_of(p, g);
#pragma unroll
      for (int q = 0; q < NS; ++q) *(u32x4*)(ops + q * kPix + at) = part[q];
      *(u32x4*)(ops + 3 * kPix + at) = xt[i];
    }
  }
  __syncthreads();
  v4f acc[4];
  float* scr = (float*)U + wave * 4 * kTile;
  double* pT = a.partT + (size_t)blockIdx.x * kL;
#define WBMM_CK_WAVE(Q)              \
  case Q:                            \
    dt_rows<Q, NS>(ops, lane, acc);  \
    __syncthreads();                 \
    dt_partial<Q>(scr, acc, pT, lane); \
    break;
  switch (wave) {   // every wave has read its operands before the tiles go over them
    WBMM_CK_WAVE(0) WBMM_CK_WAVE(1) WBMM_CK_WAVE(2) WBMM_CK_WAVE(3)
    WBMM_CK_WAVE(4) WBMM_CK_WAVE(5) WBMM_CK_WAVE(6) WBMM_CK_WAVE(7)
  }
#undef WBMM_CK_WAVE
}

int images_per_unit(int H) { return kWins / ((H / kW) * (H / kW)); }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

template <int IH>
hipError_t launch_shape(const CkptBwdArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)a.C * a.groups);
  auto go = [&](auto fn) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    return e != hipSuccess ? e : launch_main(fn, grid, dim3(kT), kLds, st, a);
  };
  if (bf16) return a.mixw ? go(k_bwd_ckpt<IH, false, true>) : go(k_bwd_ckpt<IH, false, false>);
  return a.mixw ? go(k_bwd_ckpt<IH, true, true>) : go(k_bwd_ckpt<IH, true, false>);
}

}  // namespace

// Shapes of the fused kernel; its 32-bit offsets within a unit (up to 32 images apart) must hold.
bool fast_ckpt_shape(int C, int H, int W, int w, int layout) {
  return layout == 0 && w == kW && H == W && (H == 14 || H == 28 || H == 56) &&
         (size_t)images_per_unit(H) * C * H * W < ((size_t)1 << 31);
}

size_t fast_ckpt_workspace(const BwdCkptRequest& r) {
  const int g = (r.B + images_per_unit(r.H) - 1) / images_per_unit(r.H);
  return up256((size_t)r.C * g * kL * 8) + up256((size_t)r.C * g * 9 * 8);
}

hipError_t launch_backward_ckpt_fast(const BwdCkptRequest& r, hipStream_t st) {
  CkptBwdArgs a{};
  a.B = r.B;
  a.C = r.C;
  a.groups = (r.B + images_per_unit(r.H) - 1) / images_per_unit(r.H);
  a.xc = r.xc; a.xs = r.xs; a.zc = r.zc; a.zs = r.zs;
  a.T = r.T; a.dy = r.dy; a.mixw = r.mixw; a.dx = r.dx;
  a.partT = (double*)r.ws;
  a.partW = (double*)((unsigned char*)r.ws + up256((size_t)r.C * a.groups * kL * 8));
  a.fmt = r.fmt;
  a.want_dT = r.dT != nullptr;
  a.want_dW = r.mixw && r.dmixw;
  hipError_t e = r.H == 14   ? launch_shape<14>(a, r.bf16, st)
                 : r.H == 28 ? launch_shape<28>(a, r.bf16, st)
                             : launch_shape<56>(a, r.bf16, st);
  if (e != hipSuccess || (!a.want_dT && !a.want_dW)) return e;
  return launch_bwd_reduce(a.partT, a.want_dW ? a.partW : nullptr, a.groups, r.C, kL, r.dT,
                           a.want_dW ? r.dmixw : nullptr, st);
}

}  // namespace wbmm
