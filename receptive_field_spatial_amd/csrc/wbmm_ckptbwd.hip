// The layer backward from 8-bit checkpoints for w = 14 on whole NCHW images of 14, 28 or 56 pixels
// a side (table input; fp32, or bf16 dy, T and dx), on the pieces of wbmm_ckptbwd.hpp.
//
// A workgroup takes a unit of 32 windows (whole images) of one channel through
//   dy and z loaded in 4-element pieces | mix adjoint and dWmix sums by column strips, dy -> G in LDS
//   as fp32 planes | x's codes loaded into registers, table blocks | dX | G and x transposed to
//   [pixel][window] | dT by row pairs | fp64 partial of the unit.
// Every phase's LDS lies in the same 54 KB beside G's 25 KB, so two workgroups (4 waves per SIMD)
// share a CU and one's loads and vector work run beside the other's matrix work. Partials are summed
// in a fixed order by k_bwd_reduce.
//
// What bounds it: vector issue (the adjoint, the splits into parts, the fp64 partials), then the
// matrix cores. Measured at 64 x 192 x 28 x 28 with the mix (kernel alone): fp32 66.0 us, bf16 52.8 us,
// 114 and 143 TFLOP/s of the formula's products.
#include "wbmm_ckptbwd.hpp"

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

constexpr int kW = 14, kD = kW * kW, kL = CkWin<kW>::L;
constexpr int kPix = kWins * kD;          // its pixels
constexpr int kPieces = kPix / 4;         // 4-element pieces (a piece lies in one image and group)
constexpr int kIter = (kPieces + kT - 1) / kT;
constexpr int kTile = CkWin<kW>::TILE, kBlk = CkWin<kW>::BLK;

// LDS (bytes): G | U | X, with U the table blocks (dX), dy and z (mix), or the start of the
// [pixel][window] operands (dT), which run on into X; X holds T as fp32, then x as bf16.
constexpr int kOffU = kPix * 4;
constexpr int kOffX = kOffU + 3 * kBlk * 2;
constexpr int kOffR = kOffX + kPix * 2;
constexpr int kLds = kOffR + kWaves * 4 * 9 * 4;
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
      const float s = row_sum_f32_last(active ? dw[q] : 0.f);
      if ((lane & 15) == 15) red[(wave * 4 + (lane >> 4)) * 9 + q] = s;
    }
  }
}

// dX of 16 windows and the output rows of quarter QR.
template <int IH, bool F32, int NG, int QR>
__device__ __forceinline__ void dx_quarter(const CkptBwdArgs& a, const float* G, const uint16_t* blk,
                                           size_t base, int cp, int nimg, int wu, int lane) {
  typedef Img<IH> I;
  constexpr int Y0 = CkWin<kW>::y0(QR), NY = CkWin<kW>::ny(QR);
  const int n = wu * 16 + (lane & 15), kg = lane >> 4;
  v4f acc[NY];
  dx_rows<kW, F32, NG, Y0, NY, I::IW>(G + I::win(n), blk, lane, acc);
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

  // ---- loads: T, dy, z in flight together
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
  // the unit's first element, and its place in its scale group
  const char* dyu = (const char*)a.dy + base * (F32 ? 4 : 2);
  const uint32_t og = (uint32_t)(base % kCkptGroup);
  const uint8_t *xcu = a.xc + base, *xsu = a.xs + base / kCkptGroup;
  const uint8_t *zcu = wantW ? a.zc + base : nullptr;
  const uint8_t *zsu = wantW ? a.zs + base / kCkptGroup : nullptr;
  uint32_t zw[kIter], zsc[kIter];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = 4 * (tid + it * kT), im = e / I::PLANE;
    // pieces past the unit's images read its first ones and count as zeros below
    const bool in = im < nimg;
    const uint32_t o = in ? (uint32_t)(im * cp + (e - im * I::PLANE)) : 0u, os = (og + o) / kCkptGroup;
    dv[it] = *(const raw_t*)(dyu + o * (F32 ? 4u : 2u));
    if (wantW) {
      zw[it] = *(const uint32_t*)(zcu + o);
      zsc[it] = zsu[os];
    }
    if (!in) {
#pragma unroll
      for (int j = 0; j < (F32 ? 4 : 2); ++j) dv[it][j] = 0;
      zw[it] = 0;
      zsc[it] = 127;
    }
  }
#pragma unroll
  for (int j = 0; j < TQ; ++j)
    if (tid + j * kT < kL) Tf[tid + j * kT] = tv[j];
  // x's codes, in flight across dX
  uint32_t xw[kIter], xsc[kIter];
  if (a.want_dT) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int e = 4 * (tid + it * kT), im = e / I::PLANE;
      const bool in = im < nimg;
      const uint32_t o = in ? (uint32_t)(im * cp + (e - im * I::PLANE)) : 0u;
      xw[it] = *(const uint32_t*)(xcu + o);
      xsc[it] = xsu[(og + o) / kCkptGroup];
      if (!in) xw[it] = 0, xsc[it] = 127;
    }
  }

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
#pragma unroll
      for (int w = 0; w < kWaves * 4; ++w) s += (double)red[w * 9 + tid];
      a.partW[(size_t)blockIdx.x * 9 + tid] = s;
    }
  }

  // ---- dX
  if (a.dx) {
    table_blocks<kW, NT>(Tf, (uint32_t*)U, tid);
    __syncthreads();
    const uint16_t* blk = (const uint16_t*)U;
    switch (wave >> 1) {   // 4, 4, 3 and 3 rows
      case 0: dx_quarter<IH, F32, NG, 0>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      case 1: dx_quarter<IH, F32, NG, 1>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      case 2: dx_quarter<IH, F32, NG, 2>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
      default: dx_quarter<IH, F32, NG, 3>(a, G, blk, base, cp, nimg, wave & 1, lane); break;
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
    dt_rows<kW, Q, NS>(ops, lane, acc); \
    __syncthreads();                 \
    dt_partial<kW, Q>(scr, acc, pT, lane, false); \
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

// Shapes of the fused kernel; its 32-bit byte offsets within a unit (up to 32 images apart) must hold.
bool fast_ckpt_shape(int C, int H, int W, int w, int layout) {
  return layout == 0 && w == kW && H == W && (H == 14 || H == 28 || H == 56) &&
         (size_t)images_per_unit(H) * C * H * W < ((size_t)1 << 30);
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
