// The layer backward from 8-bit checkpoints for any map size, layout and window 2 <= w <= 16 (table
// input; fp32, or bf16 dy, T and dx), on the pieces of wbmm_ckptbwd.hpp.
//
// A workgroup takes some units of 32 windows of one channel, in turn: G gathered window by window
// (with the mix: the 3 x 3 neighbourhood of every pixel read from dy, through the caches, and the
// dWmix sums taken on the way), table blocks, dX, G and x transposed to [pixel][window], dT by row
// pairs onto the workgroup's fp64 partial. Windows past the last, and pixels past the map's edge, are
// zeros and are not stored.
#include "wbmm_ckptbwd.hpp"

#include <algorithm>

namespace wbmm {

struct CkptAnyArgs {
  int H, W, units, per, groups;   // units per channel, units per workgroup, workgroups per channel
  int nwx, nwin, windows;         // windows per row, per image, in all
  size_t sb, sc, sy, sx;          // elements between images, channels, rows, columns
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

namespace {

template <int W>
struct AnyLds {
  typedef CkWin<W> C;
  static constexpr int WP = (W + 1) / 2 * 2;       // floats of a window row
  static constexpr int DP = W * WP;                // of a window
  static constexpr int PIX = kWins * C::D;
  // bytes: G | blocks then x as bf16, or the dT operands, or the tiles | dWmix sums | windows of this
  // unit and the next | dT so far | T as fp32
  static constexpr int G = (kWins * DP + 16) * 4;  // slots past the last row are read
  static constexpr int XL = 3 * C::BLK * 2;
  static constexpr int XB = kWins * DP * 2;
  static constexpr int m2(int a, int b) { return a > b ? a : b; }
  static constexpr int V = m2(XL + XB, m2(4 * PIX * 2, kWaves * 4 * C::TILE * 4));
  static constexpr int RED = G + (V + 15) / 16 * 16;
  static constexpr int WIN = RED + kWaves * 4 * 9 * 4;
  static constexpr int PT = WIN + 2 * kWins * 16;
  static constexpr int TF = PT + (C::L * 8 + 15) / 16 * 16;
  static constexpr int TOTAL = TF + (C::L * 4 + 15) / 16 * 16;
};

struct WinAt {
  uint32_t base;   // element offset of its image's channel from the unit's base
  int y0, x0;      // map position of its origin (y0 = H: no such window)
  uint32_t pad;
};

// Element o of p, by a 32-bit byte offset.
template <typename T>
__device__ __forceinline__ T at32(const void* p, uint32_t o) {
  return *(const T*)((const char*)p + o * (uint32_t)sizeof(T));
}

// dX of 16 windows and the output rows of quarter QR.
template <int W, bool F32, int QR>
__device__ __forceinline__ void dx_any(const CkptAnyArgs& a, size_t ub, const float* G,
                                       const uint16_t* blk, const WinAt* wins, int wu, int lane) {
  constexpr int Y0 = CkWin<W>::y0(QR), NY = CkWin<W>::ny(QR);
  if constexpr (NY > 0) {
    const int n = wu * 16 + (lane & 15), x = 4 * (lane >> 4);
    v4f acc[NY];
    dx_rows<W, F32, F32 ? 3 : 2, Y0, NY, AnyLds<W>::WP>(G + n * AnyLds<W>::DP, blk, lane, acc);
    const WinAt w = wins[n];
    constexpr uint32_t ES = F32 ? 4 : 2;
    char* dxu = (char*)a.dx + ub * ES;
    const uint32_t sy = (uint32_t)a.sy * ES, sx = (uint32_t)a.sx * ES;
    const uint32_t o0 = w.base * ES + (w.y0 + Y0) * sy + (w.x0 + x) * sx;
    const int rows = a.H - w.y0 - Y0;
    const int cols = (W < a.W - w.x0 ? W : a.W - w.x0) - x;
#pragma unroll
    for (int y = 0; y < NY; ++y) {
      if (y >= rows) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r >= cols) continue;
        char* at = dxu + (o0 + y * sy + r * sx);
        if constexpr (F32) *(float*)at = acc[y][r];
        else *(uint16_t*)at = f2bf(acc[y][r]);
      }
    }
  }
}

// What bounds it: vector issue and the waits between the six steps of a unit, not memory (64 x 192 x
// 33 x 33, w = 3, bf16, no mix: 272 us, 5% of the copy's rate; 64 x 96 x 28 x 28, w = 7, fp32, no mix:
// 60 us, 14%; with the mix 318 and 78 to 83). Two workgroups of 8 waves share a CU up to w = 10: three or four
// at w <= 6 spilt (w = 5, fp32 with the mix, 284 and 275 us where two took 234). Above w = 10 one runs,
// with twice the registers.
constexpr int any_waves(int w) { return w > 10 ? 2 : 4; }

template <int W, bool F32>
__global__ void __launch_bounds__(kT)
    __attribute__((amdgpu_waves_per_eu(any_waves(W), any_waves(W))))
k_bwd_ckpt_any(CkptAnyArgs a) {
  typedef CkWin<W> C;
  typedef AnyLds<W> S;
  constexpr int NT = F32 ? 3 : 1;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_a[];
  float* G = (float*)smem_a;
  unsigned char* V = smem_a + S::G;
  float* red = (float*)(smem_a + S::RED);
  double* pT = (double*)(smem_a + S::PT);
  const float* Tf = (const float*)(smem_a + S::TF);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x / a.groups, u0 = (blockIdx.x % a.groups) * a.per;
  const int u1 = u0 + a.per < a.units ? u0 + a.per : a.units;
  const bool mix = a.mixw != nullptr, wantW = mix && a.want_dW;
  float wr[9], dw[9];
#pragma unroll
  for (int q = 0; q < 9; ++q) {
    wr[q] = mix ? a.mixw[c * 9 + 8 - q] : 0.f;   // rotated by 180 degrees
    dw[q] = 0.f;
  }

  // A unit's base: its first image's channel, down to a group of the checkpoint; the host admits
  // images of which 33 stay below 2^32 bytes.
  auto unit_base = [&](int u, int& b0, uint32_t& rest) {
    b0 = (int)((unsigned)(u * kWins) / (unsigned)a.nwin);
    const size_t first = (size_t)b0 * a.sb + (size_t)c * a.sc;
    rest = (uint32_t)(first % kCkptGroup);
    return first - rest;
  };
  auto find_windows = [&](int u) {
    if (tid >= kWins || u >= u1) return;
    int b0;
    uint32_t rest;
    unit_base(u, b0, rest);
    const int n = u * kWins + tid, b = n / a.nwin, r = n - b * a.nwin, wy = r / a.nwx;
    WinAt w{(uint32_t)(b - b0) * (uint32_t)a.sb + rest, wy * W, (r - wy * a.nwx) * W, 0};
    if (n >= a.windows) w = WinAt{rest, a.H, 0, 0};
    ((WinAt*)(smem_a + S::WIN))[(u & 1) * kWins + tid] = w;
  };
  for (int q = tid; q < C::L; q += kT)
    ((float*)(smem_a + S::TF))[q] = F32 ? ((const float*)a.T)[(size_t)c * C::L + q]
                                        : bf2f(((const uint16_t*)a.T)[(size_t)c * C::L + q]);
  find_windows(u0);

  for (int u = u0; u < u1; ++u) {
    __syncthreads();   // the unit before has left LDS; this one's windows (and T) are there
    const WinAt* wins = (const WinAt*)(smem_a + S::WIN) + (u & 1) * kWins;
    int b0;
    uint32_t rest;
    const size_t ub = unit_base(u, b0, rest);
    const uint8_t* xc = a.xc + ub;
    const uint8_t* xs = a.xs + ub / kCkptGroup;
    const uint8_t* zc = a.zc + ub;
    const uint8_t* zs = a.zs + ub / kCkptGroup;
    const char* dyu = (const char*)a.dy + ub * (F32 ? 4 : 2);
    auto dy_at = [&](uint32_t o) {
      return F32 ? at32<float>(dyu, o) : bf2f(at32<uint16_t>(dyu, o));
    };
    uint16_t* xl = (uint16_t*)(V + S::XL);
    // All loads of a pixel before the first value is used, and no branches between them: one off the
    // map reads the channel's first element instead, and is zero. With a branch around each
    // neighbour 265 us at w = 5, 64 x 192 x 28 x 28, fp32 with the mix, so 234; two pixels at once 254
    // (spills), and equal or worse at the other windows.
#pragma unroll 1
    for (int q = tid; q < S::PIX; q += kT) {
      const int n = q / C::D, p = q - n * C::D, y = p / W, x = p - y * W;
      const int at = n * S::DP + y * S::WP + x;
      const WinAt w = wins[n];
      const int gy = w.y0 + y, gx = w.x0 + x;
      const bool on = gy < a.H && gx < a.W;
      const uint32_t sy = (uint32_t)a.sy, sx = (uint32_t)a.sx;
      const uint32_t oy = on ? gy * sy : 0, o = w.base + oy + (on ? gx * sx : 0);
      uint32_t xq, xe, zq, ze;
      float d[9], g = 0.f;
      if (a.want_dT) {
        xq = xc[o];
        xe = xs[o / kCkptGroup];
      }
      if (wantW) {
        zq = zc[o];
        ze = zs[o / kCkptGroup];
      }
      if (mix) {
        const bool up = on && gy > 0, down = on && gy + 1 < a.H;
        const bool left = on && gx > 0, right = on && gx + 1 < a.W;
        const uint32_t oc[3] = {left ? o - sx : o, o, right ? o + sx : o};
        const uint32_t orow[3] = {up ? 0u - sy : 0u, 0u, down ? sy : 0u};
#pragma unroll
        for (int k = 0; k < 9; ++k) d[k] = dy_at(oc[k % 3] + orow[k / 3]);
#pragma unroll
        for (int k = 0; k < 9; ++k) {
          const bool in = (k / 3 == 0 ? up : k / 3 == 2 ? down : on) &&
                          (k % 3 == 0 ? left : k % 3 == 2 ? right : on);
          d[k] = in ? d[k] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 9; ++k) g = fmaf(wr[k], d[k], g);
      } else {
        g = dy_at(o);
      }
      G[at] = on ? g : 0.f;
      if (a.want_dT) {
        const float v = ckpt_decode1(xq, a.fmt) * ckpt_factor(xe);
        xl[at] = (uint16_t)pk_bf16(on ? v : 0.f, 0.f);   // exact
      }
      if (wantW) {
        const float v = ckpt_decode1(zq, a.fmt) * ckpt_factor(ze), z = on ? v : 0.f;
#pragma unroll
        for (int k = 0; k < 9; ++k) dw[k] = fmaf(z, d[8 - k], dw[k]);
      }
    }
    if (a.dx) table_blocks<W, NT>(Tf, (uint32_t*)V, tid);
    find_windows(u + 1);
    __syncthreads();
    if (a.dx) {
      const uint16_t* blk = (const uint16_t*)V;
      switch (wave >> 1) {
        case 0: dx_any<W, F32, 0>(a, ub, G, blk, wins, wave & 1, lane); break;
        case 1: dx_any<W, F32, 1>(a, ub, G, blk, wins, wave & 1, lane); break;
        case 2: dx_any<W, F32, 2>(a, ub, G, blk, wins, wave & 1, lane); break;
        default: dx_any<W, F32, 3>(a, ub, G, blk, wins, wave & 1, lane); break;
      }
    }
    if (!a.want_dT) continue;

    __syncthreads();
    uint16_t* ops = (uint16_t*)V;
    constexpr int TI = (C::D * 4 + kT - 1) / kT;
    u32x4 xt[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int t = tid + i * kT, tt = t < C::D * 4 ? t : 0, g = tt / C::D, p = tt % C::D;
      const int o = 8 * g * S::DP + p / W * S::WP + p % W;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xt[i][j] = (uint32_t)xl[o + 2 * j * S::DP] | ((uint32_t)xl[o + (2 * j + 1) * S::DP] << 16);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int t = tid + i * kT, tt = t < C::D * 4 ? t : 0, g = tt / C::D, p = tt % C::D;
      const int o = 8 * g * S::DP + p / W * S::WP + p % W;
      u32x4 part[3];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t q3[3];
        split2<3>(G[o + 2 * j * S::DP], G[o + (2 * j + 1) * S::DP], q3);
#pragma unroll
        for (int q = 0; q < 3; ++q) part[q][j] = q3[q];
      }
      if (t < C::D * 4) {
        const int at = slot_of(p, g);
#pragma unroll
        for (int q = 0; q < 3; ++q) *(u32x4*)(ops + q * S::PIX + at) = part[q];
        *(u32x4*)(ops + 3 * S::PIX + at) = xt[i];
      }
    }
    __syncthreads();
    v4f acc[4];
    float* scr = (float*)V + wave * 4 * C::TILE;
#define WBMM_CK_WAVE(Q)                          \
  case Q:                                        \
    dt_rows<W, Q, 3>(ops, lane, acc);            \
    __syncthreads();                             \
    dt_partial<W, Q>(scr, acc, pT, lane, u > u0); \
    break;
    switch (wave) {   // every wave has read its operands before the tiles go over them
      WBMM_CK_WAVE(0) WBMM_CK_WAVE(1) WBMM_CK_WAVE(2) WBMM_CK_WAVE(3)
      WBMM_CK_WAVE(4) WBMM_CK_WAVE(5) WBMM_CK_WAVE(6) WBMM_CK_WAVE(7)
    }
#undef WBMM_CK_WAVE
  }
  if (a.want_dT) {
    __syncthreads();
    for (int q = tid; q < C::L; q += kT) a.partT[(size_t)blockIdx.x * C::L + q] = pT[q];
  }
  if (wantW) {
#pragma unroll
    for (int q = 0; q < 9; ++q) {
      const float s = row_sum_f32_last(dw[q]);
      if ((lane & 15) == 15) red[(wave * 4 + (lane >> 4)) * 9 + q] = s;
    }
    __syncthreads();
    if (tid < 9) {
      double s = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves * 4; ++w) s += (double)red[w * 9 + tid];
      a.partW[(size_t)blockIdx.x * 9 + tid] = s;
    }
  }
}

template <int W, bool F32>
hipError_t launch_any_w(const CkptAnyArgs& a, int blocks, hipStream_t st) {
  static_assert(AnyLds<W>::TOTAL <= kLdsPerCu, "one workgroup per CU at least");
  constexpr int lds = AnyLds<W>::TOTAL;
  auto fn = k_bwd_ckpt_any<W, F32>;
  const hipError_t e =
      hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  return e != hipSuccess ? e : launch_main(fn, dim3(blocks), dim3(kT), lds, st, a);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Units per channel, and how they are dealt: the workgroups per channel (at most 96, since one
// thread adds a table entry's partials, and about 2048 in all) that leave the least to the slot
// which gets the most. Of equal ones the most where a CU runs two, whose starts and ends overlap
// (64 x 192 x 24 x 24, w = 8, bf16 with the mix: 1728 workgroups of 2 units 80 us, 960 of 4 84), and the
// fewest where it runs one (64 x 64 x 40 x 40, w = 16: 256 of 5 units 111 us, 1152 of one 124).
// A thread's dWmix sums are fp32 over its workgroup's units: more workgroups where they would pass 128
// terms (to 2^20 workgroups in all, which only maps far smaller than their window reach). One chain over
// 200 units of equal terms was off by 148 half steps.
void any_units(const BwdCkptRequest& r, CkptAnyArgs& a) {
  a.nwx = (r.W + r.w - 1) / r.w;
  a.nwin = a.nwx * ((r.H + r.w - 1) / r.w);
  a.windows = r.B * a.nwin;
  a.units = (a.windows + kWins - 1) / kWins;
  const long long terms = (kWins * r.w * r.w + kT - 1) / kT;   // of a thread and unit
  const long long longest = 128 / terms;
  const long long least = std::max<long long>(
      1, std::min<long long>((a.units + longest - 1) / longest, (1 << 20) / r.C));
  const long long most =
      std::max(least, std::min<long long>({96, a.units, std::max(1, 2048 / r.C)}));
  const int resident = any_waves(r.w) / 2;   // workgroups that a CU runs at a time
  const long long slots = 256 * resident;
  long long best = -1;
  for (long long g = least; g <= most; ++g) {
    const long long per = (a.units + g - 1) / g, used = (a.units + per - 1) / per;
    const long long turns = (r.C * used + slots - 1) / slots * per;
    if (best < 0 || turns < best || (turns == best && resident > 1))
      best = turns, a.per = (int)per, a.groups = (int)used;
  }
}

}  // namespace

bool any_ckpt_shape(int B, int C, int H, int W, int w) {
  const long long nwin = (long long)((W + w - 1) / w) * ((H + w - 1) / w);
  return w >= 2 && w <= 16 && B * nwin < (1ll << 31) - kWins &&
         (double)C * H * W * 4 * (kWins + 1) < (double)(1ll << 32);   // a unit's 32-bit offsets
}

size_t any_ckpt_workspace(const BwdCkptRequest& r) {
  CkptAnyArgs a{};
  any_units(r, a);
  const size_t L = (size_t)(2 * r.w - 1) * (2 * r.w - 1);
  return up256((size_t)r.C * a.groups * L * 8) + up256((size_t)r.C * a.groups * 9 * 8);
}

hipError_t launch_backward_ckpt_any(const BwdCkptRequest& r, hipStream_t st) {
  CkptAnyArgs a{};
  any_units(r, a);
  const int L = (2 * r.w - 1) * (2 * r.w - 1);
  a.H = r.H;
  a.W = r.W;
  a.sb = (size_t)r.C * r.H * r.W;
  a.sc = r.layout == 0 ? (size_t)r.H * r.W : 1;
  a.sx = r.layout == 0 ? 1 : r.C;
  a.sy = r.W * a.sx;
  a.xc = r.xc; a.xs = r.xs; a.zc = r.zc; a.zs = r.zs;
  a.T = r.T; a.dy = r.dy; a.mixw = r.mixw; a.dx = r.dx;
  a.partT = (double*)r.ws;
  a.partW = (double*)((unsigned char*)r.ws + up256((size_t)r.C * a.groups * L * 8));
  a.fmt = r.fmt;
  a.want_dT = r.dT != nullptr;
  a.want_dW = r.mixw && r.dmixw;
  const int blocks = r.C * a.groups;
  hipError_t e = hipErrorInvalidValue;
  switch (r.w) {
#define WBMM_CK_W(N)                                                                  \
  case N:                                                                             \
    e = r.bf16 ? launch_any_w<N, false>(a, blocks, st) : launch_any_w<N, true>(a, blocks, st); \
    break;
    WBMM_CK_W(2) WBMM_CK_W(3) WBMM_CK_W(4) WBMM_CK_W(5) WBMM_CK_W(6) WBMM_CK_W(7) WBMM_CK_W(8)
    WBMM_CK_W(9) WBMM_CK_W(10) WBMM_CK_W(11) WBMM_CK_W(12) WBMM_CK_W(13) WBMM_CK_W(14)
    WBMM_CK_W(15) WBMM_CK_W(16)
#undef WBMM_CK_W
  }
  if (e != hipSuccess || (!a.want_dT && !a.want_dW)) return e;
  return launch_bwd_reduce(a.partT, a.want_dW ? a.partW : nullptr, a.groups, r.C, L, r.dT,
                           a.want_dW ? r.dmixw : nullptr, st);
}

}  // namespace wbmm
