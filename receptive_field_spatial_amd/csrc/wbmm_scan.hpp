// Gated linear recurrence, device pieces shared by the forward and backward kernels.
//
// Along one axis of a (outer, len, inner) tensor, for every (outer, inner) column:
//   a_t = sigmoid(g_t),   h_t = a_t h_{t-1} + (1 - a_t) u_t.
// A run of steps acts on the state entering it as the affine map h -> P h + H, with P the product
// of its a_t and H its result from a zero state; runs compose by
//   (P2, H2) after (P1, H1) = (P2 P1, P2 H1 + H2),
// so a column is cut into pieces whose maps are formed independently and joined in order. a_t lies
// in [0, 1]: P never overflows, and where it underflows the state entering no longer counts. The
// backward is the same recurrence from the other end: with R_t the gradient entering step t from
// step t + 1, G_t = dh_t + R_t and R_{t-1} = a_t G_t.
//
// States, gates, products and sums are fp32 whatever the tensors' type.
//
// Scan order: step s of a sequence of n steps is position s, or n - 1 - s when reversed; positions
// n .. len - 1 (padding) are never used: in their place the kernels take g = kScanPad and zeros,
// the identity map (a = 1, b = 0), and outputs there are zero.
#pragma once

#include "wbmm_ckpt.hpp"
#include "wbmm_launch.hpp"
#include "wbmm_scanplan.hpp"

namespace wbmm {

constexpr float kScanPad = 100.f; // a gate that leaves the state alone (a = 1 exactly)

struct ScanArgs {
  const void* g;
  const void* u;              // tensor, or the codes of a checkpoint when us is set
  const uint8_t* us;
  const void* dh;
  const float* carry_in;      // h0 (forward), dh_last (backward), or null
  const float* h0;            // backward without states: the initial state, or null
  const int* lens;            // or null
  void* out0;                 // h, or dg (backward)
  void* out1;                 // du (backward)
  float* carry_out;           // h_last, or dh0, or null
  float* states;              // [outer][chunks][inner]
  float2* agg;                // [maps][cols]
  float* carry_copy;          // [cols] carry_in, kept for the second launch
  int len, chunks, reverse, fmt;
  uint32_t inner, cols, rows_per_len;   // cols = outer * inner; lens[outer index / rows_per_len]
  int segs, seg_len;          // seg_len: a multiple of the workgroup's tile
  int fine, maps;             // maps per segment (of seg_len / fine steps each), maps in all
  int lanes;                  // row kernels: lanes per row (64: the workgroup's waves share a row)
  int cw;                     // column kernels: columns of a wave
  int run;                    // column kernels: neighbour groups that share memory lines
};

// a = sigmoid(g) and c = 1 - a = sigmoid(-g), each with its own relative accuracy (c from 1 - a
// would lose what a long memory lives on): with t = exp(-g), a = 1 / (1 + t) and c = t a. The
// reciprocal gets one Newton step: over hundreds of steps near a = 1 its last bit shows in the fp32
// states. exp2 is given y, the leading part of g log2(e), and t takes the rest back in, which
// otherwise costs |g| times up to 1.7 half steps of t (bf16 tensors too: their states, h_last and dh0
// are fp32). fp32: y is the rounded product and the rest its rounding and that of log2(e). BF16:
// 8 bits of g times 16 of log2(e) are exact, the rest is g times the other bits. By the roundings c is
// within 6 half steps and a within 5 (bf16 beyond |g| = 40: up to 1.6 more); measured over the range 3.6
// and 2.5, in bf16 without the correction 57, where it costs 3 of 11 instructions (64 x 784 x 192
// forward 18.9 us without, 20.0 with; 4 x 32768 x 1024 backward 378 and 380). g is held to [-87, 87],
// where a or c is the least normal number, t finite and an infinity out of the correction; the
// NaN-keeping forms let a NaN through.
template <bool BF16>
__device__ __forceinline__ void scan_gate(float g, float& a, float& c) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596299e-8f, kLn2 = 0.693147181f;
  constexpr float kL16 = 1.44268798828125f, kRest = 4.88849465e-6f;   // (log2(e) - kL16) ln(2)
  const float x =
      __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -87.f), 87.f);
  const float y = x * (BF16 ? kL16 : kL);
  const float r = BF16 ? -kRest * x : -kLn2 * fmaf(x, kLlo, fmaf(x, kL, -y));
  float t = __builtin_amdgcn_exp2f(-y);
  t = fmaf(t, r, t);
  const float d = 1.f + t;
  a = __builtin_amdgcn_rcpf(d);
  a = fmaf(a, fmaf(-d, a, 1.f), a);
  c = t * a;
}

template <typename T>
__device__ __forceinline__ float scan_widen(T v);
template <>
__device__ __forceinline__ float scan_widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float scan_widen<uint16_t>(uint16_t v) { return bf2f(v); }
template <typename T>
__device__ __forceinline__ T scan_narrow(float v);
template <>
__device__ __forceinline__ float scan_narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t scan_narrow<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}

// x of the lane that CTRL names; `id` where there is none.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float scan_dpp(float id, float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(x), CTRL,
                                                    ROW_MASK, 0xf, false));
}
__device__ __forceinline__ float scan_readlane(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// Inclusive prefix composition over each group of `lanes` lanes (a power of two; each lane's own
// map is the later one): row shifts within 16 lanes, then the two row broadcasts.
template <int CTRL, int ROW_MASK, int D>
__device__ __forceinline__ void scan_prefix_step(float& P, float& H, int li, int lanes) {
  if (lanes <= D) return;
  float ps = scan_dpp<CTRL, ROW_MASK>(1.f, P), hs = scan_dpp<CTRL, ROW_MASK>(0.f, H);
  if (D < 16 && lanes < 16) {
    ps = li < D ? 1.f : ps;
    hs = li < D ? 0.f : hs;
  }
  H = fmaf(P, hs, H);
  P *= ps;
}
__device__ __forceinline__ void scan_prefix(float& P, float& H, int li, int lanes) {
  scan_prefix_step<0x111, 0xf, 1>(P, H, li, lanes);
  scan_prefix_step<0x112, 0xf, 2>(P, H, li, lanes);
  scan_prefix_step<0x114, 0xf, 4>(P, H, li, lanes);
  scan_prefix_step<0x118, 0xf, 8>(P, H, li, lanes);
  scan_prefix_step<0x142, 0xa, 16>(P, H, li, lanes);
  scan_prefix_step<0x143, 0xc, 32>(P, H, li, lanes);
}
// The map of the lanes before this one in its group (identity for the first).
__device__ __forceinline__ void scan_before(float P, float H, int li, float& Pe, float& He) {
  Pe = scan_dpp<0x138, 0xf>(1.f, P);
  He = scan_dpp<0x138, 0xf>(0.f, H);
  Pe = li == 0 ? 1.f : Pe;
  He = li == 0 ? 0.f : He;
}

// Inclusive suffix composition (the later lanes' map is applied first, as the backward runs):
// row shifts within 16 lanes, then the totals of the later rows by lane reads.
template <int CTRL, int D>
__device__ __forceinline__ void scan_suffix_step(float& P, float& R, int li, int lanes) {
  if (lanes <= D) return;
  float ps = scan_dpp<CTRL, 0xf>(1.f, P), rs = scan_dpp<CTRL, 0xf>(0.f, R);
  if (lanes < 16) {
    ps = li + D >= lanes ? 1.f : ps;
    rs = li + D >= lanes ? 0.f : rs;
  }
  R = fmaf(P, rs, R);
  P *= ps;
}
__device__ __forceinline__ void scan_suffix(float& P, float& R, int li, int lanes, int lane) {
  scan_suffix_step<0x101, 1>(P, R, li, lanes);
  scan_suffix_step<0x102, 2>(P, R, li, lanes);
  scan_suffix_step<0x104, 4>(P, R, li, lanes);
  scan_suffix_step<0x108, 8>(P, R, li, lanes);
  if (lanes <= 16) return;
  const int row = lane >> 4;
  const float p1 = scan_readlane(P, 16), r1 = scan_readlane(R, 16);
  const float p3 = scan_readlane(P, 48), r3 = scan_readlane(R, 48);
  float ps = row == 2 ? p3 : 1.f, rs = row == 2 ? r3 : 0.f;
  if (lanes == 32) {
    ps = row == 0 ? p1 : ps;
    rs = row == 0 ? r1 : rs;
  } else {
    const float p2 = scan_readlane(P, 32), r2 = scan_readlane(R, 32);
    const float p23 = p2 * p3, r23 = fmaf(p2, r3, r2);
    ps = row == 1 ? p23 : ps;
    rs = row == 1 ? r23 : rs;
    ps = row == 0 ? p1 * p23 : ps;
    rs = row == 0 ? fmaf(p1, r23, r1) : rs;
  }
  R = fmaf(P, rs, R);
  P *= ps;
}
// The map of the lanes after this one in its group (identity for the last).
__device__ __forceinline__ void scan_after(float P, float R, int li, int lanes, float& Pe,
                                           float& Re) {
  Pe = scan_dpp<0x130, 0xf>(1.f, P);
  Re = scan_dpp<0x130, 0xf>(0.f, R);
  Pe = li + 1 == lanes ? 1.f : Pe;
  Re = li + 1 == lanes ? 0.f : Re;
}

// Steps of a sequence: its entry of lens held to [0, len], or len.
__device__ __forceinline__ int scan_steps(const ScanArgs& a, uint32_t seq) {
  if (!a.lens) return a.len;
  const int n = a.lens[seq / a.rows_per_len];
  return n < 0 ? 0 : (n > a.len ? a.len : n);
}

// ------------------------------------------------------------------ column kernels (inner > 1)
// A wave takes cw neighbouring columns (a power of two) and 64 / cw consecutive pieces of kScanK
// steps: fewer columns per wave make more workgroups of few columns, without cutting the axis.
// Addresses are a uniform base plus a byte offset of type OFF: 32 bits where a tensor has less than
// 4 GiB (one add per step, shared by the tensors), else 64.
template <typename T, typename OFF>
struct ScanCol {
  int cw, subs, sub, cl;      // columns and pieces per wave, the lane's piece and column
  uint32_t col, o, i;         // the lane's column, its sequence and place in the row
  bool active;
  int n;                      // steps of its sequence
  OFF base, start, stride;    // byte offsets of position 0 and step 0, bytes from step to step
  __device__ __forceinline__ ScanCol(const ScanArgs& a, int lane) {
    cw = a.cw;
    subs = 64 / cw;
    sub = lane / cw;
    cl = lane & (cw - 1);
    // workgroups go round the XCDs: a run of groups that share memory lines stays on one
    uint32_t group = blockIdx.x;
    const uint32_t whole = gridDim.x / (8 * a.run) * (8 * a.run);
    if (group < whole) {
      const uint32_t x = group % 8, k = group / 8;
      group = (k / a.run * 8 + x) * a.run + k % a.run;
    }
    const uint64_t c = (uint64_t)group * cw + cl;
    active = c < a.cols;
    col = active ? (uint32_t)c : a.cols - 1;
    o = col / a.inner;
    i = col - o * a.inner;
    n = scan_steps(a, o);
    const OFF row = (OFF)a.inner * sizeof(T);
    base = (OFF)o * a.len * row + (OFF)i * sizeof(T);
    start = a.reverse && n > 0 ? base + (OFF)(n - 1) * row : base;
    stride = a.reverse ? (OFF)0 - row : row;
  }
  __device__ __forceinline__ OFF at(int s) const { return start + (OFF)s * stride; }
  __device__ __forceinline__ T load(const void* p, OFF o) const {
    return *(const T*)((const char*)p + o);
  }
  __device__ __forceinline__ void store(void* p, OFF o, float v) const {
    *(T*)((char*)p + o) = scan_narrow<T>(v);
  }
  // zeros at the positions of steps s .. s + kScanK - 1 that lie past the end of the sequence
  __device__ __forceinline__ void zero(void* p, int s, int len, uint32_t inner) const {
    const OFF row = (OFF)inner * sizeof(T);
    OFF o = base + (OFF)s * row;
#pragma unroll
    for (int k = 0; k < kScanK; ++k, o += row)
      if (s + k >= n && s + k < len) store(p, o, 0.f);
  }
  // index of the kept state before step s
  __device__ __forceinline__ size_t kept(const ScanArgs& a, int s) const {
    return ((size_t)o * a.chunks + s / kScanChunk) * a.inner + i;
  }
};

// One element of u: of a map, or of a checkpoint.
template <typename T, bool CK>
struct ScanRaw {
  T r;
  uint8_t code, scale;
  template <typename OFF>
  __device__ __forceinline__ void load(const ScanArgs& a, OFF o) {
    if constexpr (CK) {
      const OFF e = o / sizeof(T);
      code = *((const uint8_t*)a.u + e);
      scale = *(a.us + e / kCkptGroup);
    } else {
      r = *(const T*)((const char*)a.u + o);
    }
  }
  __device__ __forceinline__ void clear() {
    r = T(0);
    code = 0;
    scale = 127;
  }
  __device__ __forceinline__ float widen(const ScanArgs& a) const {
    if constexpr (CK) return ckpt_decode1(code, a.fmt) * ckpt_factor(scale);
    else return scan_widen<T>(r);
  }
};

// g and u (DH: and dh) of a lane's kScanK steps from s on; past the end of the sequence a neutral gate
// and zeros.
template <typename T, bool CK, typename OFF, bool DH, bool U = true>
__device__ __forceinline__ void scan_load(const ScanArgs& a, const ScanCol<T, OFF>& cl, int s,
                                          T (&rg)[kScanK], T (&rd)[kScanK],
                                          ScanRaw<T, CK> (&ru)[kScanK]) {
  if (__all(s + kScanK <= cl.n)) {
    OFF o = cl.at(s);
#pragma unroll
    for (int k = 0; k < kScanK; ++k, o += cl.stride) {
      rg[k] = cl.load(a.g, o);
      if constexpr (DH) rd[k] = cl.load(a.dh, o);
      if constexpr (U) ru[k].load(a, o);
    }
  } else {
    // steps past the end load the last one's place (position 0 of an empty sequence) for nothing
    const T pad = scan_narrow<T>(kScanPad);
    const int last = cl.n > 0 ? cl.n - 1 : 0;
    OFF o = cl.at(s < last ? s : last);
#pragma unroll
    for (int k = 0; k < kScanK; ++k, o += s + k <= last ? cl.stride : OFF(0)) {
      const bool live = s + k < cl.n;
      const T g = cl.load(a.g, o);
      rg[k] = live ? g : pad;
      if constexpr (DH) {
        const T d = cl.load(a.dh, o);
        rd[k] = live ? d : T(0);
      }
      if constexpr (U) {
        ru[k].load(a, o);
        if (!live) ru[k].clear();
      }
    }
  }
}

// Composition over a wave's pieces (lanes cw apart): inclusive prefix, or suffix.
__device__ __forceinline__ void scan_sub_prefix(float& P, float& H, int lane, int cw) {
  for (int d = cw; d < 64; d *= 2) {
    const float ps = __shfl(P, lane - d), hs = __shfl(H, lane - d);
    H = lane >= d ? fmaf(P, hs, H) : H;
    P = lane >= d ? P * ps : P;
  }
}
__device__ __forceinline__ void scan_sub_suffix(float& P, float& R, int lane, int cw) {
  for (int d = cw; d < 64; d *= 2) {
    const float ps = __shfl(P, lane + d), rs = __shfl(R, lane + d);
    R = lane + d < 64 ? fmaf(P, rs, R) : R;
    P = lane + d < 64 ? P * ps : P;
  }
}

// ------------------------------------------------------------------ row kernels (inner = 1)
// kScanE consecutive steps of a row, in scan order; rows start at any element, so the wide
// accesses carry the element's alignment only.
template <typename T, bool REV>
struct ScanRow {
  static constexpr int E = kScanE;
  struct __attribute__((packed, aligned(sizeof(T)))) Wide { T v[E]; };
  size_t base;
  int len, n;
  __device__ __forceinline__ ScanRow(uint32_t row, int len_, int n_)
      : base((size_t)row * len_), len(len_), n(n_) {}
  __device__ __forceinline__ size_t at(int s) const { return base + (REV ? n - 1 - s : s); }
  // steps past the end of the sequence come back as `pad`
  __device__ __forceinline__ void load(const T* __restrict__ p, int s, T (&v)[E], T pad) const {
    if (s + E <= n) {
      Wide w;
      __builtin_memcpy(&w, p + at(REV ? s + E - 1 : s), sizeof(w));
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = w.v[REV ? E - 1 - k : k];
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = pad;
      if (s < n) {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (s + k < n) v[k] = p[at(s + k)];
      }
    }
  }
  // zeros at the positions past the end of the sequence
  __device__ __forceinline__ void store(T* __restrict__ p, int s, const float (&o)[E]) const {
    if (s + E <= n) {
      Wide w;
#pragma unroll
      for (int k = 0; k < E; ++k) w.v[REV ? E - 1 - k : k] = scan_narrow<T>(o[k]);
      __builtin_memcpy(p + at(REV ? s + E - 1 : s), &w, sizeof(w));
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (s + k < n) p[at(s + k)] = scan_narrow<T>(o[k]);
        else if (s + k < len) p[base + s + k] = T(0);
      }
    }
  }
};

// kScanE steps of a row's u, from the map or from a checkpoint (whose groups run through the whole
// tensor: a lane's steps lie in one or two).
template <typename T, bool REV, bool CK>
struct ScanU {
  static constexpr int E = kScanE;
  T r[CK ? 1 : E];
  uint8_t code[CK ? E : 1];
  uint32_t s0, s1;
  __device__ __forceinline__ void load(const ScanArgs& a, const ScanRow<T, REV>& rw,
                                       const ScanRow<uint8_t, REV>& rwc, int s) {
    if constexpr (CK) {
      rwc.load((const uint8_t*)a.u, s, code, 0);
      s0 = s1 = 127;
      if (s < rw.n) {   // the scales of the lane's first and last step
        const int last = s + E <= rw.n ? s + E - 1 : rw.n - 1;
        s0 = a.us[rw.at(s) / kCkptGroup];
        s1 = a.us[rw.at(last) / kCkptGroup];
      }
    } else {
      rw.load((const T*)a.u, s, r, T(0));
    }
  }
  __device__ __forceinline__ void widen(const ScanArgs& a, const ScanRow<T, REV>& rw, int s,
                                        float (&v)[E]) const {
    if constexpr (CK) {
      const float f0 = ckpt_factor(s0), f1 = ckpt_factor(s1);
      // place of the first step in its group; the second scale from where the group ends
      const int at0 = (int)(rw.at(s) % kCkptGroup);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const bool first = REV ? at0 - k >= 0 : at0 + k < kCkptGroup;
        v[k] = ckpt_decode1(code[k], a.fmt) * (first ? f0 : f1);
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = scan_widen<T>(r[k]);
    }
  }
};

// ------------------------------------------------------------------ host side
struct ScanRequest {
  int64_t outer, len, inner, n_lens;
  int bf16, reverse, fmt;
  const void* g;
  const void* u;
  const uint8_t* us;
  const void* dh;
  const float* carry_in;   // h0, or dh_last in the backward
  const float* h0;         // backward that gets no states
  const int* lens;
  void* out0;              // h, or dg; null in a forward that only forms states
  void* out1;
  float* carry_out;
  float* states;
  void* ws;
};
ScanArgs scan_args(const ScanRequest& r, const ScanPlan& p);
hipError_t launch_scan_forward(const ScanRequest& r, hipStream_t st);
hipError_t launch_scan_backward(const ScanRequest& r, hipStream_t st);

}  // namespace wbmm
