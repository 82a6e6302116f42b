// Gated linear recurrence, backward. With R_t the gradient that reaches the state h_t from step
// t + 1 (dh_last at the end),
//   G_t = dh_t + R_t,   du_t = (1 - a_t) G_t,   dg_t = a_t (1 - a_t) (h_{t-1} - u_t) G_t,
//   R_{t-1} = a_t G_t,  dh0 = R_{-1}.
// The h_{t-1} come from the states that the forward kept every 32 steps (fp32, so nothing of h's
// own rounding enters): a piece runs the recurrence again from its state, in registers, while it
// has g and u there for the gradient anyway. R runs through the same pieces in the other order,
// as the affine maps of wbmm_scan.hpp. One pass: g, u, dh read, dg, du written.
//
// What bounds it: memory, less where the axis is cut (the maps' launch reads g and dh before), vector
// issue along rows (the exponential and the reciprocal of each gate). Measured (kernel alone, rates of the bytes that have to move; a large copy reaches
// 5.05 TB/s): k_scan_cols_bwd 4 x 32768 x 1024 bf16 271 us, 5.0 TB/s, and its maps 113 us, 4.8 TB/s;
// k_scan_rows_bwd 12288 x 784 fp32 with u in 8 bits and no states 42 us, 3.9 TB/s.
#include "wbmm_scan.hpp"

#include <type_traits>

namespace wbmm {

namespace {

// A run of steps: h -> p h + h of the state, r -> p r + r of its gradient.
struct RunMap {
  float p, r, h;
};

// ------------------------------------------------------------------ columns
// As k_scan_cols. A lane's piece is half the distance between two kept states: the odd half's state
// is where the even half before it ends, one piece back in the wave, or in the wave before (then
// waves come in pairs). CK: u is a checkpoint. SELF: one tile holds the axis and no state is kept:
// the pieces' maps of the state are exchanged beside those of its gradient, from h0 (a.h0).
template <typename T, bool CK, bool SELF, typename OFF>
__global__ void __launch_bounds__(64 * scan_col_waves(true, CK, sizeof(OFF) == 8))
k_scan_cols_bwd(ScanArgs a) {
  constexpr int K = kScanK;
  static_assert(kScanChunk == 2 * K, "two pieces between states");
  extern __shared__ __attribute__((aligned(16))) RunMap smb[];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanCol<T, OFF> cl(a, lane);
  const int seg = blockIdx.y, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const int tile = NW * cl.subs * K, lofs = (wv * cl.subs + cl.sub) * K;
  const bool odd = cl.subs > 1 ? cl.sub & 1 : wv & 1;

  float carry = 0.f;
  if (seg == a.segs - 1) {
    if (a.carry_in) carry = a.carry_in[cl.col];
  } else {
    for (int j = a.maps - 1; j >= (seg + 1) * a.fine; --j) {
      const float2 m = a.agg[(size_t)j * a.cols + cl.col];
      carry = fmaf(m.x, carry, m.y);
    }
  }

  T rg[K], rd[K];
  ScanRaw<T, CK> ru[K];
  float rst = 0.f;
  auto load = [&](int s) {
    if (!SELF && !odd && s < a.len) rst = a.states[cl.kept(a, s)];
    scan_load<T, CK, OFF, true>(a, cl, s, rg, rd, ru);
  };
  int t0 = sbeg + (send - sbeg - 1) / tile * tile;
  load(t0 + lofs);
  for (int buf = 0; t0 >= sbeg; t0 -= tile, buf ^= 1) {
    const int s = t0 + lofs;
    // ev: (1 - a) u, later the gradient of g up to the factor G
    float av[K], cv[K], ev[K], dv[K], P = 1.f, Rl = 0.f, H = 0.f, h = rst;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      scan_gate<sizeof(T) == 2>(scan_widen<T>(rg[k]), av[k], cv[k]);
      ev[k] = cv[k] * ru[k].widen(a);
      dv[k] = scan_widen<T>(rd[k]);
      P *= av[k];
      H = fmaf(av[k], H, ev[k]);
    }
    Rl = dv[K - 1];
#pragma unroll
    for (int k = K - 2; k >= 0; --k) Rl = fmaf(av[k + 1], Rl, dv[k]);
    Rl *= av[0];
    if (t0 - tile >= sbeg) load(s - tile);
    float ph = P, hend = SELF ? H : fmaf(P, h, H);   // the state's map, or where the piece ends
    if (cl.subs > 1) {
      if constexpr (SELF) {
        scan_sub_prefix(ph, hend, lane, cl.cw);
      } else {
        const float b = __shfl(hend, lane - cl.cw);
        h = odd ? b : h;
      }
      scan_sub_suffix(P, Rl, lane, cl.cw);
    }
    // exchange: gradient maps of whole waves (their first piece has it), state maps or ends of
    // their last piece
    float Rt = carry, hw = SELF && a.h0 ? a.h0[cl.col] : 0.f, hs = hw;
    if (NW > 1) {
      RunMap* sb = smb + buf * NW * cl.cw;
      if (cl.subs == 1) {
        sb[wv * 64 + lane] = RunMap{P, Rl, hend};
      } else {
        if (cl.sub == 0) sb[wv * cl.cw + cl.cl].p = P, sb[wv * cl.cw + cl.cl].r = Rl;
        if (SELF && cl.sub == cl.subs - 1) sb[wv * cl.cw + cl.cl].h = hend;
      }
      __syncthreads();
      for (int w = NW - 1; w >= 0; --w) {
        const RunMap m = sb[w * cl.cw + cl.cl];
        if (w == wv) Rt = carry;
        if (!SELF && cl.subs == 1 && odd && w == wv - 1) h = m.h;
        carry = fmaf(m.p, carry, m.r);
      }
      if constexpr (SELF) {
        for (int w = 0; w < wv; ++w) {
          const RunMap m = sb[w * cl.cw + cl.cl];
          hs = fmaf(m.p, hs, m.h);
        }
      }
    } else {
      const float p = cl.subs > 1 ? __shfl(P, cl.cl) : P, r = cl.subs > 1 ? __shfl(Rl, cl.cl) : Rl;
      carry = fmaf(p, carry, r);
    }
    if (cl.subs > 1) {
      const float p = __shfl(P, lane + cl.cw), r = __shfl(Rl, lane + cl.cw);
      Rt = cl.sub + 1 < cl.subs ? fmaf(p, Rt, r) : Rt;
      if constexpr (SELF) {
        const float pe = __shfl(ph, lane - cl.cw), he = __shfl(hend, lane - cl.cw);
        hs = cl.sub > 0 ? fmaf(pe, hs, he) : hs;
      }
    }
    if constexpr (SELF) h = hs;
#pragma unroll
    for (int k = 0; k < K; ++k) {   // a c (h - u)
      const float cu = ev[k];
      ev[k] = av[k] * fmaf(cv[k], h, -cu);
      h = fmaf(av[k], h, cu);
    }
    if (cl.active && s < a.len) {
      OFF o = cl.at(s + K - 1);
      float Gt = dv[K - 1] + Rt;
      if (__all(s + K <= cl.n)) {
#pragma unroll
        for (int k = K - 1; k >= 0; --k, o -= cl.stride) {
          cl.store(a.out0, o, ev[k] * Gt);
          cl.store(a.out1, o, cv[k] * Gt);
          if (k > 0) Gt = fmaf(av[k], Gt, dv[k > 0 ? k - 1 : 0]);
        }
      } else {
#pragma unroll
        for (int k = K - 1; k >= 0; --k, o -= cl.stride) {
          if (s + k < cl.n) {
            cl.store(a.out0, o, ev[k] * Gt);
            cl.store(a.out1, o, cv[k] * Gt);
          }
          if (k > 0) Gt = fmaf(av[k], Gt, dv[k > 0 ? k - 1 : 0]);
        }
        cl.zero(a.out0, s, a.len, a.inner);
        cl.zero(a.out1, s, a.len, a.inner);
      }
    }
  }
  if (seg == 0 && wv == 0 && cl.sub == 0 && cl.active && a.carry_out) a.carry_out[cl.col] = carry;
}

// The maps after the first segment's; the last has dh_last folded in (P = 0).
template <typename T, typename OFF>
__global__ void __launch_bounds__(64 * scan_map_waves(false)) k_scan_cols_bwd_agg(ScanArgs a) {
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sma[];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanCol<T, OFF> cl(a, lane);
  const int seg = blockIdx.y + a.fine, flen = a.seg_len / a.fine, part = flen / (NW * cl.subs);   // K's multiple
  const int sbeg = seg * flen + (wv * cl.subs + cl.sub) * part;
  float P = 1.f, Rl = 0.f;
  T rg[K], rd[K];
  ScanRaw<T, false> none[K];
  scan_load<T, false, OFF, true, false>(a, cl, sbeg + part - K, rg, rd, none);
  for (int it = part - K; it >= 0; it -= K) {
    float gv[K], dv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) gv[k] = scan_widen<T>(rg[k]), dv[k] = scan_widen<T>(rd[k]);
    if (it > 0) scan_load<T, false, OFF, true, false>(a, cl, sbeg + it - K, rg, rd, none);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      float aa, c;
      scan_gate<sizeof(T) == 2>(gv[k], aa, c);
      Rl = aa * (dv[k] + Rl);
      P *= aa;
    }
  }
  if (cl.subs > 1) scan_sub_suffix(P, Rl, lane, cl.cw);
  if (cl.sub == 0) sma[wv * cl.cw + cl.cl] = make_float2(P, Rl);
  __syncthreads();
  if (wv == 0 && cl.sub == 0 && cl.active) {
    float p = 1.f, r = 0.f;
    for (int w = NW - 1; w >= 0; --w) {
      const float2 m = sma[w * cl.cw + cl.cl];
      r = fmaf(m.x, r, m.y);
      p *= m.x;
    }
    if (seg == a.maps - 1) {
      r = fmaf(p, a.carry_in ? a.carry_in[cl.col] : 0.f, r);
      p = 0.f;
    }
    a.agg[(size_t)seg * a.cols + cl.col] = make_float2(p, r);
  }
}

// ------------------------------------------------------------------ rows
// As k_scan_rows. A lane's state follows from the kept one of its 32 steps through the maps of
// the (up to three) lanes before it, or (SELF: one tile holds the row) from h0 through the maps of
// all lanes before it. CK: u is a checkpoint. AGG: only the maps.
template <typename T, bool REV, int LANES, bool CK, bool SELF, bool AGG>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_rows_bwd(ScanArgs a) {
  constexpr int E = kScanE;
  static_assert(kScanChunk == 4 * E, "four lanes between states");
  __shared__ RunMap sm[2][kScanWaves];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const T pad = scan_narrow<T>(kScanPad);
  const int lanes = LANES ? LANES : a.lanes, li = lane & (lanes - 1);
  uint64_t r64 = blockIdx.x;
  if (!LANES) r64 = ((uint64_t)blockIdx.x * NW + wv) * (64 / lanes) + lane / lanes;
  const bool active = r64 < a.cols;
  const uint32_t row = active ? (uint32_t)r64 : a.cols - 1;
  const int n = scan_steps(a, row);
  const ScanRow<T, REV> rw(row, a.len, n);
  const ScanRow<uint8_t, REV> rwc(row, a.len, n);
  const int slen = AGG ? a.seg_len / a.fine : a.seg_len;
  const int seg = LANES ? (int)blockIdx.y + (AGG ? a.fine : 0) : 0, sbeg = seg * slen;
  const int send = sbeg + slen < a.len ? sbeg + slen : a.len;
  const int nseg = AGG ? a.maps : a.segs;
  const int tile = LANES ? NW * 64 * E : 64 * E;
  const int lofs = LANES ? (wv * 64 + lane) * E : li * E;
  const T* gp = (const T*)a.g;
  const T* dp = (const T*)a.dh;

  float carry = 0.f, carryP = 1.f, h0 = SELF && a.h0 ? a.h0[row] : 0.f;
  if (seg == nseg - 1) {
    carry = a.carry_in ? a.carry_in[row] : 0.f;
  } else if (!AGG) {
    for (int j = a.maps - 1; j >= (seg + 1) * a.fine; --j) {
      const float2 m = a.agg[(size_t)j * a.cols + row];
      carry = fmaf(m.x, carry, m.y);
    }
  }
  T rg[E], rd[E];
  ScanU<T, REV, CK> ru;
  float kept = 0.f;
  auto load = [&](int s) {
    rw.load(gp, s, rg, pad);
    rw.load(dp, s, rd, T(0));
    if constexpr (!AGG) {
      ru.load(a, rw, rwc, s);
      if (!SELF && s < a.len) kept = a.states[(size_t)row * a.chunks + s / kScanChunk];
    }
  };
  int t0 = sbeg + (send - sbeg - 1) / tile * tile;
  load(t0 + lofs);
  for (int buf = 0; t0 >= sbeg; t0 -= tile, buf ^= 1) {
    const int s = t0 + lofs;
    float av[E], cv[E], ev[E], dv[E], P = 1.f, Rl = 0.f, H = 0.f;
    if constexpr (!AGG) ru.widen(a, rw, s, ev);   // u for now
#pragma unroll
    for (int k = 0; k < E; ++k) {
      scan_gate<sizeof(T) == 2>(scan_widen<T>(rg[k]), av[k], cv[k]);
      dv[k] = scan_widen<T>(rd[k]);
      P *= av[k];
      if constexpr (!AGG) {
        ev[k] *= cv[k];
        H = fmaf(av[k], H, ev[k]);
      }
    }
    Rl = dv[E - 1];
#pragma unroll
    for (int k = E - 2; k >= 0; --k) Rl = fmaf(av[k + 1], Rl, dv[k]);
    Rl *= av[0];
    float h = 0.f;
    float ph = P, hh = H, pe, he;
    if constexpr (SELF) {
      scan_prefix(ph, hh, li, lanes);
    } else if constexpr (!AGG) {   // from the state kept for its group of four lanes
      const int q = lanes < 4 ? lanes : 4, qi = lane & (q - 1);
      if (q > 1) {
        pe = scan_dpp<0x111, 0xf>(1.f, ph);
        he = scan_dpp<0x111, 0xf>(0.f, hh);
        hh = qi >= 1 ? fmaf(ph, he, hh) : hh;
        ph = qi >= 1 ? ph * pe : ph;
      }
      if (q > 2) {
        pe = scan_dpp<0x112, 0xf>(1.f, ph);
        he = scan_dpp<0x112, 0xf>(0.f, hh);
        hh = qi >= 2 ? fmaf(ph, he, hh) : hh;
        ph = qi >= 2 ? ph * pe : ph;
      }
      scan_before(ph, hh, qi, pe, he);
      h = fmaf(pe, kept, he);
    }
    if (t0 - tile >= sbeg) load(s - tile);
    scan_suffix(P, Rl, li, lanes, lane);
    float Rt;
    if (LANES) {
      const float tp = scan_readlane(P, 0), tr = scan_readlane(Rl, 0);
      if (NW > 1) {
        const float th = SELF ? scan_readlane(hh, 63) : 0.f;
        if (lane == 0) sm[buf][wv] = RunMap{tp, tr, th};
        __syncthreads();
        Rt = 0.f;
        for (int w = NW - 1; w >= 0; --w) {
          const RunMap m = sm[buf][w];
          if (w == wv) Rt = carry;
          carry = fmaf(m.p, carry, m.r);
          carryP *= m.p;
        }
        if constexpr (SELF)
          for (int w = 0; w < wv; ++w) h0 = fmaf(sm[buf][w].p, h0, sm[buf][w].h);
      } else {
        Rt = carry;
        carry = fmaf(tp, carry, tr);
        carryP *= tp;
      }
    } else {
      Rt = carry;
    }
    if constexpr (!AGG) {
      if constexpr (SELF) {
        scan_before(ph, hh, li, pe, he);
        h = fmaf(pe, h0, he);
      }
      float re;
      scan_after(P, Rl, li, lanes, pe, re);
      if (!LANES) carry = fmaf(P, Rt, Rl);   // the group's first lane has the row's dh0
      Rt = fmaf(pe, Rt, re);
      if (active && s < a.len) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float cu = ev[k];   // (1 - a) u
          ev[k] = av[k] * fmaf(cv[k], h, -cu);
          h = fmaf(av[k], h, cu);
        }
#pragma unroll
        for (int k = E - 1; k >= 0; --k) {
          const float G = k == E - 1 ? dv[k] + Rt : fmaf(av[k + 1 < E ? k + 1 : k], Rt, dv[k]);
          ev[k] *= G;
          cv[k] *= G;
          Rt = G;
        }
        rw.store((T*)a.out0, s, ev);
        rw.store((T*)a.out1, s, cv);
      }
    }
  }
  const bool writer = LANES ? threadIdx.x == 0 : li == 0;
  if constexpr (AGG) {
    if (writer)
      a.agg[(size_t)seg * a.cols + row] = make_float2(seg == nseg - 1 ? 0.f : carryP, carry);
  } else {
    if (writer && active && seg == 0 && a.carry_out) a.carry_out[row] = carry;
  }
}

template <typename T, bool REV, bool CK, bool SELF>
hipError_t launch_rows(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const dim3 block(64 * p.waves);
  if (a.lanes < 64) {
    const uint32_t per = (uint32_t)p.waves * (64 / a.lanes);
    k_scan_rows_bwd<T, REV, 0, CK, SELF, false><<<dim3((a.cols + per - 1) / per), block, 0, st>>>(a);
    return hipGetLastError();
  }
  if (p.segs > 1) {
    k_scan_rows_bwd<T, REV, 64, false, false, true><<<dim3(a.cols, (p.segs - 1) * p.fine), block, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_rows_bwd<T, REV, 64, CK, SELF, false><<<dim3(a.cols, p.segs), block, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool CK, bool SELF, typename OFF>
hipError_t launch_cols(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const uint32_t groups = (a.cols + a.cw - 1) / a.cw;
  if (p.segs > 1) {
    constexpr int mw = scan_map_waves(false);
    k_scan_cols_bwd_agg<T, OFF><<<dim3(groups, (p.segs - 1) * p.fine), 64 * mw,
                                  mw * a.cw * sizeof(float2), st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  static_assert(2 * scan_col_waves(true, false, false) * 64 * sizeof(RunMap) <= 64 * 1024, "LDS of a launch");
  k_scan_cols_bwd<T, CK, SELF, OFF><<<dim3(groups, p.segs), 64 * p.waves,
                                      2 * p.waves * a.cw * sizeof(RunMap), st>>>(a);
  return hipGetLastError();
}

template <typename T, bool CK, bool SELF>
hipError_t launch_backward_t(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  if (p.rows)
    return a.reverse ? launch_rows<T, true, CK, SELF>(a, p, st) : launch_rows<T, false, CK, SELF>(a, p, st);
  return p.wide ? launch_cols<T, CK, SELF, uint64_t>(a, p, st)
                : launch_cols<T, CK, SELF, uint32_t>(a, p, st);
}

}  // namespace

hipError_t launch_scan_backward(const ScanRequest& r, hipStream_t st) {
  const ScanPlan p = scan_plan(r.outer, r.len, r.inner, r.bf16, r.states ? 1 : 2, r.us != nullptr);
  ScanArgs a = scan_args(r, p);
  const bool self = !r.states && p.self;
  if (!r.states && !self) {   // run the forward for its states, into the workspace
    ScanRequest f = r;
    f.carry_in = r.h0;
    f.carry_out = nullptr;
    f.out0 = f.out1 = nullptr;
    f.states = (float*)r.ws;
    const size_t kept = (size_t)a.cols * a.chunks * 4;
    f.ws = (unsigned char*)r.ws + (kept + 15) / 16 * 16;
    const hipError_t e = launch_scan_forward(f, st);
    if (e != hipSuccess) return e;
    ScanRequest b = r;
    b.states = f.states;
    b.ws = f.ws;
    a = scan_args(b, p);
  }
  auto go = [&](auto ck, auto sf) {
    return r.bf16 ? launch_backward_t<uint16_t, decltype(ck)::value, decltype(sf)::value>(a, p, st)
                  : launch_backward_t<float, decltype(ck)::value, decltype(sf)::value>(a, p, st);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (r.us) return self ? go(Yes{}, Yes{}) : go(Yes{}, No{});
  return self ? go(No{}, Yes{}) : go(No{}, No{});
}

}  // namespace wbmm
