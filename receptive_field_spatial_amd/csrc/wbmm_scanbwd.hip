// Gated linear recurrence, backward. With R_t the gradient that reaches the state h_t from step
// t + 1 (dh_last at the end),
//   G_t = dh_t + R_t,   du_t = (1 - a_t) G_t,   dg_t = a_t (1 - a_t) (h_{t-1} - u_t) G_t,
//   R_{t-1} = a_t G_t,  dh0 = R_{-1}.
// The h_{t-1} come from the states that the forward kept every 32 steps (fp32, so nothing of h's
// own rounding enters): a piece runs the recurrence again from its state, in registers, while it
// has g and u there for the gradient anyway. R runs through the same pieces in the other order,
// as the affine maps of wbmm_scan.hpp. One pass: g, u, dh read, dg, du written.
#include "wbmm_scan.hpp"

namespace wbmm {

namespace {

struct SegMap {
  float p, r, h;
};

// ------------------------------------------------------------------ columns
// A wave's tile is half the distance between two states: the wave of an odd half gets its state
// from the wave before it, beside the maps that are exchanged anyway, so waves come in pairs.
// CK: u is a checkpoint.
template <typename T, int V, bool CK>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_cols_bwd(ScanArgs a) {
  typedef typename ScanVec<T, V>::type R;
  constexpr int K = kScanK;
  static_assert(kScanChunk == 2 * K, "two tiles between states");
  extern __shared__ __attribute__((aligned(16))) SegMap smb[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, NW = blockDim.x >> 6;
  const ScanCol<V> cl(a, blockIdx.x, lane);
  const int seg = blockIdx.y, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const T* gp = (const T*)a.g;
  const T* dp = (const T*)a.dh;
  T* dgp = (T*)a.out0;
  T* dup = (T*)a.out1;

  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  if (seg == a.segs - 1) {
    if (a.carry_in) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = a.carry_in[cl.col + v];
    }
  } else {
    for (int j = a.segs - 1; j > seg; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 m = a.agg[(size_t)j * a.cols + cl.col + v];
        carry[v] = fmaf(m.x, carry[v], m.y);
      }
  }

  R rg[K], rd[K];
  typename ScanCol<V>::template Raw<T, CK> ru[K];
  auto load = [&](int s) {
    const bool full = __all(s + K <= cl.n);
    size_t off = cl.start + (long long)s * cl.stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t o = full ? off : cl.at(s + k);
      rg[k] = *(const R*)(gp + o);
      rd[k] = *(const R*)(dp + o);
      ru[k].load(a, o);
      off += cl.stride;
    }
  };
  const int tile = NW * K;
  int t0 = sbeg + (send - sbeg - 1) / tile * tile;
  load(t0 + wv * K);
  for (int buf = 0; t0 >= sbeg; t0 -= tile, buf ^= 1) {
    const int s = t0 + wv * K;
    float av[K][V], cv[K][V], ev[K][V], dv[K][V], P[V], Rl[V], h[V];
    const bool even = (wv & 1) == 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      Rl[v] = 0.f;
      h[v] = 0.f;
      if (even && s < a.len)
        h[v] = a.states[((size_t)cl.o * a.chunks + s / kScanChunk) * a.inner + cl.i + v];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[V], d[V];
      scan_unpack<V>(rg[k], g);
      scan_unpack<V>(rd[k], d);
      ru[k].widen(a, ev[k]);   // u for now
      const bool live = s + k < cl.n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float aa, cc;
        scan_gate(g[v], aa, cc);
        av[k][v] = live ? aa : 1.f;
        cv[k][v] = live ? cc : 0.f;
        dv[k][v] = live ? d[v] : 0.f;
        ev[k][v] = live ? ev[k][v] : 0.f;
        P[v] *= av[k][v];
      }
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
#pragma unroll
      for (int v = 0; v < V; ++v) Rl[v] = av[k][v] * (dv[k][v] + Rl[v]);
    // the gradient of g up to the factor G; the state runs along
    auto run = [&]() {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float u = ev[k][v];
          ev[k][v] = av[k][v] * cv[k][v] * (h[v] - u);
          h[v] = fmaf(av[k][v], h[v], cv[k][v] * u);
        }
    };
    if (even) run();
    if (t0 - tile >= sbeg) load(s - tile);
    SegMap* sb = smb + (size_t)buf * NW * 64 * V;
#pragma unroll
    for (int v = 0; v < V; ++v) sb[(wv * 64 + lane) * V + v] = SegMap{P[v], Rl[v], h[v]};
    __syncthreads();
    float Rt[V];
    for (int w = NW - 1; w >= 0; --w)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const SegMap m = sb[(w * 64 + lane) * V + v];
        if (w == wv) Rt[v] = carry[v];
        if (w == wv - 1 && !even) h[v] = m.h;
        carry[v] = fmaf(m.p, carry[v], m.r);
      }
    if (!even) run();
    if (cl.active && s < a.len) {
      size_t off = cl.start + (long long)(s + K - 1) * cl.stride;
#pragma unroll
      for (int k = K - 1; k >= 0; --k) {
        float dg[V], du[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float G = dv[k][v] + Rt[v];
          dg[v] = ev[k][v] * G;
          du[v] = cv[k][v] * G;
          Rt[v] = av[k][v] * G;
        }
        if (s + k < cl.n) {
          *(R*)(dgp + off) = scan_pack<R, V>(dg);
          *(R*)(dup + off) = scan_pack<R, V>(du);
        }
        off -= cl.stride;
      }
      if (s + K > cl.n) {
        cl.template zero<R>(dgp, s, a.len, a.inner);
        cl.template zero<R>(dup, s, a.len, a.inner);
      }
    }
  }
  if (seg == 0 && wv == 0 && cl.active && a.carry_out) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.carry_out[cl.col + v] = carry[v];
  }
}

// Maps of segments 1 .. segs - 1 (blockIdx.y + 1); the last one's has dh_last folded in (P = 0).
template <typename T, int V>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_cols_bwd_agg(ScanArgs a) {
  typedef typename ScanVec<T, V>::type R;
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sma[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, NW = blockDim.x >> 6;
  const ScanCol<V> cl(a, blockIdx.x, lane);
  const int seg = blockIdx.y + 1, part = a.seg_len / NW;   // a multiple of K
  const int sbeg = seg * a.seg_len + wv * part;
  const T* gp = (const T*)a.g;
  const T* dp = (const T*)a.dh;
  float P[V], Rl[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.f, Rl[v] = 0.f;
  for (int s = sbeg + part - K; s >= sbeg; s -= K) {
    R rg[K], rd[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t off = cl.at(s + k);
      rg[k] = *(const R*)(gp + off);
      rd[k] = *(const R*)(dp + off);
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      float g[V], d[V];
      scan_unpack<V>(rg[k], g);
      scan_unpack<V>(rd[k], d);
      const bool live = s + k < cl.n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float aa, cc;
        scan_gate(g[v], aa, cc);
        Rl[v] = live ? aa * (d[v] + Rl[v]) : Rl[v];
        P[v] = live ? P[v] * aa : P[v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sma[(wv * 64 + lane) * V + v] = make_float2(P[v], Rl[v]);
  __syncthreads();
  if (wv == 0 && cl.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p = 1.f, r = 0.f;
      for (int w = NW - 1; w >= 0; --w) {
        const float2 m = sma[(w * 64 + lane) * V + v];
        r = fmaf(m.x, r, m.y);
        p *= m.x;
      }
      if (seg == a.segs - 1) {
        r = fmaf(p, a.carry_in ? a.carry_in[cl.col + v] : 0.f, r);
        p = 0.f;
      }
      a.agg[(size_t)seg * a.cols + cl.col + v] = make_float2(p, r);
    }
  }
}

// ------------------------------------------------------------------ rows
// As k_scan_rows. A lane's state follows from the kept one of its 32 steps through the maps of
// the (up to three) lanes before it. CK: u is a checkpoint. AGG: maps of segments 1 .. segs - 1.
template <typename T, bool REV, int LANES, bool CK, bool AGG>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_rows_bwd(ScanArgs a) {
  constexpr int E = kScanE;
  static_assert(kScanChunk == 4 * E, "four lanes between states");
  __shared__ float2 sm[2][kScanWaves];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, NW = blockDim.x >> 6;
  const int lanes = LANES ? LANES : a.lanes, li = lane & (lanes - 1);
  uint64_t r64 = blockIdx.x;
  if (!LANES) r64 = ((uint64_t)blockIdx.x * NW + wv) * (64 / lanes) + lane / lanes;
  const bool active = r64 < a.cols;
  const uint32_t row = active ? (uint32_t)r64 : a.cols - 1;
  const int n = scan_steps(a, row);
  const ScanRow<T, REV> rw(row, a.len, n);
  const ScanRow<uint8_t, REV> rwc(row, a.len, n);
  const int seg = LANES ? (int)blockIdx.y + (AGG ? 1 : 0) : 0, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const int tile = LANES ? NW * 64 * E : 64 * E;
  const int lofs = LANES ? (wv * 64 + lane) * E : li * E;
  const T* gp = (const T*)a.g;
  const T* dp = (const T*)a.dh;

  float carry = 0.f, carryP = 1.f;
  if (seg == a.segs - 1) {
    carry = a.carry_in ? a.carry_in[row] : 0.f;
  } else if (!AGG) {
    for (int j = a.segs - 1; j > seg; --j) {
      const float2 m = a.agg[(size_t)j * a.cols + row];
      carry = fmaf(m.x, carry, m.y);
    }
  }
  T rg[E], rd[E];
  ScanU<T, REV, CK> ru;
  float kept = 0.f;
  auto load = [&](int s) {
    rw.load(gp, s, rg);
    rw.load(dp, s, rd);
    if constexpr (!AGG) {
      ru.load(a, rw, rwc, s);
      if (s < a.len) kept = a.states[(size_t)row * a.chunks + s / kScanChunk];
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
      float aa, cc;
      scan_gate(scan_widen<T>(rg[k]), aa, cc);
      const bool live = s + k < n;
      av[k] = live ? aa : 1.f;
      cv[k] = live ? cc : 0.f;
      dv[k] = live ? scan_widen<T>(rd[k]) : 0.f;
      P *= av[k];
      if constexpr (!AGG) {
        ev[k] = live ? ev[k] : 0.f;
        H = fmaf(av[k], H, cv[k] * ev[k]);
      }
    }
#pragma unroll
    for (int k = E - 1; k >= 0; --k) Rl = av[k] * (dv[k] + Rl);
    float h = 0.f;
    if constexpr (!AGG) {   // the lane's state, from the one kept for its group of four lanes
      const int q = lanes < 4 ? lanes : 4, qi = lane & (q - 1);
      float ph = P, hh = H, pe, he;
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
        if (lane == 0) sm[buf][wv] = make_float2(tp, tr);
        __syncthreads();
        Rt = 0.f;
        for (int w = NW - 1; w >= 0; --w) {
          const float2 m = sm[buf][w];
          if (w == wv) Rt = carry;
          carry = fmaf(m.x, carry, m.y);
          carryP *= m.x;
        }
      } else {
        Rt = carry;
        carry = fmaf(tp, carry, tr);
        carryP *= tp;
      }
    } else {
      Rt = carry;
    }
    if constexpr (!AGG) {
      float pe, re;
      scan_after(P, Rl, li, lanes, pe, re);
      if (!LANES) carry = fmaf(P, Rt, Rl);   // the group's first lane has the row's dh0
      Rt = fmaf(pe, Rt, re);
      if (active && s < a.len) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float u = ev[k];
          ev[k] = av[k] * cv[k] * (h - u);
          h = fmaf(av[k], h, cv[k] * u);
        }
#pragma unroll
        for (int k = E - 1; k >= 0; --k) {
          const float G = dv[k] + Rt;
          ev[k] *= G;
          cv[k] *= G;
          Rt = av[k] * G;
        }
        rw.store((T*)a.out0, s, ev);
        rw.store((T*)a.out1, s, cv);
      }
    }
  }
  const bool writer = LANES ? threadIdx.x == 0 : li == 0;
  if constexpr (AGG) {
    if (writer)
      a.agg[(size_t)seg * a.cols + row] = make_float2(seg == a.segs - 1 ? 0.f : carryP, carry);
  } else {
    if (writer && active && seg == 0 && a.carry_out) a.carry_out[row] = carry;
  }
}

template <typename T, bool REV>
hipError_t launch_rows(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const dim3 block(64 * p.waves);
  if (a.lanes < 64) {
    const uint32_t per = (uint32_t)p.waves * (64 / a.lanes);
    const dim3 grid((a.cols + per - 1) / per);
    if (a.us)
      k_scan_rows_bwd<T, REV, 0, true, false><<<grid, block, 0, st>>>(a);
    else
      k_scan_rows_bwd<T, REV, 0, false, false><<<grid, block, 0, st>>>(a);
    return hipGetLastError();
  }
  if (p.segs > 1) {
    k_scan_rows_bwd<T, REV, 64, false, true><<<dim3(a.cols, p.segs - 1), block, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(a.cols, p.segs);
  if (a.us)
    k_scan_rows_bwd<T, REV, 64, true, false><<<grid, block, 0, st>>>(a);
  else
    k_scan_rows_bwd<T, REV, 64, false, false><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_cols(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const uint32_t groups = (uint32_t)(((uint64_t)a.cols + 64 * V - 1) / (64 * V));
  const dim3 block(64 * p.waves);
  const unsigned per = p.waves * 64 * V;
  if (p.segs > 1) {
    k_scan_cols_bwd_agg<T, V><<<dim3(groups, p.segs - 1), block, per * sizeof(float2), st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(groups, p.segs);
  const unsigned lds = 2 * per * sizeof(SegMap);
  static_assert(2 * kScanWaves * 64 * V * sizeof(SegMap) <= 64 * 1024, "LDS of a launch");
  if (a.us)
    k_scan_cols_bwd<T, V, true><<<grid, block, lds, st>>>(a);
  else
    k_scan_cols_bwd<T, V, false><<<grid, block, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_backward(const ScanRequest& r, hipStream_t st) {
  const ScanPlan p = scan_plan(r.outer, r.len, r.inner, 1, true);
  ScanArgs a = scan_args(r, p);
  if (!r.states) {   // run the forward for its states, into the workspace
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
  if (p.rows) {
    if (r.bf16) return r.reverse ? launch_rows<uint16_t, true>(a, p, st) : launch_rows<uint16_t, false>(a, p, st);
    return r.reverse ? launch_rows<float, true>(a, p, st) : launch_rows<float, false>(a, p, st);
  }
  return r.bf16 ? launch_cols<uint16_t, 1>(a, p, st) : launch_cols<float, 1>(a, p, st);
}

}  // namespace wbmm
