// Gated linear recurrence, forward: the kernels for columns (inner > 1), for rows (inner = 1) and
// for a single step, and the launch rules that forward and backward share.
//
// One pass over the data: a workgroup's waves take consecutive pieces of its columns (or of its
// row), form their pieces' affine maps in registers, pass them through LDS, and each applies the
// state that reaches its piece: g and u are read once, h written once. The next tile's loads are
// issued before the exchange of the current one. Only where the columns are too few to fill the
// chip is the axis cut into segments over several workgroups; a first launch then forms the
// segments' maps (reading g and u a second time), and every workgroup of the second one joins the
// maps before its own, in order.
#include "wbmm_scan.hpp"

#include <algorithm>

namespace wbmm {

namespace {

// ------------------------------------------------------------------ columns
// CK: u is a checkpoint. Without out0 only the states (and the last one) are formed.
template <typename T, int V, bool CK>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_cols(ScanArgs a) {
  typedef typename ScanVec<T, V>::type R;
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sm[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, NW = blockDim.x >> 6;
  const ScanCol<V> cl(a, blockIdx.x, lane);
  const int seg = blockIdx.y, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const T* gp = (const T*)a.g;
  T* hp = (T*)a.out0;

  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  if (seg == 0) {
    const float* ci = a.segs > 1 ? a.carry_copy : a.carry_in;
    if (ci) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = ci[cl.col + v];
    }
  } else {
    for (int j = 0; j < seg; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 m = a.agg[(size_t)j * a.cols + cl.col + v];
        carry[v] = fmaf(m.x, carry[v], m.y);
      }
  }

  R rg[K];
  typename ScanCol<V>::template Raw<T, CK> ru[K];
  auto load = [&](int s) {
    if (__all(s + K <= cl.n)) {
      size_t off = cl.start + (long long)s * cl.stride;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        rg[k] = *(const R*)(gp + off);
        ru[k].load(a, off);
        off += cl.stride;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const size_t off = cl.at(s + k);
        rg[k] = *(const R*)(gp + off);
        ru[k].load(a, off);
      }
    }
  };
  load(sbeg + wv * K);
  int buf = 0;
  for (int t0 = sbeg; t0 < send; t0 += NW * K, buf ^= 1) {
    const int s = t0 + wv * K;
    float av[K][V], bv[K][V], P[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[V], u[V];
      scan_unpack<V>(rg[k], g);
      ru[k].widen(a, u);
      const bool live = s + k < cl.n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float aa, cc;
        scan_gate(g[v], aa, cc);
        av[k][v] = live ? aa : 1.f;
        bv[k][v] = live ? cc * u[v] : 0.f;
        H[v] = fmaf(av[k][v], H[v], bv[k][v]);
        P[v] *= av[k][v];
      }
    }
    if (t0 + NW * K < send) load(s + NW * K);
    float start[V];
    if (NW > 1) {
      float2* sb = sm + (size_t)buf * NW * 64 * V;
#pragma unroll
      for (int v = 0; v < V; ++v) sb[(wv * 64 + lane) * V + v] = make_float2(P[v], H[v]);
      __syncthreads();
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float2 m = sb[(w * 64 + lane) * V + v];
          if (w == wv) start[v] = carry[v];
          carry[v] = fmaf(m.x, carry[v], m.y);
        }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        start[v] = carry[v];
        carry[v] = fmaf(P[v], carry[v], H[v]);
      }
    }
    if (cl.active && s < a.len) {
      if (a.states && s % kScanChunk == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          a.states[((size_t)cl.o * a.chunks + s / kScanChunk) * a.inner + cl.i + v] = start[v];
      }
      float h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = start[v];
      size_t off = cl.start + (long long)s * cl.stride;
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(av[k][v], h[v], bv[k][v]);
        if (hp && s + k < cl.n) *(R*)(hp + off) = scan_pack<R, V>(h);
        off += cl.stride;
      }
      if (hp && s + K > cl.n) cl.template zero<R>(hp, s, a.len, a.inner);
    }
  }
  if (seg == a.segs - 1 && wv == 0 && cl.active && a.carry_out) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.carry_out[cl.col + v] = carry[v];
  }
}

// Maps of segments 0 .. segs - 2; segment 0's has the initial state folded in (P = 0).
template <typename T, int V, bool CK>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_cols_agg(ScanArgs a) {
  typedef typename ScanVec<T, V>::type R;
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sm[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, NW = blockDim.x >> 6;
  const ScanCol<V> cl(a, blockIdx.x, lane);
  const int seg = blockIdx.y, part = a.seg_len / NW;   // a multiple of K
  const int sbeg = seg * a.seg_len + wv * part;
  const T* gp = (const T*)a.g;
  float P[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f;
  for (int s = sbeg; s < sbeg + part; s += K) {
    R rg[K];
    typename ScanCol<V>::template Raw<T, CK> ru[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t off = cl.at(s + k);
      rg[k] = *(const R*)(gp + off);
      ru[k].load(a, off);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[V], u[V];
      scan_unpack<V>(rg[k], g);
      ru[k].widen(a, u);
      const bool live = s + k < cl.n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float aa, cc;
        scan_gate(g[v], aa, cc);
        H[v] = live ? fmaf(aa, H[v], cc * u[v]) : H[v];
        P[v] = live ? P[v] * aa : P[v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sm[(wv * 64 + lane) * V + v] = make_float2(P[v], H[v]);
  __syncthreads();
  if (wv == 0 && cl.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p = 1.f, h = 0.f;
      for (int w = 0; w < NW; ++w) {
        const float2 m = sm[(w * 64 + lane) * V + v];
        h = fmaf(m.x, h, m.y);
        p *= m.x;
      }
      if (seg == 0) {
        const float c0 = a.carry_in ? a.carry_in[cl.col + v] : 0.f;
        h = fmaf(p, c0, h);
        p = 0.f;
        a.carry_copy[cl.col + v] = c0;
      }
      a.agg[(size_t)seg * a.cols + cl.col + v] = make_float2(p, h);
    }
  }
}

// ------------------------------------------------------------------ rows
// LANES = 64: the waves of the workgroup take consecutive 512-step pieces of one row; LANES = 0:
// a.lanes lanes per row (the row fits in a.lanes * kScanE steps) and 64 / a.lanes rows per wave.
// AGG: only the maps of segments 0 .. segs - 2 (as k_scan_cols_agg).
template <typename T, bool REV, int LANES, bool CK, bool AGG>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_rows(ScanArgs a) {
  constexpr int E = kScanE;
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
  const int seg = LANES ? blockIdx.y : 0, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const int tile = LANES ? NW * 64 * E : 64 * E;
  const int lofs = LANES ? (wv * 64 + lane) * E : li * E;
  const T* gp = (const T*)a.g;

  float carry = 0.f, carryP = 1.f, c0 = 0.f;
  if (seg == 0) {
    const float* ci = a.segs > 1 && !AGG ? a.carry_copy : a.carry_in;
    c0 = ci ? ci[row] : 0.f;
    carry = c0;
  } else if (!AGG) {
    for (int j = 0; j < seg; ++j) {
      const float2 m = a.agg[(size_t)j * a.cols + row];
      carry = fmaf(m.x, carry, m.y);
    }
  }
  T rg[E];
  ScanU<T, REV, CK> ru;
  rw.load(gp, sbeg + lofs, rg);
  ru.load(a, rw, rwc, sbeg + lofs);
  int buf = 0;
  for (int t0 = sbeg; t0 < send; t0 += tile, buf ^= 1) {
    const int s = t0 + lofs;
    float av[E], bv[E], P = 1.f, H = 0.f;
    ru.widen(a, rw, s, bv);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      float aa, cc;
      scan_gate(scan_widen<T>(rg[k]), aa, cc);
      const bool live = s + k < n;
      av[k] = live ? aa : 1.f;
      bv[k] = live ? cc * bv[k] : 0.f;
      H = fmaf(av[k], H, bv[k]);
      P *= av[k];
    }
    if (t0 + tile < send) {
      rw.load(gp, s + tile, rg);
      ru.load(a, rw, rwc, s + tile);
    }
    scan_prefix(P, H, li, lanes);
    float start;
    if (LANES) {
      const float tp = scan_readlane(P, 63), th = scan_readlane(H, 63);
      if (NW > 1) {
        if (lane == 0) sm[buf][wv] = make_float2(tp, th);
        __syncthreads();
        start = 0.f;
        for (int w = 0; w < NW; ++w) {
          const float2 m = sm[buf][w];
          if (w == wv) start = carry;
          carry = fmaf(m.x, carry, m.y);
          carryP *= m.x;
        }
      } else {
        start = carry;
        carry = fmaf(tp, carry, th);
        carryP *= tp;
      }
    } else {
      start = carry;
    }
    if constexpr (!AGG) {
      float pe, he;
      scan_before(P, H, li, pe, he);
      float h = fmaf(pe, start, he);
      if (!LANES) carry = fmaf(P, start, H);   // the group's last lane has the row's last state
      if (active && s < a.len) {
        if (a.states && s % kScanChunk == 0)
          a.states[(size_t)row * a.chunks + s / kScanChunk] = h;
        float o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
          h = fmaf(av[k], h, bv[k]);
          o[k] = h;
        }
        if (a.out0) rw.store((T*)a.out0, s, o);
      }
    }
  }
  const bool writer = LANES ? threadIdx.x == 0 : li == lanes - 1;
  if constexpr (AGG) {
    if (writer) {
      if (seg == 0) a.carry_copy[row] = c0;
      a.agg[(size_t)seg * a.cols + row] = make_float2(seg == 0 ? 0.f : carryP, carry);
    }
  } else {
    if (writer && active && seg == a.segs - 1 && a.carry_out) a.carry_out[row] = carry;
  }
}

// ------------------------------------------------------------------ one step (len = 1)
template <typename T>
__global__ void __launch_bounds__(kThreads) k_scan_step(ScanArgs a) {
  const uint64_t c = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.cols) return;
  const float h0 = a.carry_in ? a.carry_in[c] : 0.f;
  float aa, cc;
  scan_gate(scan_widen<T>(((const T*)a.g)[c]), aa, cc);
  const float h = fmaf(aa, h0, cc * scan_widen<T>(((const T*)a.u)[c]));
  const bool live = scan_steps(a, (uint32_t)(c / a.inner)) > 0;
  ((T*)a.out0)[c] = scan_narrow<T>(live ? h : 0.f);
  if (a.carry_out) a.carry_out[c] = live ? h : h0;
  if (a.states) a.states[c] = h0;
}

template <typename T, bool REV, bool CK>
hipError_t launch_rows(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const dim3 block(64 * p.waves);
  if (a.lanes < 64) {
    const uint32_t per = (uint32_t)p.waves * (64 / a.lanes);
    k_scan_rows<T, REV, 0, CK, false><<<dim3((a.cols + per - 1) / per), block, 0, st>>>(a);
    return hipGetLastError();
  }
  if (p.segs > 1) {
    k_scan_rows<T, REV, 64, CK, true><<<dim3(a.cols, p.segs - 1), block, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_rows<T, REV, 64, CK, false><<<dim3(a.cols, p.segs), block, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int V, bool CK>
hipError_t launch_cols(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const uint32_t groups = (uint32_t)(((uint64_t)a.cols + 64 * V - 1) / (64 * V));
  const dim3 block(64 * p.waves);
  const unsigned lds = p.waves * 64 * V * sizeof(float2);
  if (p.segs > 1) {
    k_scan_cols_agg<T, V, CK><<<dim3(groups, p.segs - 1), block, lds, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_cols<T, V, CK><<<dim3(groups, p.segs), block, 2 * lds, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool CK>
hipError_t launch_forward(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  if (p.rows)
    return a.reverse ? launch_rows<T, true, CK>(a, p, st) : launch_rows<T, false, CK>(a, p, st);
  if constexpr (sizeof(T) == 2) {
    if (p.V == 2) return launch_cols<T, 2, CK>(a, p, st);
  }
  return launch_cols<T, 1, CK>(a, p, st);
}

}  // namespace

int scan_pow2(long long v) {  // least power of two >= v, at least 1
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Launch shape. Waves per workgroup: as many as the axis has pieces for, up to kScanWaves, and
// only as many as it takes to put kWantWaves on the chip. Where that is not reached, segments.
ScanPlan scan_plan(int64_t outer, int64_t len, int64_t inner, int V, bool backward) {
  constexpr long long kWantWaves = 4096, kSegWaves = 1024;
  ScanPlan p{};
  p.V = V;
  p.rows = inner == 1;
  p.segs = 1;
  const int piece = p.rows ? 64 * kScanE : kScanK;
  long long units;   // workgroups without segments
  if (p.rows) {
    p.lanes = len >= 32 * kScanE + 1 ? 64 : scan_pow2((len + kScanE - 1) / kScanE);
    if (p.lanes < 64) {
      p.waves = 4;
      p.seg_len = 64 * kScanE;
      return p;
    }
    units = outer;
  } else {
    p.lanes = 64;
    units = (outer * inner + 64 * V - 1) / (64 * V);
  }
  const int least = !p.rows && backward ? 2 : 1;   // the backward's waves work in pairs there
  const int most = std::max(least, std::min(kScanWaves, scan_pow2((len + piece - 1) / piece)));
  p.waves = (int)std::min<long long>(most, std::max<long long>(least, scan_pow2((kWantWaves + units - 1) / units)));
  const long long tile = (long long)p.waves * piece;
  if (units * p.waves < kSegWaves) {
    const long long tiles = (len + tile - 1) / tile;
    long long segs = std::min<long long>({(2 * kSegWaves + units * p.waves - 1) / (units * p.waves),
                                          (tiles + 1) / 2, 64});
    if (segs > 1) {
      const long long per = (tiles + segs - 1) / segs;
      p.segs = (int)((tiles + per - 1) / per);
      p.seg_len = (int)(per * tile);
      return p;
    }
  }
  p.seg_len = (int)((len + tile - 1) / tile * tile);
  return p;
}

int scan_vec(const ScanRequest& r) {   // columns per lane of the forward
  const uintptr_t p = (uintptr_t)r.g | (uintptr_t)r.u | (uintptr_t)r.out0;
  return r.bf16 && r.inner % 2 == 0 && p % 4 == 0 ? 2 : 1;
}

namespace {
size_t maps_bytes(const ScanPlan& p, size_t cols) { return p.segs > 1 ? cols * (8 * p.segs + 4) : 0; }
}  // namespace

size_t scan_workspace(int64_t outer, int64_t len, int64_t inner) {
  // the type and the alignment are not arguments: the larger need
  const size_t cols = (size_t)(outer * inner);
  return std::max(maps_bytes(scan_plan(outer, len, inner, 1, false), cols),
                  maps_bytes(scan_plan(outer, len, inner, 2, false), cols));
}

size_t scan_backward_workspace(int64_t outer, int64_t len, int64_t inner, bool has_states) {
  const size_t cols = (size_t)(outer * inner);
  const size_t maps = maps_bytes(scan_plan(outer, len, inner, 1, true), cols);
  if (has_states) return maps;
  // states (whole 16 bytes), then the maps of either launch
  const size_t kept = cols * ((len + kScanChunk - 1) / kScanChunk) * 4;
  return (kept + 15) / 16 * 16 + std::max(maps, scan_workspace(outer, len, inner));
}

ScanArgs scan_args(const ScanRequest& r, const ScanPlan& p) {
  ScanArgs a{};
  a.g = r.g;
  a.u = r.u;
  a.us = r.us;
  a.fmt = r.fmt;
  a.dh = r.dh;
  a.carry_in = r.carry_in;
  a.lens = r.lens;
  a.out0 = r.out0;
  a.out1 = r.out1;
  a.carry_out = r.carry_out;
  a.states = r.states;
  a.len = (int)r.len;
  a.chunks = (int)((r.len + kScanChunk - 1) / kScanChunk);
  a.reverse = r.reverse;
  a.inner = (uint32_t)r.inner;
  a.cols = (uint32_t)(r.outer * r.inner);
  a.rows_per_len = r.lens ? (uint32_t)(r.outer / r.n_lens) : 1;
  a.segs = p.segs;
  a.seg_len = p.seg_len;
  a.lanes = p.lanes;
  a.agg = (float2*)r.ws;
  a.carry_copy = r.ws ? (float*)r.ws + (size_t)2 * p.segs * a.cols : nullptr;
  return a;
}

hipError_t launch_scan_forward(const ScanRequest& r, hipStream_t st) {
  const int V = scan_vec(r);
  const ScanPlan p = scan_plan(r.outer, r.len, r.inner, V, false);
  const ScanArgs a = scan_args(r, p);
  if (r.len == 1 && r.out0) {
    const dim3 grid((unsigned)(((uint64_t)a.cols + kThreads - 1) / kThreads));
    if (r.bf16)
      k_scan_step<uint16_t><<<grid, kThreads, 0, st>>>(a);
    else
      k_scan_step<float><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  if (r.bf16) return r.us ? launch_forward<uint16_t, true>(a, p, st) : launch_forward<uint16_t, false>(a, p, st);
  return r.us ? launch_forward<float, true>(a, p, st) : launch_forward<float, false>(a, p, st);
}

}  // namespace wbmm
