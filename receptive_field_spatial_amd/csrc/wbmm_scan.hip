// Gated linear recurrence, forward: the kernels for columns (inner > 1), for rows (inner = 1) and
// for a single step.
//
// One pass over the data: a workgroup's waves take consecutive pieces of its columns (or of its
// row), form their pieces' affine maps in registers, pass them through LDS, and each applies the
// state that reaches its piece: g and u are read once, h written once. The next tile's loads are
// issued before the exchange of the current one. Only where the columns are too few to fill the
// chip is the axis cut into segments over several workgroups; a first launch then forms the maps of
// the segments, or of finer parts of them (reading g and u a second time), and every workgroup of the
// second one joins the maps before its own, in order.
//
// What bounds it: memory on large tensors, one launch and its chain of loads and exchanges on small
// ones. Measured (kernel alone; rates of the bytes that have to move, a large copy reaches 5.05 TB/s):
// k_scan_cols 64 x 784 x 192 bf16 20 us, 3.0 TB/s; k_scan_rows 256 x 16384 fp32, reversed, 13.6 us,
// 3.7 TB/s; k_scan_cols 13 x 1531 x 97 fp32, ragged, 16 us; k_scan_step 8 x 192 bf16 2.3 us.
#include "wbmm_scan.hpp"

namespace wbmm {

namespace {

// ------------------------------------------------------------------ columns
// CK: u is a checkpoint. Without out0 only the states (and the last one) are formed.
template <typename T, bool CK, typename OFF>
__global__ void __launch_bounds__(64 * scan_col_waves(false, CK, false))
k_scan_cols(ScanArgs a) {
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sm[];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanCol<T, OFF> cl(a, lane);
  const int seg = blockIdx.y, sbeg = seg * a.seg_len;
  const int send = sbeg + a.seg_len < a.len ? sbeg + a.seg_len : a.len;
  const int tile = NW * cl.subs * K, lofs = (wv * cl.subs + cl.sub) * K;

  float carry = 0.f;
  if (seg == 0) {
    const float* ci = a.segs > 1 ? a.carry_copy : a.carry_in;
    if (ci) carry = ci[cl.col];
  } else {
    for (int j = 0; j < seg * a.fine; ++j) {
      const float2 m = a.agg[(size_t)j * a.cols + cl.col];
      carry = fmaf(m.x, carry, m.y);
    }
  }

  T rg[K];
  ScanRaw<T, CK> ru[K];
  auto load = [&](int s) { scan_load<T, CK, OFF, false>(a, cl, s, rg, rg, ru); };
  load(sbeg + lofs);
  int buf = 0;
  for (int t0 = sbeg; t0 < send; t0 += tile, buf ^= 1) {
    const int s = t0 + lofs;
    float av[K], bv[K], P = 1.f, H = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float c;
      scan_gate<sizeof(T) == 2>(scan_widen<T>(rg[k]), av[k], c);
      bv[k] = c * ru[k].widen(a);
      H = fmaf(av[k], H, bv[k]);
      P *= av[k];
    }
    if (t0 + tile < send) load(s + tile);
    float start = carry;
    if (cl.subs > 1) scan_sub_prefix(P, H, lane, cl.cw);
    if (NW > 1) {
      float2* sb = sm + buf * NW * cl.cw;
      if (cl.sub == cl.subs - 1) sb[wv * cl.cw + cl.cl] = make_float2(P, H);
      __syncthreads();
      for (int w = 0; w < NW; ++w) {
        const float2 m = sb[w * cl.cw + cl.cl];
        if (w == wv) start = carry;
        carry = fmaf(m.x, carry, m.y);
      }
    } else {
      const float p = cl.subs > 1 ? __shfl(P, 64 - cl.cw + cl.cl) : P;
      const float h = cl.subs > 1 ? __shfl(H, 64 - cl.cw + cl.cl) : H;
      carry = fmaf(p, carry, h);
    }
    if (cl.subs > 1) {
      const float p = __shfl(P, lane - cl.cw), h = __shfl(H, lane - cl.cw);
      start = cl.sub > 0 ? fmaf(p, start, h) : start;
    }
    if (cl.active && s < a.len) {
      if (a.states && s % kScanChunk == 0) a.states[cl.kept(a, s)] = start;
      float h = start;
      if (a.out0) {
        OFF o = cl.at(s);
        if (__all(s + K <= cl.n)) {
#pragma unroll
          for (int k = 0; k < K; ++k, o += cl.stride) {
            h = fmaf(av[k], h, bv[k]);
            cl.store(a.out0, o, h);
          }
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k, o += cl.stride) {
            h = fmaf(av[k], h, bv[k]);
            if (s + k < cl.n) cl.store(a.out0, o, h);
          }
          cl.zero(a.out0, s, a.len, a.inner);
        }
      }
    }
  }
  if (seg == a.segs - 1 && wv == 0 && cl.sub == 0 && cl.active && a.carry_out)
    a.carry_out[cl.col] = carry;
}

// The maps before the last segment's; the first has the initial state folded in (P = 0).
template <typename T, bool CK, typename OFF>
__global__ void __launch_bounds__(64 * scan_map_waves(CK)) k_scan_cols_agg(ScanArgs a) {
  constexpr int K = kScanK;
  extern __shared__ __attribute__((aligned(16))) float2 sm[];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanCol<T, OFF> cl(a, lane);
  const int seg = blockIdx.y, flen = a.seg_len / a.fine, part = flen / (NW * cl.subs);   // K's multiple
  const int sbeg = seg * flen + (wv * cl.subs + cl.sub) * part;
  float P = 1.f, H = 0.f;
  T rg[K];
  ScanRaw<T, CK> ru[K];
  scan_load<T, CK, OFF, false>(a, cl, sbeg, rg, rg, ru);
  for (int it = 0; it < part; it += K) {
    float gv[K], uv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) gv[k] = scan_widen<T>(rg[k]), uv[k] = ru[k].widen(a);
    if (it + K < part) scan_load<T, CK, OFF, false>(a, cl, sbeg + it + K, rg, rg, ru);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float aa, c;
      scan_gate<sizeof(T) == 2>(gv[k], aa, c);
      H = fmaf(aa, H, c * uv[k]);
      P *= aa;
    }
  }
  if (cl.subs > 1) scan_sub_prefix(P, H, lane, cl.cw);
  if (cl.sub == cl.subs - 1) sm[wv * cl.cw + cl.cl] = make_float2(P, H);
  __syncthreads();
  if (wv == 0 && cl.sub == 0 && cl.active) {
    float p = 1.f, h = 0.f;
    for (int w = 0; w < NW; ++w) {
      const float2 m = sm[w * cl.cw + cl.cl];
      h = fmaf(m.x, h, m.y);
      p *= m.x;
    }
    if (seg == 0) {
      const float c0 = a.carry_in ? a.carry_in[cl.col] : 0.f;
      h = fmaf(p, c0, h);
      p = 0.f;
      a.carry_copy[cl.col] = c0;
    }
    a.agg[(size_t)seg * a.cols + cl.col] = make_float2(p, h);
  }
}

// ------------------------------------------------------------------ rows
// LANES = 64: the waves of the workgroup take consecutive 512-step pieces of one row; LANES = 0:
// a.lanes lanes per row (the row fits in a.lanes * kScanE steps) and 64 / a.lanes rows per wave.
// AGG: only the maps (as k_scan_cols_agg).
template <typename T, bool REV, int LANES, bool CK, bool AGG>
__global__ void __launch_bounds__(64 * kScanWaves) k_scan_rows(ScanArgs a) {
  constexpr int E = kScanE;
  __shared__ float2 sm[2][kScanWaves];
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
  const int seg = LANES ? blockIdx.y : 0, sbeg = seg * slen;
  const int send = sbeg + slen < a.len ? sbeg + slen : a.len;
  const int tile = LANES ? NW * 64 * E : 64 * E;
  const int lofs = LANES ? (wv * 64 + lane) * E : li * E;
  const T* gp = (const T*)a.g;

  float carry = 0.f, carryP = 1.f, c0 = 0.f;
  if (seg == 0) {
    const float* ci = a.segs > 1 && !AGG ? a.carry_copy : a.carry_in;
    c0 = ci ? ci[row] : 0.f;
    carry = c0;
  } else if (!AGG) {
    for (int j = 0; j < seg * a.fine; ++j) {
      const float2 m = a.agg[(size_t)j * a.cols + row];
      carry = fmaf(m.x, carry, m.y);
    }
  }
  T rg[E];
  ScanU<T, REV, CK> ru;
  rw.load(gp, sbeg + lofs, rg, pad);
  ru.load(a, rw, rwc, sbeg + lofs);
  int buf = 0;
  for (int t0 = sbeg; t0 < send; t0 += tile, buf ^= 1) {
    const int s = t0 + lofs;
    float av[E], bv[E], P = 1.f, H = 0.f;
    ru.widen(a, rw, s, bv);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      float c;
      scan_gate<sizeof(T) == 2>(scan_widen<T>(rg[k]), av[k], c);
      bv[k] *= c;
      H = fmaf(av[k], H, bv[k]);
      P *= av[k];
    }
    if (t0 + tile < send) {
      rw.load(gp, s + tile, rg, pad);
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
  scan_gate<sizeof(T) == 2>(scan_widen<T>(((const T*)a.g)[c]), aa, cc);
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
    k_scan_rows<T, REV, 64, CK, true><<<dim3(a.cols, (p.segs - 1) * p.fine), block, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_rows<T, REV, 64, CK, false><<<dim3(a.cols, p.segs), block, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool CK, typename OFF>
hipError_t launch_cols(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const uint32_t groups = (a.cols + a.cw - 1) / a.cw;
  const unsigned lds = a.cw * sizeof(float2);
  if (p.segs > 1) {
    constexpr int mw = scan_map_waves(CK);
    k_scan_cols_agg<T, CK, OFF><<<dim3(groups, (p.segs - 1) * p.fine), 64 * mw, mw * lds, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_cols<T, CK, OFF><<<dim3(groups, p.segs), 64 * p.waves, 2 * p.waves * lds, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool CK>
hipError_t launch_forward(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  if (p.rows)
    return a.reverse ? launch_rows<T, true, CK>(a, p, st) : launch_rows<T, false, CK>(a, p, st);
  return p.wide ? launch_cols<T, CK, uint64_t>(a, p, st) : launch_cols<T, CK, uint32_t>(a, p, st);
}

}  // namespace

ScanArgs scan_args(const ScanRequest& r, const ScanPlan& p) {
  ScanArgs a{};
  a.g = r.g;
  a.u = r.u;
  a.us = r.us;
  a.fmt = r.fmt;
  a.dh = r.dh;
  a.carry_in = r.carry_in;
  a.h0 = r.h0;
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
  a.fine = p.fine;
  a.maps = p.segs * p.fine;
  a.seg_len = p.seg_len;
  a.lanes = p.lanes;
  a.cw = p.cw;
  a.run = p.run;
  a.agg = (float2*)r.ws;
  a.carry_copy = r.ws ? (float*)r.ws + (size_t)2 * a.maps * a.cols : nullptr;
  return a;
}

hipError_t launch_scan_forward(const ScanRequest& r, hipStream_t st) {
  const ScanPlan p = scan_plan(r.outer, r.len, r.inner, r.bf16, 0, r.us != nullptr);
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
