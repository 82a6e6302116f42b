// Gated delta rule, forward: what each chunk computes on its own (k_delta_prep), the walk along the
// chunks (k_delta_walk), and single steps (k_delta_step).
#include "wbmm_deltadev.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

// ---------------------------------------------------------------------------- chunks on their own
// One workgroup of 4 waves per chunk of a head: T, P and the gates. Wave j takes column tile j of the
// 64 x 64 matrices. (I + A)^-1 in fp32 on v_mfma_f32_16x16x4f32: its diagonal tiles by doubling, with N
// = -A_jj: (I + N)(I + N^2)(I + N^4)(I + N^8), N^16 = 0; below them T_ij = T_ii sum_k N_ik T_kj, down the
// column, which needs no other wave's column. With terms in the order 4 q + s, s the product's number,
// a result is the next product's B operand as it lies, and the A operand of its transpose.
__device__ __forceinline__ v4f mm16(const v4f& a, const v4f& b, v4f acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma_f32(a[s], b[s], acc);
  return acc;
}

template <typename T>
__device__ __forceinline__ float elem(const void* p, size_t i) { return load_f32<T>((const T*)p, i); }

template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(256) k_delta_prep(DeltaArgs a) {
  constexpr int PI = DeltaType<T>::PI, KS = DK / 32;
  using Quad = typename DeltaType<T>::Quad;
  __shared__ double s_cum[kDeltaChunk];
  __shared__ float s_b[kDeltaChunk];
  __shared__ float s_n[6][16][20];      // N_ij, j < i
  __shared__ float s_t[4][16][20];      // T_ii
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, gq = lane >> 4;
  const int ch = blockIdx.x, bh = ch / a.chunks, c = ch - bh * a.chunks;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const DeltaSeq sq = delta_seq(a, b);
  const int t0 = c * kDeltaChunk;
  if (t0 >= sq.n) return;

  // gates: lane = step. log a = min(g, 0) - log(1 + exp(-|g|)), g held to [-87, 87] (NaN passes)
  double cum;
  float be, na;
  {
    const int t = t0 + lane;
    const size_t at = ((size_t)b * a.L + sq.pos(t)) * a.H + h;
    float g = elem<T>(a.g, at);
    const float x = elem<T>(a.beta, at);
    g = __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -87.f), 87.f);
    const float e = expf(-fabsf(g));
    const float la = fminf(g, 0.f) - log1pf(e);
    na = (g > 0.f ? e : 1.f) / (1.f + e);
    be = 1.f / (1.f + expf(-x));
    const bool live = sq.live(t);
    cum = live ? (double)(g == g ? la : g) : 0.0;
    na = live ? na : 0.f;
    be = live ? be : 0.f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double o = __shfl_up(cum, d);
      cum += lane >= d ? o : 0.0;
    }
  }
  if (w == 0) {
    s_cum[lane] = cum;
    s_b[lane] = be;
    DeltaGates& gt = a.gates[ch];
    gt.cum[lane] = cum;
    gt.gam[lane] = expf((float)cum);
    gt.end[lane] = expf((float)(__shfl(cum, 63) - cum));
    gt.b[lane] = be;
    gt.na[lane] = na;
  }

  // K_i K_w^T and Q_i K_w^T for row tiles i >= w
  auto tile_of = [&](const void* src, int i, Frag<PI> (&f)[KS]) {
    const int t = t0 + 16 * i + row;
    const T* p = (const T*)src + (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk;
    const bool live = sq.live(t);
    Quad x[KS][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) x[s][e] = load4<VEC>(p, 32 * s + 16 * e + 4 * gq, a.dk, live);
#pragma unroll
    for (int s = 0; s < KS; ++s) f[s] = join<PI>(to_half(x[s][0]), to_half(x[s][1]));
  };
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  v4f kk[4], qk[4];
  {
    Frag<PI> kw[KS];
    tile_of(a.k, w, kw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kk[i] = qk[i] = zero;
      if (i < w) continue;
      Frag<PI> f[KS];
      if (i == w) {
#pragma unroll
        for (int s = 0; s < KS; ++s) f[s] = kw[s];
      } else {
        tile_of(a.k, i, f);
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) kk[i] = mma<PI, PI>(f[s], kw[s], kk[i]);
      tile_of(a.q, i, f);
#pragma unroll
      for (int s = 0; s < KS; ++s) qk[i] = mma<PI, PI>(f[s], kw[s], qk[i]);
    }
  }
  __syncthreads();

  float* Pm = a.P + (size_t)ch * kDeltaTri;
  float* Tm = a.T + (size_t)ch * kDeltaTri;
  const double cc = s_cum[16 * w + row];
  const float bc = s_b[16 * w + row];
  v4f n, nt;        // N_ww and its transpose
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 4 * gq + r;
      const double d = s_cum[16 * i + m] - cc;
      const float dec = expf((float)(i == w && m < row ? -d : d));   // the transpose's above the diagonal
      Pm[tri(i, w) + m * 16 + row] = i > w || m >= row ? dec * qk[i][r] : 0.f;
      if (i == w) {
        n[r] = m > row ? -(s_b[16 * i + m] * dec * kk[i][r]) : 0.f;
        nt[r] = m < row ? -(bc * dec * kk[i][r]) : 0.f;
      } else {
        s_n[i * (i - 1) / 2 + w][m][row] = -(s_b[16 * i + m] * dec * kk[i][r]);
      }
    }
  }

  v4f t, tt;        // T_ww and its transpose
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float one = 4 * gq + r == row ? 1.f : 0.f;
    t[r] = one + n[r];
    tt[r] = one + nt[r];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {      // T (I + N^2), (I + N^4), (I + N^8)
    const v4f n2 = mm16(nt, n, zero), n2t = mm16(n, nt, zero);
    n = n2;
    nt = n2t;
    const v4f u = mm16(tt, n, t), ut = mm16(n, tt, tt);
    t = u;
    tt = ut;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) s_t[w][4 * gq + r][row] = t[r];
  __syncthreads();

  v4f col[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) col[i] = zero;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) continue;
    if (i == w) {
      col[i] = t;
    } else {
      v4f y = zero;
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k >= w && k < i) y = mm16(*(const v4f*)&s_n[i * (i - 1) / 2 + k][row][4 * gq], col[k], y);
      col[i] = mm16(*(const v4f*)&s_t[i][row][4 * gq], y, zero);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) Tm[tri(i, w) + (4 * gq + r) * 16 + row] = col[i][r] * bc;
  }
}

// ---------------------------------------------------------------------------- the walk
// One workgroup per head and 16 columns of dv; the 4 waves share a chunk's work: wave w has row tile w of
// the 64 steps and OWN of the state's row tiles. Three hand-overs per chunk, each through LDS: the state
// (as B operands of K S and Q S), X = V - diag(y) K S, and U.
template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(256) k_delta_walk(DeltaArgs a) {
  constexpr int PI = DeltaType<T>::PI, PO = DeltaType<T>::PO;
  constexpr int KS = DK / 32, NT = DK / 16, OWN = (NT + 3) / 4, BLK = 64 * DK / 16 / 256;
  constexpr int BLKS = BLK < 1 ? 1 : BLK;
  using Quad = typename DeltaType<T>::Quad;
  constexpr int kTileB = 2 * PI * 1024 + 16;    // of K^T: two frags, staggered over the banks
  __shared__ __attribute__((aligned(16))) unsigned char s_s[KS * 3 * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_x[2 * 3 * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_u[2 * PO * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_e[2 * 3 * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_kt[NT * kTileB];
  const int bh = blockIdx.x;
  if (bh >= a.B * a.H) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, gq = lane >> 4;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const DeltaSeq sq = delta_seq(a, b);
  const int col = blockIdx.y * 16 + row;
  const bool in = col < a.dv;
  const int nch = (sq.n + kDeltaChunk - 1) / kDeltaChunk;
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};

  const size_t sdim = (size_t)a.dk * a.dv;
  v4f S[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    S[i] = zero;
    const int tile = w * OWN + i;
    if (tile < NT && a.s0 && in)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * tile + 4 * gq + r;
        if (k < a.dk) S[i][r] = a.s0[bh * sdim + (size_t)k * a.dv + col];
      }
  }
  auto put_state = [&](float* to) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int tile = w * OWN + i;
      if (tile < NT && in)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 16 * tile + 4 * gq + r;
          if (k < a.dk) to[(size_t)k * a.dv + col] = S[i][r];
        }
    }
  };
  auto share_state = [&] {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int tile = w * OWN + i;
      if (tile < NT)
        lds_half<3>(s_s, tile >> 1, lane, tile & 1, split4<3>(S[i][0], S[i][1], S[i][2], S[i][3]));
    }
  };
  share_state();

  // of a chunk, loaded while the one before is computed
  struct Chunk {
    Quad k[KS][2], q[KS][2], kb[BLKS][4];
    float t[2][8], p[2][8], v[4], gam[4], end[4], last;
  };
  const bool out = a.o != nullptr;
  auto load = [&](int c, Chunk& x) {
    const int ch = bh * a.chunks + c, t0 = c * kDeltaChunk;
    {
      const int t = t0 + 16 * w + row;
      const size_t at = (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk;
      const bool live = sq.live(t);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x.k[s][e] = load4<VEC>((const T*)a.k + at, 32 * s + 16 * e + 4 * gq, a.dk, live);
          if (out) x.q[s][e] = load4<VEC>((const T*)a.q + at, 32 * s + 16 * e + 4 * gq, a.dk, live);
        }
    }
#pragma unroll
    for (int m = 0; m < BLKS; ++m) {
      const int id = threadIdx.x + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (BLK >= 1 || tg < 16)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + 4 * tg + j;
          const size_t at = (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk;
          x.kb[m][j] = load4<VEC>((const T*)a.k + at, 4 * dg, a.dk, sq.live(t));
        }
    }
    const float *Tm = a.T + (size_t)ch * kDeltaTri, *Pm = a.P + (size_t)ch * kDeltaTri;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (2 * s <= w) {
        tri_rows(Tm, w, s, lane, x.t[s]);
        if (out) tri_rows(Pm, w, s, lane, x.p[s]);
      }
    const DeltaGates& gt = a.gates[ch];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * w + 4 * gq + r, t = t0 + m;
      x.gam[r] = gt.gam[m];
      x.end[r] = gt.end[m];
      const float v = elem<T>(a.v, (((size_t)b * a.L + sq.pos(t)) * a.H + h) * a.dv + (in ? col : 0));
      x.v[r] = in && sq.live(t) ? v : 0.f;
    }
    x.last = gt.gam[kDeltaChunk - 1];
  };

  Chunk x, y;
  if (nch > 0) load(0, x);
  __syncthreads();
  for (int c = 0; c < nch; ++c) {
    if (c + 1 < nch) load(c + 1, y);
    if (a.states) put_state(a.states + ((size_t)bh * a.chunks + c) * sdim);
    // K S and Q S; K^T for the update
    v4f ks = zero, qs = zero;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const Frag<3> f = lds_frag<3>(s_s, s, lane);
      ks = mma<PI, 3>(join<PI>(to_half(x.k[s][0]), to_half(x.k[s][1])), f, ks);
      if (out)
        qs = mma<PI, PO>(join<PI>(to_half(x.q[s][0]), to_half(x.q[s][1])), lead<PO>(f), qs);
    }
    lds_half<3>(s_x, w >> 1, lane, w & 1,
                split4<3>(x.v[0] - x.gam[0] * ks[0], x.v[1] - x.gam[1] * ks[1],
                          x.v[2] - x.gam[2] * ks[2], x.v[3] - x.gam[3] * ks[3]));
#pragma unroll
    for (int m = 0; m < BLKS; ++m) {
      const int id = threadIdx.x + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (BLK >= 1 || tg < 16) {
        Half<PI> cl[4];
        transpose4(x.kb[m], cl);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 4 * dg + j;
          lds_half<PI>(s_kt + (k >> 4) * kTileB, tg >> 3, (tg & 3) * 16 + (k & 15), (tg >> 2) & 1,
                       cl[j]);
        }
      }
    }
    __syncthreads();
    v4f u = zero;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (2 * s <= w) u = mma<3, 3>(split8<3>(x.t[s]), lds_frag<3>(s_x, s, lane), u);
    if (out) lds_half<PO>(s_u, w >> 1, lane, w & 1, split4<PO>(u[0], u[1], u[2], u[3]));
    lds_half<3>(s_e, w >> 1, lane, w & 1,
                split4<3>(x.end[0] * u[0], x.end[1] * u[1], x.end[2] * u[2], x.end[3] * u[3]));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int tile = w * OWN + i;
      if (tile < NT) {
        S[i] *= x.last;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          S[i] = mma<PI, 3>(lds_frag<PI>(s_kt + tile * kTileB, s, lane), lds_frag<3>(s_e, s, lane),
                            S[i]);
      }
    }
    share_state();
    if (out) {
      v4f pu = zero;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (2 * s <= w) pu = mma<PO, PO>(split8<PO>(x.p[s]), lds_frag<PO>(s_u, s, lane), pu);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = c * kDeltaChunk + 16 * w + 4 * gq + r;
        if (in && sq.live(t))
          put1((T*)a.o + (((size_t)b * a.L + sq.pos(t)) * a.H + h) * a.dv + col,
               a.scale * fmaf(x.gam[r], qs[r], pu[r]));
      }
    }
    x = y;
    __syncthreads();
  }
  if (a.s_last) put_state(a.s_last + bh * sdim);
  if (a.states)
    for (int c = nch; c < a.chunks; ++c) put_state(a.states + ((size_t)bh * a.chunks + c) * sdim);
  if (out && in)
    for (int t = sq.n + (threadIdx.x >> 4); t < a.L; t += 16)
      put1((T*)a.o + (((size_t)b * a.L + t) * a.H + h) * a.dv + col, 0.f);
}

// ---------------------------------------------------------------------------- single steps
// A wave per head and 16 columns: lane 4 i + c has rows i, i + 16, ... of four of them in registers.
template <typename T, int RW>
__global__ void __launch_bounds__(64) k_delta_step(DeltaArgs a) {
  const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const int lane = threadIdx.x, i0 = lane >> 2, col = blockIdx.y * 16 + 4 * (lane & 3);
  const DeltaSeq sq = delta_seq(a, b);
  const size_t sdim = (size_t)a.dk * a.dv;
  float S[RW][4];
  auto get = [&](const float* from) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int k = i0 + 16 * i;
      const size_t at = bh * sdim + (size_t)(k < a.dk ? k : 0) * a.dv;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = from[at + (col + j < a.dv ? col + j : 0)];
        S[i][j] = k < a.dk && col + j < a.dv ? s : 0.f;
      }
    }
  };
  auto put = [&](float* to) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int k = i0 + 16 * i;
      if (k < a.dk)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < a.dv) to[(size_t)k * a.dv + col + j] = S[i][j];
    }
  };
  if (a.s0) {
    get(a.s0);
  } else {
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = 0.f;
  }
  if (a.states) put(a.states + (size_t)bh * a.chunks * sdim);
  for (int t = 0; t < sq.n; ++t) {
    const size_t pos = (size_t)b * a.L + sq.pos(t), kat = (pos * a.Hk + hk) * a.dk;
    const size_t vat = (pos * a.H + h) * a.dv, gat = pos * a.H + h;
    float q[RW], k[RW], v[4];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = i0 + 16 * i;
      k[i] = elem<T>(a.k, kat + (r < a.dk ? r : 0));
      q[i] = elem<T>(a.q, kat + (r < a.dk ? r : 0));
      k[i] = r < a.dk ? k[i] : 0.f;
      q[i] = r < a.dk ? q[i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = elem<T>(a.v, vat + (col + j < a.dv ? col + j : 0));
    float g = elem<T>(a.g, gat);
    g = __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -87.f), 87.f);
    const float be = 1.f / (1.f + expf(-elem<T>(a.beta, gat)));
    const float al = 1.f / (1.f + expf(-g));
    float x[4], o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = 0.f;
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        S[i][j] *= al;
        x[j] = fmaf(k[i], S[i][j], x[j]);
      }
    }
#pragma unroll
    for (int d = 4; d < 64; d *= 2)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = be * (v[j] - x[j]);
      o[j] = 0.f;
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        S[i][j] = fmaf(k[i], u, S[i][j]);
        o[j] = fmaf(q[i], S[i][j], o[j]);
      }
    }
#pragma unroll
    for (int d = 4; d < 64; d *= 2)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], d);
    if (i0 == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < a.dv) put1((T*)a.o + vat + col + j, a.scale * o[j]);
  }
  if (a.s_last) put(a.s_last + bh * sdim);
  for (int t = sq.n + i0; t < a.L; t += 16)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < a.dv) put1((T*)a.o + (((size_t)b * a.L + t) * a.H + h) * a.dv + col + j, 0.f);
}

constexpr int kDeltaSteps = 8;     // longest sequences that go step by step

int64_t chunks_of(int64_t L) { return (L + kDeltaChunk - 1) / kDeltaChunk; }

template <typename T, typename F>
void with_dk(int dk, bool vec, F f) {
  auto go = [&](auto d) {
    if (vec) f(d, std::true_type());
    else f(d, std::false_type());
  };
  if (dk <= 32) go(std::integral_constant<int, 32>());
  else if (dk <= 64) go(std::integral_constant<int, 64>());
  else go(std::integral_constant<int, 128>());
}

template <typename T>
void prep_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  with_dk<T>(a.dk, vec, [&](auto d, auto v) {
    k_delta_prep<T, decltype(d)::value, decltype(v)::value>
        <<<dim3(a.B * a.H * a.chunks), 256, 0, st>>>(a);
  });
}
template <typename T>
void walk_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  // heads side by side in steps of 8: a head's columns then lie on one XCD and share its L2
  const dim3 grid((a.B * a.H + 7) / 8 * 8, (a.dv + 15) / 16);
  with_dk<T>(a.dk, vec, [&](auto d, auto v) {
    k_delta_walk<T, decltype(d)::value, decltype(v)::value><<<grid, 256, 0, st>>>(a);
  });
}
template <typename T>
void step_t(const DeltaArgs& a, hipStream_t st) {
  const dim3 grid(a.B * a.H, (a.dv + 15) / 16);
  if (a.dk <= 32) k_delta_step<T, 2><<<grid, 64, 0, st>>>(a);
  else if (a.dk <= 64) k_delta_step<T, 4><<<grid, 64, 0, st>>>(a);
  else k_delta_step<T, 8><<<grid, 64, 0, st>>>(a);
}

}  // namespace

DeltaArgs delta_args(const DeltaRequest& r) {
  DeltaArgs a{};
  a.q = r.q; a.k = r.k; a.v = r.v; a.g = r.g; a.beta = r.beta; a.dout = r.dout;
  a.s0 = r.s0; a.ds_last = r.ds_last; a.lens = r.lens; a.o = r.o; a.s_last = r.s_last;
  a.states = r.states; a.dq = r.dq; a.dkey = r.dkey; a.dval = r.dval; a.dg = r.dg;
  a.dbeta = r.dbeta; a.ds0 = r.ds0;
  a.B = (int)r.B; a.L = (int)r.L; a.Hk = r.Hk; a.H = r.H; a.dk = r.dk; a.dv = r.dv;
  a.rep = r.H / r.Hk; a.chunks = (int)chunks_of(r.L); a.reverse = r.reverse; a.scale = r.scale;
  const size_t n = (size_t)r.B * r.H * a.chunks;
  unsigned char* ws = (unsigned char*)r.ws;
  a.T = (float*)ws;
  a.P = a.T + n * kDeltaTri;
  a.gates = (DeltaGates*)(a.P + n * kDeltaTri);
  return a;
}

bool delta_vec(const DeltaRequest& r) {
  const uintptr_t m = r.bf16 ? 7 : 15;
  auto al = [](const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) == 0; };
  return r.dk % 4 == 0 && r.dv % 4 == 0 && al(r.q, m) && al(r.k, m) && al(r.v, m) &&
         al(r.dout, m) && al(r.states, 15);
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool bf16, bool vec, hipStream_t st) {
  if (bf16) prep_t<uint16_t>(a, vec, st);
  else prep_t<float>(a, vec, st);
  return hipGetLastError();
}
hipError_t launch_delta_walk(const DeltaArgs& a, bool bf16, bool vec, hipStream_t st) {
  if (bf16) walk_t<uint16_t>(a, vec, st);
  else walk_t<float>(a, vec, st);
  return hipGetLastError();
}

size_t delta_forward_workspace(int64_t B, int64_t L, int H, int dk, int dv) {
  if (L <= kDeltaSteps) return 0;
  return (size_t)B * H * chunks_of(L) * (2 * kDeltaTri * 4 + sizeof(DeltaGates));
}

hipError_t launch_delta_forward(const DeltaRequest& r, hipStream_t st) {
  const DeltaArgs a = delta_args(r);
  if (r.L <= kDeltaSteps) {
    if (r.bf16) step_t<uint16_t>(a, st);
    else step_t<float>(a, st);
    return hipGetLastError();
  }
  const bool vec = delta_vec(r);
  const hipError_t e = launch_delta_prep(a, r.bf16, vec, st);
  return e != hipSuccess ? e : launch_delta_walk(a, r.bf16, vec, st);
}

}  // namespace wbmm
