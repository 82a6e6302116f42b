// Gated delta rule, backward: the walk along the chunks from the last to the first
// (k_delta_walk_bwd), and what each chunk computes on its own then (k_delta_grads).
#include "wbmm_deltadev.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

template <typename T>
__device__ __forceinline__ float elem(const void* p, size_t i) { return load_f32<T>((const T*)p, i); }

// ---------------------------------------------------------------------------- the walk back
// As the forward's walk: one workgroup per head and 16 columns of dv, wave w with row tile w of the 64
// steps and OWN row tiles of D. Hand-overs per chunk: D, then dU (with diag(y) G beside it), then
// diag(y) R. D after each chunk and R stay in the workspace for k_delta_grads.
template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(256) k_delta_walk_bwd(DeltaArgs a) {
  constexpr int PI = DeltaType<T>::PI;
  constexpr int KS = DK / 32, NT = DK / 16, OWN = (NT + 3) / 4, BLK = 64 * DK / 16 / 256;
  constexpr int BLKS = BLK < 1 ? 1 : BLK;
  using Quad = typename DeltaType<T>::Quad;
  constexpr int kTileB = 2 * PI * 1024 + 16;
  __shared__ __attribute__((aligned(16))) unsigned char s_d[KS * 3 * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_x[2 * 3 * 1024];   // dU
  __shared__ __attribute__((aligned(16))) unsigned char s_g[2 * 3 * 1024];   // diag(y) G
  __shared__ __attribute__((aligned(16))) unsigned char s_r[2 * 3 * 1024];   // -diag(y) R
  __shared__ __attribute__((aligned(16))) unsigned char s_kt[NT * kTileB];
  __shared__ __attribute__((aligned(16))) unsigned char s_qt[NT * kTileB];
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
  v4f D[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    D[i] = zero;
    const int tile = w * OWN + i;
    if (tile < NT && a.ds_last && in)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * tile + 4 * gq + r;
        if (k < a.dk) D[i][r] = a.ds_last[bh * sdim + (size_t)k * a.dv + col];
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
          if (k < a.dk) to[(size_t)k * a.dv + col] = D[i][r];
        }
    }
  };
  auto share_state = [&] {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int tile = w * OWN + i;
      if (tile < NT)
        lds_half<3>(s_d, tile >> 1, lane, tile & 1, split4<3>(D[i][0], D[i][1], D[i][2], D[i][3]));
    }
  };
  share_state();

  struct Chunk {
    Quad k[KS][2], kb[BLKS][4], qb[BLKS][4];
    float t[2][8], p[2][8], g[2][8], gam[4], end[4], last;
  };
  auto load = [&](int c, Chunk& x) {
    const int ch = bh * a.chunks + c, t0 = c * kDeltaChunk;
    {
      const int t = t0 + 16 * w + row;
      const size_t at = (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk;
      const bool live = sq.live(t);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x.k[s][e] = load4<VEC>((const T*)a.k + at, 32 * s + 16 * e + 4 * gq, a.dk, live);
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
          x.qb[m][j] = load4<VEC>((const T*)a.q + at, 4 * dg, a.dk, sq.live(t));
        }
    }
    const float *Tm = a.T + (size_t)ch * kDeltaTri, *Pm = a.P + (size_t)ch * kDeltaTri;
    const DeltaGates& gt = a.gates[ch];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (2 * s + 1 >= w) {
        tri_cols(Tm, w, s, lane, x.t[s]);
        tri_cols(Pm, w, s, lane, x.p[s]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = t0 + 32 * s + (j < 4 ? 0 : 16) + 4 * gq + (j & 3);
          const float v =
              elem<T>(a.dout, (((size_t)b * a.L + sq.pos(t)) * a.H + h) * a.dv + (in ? col : 0));
          x.g[s][j] = in && sq.live(t) ? v : 0.f;
        }
      }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * w + 4 * gq + r;
      x.gam[r] = gt.gam[m];
      x.end[r] = gt.end[m];
    }
    x.last = gt.gam[kDeltaChunk - 1];
  };

  Chunk x, y;
  if (nch > 0) load(nch - 1, x);
  __syncthreads();
  for (int c = nch - 1; c >= 0; --c) {
    const int ch = bh * a.chunks + c;
    if (c > 0) load(c - 1, y);
    put_state(a.D + (size_t)ch * sdim);
    v4f kd = zero, pg = zero;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      kd = mma<PI, 3>(join<PI>(to_half(x.k[s][0]), to_half(x.k[s][1])), lds_frag<3>(s_d, s, lane), kd);
    v4f gy = zero;      // diag(y) G of this wave's rows
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s + 1 >= w) pg = mma<3, PI>(split8<3>(x.p[s]), split8<PI>(x.g[s]), pg);
      if (s == w >> 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          gy[r] = a.scale * x.gam[r] * ((w & 1) ? x.g[s][4 + r] : x.g[s][r]);
      }
    }
    lds_half<3>(s_x, w >> 1, lane, w & 1,
                split4<3>(fmaf(a.scale, pg[0], x.end[0] * kd[0]), fmaf(a.scale, pg[1], x.end[1] * kd[1]),
                          fmaf(a.scale, pg[2], x.end[2] * kd[2]), fmaf(a.scale, pg[3], x.end[3] * kd[3])));
    lds_half<3>(s_g, w >> 1, lane, w & 1, split4<3>(gy[0], gy[1], gy[2], gy[3]));
#pragma unroll
    for (int m = 0; m < BLKS; ++m) {
      const int id = threadIdx.x + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (BLK >= 1 || tg < 16) {
        Half<PI> ck[4], cq[4];
        transpose4(x.kb[m], ck);
        transpose4(x.qb[m], cq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 4 * dg + j, at = (k >> 4) * kTileB, ln = (tg & 3) * 16 + (k & 15);
          lds_half<PI>(s_kt + at, tg >> 3, ln, (tg >> 2) & 1, ck[j]);
          lds_half<PI>(s_qt + at, tg >> 3, ln, (tg >> 2) & 1, cq[j]);
        }
      }
    }
    __syncthreads();
    v4f rr = zero;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (2 * s + 1 >= w) rr = mma<3, 3>(split8<3>(x.t[s]), lds_frag<3>(s_x, s, lane), rr);
    lds_half<3>(s_r, w >> 1, lane, w & 1,
                split4<3>(-x.gam[0] * rr[0], -x.gam[1] * rr[1], -x.gam[2] * rr[2], -x.gam[3] * rr[3]));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * w + 4 * gq + r, t = c * kDeltaChunk + m;
      if (in) {
        a.R[((size_t)ch * kDeltaChunk + m) * a.dv + col] = rr[r];
        if (sq.live(t))
          put1((T*)a.dval + (((size_t)b * a.L + sq.pos(t)) * a.H + h) * a.dv + col, rr[r]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int tile = w * OWN + i;
      if (tile < NT) {
        D[i] *= x.last;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          D[i] = mma<PI, 3>(lds_frag<PI>(s_qt + tile * kTileB, s, lane), lds_frag<3>(s_g, s, lane),
                            D[i]);
          D[i] = mma<PI, 3>(lds_frag<PI>(s_kt + tile * kTileB, s, lane), lds_frag<3>(s_r, s, lane),
                            D[i]);
        }
      }
    }
    share_state();
    x = y;
    __syncthreads();
  }
  if (a.ds0) put_state(a.ds0 + bh * sdim);
  if (in)
    for (int t = sq.n + (threadIdx.x >> 4); t < a.L; t += 16)
      put1((T*)a.dval + (((size_t)b * a.L + t) * a.H + h) * a.dv + col, 0.f);
}

// ---------------------------------------------------------------------------- chunks on their own
// One workgroup of 8 waves per chunk of a key head, its heads one after the other. Wave (w, hf) has row
// tile w of the 64 steps, and of everything along dk the half hf; the (64 x 64) dP is hf = 0's and N hf =
// 1's. dv is walked in pieces of 32 columns, whose S0 and D are staged in LDS as operands.
template <typename T, int DK, bool VEC>
struct GradLds {
  static constexpr int PI = DeltaType<T>::PI, PO = DeltaType<T>::PO, NT = DK / 16, KS = DK / 32;
  static constexpr int sn = 0;                            // S0, terms along dv: NT frags
  static constexpr int sk = sn + NT * PO * 1024;          // S0, terms along dk: KS x 2
  static constexpr int dn = sk + KS * 2 * PO * 1024;      // D, terms along dv: NT
  static constexpr int xf = dn + NT * PO * 1024;          // X: 2 x 2
  static constexpr int uf = xf + 4 * PO * 1024;           // U as rows: 4
  static constexpr int walk = uf + 4 * PO * 1024;
  static constexpr int kt = 0;                            // afterwards: K^T and Q^T, NT x 2 each
  static constexpr int kTileB = 2 * PI * 1024 + 16;
  static constexpr int qt = kt + NT * kTileB;
  static constexpr int after = qt + NT * kTileB;
  static constexpr int mat = walk > after ? walk : after; // dP and N: 64 rows of 68 floats each
  static constexpr int red = mat + 2 * 64 * 68 * 4;       // row sums
  static constexpr int bytes = red + (2 * 4 + 2) * 64 * 4;
};

// Sum over the 16 lanes of a row of lanes, in each of them.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) v += __shfl_xor(v, d);
  return v;
}

template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(512) k_delta_grads(DeltaArgs a) {
  using Lds = GradLds<T, DK, VEC>;
  constexpr int PI = Lds::PI, PO = Lds::PO, KS = Lds::KS, NT = Lds::NT, NTH = NT / 2;
  using Quad = typename DeltaType<T>::Quad;
  extern __shared__ __attribute__((aligned(16))) unsigned char sm[];
  float* mat = (float*)(sm + Lds::mat);
  float* red = (float*)(sm + Lds::red);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), w = wid & 3, hf = wid >> 2;
  const int row = lane & 15, gq = lane >> 4;
  const int c = blockIdx.x % a.chunks, bk = blockIdx.x / a.chunks;
  const int b = bk / a.Hk, hk = bk - b * a.Hk;
  const DeltaSeq sq = delta_seq(a, b);
  const int t0 = c * kDeltaChunk;
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  const size_t sdim = (size_t)a.dk * a.dv;
  // positions of rows: this lane's as an operand's row, and its four as a result's
  const int tr = t0 + 16 * w + row;
  const bool live_r = sq.live(tr);
  const size_t pos_r = (size_t)b * a.L + sq.pos(tr);

  if (t0 >= sq.n) {   // past the end: zeros at the chunk's own positions
    for (int i = tid; i < kDeltaChunk; i += 512) {
      const int t = t0 + i;
      if (t >= a.L) break;
      const size_t p = (size_t)b * a.L + t;
      for (int k = 0; k < a.dk; ++k) {
        put1((T*)a.dq + (p * a.Hk + hk) * a.dk + k, 0.f);
        put1((T*)a.dkey + (p * a.Hk + hk) * a.dk + k, 0.f);
      }
      for (int j = 0; j < a.rep; ++j) {
        put1((T*)a.dg + p * a.H + hk * a.rep + j, 0.f);
        put1((T*)a.dbeta + p * a.H + hk * a.rep + j, 0.f);
      }
    }
    return;
  }

  Frag<PI> kf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const T* p = (const T*)a.k + (pos_r * a.Hk + hk) * a.dk;
    kf[s] = join<PI>(to_half(load4<VEC>(p, 32 * s + 4 * gq, a.dk, live_r)),
                     to_half(load4<VEC>(p, 32 * s + 16 + 4 * gq, a.dk, live_r)));
  }
  v4f dqs[NTH], dks[NTH];
#pragma unroll
  for (int i = 0; i < NTH; ++i) dqs[i] = dks[i] = zero;

  for (int j = 0; j < a.rep; ++j) {
    const int h = hk * a.rep + j, ch = (b * a.H + h) * a.chunks + c;
    const DeltaGates& gt = a.gates[ch];
    const float* S0 = a.states + (size_t)ch * sdim;
    const float* D1 = a.D + (size_t)ch * sdim;
    const float* R = a.R + (size_t)ch * kDeltaChunk * a.dv;
    const float* Tm = a.T + (size_t)ch * kDeltaTri;
    float gam[4], end[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gam[r] = gt.gam[16 * w + 4 * gq + r];
      end[r] = gt.end[16 * w + 4 * gq + r];
    }
    v4f dq[NTH], rowg[NTH], colg[NTH], pn[4];
#pragma unroll
    for (int i = 0; i < NTH; ++i) dq[i] = rowg[i] = colg[i] = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) pn[i] = zero;
    float rv = 0.f, sd = 0.f;     // v.R of row tr; <S0, D>

    for (int n0 = 0; n0 < a.dv; n0 += 32) {
      __syncthreads();            // the last piece's (or head's) operands have been read
      {
        // 4 x 4 blocks of S0 (threads below 256) and of D (the others)
        const bool second = tid >= 256;
        for (int id = tid & 255; id < DK * 2; id += 256) {
          const int n4 = id & 7, k4 = id >> 3, n = n0 + 4 * n4;
          v4f m[4], s[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int k = 4 * k4 + r;
            const size_t at = (size_t)(k < a.dk ? k : 0) * a.dv;
            s[r] = load4<VEC>(S0 + at, n, a.dv, k < a.dk);
            m[r] = second ? load4<VEC>(D1 + at, n, a.dv, k < a.dk) : s[r];
          }
          unsigned char* to = sm + (second ? Lds::dn : Lds::sn);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            lds_half<PO>(to, k4 >> 2, (n4 & 3) * 16 + 4 * (k4 & 3) + r, n4 >> 2,
                         split4<PO>(m[r][0], m[r][1], m[r][2], m[r][3]));
            if (second)
              sd += s[r][0] * m[r][0] + s[r][1] * m[r][1] + s[r][2] * m[r][2] + s[r][3] * m[r][3];
            else
              lds_half<PO>(sm + Lds::sk, (k4 >> 3) * 2 + (n4 >> 2),
                           (k4 & 3) * 16 + 4 * (n4 & 3) + r, (k4 >> 2) & 1,
                           split4<PO>(m[0][r], m[1][r], m[2][r], m[3][r]));
          }
        }
      }
      // rows of do and R (operands), v as a result lies
      const int n = n0 + 16 * hf + row;
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + 16 * w + 4 * gq + r;
        const float e = elem<T>(a.v, (((size_t)b * a.L + sq.pos(t)) * a.H + h) * a.dv +
                                         (n < a.dv ? n : 0));
        v[r] = n < a.dv && sq.live(t) ? e : 0.f;
      }
      const size_t vrow = (pos_r * a.H + h) * a.dv;
      const Quad g0 = load4<VEC>((const T*)a.dout + vrow, n0 + 4 * gq, a.dv, live_r);
      const Quad g1 = load4<VEC>((const T*)a.dout + vrow, n0 + 16 + 4 * gq, a.dv, live_r);
      const float* rp = R + (size_t)(16 * w + row) * a.dv;
      const v4f r0 = load4<VEC>(rp, n0 + 4 * gq, a.dv, live_r);
      const v4f r1 = load4<VEC>(rp, n0 + 16 + 4 * gq, a.dv, live_r);
      const Frag<PI> gf = join<PI>(to_half(g0), to_half(g1));
      const Frag<PO> rf = join<PO>(split4<PO>(r0[0], r0[1], r0[2], r0[3]),
                                   split4<PO>(r1[0], r1[1], r1[2], r1[3]));
      if (hf == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int na = n0 + 4 * gq + i, nb = na + 16;
          const float va = elem<T>(a.v, vrow + (na < a.dv ? na : 0));
          const float vb = elem<T>(a.v, vrow + (nb < a.dv ? nb : 0));
          rv += na < a.dv && live_r ? r0[i] * va : 0.f;
          rv += nb < a.dv && live_r ? r1[i] * vb : 0.f;
        }
      }
      __syncthreads();
      // X = V - diag(y) K S0, this wave's 16 rows and 16 columns
      v4f ks = zero;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        ks = mma<PI, PO>(kf[s], lds_frag<PO>(sm + Lds::sk, 2 * s + hf, lane), ks);
      lds_half<PO>(sm + Lds::xf, (w >> 1) * 2 + hf, lane, w & 1,
                   split4<PO>(v[0] - gam[0] * ks[0], v[1] - gam[1] * ks[1], v[2] - gam[2] * ks[2],
                              v[3] - gam[3] * ks[3]));
      __syncthreads();
      v4f u = zero;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (2 * s <= w) {
          float t[8];
          tri_rows(Tm, w, s, lane, t);
          u = mma<PO, PO>(split8<PO>(t), lds_frag<PO>(sm + Lds::xf, 2 * s + hf, lane), u);
        }
      {   // U as rows: entry (16 w + 4 gq + r, 16 hf + row) of the piece
        uint32_t lo[PO], hi[PO];
        split2<PO>(u[0], u[1], lo);
        split2<PO>(u[2], u[3], hi);
#pragma unroll
        for (int p = 0; p < PO; ++p) {
          unsigned char* to = sm + Lds::uf + (w * PO + p) * 1024 + ((row >> 2) * 16 + 4 * gq) * 16 +
                              hf * 8 + (row & 3) * 2;
          *(uint16_t*)(to) = (uint16_t)lo[p];
          *(uint16_t*)(to + 16) = (uint16_t)(lo[p] >> 16);
          *(uint16_t*)(to + 32) = (uint16_t)hi[p];
          *(uint16_t*)(to + 48) = (uint16_t)(hi[p] >> 16);
        }
      }
      __syncthreads();
      const Frag<PO> uw = lds_frag<PO>(sm + Lds::uf, w, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= w) {
          const Frag<PO> ui = lds_frag<PO>(sm + Lds::uf, i, lane);
          if (hf == 0) pn[i] = mma<PI, PO>(gf, ui, pn[i]);
          else pn[i] = mma<PO, PO>(rf, ui, pn[i]);
        }
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        const Frag<PO> sf = lds_frag<PO>(sm + Lds::sn, hf * NTH + i, lane);
        dq[i] = mma<PI, PO>(gf, sf, dq[i]);
        rowg[i] = mma<PO, PO>(rf, sf, rowg[i]);
        colg[i] = mma<PO, PO>(uw, lds_frag<PO>(sm + Lds::dn, hf * NTH + i, lane), colg[i]);
      }
    }

    // dP and N to LDS, with their decays
    float cend = 0.f;             // sum over this lane's entries of k.(U D^T y_C / y): the rest of <S_C, D>
    float kd[NTH][4], qd[NTH][4];
    {
      const float one = hf == 0 ? a.scale : -1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= w) {
          const double cc = gt.cum[16 * i + row];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int m = 16 * w + 4 * gq + r, nn = 16 * i + row;
            const float dec = expf((float)(gt.cum[m] - cc));
            mat[hf * 64 * 68 + m * 68 + nn] = (hf == 0 ? nn <= m : nn < m) ? one * dec * pn[i][r] : 0.f;
          }
        }
    }
    __syncthreads();              // also: the pieces' operands have been read
    {
      const bool second = tid >= 256;
      for (int id = tid & 255; id < DK * 4; id += 256) {
        const int dg = id % (DK / 4), tg = id / (DK / 4);
        Quad m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = t0 + 4 * tg + r;
          const size_t at = (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk;
          m[r] = load4<VEC>((const T*)(second ? a.q : a.k) + at, 4 * dg, a.dk, sq.live(t));
        }
        Half<PI> cl[4];
        transpose4(m, cl);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 4 * dg + r;
          lds_half<PI>(sm + (second ? Lds::qt : Lds::kt) + (k >> 4) * Lds::kTileB, tg >> 3,
                       (tg & 3) * 16 + (k & 15), (tg >> 2) & 1, cl[r]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NTH; ++i) {
      const int k = 16 * (hf * NTH + i) + row;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + 16 * w + 4 * gq + r;
        const size_t at = (((size_t)b * a.L + sq.pos(t)) * a.Hk + hk) * a.dk + (k < a.dk ? k : 0);
        const float e = elem<T>(a.k, at), f = elem<T>(a.q, at);
        const bool ok = k < a.dk && sq.live(t);
        kd[i][r] = ok ? e : 0.f;
        qd[i][r] = ok ? f : 0.f;
        dq[i][r] *= a.scale * gam[r];
        rowg[i][r] *= -gam[r];
        colg[i][r] *= end[r];
        cend += kd[i][r] * colg[i][r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s <= w) {
        float p[8], q[8];
        const float* m = mat + (16 * w + row) * 68 + 32 * s + 4 * gq;
        const v4f a0 = *(const v4f*)m, b0 = *(const v4f*)(m + 64 * 68);
        v4f a1 = zero, b1 = zero;
        if (2 * s + 1 <= w) a1 = *(const v4f*)(m + 16), b1 = *(const v4f*)(m + 64 * 68 + 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = a0[e], p[4 + e] = a1[e], q[e] = b0[e], q[4 + e] = b1[e];
        const Frag<PO> pf = split8<PO>(p), nf = split8<PO>(q);
#pragma unroll
        for (int i = 0; i < NTH; ++i) {
          const Frag<PI> kt = lds_frag<PI>(sm + Lds::kt + (hf * NTH + i) * Lds::kTileB, s, lane);
          dq[i] = mma<PO, PI>(pf, kt, dq[i]);
          rowg[i] = mma<PO, PI>(nf, kt, rowg[i]);
        }
      }
      if (2 * s + 1 >= w) {
        float p[8], q[8];
        const float* m = mat + (32 * s + 4 * gq) * 68 + 16 * w + row;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = 2 * s >= w ? m[e * 68] : 0.f;
          q[e] = 2 * s >= w ? m[(64 + e) * 68] : 0.f;
          p[4 + e] = m[(16 + e) * 68];
          q[4 + e] = m[(80 + e) * 68];
        }
        const Frag<PO> pf = split8<PO>(p), nf = split8<PO>(q);
#pragma unroll
        for (int i = 0; i < NTH; ++i) {
          const int at = (hf * NTH + i) * Lds::kTileB;
          colg[i] = mma<PO, PI>(pf, lds_frag<PI>(sm + Lds::qt + at, s, lane), colg[i]);
          colg[i] = mma<PO, PI>(nf, lds_frag<PI>(sm + Lds::kt + at, s, lane), colg[i]);
        }
      }
    }
    // row sums: q.dq - k.col, k.row, and over all rows <S_C, D>
    float z0[4], z1[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      z0[r] = z1[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        z0[r] += qd[i][r] * dq[i][r] - kd[i][r] * colg[i][r];
        z1[r] += kd[i][r] * rowg[i][r];
      }
      z0[r] = sum16(z0[r]);
      z1[r] = sum16(z1[r]);
    }
    rv += __shfl_xor(rv, 16);
    rv += __shfl_xor(rv, 32);
    float tot = fmaf(gt.gam[kDeltaChunk - 1], sd, cend);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) tot += __shfl_xor(tot, d);
    if (row == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        red[hf * 64 + 16 * w + 4 * gq + r] = z0[r];
        red[(2 + hf) * 64 + 16 * w + 4 * gq + r] = z1[r];
      }
    if (hf == 0 && gq == 0) red[4 * 64 + 16 * w + row] = rv;
    if (lane == 0) red[5 * 64 + wid] = tot;
#pragma unroll
    for (int i = 0; i < NTH; ++i) {
      dqs[i] += dq[i];
      dks[i] += rowg[i] + colg[i];
    }
    __syncthreads();
    if (wid == 0) {
      const float rowk = red[2 * 64 + lane] + red[3 * 64 + lane];
      double d = (double)(red[lane] + red[64 + lane]) + (double)rowk;
      if (lane == 63)
        for (int i = 0; i < 8; ++i) d += (double)red[5 * 64 + i];
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const double o = __shfl_down(d, s);
        d += lane + s < 64 ? o : 0.0;
      }
      const int t = t0 + lane;
      const float dg = (float)d * gt.na[lane];
      const float db = (red[4 * 64 + lane] + rowk) * (1.f - gt.b[lane]);
      if (t < a.L) {
        const bool live = sq.live(t);
        const size_t at = ((size_t)b * a.L + (live ? sq.pos(t) : t)) * a.H + h;
        put1((T*)a.dg + at, live ? dg : 0.f);
        put1((T*)a.dbeta + at, live ? db : 0.f);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NTH; ++i) {
    const int k = 16 * (hf * NTH + i) + row;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 16 * w + 4 * gq + r;
      if (k < a.dk && t < a.L) {
        const bool live = sq.live(t);
        const size_t at = (((size_t)b * a.L + (live ? sq.pos(t) : t)) * a.Hk + hk) * a.dk + k;
        put1((T*)a.dq + at, live ? dqs[i][r] : 0.f);
        put1((T*)a.dkey + at, live ? dks[i][r] : 0.f);
      }
    }
  }
}

template <typename F>
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
hipError_t backward_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  const dim3 grid((a.B * a.H + 7) / 8 * 8, (a.dv + 15) / 16);
  hipError_t e = hipSuccess;
  with_dk(a.dk, vec, [&](auto d, auto v) {
    constexpr int DK = decltype(d)::value;
    constexpr bool VEC = decltype(v)::value;
    k_delta_walk_bwd<T, DK, VEC><<<grid, 256, 0, st>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return;
    constexpr int bytes = GradLds<T, DK, VEC>::bytes;
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    e = hipFuncSetAttribute((const void*)k_delta_grads<T, DK, VEC>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return;
    k_delta_grads<T, DK, VEC><<<dim3(a.B * a.Hk * a.chunks), 512, bytes, st>>>(a);
    e = hipGetLastError();
  });
  return e;
}

struct BwdWs {
  size_t D, R, states, total;
};
BwdWs bwd_ws(int64_t B, int64_t L, int H, int dk, int dv, bool has_states) {
  const size_t n = (size_t)B * H * ((L + kDeltaChunk - 1) / kDeltaChunk);
  auto al = [](size_t v) { return (v + 255) / 256 * 256; };
  BwdWs w{};
  size_t o = al(n * (2 * kDeltaTri * 4 + sizeof(DeltaGates)));
  w.D = o;
  o += al(n * dk * dv * 4);
  w.R = o;
  o += al(n * kDeltaChunk * dv * 4);
  w.states = o;
  if (!has_states) o += al(n * dk * dv * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t delta_backward_workspace(int64_t B, int64_t L, int H, int dk, int dv, bool has_states) {
  return bwd_ws(B, L, H, dk, dv, has_states).total;
}

hipError_t launch_delta_backward(const DeltaRequest& r, hipStream_t st) {
  DeltaArgs a = delta_args(r);
  const BwdWs w = bwd_ws(r.B, r.L, r.H, r.dk, r.dv, r.states != nullptr);
  unsigned char* ws = (unsigned char*)r.ws;
  a.D = (float*)(ws + w.D);
  a.R = (float*)(ws + w.R);
  const bool vec = delta_vec(r);
  hipError_t e = launch_delta_prep(a, r.bf16, vec, st);
  if (e == hipSuccess && !a.states) {
    a.states = (float*)(ws + w.states);
    e = launch_delta_walk(a, r.bf16, vec, st);   // states only: a.o is null
  }
  if (e != hipSuccess) return e;
  return r.bf16 ? backward_t<uint16_t>(a, vec, st) : backward_t<float>(a, vec, st);
}

}  // namespace wbmm
