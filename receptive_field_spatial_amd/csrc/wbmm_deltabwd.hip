// Gated delta rule, backward: the walk along the chunks from the last to the first
// (k_delta_walk_bwd), and what each chunk computes on its own then (k_delta_grads).
#include "wbmm_deltadev.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

// ---------------------------------------------------------------------------- the walk back
// As the forward's walk: one workgroup per head and 16 columns of dv, wave w with row tile w of the 64
// steps and OWN row tiles of D. Hand-overs per chunk: D, then dU (with diag(y) G beside it), then
// diag(y) R. D after each chunk and R stay in the workspace for k_delta_grads.
template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(256) k_delta_walk_bwd(DeltaArgs a) {
  using Ty = DeltaType<T, VEC>;
  constexpr int PI = Ty::PI;
  constexpr int KS = DK / 32, NT = DK / 16, OWN = (NT + 3) / 4, BLK = 64 * DK / 16 / 256;
  constexpr int BLKS = BLK < 1 ? 1 : BLK;
  constexpr int kTileB = 2 * PI * 1024 + 16;
  __shared__ __attribute__((aligned(16))) unsigned char s_d[KS * 3 * 1024];
  __shared__ __attribute__((aligned(16))) unsigned char s_o[2 * PI * 1024];  // do
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
  const uint32_t kstride = (uint32_t)(a.Hk * a.dk) * sizeof(T), vstride = (uint32_t)(a.H * a.dv) * sizeof(T);

  const size_t sdim = (size_t)a.dk * a.dv;
  v4f D[OWN];
  uint32_t soff[OWN][4], roff[4];
#pragma unroll
  for (int i = 0; i < OWN; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int k = 16 * (w * OWN + i) + 4 * gq + r;
      const bool own = w * OWN + i < NT && k < a.dk && in;
      soff[i][r] = own ? (uint32_t)(k * a.dv + col) * 4 : kNowhere;
      D[i][r] = a.ds_last ? buf_load<float>(delta_buf(a.ds_last + bh * sdim), soff[i][r]) : 0.f;
    }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    roff[r] = in ? (uint32_t)((16 * w + 4 * gq + r) * a.dv + col) * 4 : kNowhere;
  auto put_state = [&](float* to) {
    const auto buf = delta_buf(to);
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) buf_store(buf, soff[i][r], D[i][r], 0.f);
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
    typename Ty::Raw k[KS][2], kb[BLKS][4], qb[BLKS][4];
    Frag<3> t[2], p[2];
    T g[4];
    float gam[4], end[4], last;
  } x;
  uint32_t koff = 0, boff[BLKS][4], voff[4];
  auto offsets = [&](const DeltaRows& rows) {
    koff = rows.off(16 * w + row, kstride);
#pragma unroll
    for (int m = 0; m < BLKS; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        boff[m][j] = rows.off(4 * ((threadIdx.x + 256 * m) / (DK / 4)) + j, kstride);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      voff[r] = in ? rows.off(16 * w + 4 * gq + r, vstride) + col * sizeof(T) : kNowhere;
  };
  // frags of row tiles 2 and 3 have terms from 32 on only (loaded twice, as in the forward)
  const int first = w >= 2 ? 1 : 0;
  auto load_rows = [&](int c) {
    const size_t low = delta_low(a, sq, b, c), ch = (size_t)bh * a.chunks + c;
    const auto kbuf = delta_buf((const T*)a.k + (low * a.Hk + hk) * a.dk);
    const auto qbuf = delta_buf((const T*)a.q + (low * a.Hk + hk) * a.dk);
    const auto obuf = delta_buf((const T*)a.dout + (low * a.H + h) * a.dv);
#pragma unroll
    for (int r = 0; r < 4; ++r) x.g[r] = buf_load<T>(obuf, voff[r]);
    const unsigned char* Pm = a.Pt + ch * kDeltaTtBytes;
    x.p[0] = mem_frag<3>(Pm, trit_frag(w, first), lane);
    x.p[1] = mem_frag<3>(Pm, trit_frag(w, 1), lane);
    const DeltaGates& gt = a.gates[ch];
    *(v4f*)x.gam = *(const v4f*)&gt.gam[16 * w + 4 * gq];
    *(v4f*)x.end = *(const v4f*)&gt.end[16 * w + 4 * gq];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x.k[s][e] = raw4<T, VEC>(kbuf, koff, 32 * s + 16 * e + 4 * gq, a.dk);
#pragma unroll
    for (int m = 0; m < BLKS; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 4 * ((threadIdx.x + 256 * m) % (DK / 4));
        x.kb[m][j] = raw4<T, VEC>(kbuf, boff[m][j], at, a.dk);
        x.qb[m][j] = raw4<T, VEC>(qbuf, boff[m][j], at, a.dk);
      }
  };
  auto load_t = [&](int c) {
    const unsigned char* Tm = a.Tt + ((size_t)bh * a.chunks + c) * kDeltaTtBytes;
    x.t[0] = mem_frag<3>(Tm, trit_frag(w, first), lane);
    x.t[1] = mem_frag<3>(Tm, trit_frag(w, 1), lane);
  };
  auto load_last = [&](int c) {
    x.last = a.gates[(size_t)bh * a.chunks + c].gam[kDeltaChunk - 1];
  };
  auto share_do = [&] {
    lds_half<PI>(s_o, w >> 1, lane, w & 1,
                 split4<PI>(wide(x.g[0]), wide(x.g[1]), wide(x.g[2]), wide(x.g[3])));
  };

  if (nch > 0) {
    offsets(delta_rows(sq, nch - 1));
    load_rows(nch - 1);
    load_t(nch - 1);
    load_last(nch - 1);
    share_do();
  }
  __syncthreads();
  for (int c = nch - 1; c >= 0; --c) {
    const size_t ch = (size_t)bh * a.chunks + c;
    const int next = c > 0 ? c - 1 : 0;         // the last one loads itself again
    put_state(a.D + ch * sdim);
    v4f kd = zero, pg = zero;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      kd = mma<PI, 3>(operand<PI>(x.k[s][0], x.k[s][1]), lds_frag<3>(s_d, s, lane), kd);
    if (w < 2) pg = mma<3, PI>(x.p[0], lds_frag<PI>(s_o, 0, lane), pg);
    pg = mma<3, PI>(x.p[1], lds_frag<PI>(s_o, 1, lane), pg);
    lds_half<3>(s_x, w >> 1, lane, w & 1,
                split4<3>(fmaf(a.scale, pg[0], x.end[0] * kd[0]), fmaf(a.scale, pg[1], x.end[1] * kd[1]),
                          fmaf(a.scale, pg[2], x.end[2] * kd[2]), fmaf(a.scale, pg[3], x.end[3] * kd[3])));
    float gam[4], gy[4];
    uint32_t voff0[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gam[r] = x.gam[r];
      gy[r] = a.scale * gam[r] * wide(x.g[r]);
      voff0[r] = voff[r];
    }
    lds_half<3>(s_g, w >> 1, lane, w & 1, split4<3>(gy[0], gy[1], gy[2], gy[3]));
#pragma unroll
    for (int m = 0; m < BLKS; ++m) {
      const int id = threadIdx.x + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (BLK >= 1 || tg < 16) {
        Half<PI> qk[4], qq[4], ck[4], cq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qk[j] = to_half(quad(x.kb[m][j])), qq[j] = to_half(quad(x.qb[m][j]));
        transpose4(qk, ck);
        transpose4(qq, cq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 4 * dg + j, at = (k >> 4) * kTileB, ln = (tg & 3) * 16 + (k & 15);
          lds_half<PI>(s_kt + at, tg >> 3, ln, (tg >> 2) & 1, ck[j]);
          lds_half<PI>(s_qt + at, tg >> 3, ln, (tg >> 2) & 1, cq[j]);
        }
      }
    }
    if (c == nch - 1) offsets(delta_rows(sq, next));
    load_rows(next);
    __syncthreads();
    v4f rr = zero;
    if (w < 2) rr = mma<3, 3>(x.t[0], lds_frag<3>(s_x, 0, lane), rr);
    rr = mma<3, 3>(x.t[1], lds_frag<3>(s_x, 1, lane), rr);
    lds_half<3>(s_r, w >> 1, lane, w & 1,
                split4<3>(-gam[0] * rr[0], -gam[1] * rr[1], -gam[2] * rr[2], -gam[3] * rr[3]));
    load_t(next);
    const auto rbuf = delta_buf(a.R + ch * kDeltaChunk * a.dv);
    const auto vbuf = delta_buf((T*)a.dval + (delta_low(a, sq, b, c) * a.H + h) * a.dv);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      buf_store(rbuf, roff[r], rr[r], 0.f);
      buf_store(vbuf, voff0[r], rr[r], T());
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
    load_last(next);
    share_do();
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
  static constexpr int PI = DeltaType<T, VEC>::PI, PO = DeltaType<T, VEC>::PO, NT = DK / 16, KS = DK / 32;
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
  static constexpr int bytes = red + 7 * 64 * 4;
};

// Sum over the 16 lanes of a row of lanes, in its last one.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16_last(float x) {
  x = dpp_add<0x111>(x);
  x = dpp_add<0x112>(x);
  x = dpp_add<0x114>(x);
  return dpp_add<0x118>(x);
}

template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(512) k_delta_grads(DeltaArgs a) {
  using Lds = GradLds<T, DK, VEC>;
  using Ty = DeltaType<T, VEC>;
  using Fy = DeltaType<float, VEC>;
  constexpr int PI = Lds::PI, PO = Lds::PO, KS = Lds::KS, NT = Lds::NT, NTH = NT / 2;
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

  // positions from the end of the sequence on that this chunk covers: zeros
  {
    const int from = t0 > sq.n ? t0 : sq.n, to = t0 + kDeltaChunk < a.L ? t0 + kDeltaChunk : a.L;
    for (int t = from + wid; t < to; t += 8) {
      const size_t p = (size_t)b * a.L + t;
      for (int k = lane; k < a.dk; k += 64) {
        put1((T*)a.dq + (p * a.Hk + hk) * a.dk + k, 0.f);
        put1((T*)a.dkey + (p * a.Hk + hk) * a.dk + k, 0.f);
      }
      for (int j = lane; j < a.rep; j += 64) {
        put1((T*)a.dg + p * a.H + hk * a.rep + j, 0.f);
        put1((T*)a.dbeta + p * a.H + hk * a.rep + j, 0.f);
      }
    }
  }
  if (t0 >= sq.n) return;
  const DeltaRows rows = delta_rows(sq, c);
  const size_t low = delta_low(a, sq, b, c);
  const uint32_t kstride = (uint32_t)(a.Hk * a.dk) * sizeof(T), vstride = (uint32_t)(a.H * a.dv) * sizeof(T);
  const auto kbuf = delta_buf((const T*)a.k + (low * a.Hk + hk) * a.dk);
  const auto qbuf = delta_buf((const T*)a.q + (low * a.Hk + hk) * a.dk);
  const uint32_t krow = rows.off(16 * w + row, kstride), vrow = rows.off(16 * w + row, vstride);

  Frag<PI> kf[KS];
  {
    typename Ty::Raw k[KS][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) k[s][e] = raw4<T, VEC>(kbuf, krow, 32 * s + 16 * e + 4 * gq, a.dk);
#pragma unroll
    for (int s = 0; s < KS; ++s) kf[s] = operand<PI>(k[s][0], k[s][1]);
  }
  v4f dqs[NTH], dks[NTH];
#pragma unroll
  for (int i = 0; i < NTH; ++i) dqs[i] = dks[i] = zero;

  for (int j = 0; j < a.rep; ++j) {
    const int h = hk * a.rep + j;
    const size_t ch = (size_t)(b * a.H + h) * a.chunks + c;
    const DeltaGates& gt = a.gates[ch];
    const auto sbuf = delta_buf(a.states + ch * sdim), dbuf = delta_buf(a.D + ch * sdim);
    const auto rbuf = delta_buf(a.R + ch * kDeltaChunk * a.dv);
    const auto vbuf = delta_buf((const T*)a.v + (low * a.H + h) * a.dv);
    const auto gbuf = delta_buf((const T*)a.dout + (low * a.H + h) * a.dv);
    const unsigned char* Tm = a.T + ch * delta_t_bytes(PI == 1, true);
    const Frag<PO> tf0 = mem_frag<PO>(Tm, tri_frag(w, 0), lane);
    const Frag<PO> tf1 = mem_frag<PO>(Tm, tri_frag(w, w >> 1), lane);
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
    float rv[4] = {0.f, 0.f, 0.f, 0.f}, sd = 0.f;     // v.R of this lane's rows; <S0, D>

    for (int n0 = 0; n0 < a.dv; n0 += 32) {
      // 4 x 4 blocks of S0 (threads below 256) and of D (the others); rows of do and R as operands; v and
      // R as results lie
      constexpr int kBlk = (DK * 2 + 255) / 256;
      const bool second = tid >= 256;
      typename Fy::Raw ms[kBlk][4], md[kBlk][4];
#pragma unroll
      for (int m = 0; m < kBlk; ++m) {
        const int id = (tid & 255) + 256 * m, n4 = id & 7, k4 = id >> 3;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 4 * k4 + r;
          const uint32_t off = k < a.dk ? (uint32_t)(k * a.dv) * 4 : kNowhere;
          ms[m][r] = raw4<float, VEC>(sbuf, off, n0 + 4 * n4, a.dv);
          if (second) md[m][r] = raw4<float, VEC>(dbuf, off, n0 + 4 * n4, a.dv);
        }
      }
      const auto g0 = raw4<T, VEC>(gbuf, vrow, n0 + 4 * gq, a.dv);
      const auto g1 = raw4<T, VEC>(gbuf, vrow, n0 + 16 + 4 * gq, a.dv);
      const uint32_t rrow = (uint32_t)((16 * w + row) * a.dv) * 4;
      const v4f r0 = raw4<float, VEC>(rbuf, rrow, n0 + 4 * gq, a.dv);
      const v4f r1 = raw4<float, VEC>(rbuf, rrow, n0 + 16 + 4 * gq, a.dv);
      const int n = n0 + 16 * hf + row;
      T v[4];
      float rd[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * w + 4 * gq + r;
        v[r] = buf_load<T>(vbuf, n < a.dv ? rows.off(m, vstride) + n * sizeof(T) : kNowhere);
        rd[r] = buf_load<float>(rbuf, n < a.dv ? (uint32_t)(m * a.dv + n) * 4 : kNowhere);
      }
      __syncthreads();            // the last piece's (or head's) operands have been read
#pragma unroll
      for (int m = 0; m < kBlk; ++m) {
        const int id = (tid & 255) + 256 * m, n4 = id & 7, k4 = id >> 3;
        if (DK * 2 % 256 == 0 || id < DK * 2) {
          if (second) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const v4f d = md[m][r], s = ms[m][r];
              lds_half<PO>(sm + Lds::dn, k4 >> 2, (n4 & 3) * 16 + 4 * (k4 & 3) + r, n4 >> 2,
                           split4<PO>(d[0], d[1], d[2], d[3]));
              sd += s[0] * d[0] + s[1] * d[1] + s[2] * d[2] + s[3] * d[3];
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const v4f s = ms[m][r];
              lds_half<PO>(sm + Lds::sn, k4 >> 2, (n4 & 3) * 16 + 4 * (k4 & 3) + r, n4 >> 2,
                           split4<PO>(s[0], s[1], s[2], s[3]));
              lds_half<PO>(sm + Lds::sk, (k4 >> 3) * 2 + (n4 >> 2), (k4 & 3) * 16 + 4 * (n4 & 3) + r,
                           (k4 >> 2) & 1,
                           split4<PO>(ms[m][0][r], ms[m][1][r], ms[m][2][r], ms[m][3][r]));
            }
          }
        }
      }
      const Frag<PI> gf = operand<PI>(g0, g1);
      const Frag<PO> rf = join<PO>(split4<PO>(r0[0], r0[1], r0[2], r0[3]),
                                   split4<PO>(r1[0], r1[1], r1[2], r1[3]));
      __syncthreads();
      // X = V - diag(y) K S0, this wave's 16 rows and 16 columns
      v4f ks = zero;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        ks = mma<PI, PO>(kf[s], lds_frag<PO>(sm + Lds::sk, 2 * s + hf, lane), ks);
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = wide(v[r]) - gam[r] * ks[r];
        rv[r] = fmaf(rd[r], wide(v[r]), rv[r]);
      }
      lds_half<PO>(sm + Lds::xf, (w >> 1) * 2 + hf, lane, w & 1, split4<PO>(x[0], x[1], x[2], x[3]));
      __syncthreads();
      v4f u = mma<PO, PO>(tf0, lds_frag<PO>(sm + Lds::xf, hf, lane), zero);
      if (w >= 2) u = mma<PO, PO>(tf1, lds_frag<PO>(sm + Lds::xf, 2 + hf, lane), u);
      {   // U as rows: entry (16 w + 4 gq + r, 16 hf + row) of the piece
        const Half<PO> uh = split4<PO>(u[0], u[1], u[2], u[3]);
#pragma unroll
        for (int p = 0; p < PO; ++p) {
          unsigned char* to = sm + Lds::uf + (w * PO + p) * 1024 + ((row >> 2) * 16 + 4 * gq) * 16 +
                              hf * 8 + (row & 3) * 2;
          *(uint16_t*)(to) = (uint16_t)uh.p[p].x;
          *(uint16_t*)(to + 16) = (uint16_t)(uh.p[p].x >> 16);
          *(uint16_t*)(to + 32) = (uint16_t)uh.p[p].y;
          *(uint16_t*)(to + 48) = (uint16_t)(uh.p[p].y >> 16);
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

    // K and Q by 4 x 4 blocks, for their transposes; as results lie
    constexpr int kBlk = (DK * 4 + 255) / 256;
    typename Ty::Raw mb[kBlk][4];
#pragma unroll
    for (int m = 0; m < kBlk; ++m) {
      const int id = (tid & 255) + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        mb[m][r] = raw4<T, VEC>(tid >= 256 ? qbuf : kbuf,
                                tg < 16 ? rows.off(4 * tg + r, kstride) : kNowhere, 4 * dg, a.dk);
    }
    T kr[NTH][4], qr[NTH][4];
#pragma unroll
    for (int i = 0; i < NTH; ++i) {
      const int k = 16 * (hf * NTH + i) + row;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t off =
            k < a.dk ? rows.off(16 * w + 4 * gq + r, kstride) + k * sizeof(T) : kNowhere;
        kr[i][r] = buf_load<T>(kbuf, off);
        qr[i][r] = buf_load<T>(qbuf, off);
      }
    }
    // dP and N to LDS, with their decays
    {
      const float one = hf == 0 ? a.scale : -1.f;
      double cm[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) cm[r] = gt.cum[16 * w + 4 * gq + r];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= w) {
          const double cc = gt.cum[16 * i + row];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int m = 16 * w + 4 * gq + r, nn = 16 * i + row;
            const bool low_ = hf == 0 ? nn <= m : nn < m;
            const float dec = expf(low_ ? (float)(cm[r] - cc) : 0.f);
            mat[hf * 64 * 68 + m * 68 + nn] = low_ ? one * dec * pn[i][r] : 0.f;
          }
        }
    }
    __syncthreads();              // the pieces' operands have been read
#pragma unroll
    for (int m = 0; m < kBlk; ++m) {
      const int id = (tid & 255) + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (tg < 16) {
        Half<PI> q[4], cl[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) q[r] = to_half(quad(mb[m][r]));
        transpose4(q, cl);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 4 * dg + r;
          lds_half<PI>(sm + (tid >= 256 ? Lds::qt : Lds::kt) + (k >> 4) * Lds::kTileB, tg >> 3,
                       (tg & 3) * 16 + (k & 15), (tg >> 2) & 1, cl[r]);
        }
      }
    }
    float cend = 0.f;             // this lane's part of k.(U D^T y_C / y): the rest of <S_C, D>
#pragma unroll
    for (int i = 0; i < NTH; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dq[i][r] *= a.scale * gam[r];
        rowg[i][r] *= -gam[r];
        colg[i][r] *= end[r];
        cend = fmaf(wide(kr[i][r]), colg[i][r], cend);
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
    // row sums: q.dq - k.col, k.row, v.R, and over all rows <S_C, D>
    float z[3][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      z[0][r] = z[1][r] = 0.f;
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        z[0][r] += wide(qr[i][r]) * dq[i][r] - wide(kr[i][r]) * colg[i][r];
        z[1][r] += wide(kr[i][r]) * rowg[i][r];
      }
      z[2][r] = rv[r];
#pragma unroll
      for (int e = 0; e < 3; ++e) z[e][r] = sum16_last(z[e][r]);
    }
    float tot = fmaf(gt.gam[kDeltaChunk - 1], sd, cend);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) tot += __shfl_xor(tot, d);
    if (row == 15)
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[(2 * e + hf) * 64 + 16 * w + 4 * gq + r] = z[e][r];
    if (lane == 0) red[6 * 64 + wid] = tot;
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
        for (int i = 0; i < 8; ++i) d += (double)red[6 * 64 + i];
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const double o = __shfl_down(d, s);
        d += lane + s < 64 ? o : 0.0;
      }
      const uint32_t off = rows.off(lane, (uint32_t)a.H * sizeof(T));
      buf_store(delta_buf((T*)a.dg + low * a.H + h), off, (float)d * gt.na[lane], T());
      buf_store(delta_buf((T*)a.dbeta + low * a.H + h), off,
                (red[4 * 64 + lane] + red[5 * 64 + lane] + rowk) * (1.f - gt.b[lane]), T());
    }
  }
  const auto dqbuf = delta_buf((T*)a.dq + (low * a.Hk + hk) * a.dk);
  const auto dkbuf = delta_buf((T*)a.dkey + (low * a.Hk + hk) * a.dk);
#pragma unroll
  for (int i = 0; i < NTH; ++i) {
    const int k = 16 * (hf * NTH + i) + row;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t off =
          k < a.dk ? rows.off(16 * w + 4 * gq + r, kstride) + k * sizeof(T) : kNowhere;
      buf_store(dqbuf, off, dqs[i][r], T());
      buf_store(dkbuf, off, dks[i][r], T());
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
  size_t T, Tt, Pt, gates, D, R, states, total;
};
// T has room for the three parts that forming the states again takes; the gradients' T follows it there.
BwdWs bwd_ws(int64_t B, int64_t L, int H, int dk, int dv, bool bf16, bool has_states) {
  const size_t n = (size_t)B * H * ((L + kDeltaChunk - 1) / kDeltaChunk);
  BwdWs w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  w.T = take(n * delta_t_bytes(bf16, has_states));
  w.Tt = take(n * kDeltaTtBytes);
  w.Pt = take(n * kDeltaTtBytes);
  w.gates = take(n * sizeof(DeltaGates));
  w.D = take(n * dk * dv * 4);
  w.R = take(n * kDeltaChunk * dv * 4);
  w.states = take(has_states ? 0 : n * dk * dv * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t delta_backward_workspace(int64_t B, int64_t L, int H, int dk, int dv, bool bf16,
                                bool has_states) {
  return bwd_ws(B, L, H, dk, dv, bf16, has_states).total;
}

hipError_t launch_delta_backward(const DeltaRequest& r, hipStream_t st) {
  DeltaArgs a = delta_args(r);
  const BwdWs w = bwd_ws(r.B, r.L, r.H, r.dk, r.dv, r.bf16, r.states != nullptr);
  unsigned char* ws = (unsigned char*)r.ws;
  a.T = ws + w.T;
  a.Tt = ws + w.Tt;
  a.Pt = ws + w.Pt;
  a.gates = (DeltaGates*)(ws + w.gates);
  a.D = (float*)(ws + w.D);
  a.R = (float*)(ws + w.R);
  const bool vec = delta_vec(r);
  hipError_t e = hipSuccess;
  if (!a.states) {               // a.o is null: the walk forms the states only
    a.states = (float*)(ws + w.states);
    e = launch_delta_prep(a, r.bf16, vec, kPrepStates, st);
    if (e == hipSuccess) e = launch_delta_walk(a, r.bf16, vec, st);
  }
  if (e == hipSuccess) e = launch_delta_prep(a, r.bf16, vec, kPrepBackward, st);
  if (e != hipSuccess) return e;
  return r.bf16 ? backward_t<uint16_t>(a, vec, st) : backward_t<float>(a, vec, st);
}

}  // namespace wbmm
