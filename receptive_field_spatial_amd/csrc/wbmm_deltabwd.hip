// Gated delta rule, backward: the walk along the chunks from the last to the first
// (k_delta_walk_bwd), and what each chunk computes on its own then (k_delta_grads).
#include "wbmm_deltadev.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

// ---------------------------------------------------------------------------- the walk back
// As the forward's walk: one workgroup per head and NC tiles of 16 columns of dv, four walkers and four helpers.
//        walkers                                         helpers
//   A    dU = P^T G + diag(y_C / y) K D                  M = Q^T diag(y) G
//   B    R = T^T dU (= dv)                               P^T G, K, K^T, Q^T and diag(y) G of the next chunk
//   C    D = y_C D + M - K^T diag(y) R                   do of the one after
// D after each chunk and R stay in the workspace for k_delta_grads. Bound as the forward's, with D and R to store:
// 192 heads of 64, 784 steps, bf16: 70 to 75 us with four tiles a workgroup, 85 to 88 with two, 98 to 102 with one; 30 heads
// of 48 x 40 over 1531 steps, fp32: 75 us, 3.1 a chunk.
template <typename T, int DK, int NC>
struct BackLds {
  static constexpr int PI = DeltaType<T, true>::PI, KS = DK / 32, NT = DK / 16;
  static constexpr int d = 0;                              // D
  static constexpr int x = d + NC * KS * 3 * 1024;              // dU
  static constexpr int r = x + NC * 2 * 3 * 1024;               // -diag(y) R
  static constexpr int g = r + NC * 2 * 3 * 1024;               // diag(y) G
  static constexpr int o = g + NC * 2 * 3 * 1024;               // do
  static constexpr int m = o + NC * 2 * PI * 1024;              // M, as results lie
  static constexpr int pg = m + NC * NT * 1024;                 // P^T G, as results lie
  static constexpr int qt = pg + NC * 4 * 1024;                 // Q^T
  static constexpr int cols = NT * kTileBytes<PI>;
  static constexpr int kt = qt + cols;                     // K^T, of two chunks where they fit
  static constexpr int rows = 4 * KS * PI * 1024;
  // fp32 with 96 < dk: the walkers load K's rows themselves
  static constexpr bool direct = kt + cols + rows > 160 * 1024;
  static constexpr bool two = !direct && kt + 2 * cols + rows <= 160 * 1024;
  static constexpr int k = kt + (two ? 2 : 1) * cols;      // K
  static constexpr int bytes = k + (direct ? 0 : rows);
};

template <typename T, int DK, bool VEC, int NC>
__global__ void __launch_bounds__(512) k_delta_walk_bwd(DeltaArgs a) {
  using Ty = DeltaType<T, VEC>;
  using Lds = BackLds<T, DK, NC>;
  constexpr int PI = Ty::PI, KS = DK / 32, NT = DK / 16, OWN = (NT + 3) / 4;
  constexpr bool TWO = Lds::two, DIRECT = Lds::direct;
  constexpr int kD = KS * 3 * 1024, kX = 2 * 3 * 1024, kO = 2 * PI * 1024, kM = NT * 1024;   // of a column tile
  extern __shared__ __attribute__((aligned(16))) unsigned char sm[];
  const DeltaWalkAt at = delta_walk_at((a.dv + 16 * NC - 1) / (16 * NC));
  const int bh = at.bh;
  if (bh >= a.B * a.H) return;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wid & 3, row = lane & 15, gq = lane >> 4;
  const bool walker = wid < 4;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const DeltaSeq sq = delta_seq(a, b);
  const int col = at.tile * (16 * NC) + row;
  const bool in = col < a.dv;
  const int nch = (sq.n + kDeltaChunk - 1) / kDeltaChunk, endc = nch - 1;
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  const uint32_t kstride = (uint32_t)(a.Hk * a.dk) * sizeof(T), vstride = (uint32_t)(a.H * a.dv) * sizeof(T);
  const size_t sdim = (size_t)a.dk * a.dv;
  // frags of row tiles 2 and 3 have terms from 32 on only (loaded twice, as in the forward)
  const int first = w >= 2 ? 1 : 0;
  auto value_offsets = [&](const DeltaRows& rows, uint32_t (&off)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      off[r] = in ? rows.off(16 * w + 4 * gq + r, vstride) + col * sizeof(T) : kNowhere;
  };

  if (walker) {
    v4f D[NC][OWN];
    uint32_t soff[OWN][4], roff[4], voff[4], koff = 0;
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = walk_entry(w * OWN + i, 4 * gq + r);
        const bool own = w * OWN + i < NT && k < a.dk && in;
        soff[i][r] = own ? (uint32_t)(k * a.dv + col) * 4 : kNowhere;
#pragma unroll
        for (int n = 0; n < NC; ++n)
          D[n][i][r] = a.ds_last ? buf_load<float>(delta_buf(a.ds_last + bh * sdim), soff[i][r] + 64 * n) : 0.f;
      }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      roff[r] = in ? (uint32_t)((16 * w + 4 * gq + r) * a.dv + col) * 4 : kNowhere;
    auto put_state = [&](float* to) {
      const auto buf = delta_buf(to);
#pragma unroll
      for (int i = 0; i < OWN; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int n = 0; n < NC; ++n) buf_store(buf, soff[i][r] + 64 * n, D[n][i][r], 0.f);
    };
    auto share_state = [&] {
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const int tile = w * OWN + i;
        if (tile < NT)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            lds_half<3>(sm + Lds::d + n * kD, tile >> 1, lane, tile & 1,
                        split4<3>(D[n][i][0], D[n][i][1], D[n][i][2], D[n][i][3]));
      }
    };
    Frag<3> t[2];
    Raw8<T, VEC> k[DIRECT ? KS : 1];
    v4f gam = zero, end = zero;
    float last = 1.f;
    auto load_k = [&](int c) {
      if constexpr (DIRECT) {
        if (c == endc || c == endc - 1) koff = delta_rows(sq, c).off(16 * w + row, kstride);
        const auto kbuf = delta_buf((const T*)a.k + (delta_low(a, sq, b, c) * a.Hk + hk) * a.dk);
#pragma unroll
        for (int s = 0; s < KS; ++s) k[s] = raw8<T, VEC>(kbuf, koff, 32 * s + 8 * gq, a.dk);
      }
      end = *(const v4f*)&a.gates[(size_t)bh * a.chunks + c].end[16 * w + 4 * gq];
    };
    auto load_t = [&](int c) {
      const size_t ch = (size_t)bh * a.chunks + c;
      const unsigned char* Tm = a.Tt + ch * kDeltaTtBytes;
      t[0] = mem_frag<3>(Tm, trit_frag(w, first), lane);
      t[1] = mem_frag<3>(Tm, trit_frag(w, 1), lane);
      gam = *(const v4f*)&a.gates[ch].gam[16 * w + 4 * gq];
    };
    auto load_last = [&](int c) {
      last = a.gates[(size_t)bh * a.chunks + c].gam[kDeltaChunk - 1];
    };
    if (nch > 0) {
      value_offsets(delta_rows(sq, endc), voff);
      load_k(endc);
      load_t(endc);
      load_last(endc);
    }
    share_state();
    __syncthreads();
    __syncthreads();
    __syncthreads();
    for (int c = endc; c >= 0; --c) {
      const size_t ch = (size_t)bh * a.chunks + c;
      const int next = c > 0 ? c - 1 : 0;
      put_state(a.D + ch * sdim);
      v4f kp[NC][KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Frag<PI> f;
        if constexpr (DIRECT) {
          Half<PI> lo, hi;
          halves<PI>(k[s], lo, hi);
          f = join<PI>(lo, hi);
        } else {
          f = lds_frag<PI>(sm + Lds::k, w * KS + s, lane);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) kp[n][s] = mma<PI, 3>(f, lds_frag<3>(sm + Lds::d + n * kD, s, lane), zero);
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        v4f kd = zero;
#pragma unroll
        for (int s = 0; s < KS; ++s) kd += kp[n][s];
        const v4f pg = *(const v4f*)(sm + Lds::pg + (4 * n + w) * 1024 + lane * 16);
        lds_half<3>(sm + Lds::x + n * kX, w >> 1, lane, w & 1,
                    split4<3>(fmaf(end[0], kd[0], pg[0]), fmaf(end[1], kd[1], pg[1]),
                              fmaf(end[2], kd[2], pg[2]), fmaf(end[3], kd[3], pg[3])));
      }
      load_k(next);
      __syncthreads();
      v4f rr[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) rr[n] = mma_short(t[1], lds_frag<3>(sm + Lds::x + n * kX, 1, lane));
      if (w < 2)
#pragma unroll
        for (int n = 0; n < NC; ++n) rr[n] += mma_short(t[0], lds_frag<3>(sm + Lds::x + n * kX, 0, lane));
#pragma unroll
      for (int n = 0; n < NC; ++n)
        lds_half<3>(sm + Lds::r + n * kX, w >> 1, lane, w & 1,
                    split4<3>(-gam[0] * rr[n][0], -gam[1] * rr[n][1], -gam[2] * rr[n][2], -gam[3] * rr[n][3]));
      load_t(next);
      const auto rbuf = delta_buf(a.R + ch * kDeltaChunk * a.dv);
      const auto vbuf = delta_buf((T*)a.dval + (delta_low(a, sq, b, c) * a.H + h) * a.dv);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          buf_store(rbuf, roff[r] + 64 * n, rr[n][r], 0.f);
          buf_store(vbuf, voff[r] + 16 * n * sizeof(T), rr[n][r], T());
        }
      if (c == endc) value_offsets(delta_rows(sq, next), voff);
      __syncthreads();
      const unsigned char* kt = sm + Lds::kt + (TWO ? c & 1 : 0) * Lds::cols;
      v4f more[NC][OWN];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
          D[n][i] *= last;
          more[n][i] = w * OWN + i < NT
                           ? *(const v4f*)(sm + Lds::m + n * kM + (w * OWN + i) * 1024 + lane * 16) : zero;
        }
      load_last(next);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<3> f[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) f[n] = lds_frag<3>(sm + Lds::r + n * kX, s, lane);
#pragma unroll
        for (int i = 0; i < OWN; ++i)
          if (w * OWN + i < NT) {
            const Frag<PI> kf = lds_frag<PI>(kt + (w * OWN + i) * kTileBytes<PI>, s, lane);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              v4f& to = s ? more[n][i] : D[n][i];
              to = mma<PI, 3>(kf, f[n], to);
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < OWN; ++i) D[n][i] += more[n][i];
      share_state();
      __syncthreads();
    }
    if (a.ds0) put_state(a.ds0 + bh * sdim);
  } else {
    const int id = threadIdx.x - 256, dg = id % (DK / 8), tg = id / (DK / 8);
    const bool block = tg < 16;      // a 4 x 8 block of K and of Q
    Raw8<T, VEC> kb[4], qb[4];
    Frag<3> p[2];
    uint32_t g[NC][4], g2[NC][4];    // do of the next chunk and of the one after
    v4f gam = zero;
    uint32_t boff[4], goff[4];
    auto load_kq = [&](int c) {
      if (c == endc || c == endc - 1) {
        const DeltaRows rows = delta_rows(sq, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) boff[j] = block ? rows.off(4 * tg + j, kstride) : kNowhere;
      }
      const size_t at = (delta_low(a, sq, b, c) * a.Hk + hk) * a.dk;
      const auto kbuf = delta_buf((const T*)a.k + at), qbuf = delta_buf((const T*)a.q + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) kb[j] = raw8<T, VEC>(kbuf, boff[j], 8 * dg, a.dk);
#pragma unroll
      for (int j = 0; j < 4; ++j) qb[j] = raw8<T, VEC>(qbuf, boff[j], 8 * dg, a.dk);
      gam = *(const v4f*)&a.gates[(size_t)bh * a.chunks + c].gam[16 * w + 4 * gq];
    };
    auto load_g = [&](int c, uint32_t (&to)[NC][4]) {
      if (c == endc || c == endc - 1) value_offsets(delta_rows(sq, c), goff);
      const auto obuf = delta_buf((const T*)a.dout + (delta_low(a, sq, b, c) * a.H + h) * a.dv);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < NC; ++n) to[n][r] = raw1<T>(obuf, goff[r] + 16 * n * sizeof(T));
    };
    auto load_p = [&](int c) {
      const unsigned char* Pm = a.Pt + ((size_t)bh * a.chunks + c) * kDeltaTtBytes;
      p[0] = mem_frag<3>(Pm, trit_frag(w, first), lane);
      p[1] = mem_frag<3>(Pm, trit_frag(w, 1), lane);
    };
    auto share_k = [&](int c, bool as_rows, bool as_cols) {
      Half<PI> lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) halves<PI>(kb[j], lo[j], hi[j]);
      if (block && as_rows && !DIRECT) lds_rows<PI, KS>(sm + Lds::k, tg, dg, lo, hi);
      if (block && as_cols) lds_cols<PI>(sm + Lds::kt + (TWO ? c & 1 : 0) * Lds::cols, tg, dg, lo, hi);
    };
    auto share_q = [&] {
      Half<PI> lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) halves<PI>(qb[j], lo[j], hi[j]);
      if (block) lds_cols<PI>(sm + Lds::qt, tg, dg, lo, hi);
    };
    auto share_g = [&] {             // diag(y) G
#pragma unroll
      for (int n = 0; n < NC; ++n)
        lds_half<3>(sm + Lds::g + n * kX, w >> 1, lane, w & 1,
                    split4<3>(a.scale * gam[0] * wide1<T>(g[n][0]), a.scale * gam[1] * wide1<T>(g[n][1]),
                              a.scale * gam[2] * wide1<T>(g[n][2]), a.scale * gam[3] * wide1<T>(g[n][3])));
    };
    auto share_o = [&](const uint32_t (&o)[NC][4]) {
#pragma unroll
      for (int n = 0; n < NC; ++n)
        lds_half<PI>(sm + Lds::o + n * kO, w >> 1, lane, w & 1,
                     split4<PI>(wide1<T>(o[n][0]), wide1<T>(o[n][1]), wide1<T>(o[n][2]), wide1<T>(o[n][3])));
    };
    auto form_pg = [&] {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        v4f pg = zero;
        if (w < 2) pg = mma<3, PI>(p[0], lds_frag<PI>(sm + Lds::o + n * kO, 0, lane), pg);
        pg = mma<3, PI>(p[1], lds_frag<PI>(sm + Lds::o + n * kO, 1, lane), pg);
        *(v4f*)(sm + Lds::pg + (4 * n + w) * 1024 + lane * 16) = pg * a.scale;
      }
    };
    auto next_g = [&] {
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) g[n][r] = g2[n][r];
    };
    auto back = [&](int c, int by) { return c >= by ? c - by : 0; };
    if (nch > 0) {
      load_kq(endc);
      load_g(endc, g);
      load_p(endc);
      load_g(back(endc, 1), g2);
      share_k(endc, true, TWO);
      share_q();
      share_g();
      share_o(g);
    }
    __syncthreads();
    if (nch > 0) form_pg();
    __syncthreads();
    if (nch > 0) {
      share_o(g2);
      next_g();
      load_p(back(endc, 1));
      load_g(back(endc, 2), g2);
      if (TWO) load_kq(back(endc, 1));
    }
    __syncthreads();
    for (int c = endc; c >= 0; --c) {
      // M: its row tiles over the four waves
#pragma unroll
      for (int i = 0; i < OWN; ++i)
        if (w * OWN + i < NT) {
          v4f m[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) m[n] = zero;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const Frag<PI> f = lds_frag<PI>(sm + Lds::qt + (w * OWN + i) * kTileBytes<PI>, s, lane);
#pragma unroll
            for (int n = 0; n < NC; ++n) m[n] = mma<PI, 3>(f, lds_frag<3>(sm + Lds::g + n * kX, s, lane), m[n]);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n)
            *(v4f*)(sm + Lds::m + n * kM + (w * OWN + i) * 1024 + lane * 16) = m[n];
        }
      if (!TWO) {
        share_k(c, false, true);
        load_kq(back(c, 1));
      }
      __syncthreads();
      form_pg();
      load_p(back(c, 2));
      share_k(c - 1, true, TWO);     // this chunk's rows, Q^T and G have been read
      share_q();
      share_g();
      if (TWO) load_kq(back(c, 2));
      __syncthreads();
      share_o(g2);
      next_g();
      load_g(back(c, 3), g2);
      __syncthreads();
    }
    if (in)
      for (int t = sq.n + (id >> 4); t < a.L; t += 16)
#pragma unroll
        for (int n = 0; n < NC; ++n)
          put1((T*)a.dval + (((size_t)b * a.L + t) * a.H + h) * a.dv + col + 16 * n, 0.f);
  }
}

// ---------------------------------------------------------------------------- chunks on their own
// One workgroup of 8 waves per chunk of a key head, its heads one after the other. Wave (w, hf) has row
// tile w of the 64 steps, and of everything along dk the half hf; the (64 x 64) dP is hf = 0's and N hf =
// 1's. dv is walked in pieces of 32 columns, whose S0 and D are staged in LDS as operands. Bound by vector
// issue (2000 instructions a wave and chunk, 59 % of the cycles; the matrix cores 17 %): splitting S0, D, dP and N,
// transposes, decays, row sums. 2496 chunks of one head of 64, bf16: 132 us (110 with two parts of what now has three);
// 240 of three heads, fp32: 47.
template <typename T, int DK, bool VEC>
struct GradLds {
  static constexpr int PI = DeltaType<T, VEC>::PI, NT = DK / 16, KS = DK / 32;
  static constexpr int sn = 0;                            // S0, terms along dv: NT frags
  static constexpr int sk = sn + NT * 3 * 1024;          // S0, terms along dk: KS x 2
  static constexpr int dn = sk + KS * 2 * 3 * 1024;      // D, terms along dv: NT
  static constexpr int xf = dn + NT * 3 * 1024;          // X: 2 x 2
  static constexpr int uf = xf + 4 * 3 * 1024;           // U as rows: 4
  static constexpr int walk = uf + 4 * 3 * 1024;
  static constexpr int kt = 0;                            // afterwards: K^T and Q^T, NT x 2 each
  static constexpr int kTileB = 2 * PI * 1024;
  static constexpr int qt = kt + NT * kTileB;
  static constexpr int after = qt + NT * kTileB;
  static constexpr int mat = after;                       // and dP and N: 64 rows of 68 floats each
  static constexpr int end = mat + 2 * 64 * 68 * 4;
  static constexpr int red = walk > end ? walk : end;     // row sums
  static constexpr int bytes = red + 7 * 64 * 4;
};

// x, as a value that the compiler forms where it is used: offsets derived from it are not kept in registers
// over a whole loop.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The sum of the products of this lane's 8 entries.
template <int P>
__device__ __forceinline__ float dot(const Frag<P>& a, const Frag<P>& b) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = 0.f, y = 0.f, z = 0.f, t = 0.f;
#pragma unroll
    for (int p = P - 1; p >= 0; --p) {
      x += __uint_as_float(a.p[p][j] << 16);
      y += __uint_as_float(b.p[p][j] << 16);
      z += __uint_as_float(a.p[p][j] & 0xffff0000u);
      t += __uint_as_float(b.p[p][j] & 0xffff0000u);
    }
    s = fmaf(x, y, fmaf(z, t, s));
  }
  return s;
}

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

template <typename T, int DK, bool VEC, bool ONE>
__global__ void __launch_bounds__(512, (DK < 128 && DeltaType<T, VEC>::PI == 1 ? 4 : 2)) k_delta_grads(DeltaArgs a) {
  using Lds = GradLds<T, DK, VEC>;
  using Ty = DeltaType<T, VEC>;
  using Fy = DeltaType<float, VEC>;
  constexpr int PI = Lds::PI, PM = Ty::PM, KS = Lds::KS, NT = Lds::NT, NTH = NT / 2;
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
  const uint32_t krow = rows.off(16 * w + row, kstride);

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

  for (int j = 0; j < (ONE ? 1 : a.rep); ++j) {
    const int h = hk * a.rep + j;
    const size_t ch = (size_t)(b * a.H + h) * a.chunks + c;
    const DeltaGates& gt = a.gates[ch];
    const auto sbuf = delta_buf(a.states + ch * sdim), dbuf = delta_buf(a.D + ch * sdim);
    const auto rbuf = delta_buf(a.R + ch * kDeltaChunk * a.dv);
    const auto vbuf = delta_buf((const T*)a.v + (low * a.H + h) * a.dv);
    const auto gbuf = delta_buf((const T*)a.dout + (low * a.H + h) * a.dv);
    const unsigned char* Tm = a.T + ch * delta_t_bytes(PI == 1, true);
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

    // Of a piece: 4 x 4 blocks of S0 (threads below 256) or of D (the others), rows of do and R as
    // operands, v and R as results lie. (The next piece's in flight meanwhile would take 36 more registers, and
    // with them one of the two workgroups of a CU.)
    constexpr int kBlk = (DK * 2 + 255) / 256;
    const bool second = hf == 1;     // the same for a whole wave, and known to be
    const auto mbuf = second ? dbuf : sbuf;
    typename Fy::Raw ms[kBlk][4];
    typename Ty::Raw g0, g1;
    v4f r0, r1;
    uint32_t v[4];
    float rd[4];
    auto load_piece = [&](int n0) {
      const int tid = here(threadIdx.x), lane = tid & 63, row = lane & 15, gq = lane >> 4;
      const uint32_t vrow = rows.off(16 * w + row, vstride);
#pragma unroll
      for (int m = 0; m < kBlk; ++m) {
        const int id = (tid & 255) + 256 * m, n4 = id & 7, k4 = id >> 3;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 4 * k4 + r;
          ms[m][r] = raw4<float, VEC>(mbuf, k < a.dk ? (uint32_t)(k * a.dv) * 4 : kNowhere, n0 + 4 * n4,
                                      a.dv);
        }
      }
      g0 = raw4<T, VEC>(gbuf, vrow, n0 + 4 * gq, a.dv);
      g1 = raw4<T, VEC>(gbuf, vrow, n0 + 16 + 4 * gq, a.dv);
      const uint32_t rrow = (uint32_t)((16 * w + row) * a.dv) * 4;
      r0 = raw4<float, VEC>(rbuf, rrow, n0 + 4 * gq, a.dv);
      r1 = raw4<float, VEC>(rbuf, rrow, n0 + 16 + 4 * gq, a.dv);
      const int n = n0 + 16 * hf + row;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * w + 4 * gq + r;
        v[r] = raw1<T>(vbuf, n < a.dv ? rows.off(m, vstride) + n * sizeof(T) : kNowhere);
        rd[r] = buf_load<float>(rbuf, n < a.dv ? (uint32_t)(m * a.dv + n) * 4 : kNowhere);
      }
    };
    for (int n0 = 0; n0 < a.dv; n0 += 32) {
      const int tid = here(threadIdx.x), lane = tid & 63, row = lane & 15, gq = lane >> 4;
      load_piece(n0);
      __syncthreads();            // the last piece's (or head's) operands have been read
#pragma unroll
      for (int m = 0; m < kBlk; ++m) {
        const int id = (tid & 255) + 256 * m, n4 = id & 7, k4 = id >> 3;
        if (DK * 2 % 256 == 0 || id < DK * 2) {
          unsigned char* to = sm + (second ? Lds::dn : Lds::sn);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            lds_half<3>(to, k4 >> 2, (n4 & 3) * 16 + 4 * (k4 & 3) + r, n4 >> 2,
                         split4<3>(ms[m][r][0], ms[m][r][1], ms[m][r][2], ms[m][r][3]));
          if (!second)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              lds_half<3>(sm + Lds::sk, (k4 >> 3) * 2 + (n4 >> 2), (k4 & 3) * 16 + 4 * (n4 & 3) + r,
                           (k4 >> 2) & 1,
                           split4<3>(ms[m][0][r], ms[m][1][r], ms[m][2][r], ms[m][3][r]));
        }
      }
      const Frag<PI> gf = operand<PI>(g0, g1);
      const Frag<3> rf = join<3>(split4<3>(r0[0], r0[1], r0[2], r0[3]),
                                   split4<3>(r1[0], r1[1], r1[2], r1[3]));
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = wide1<T>(v[r]);
        rv[r] = fmaf(rd[r], x[r], rv[r]);
      }
      // for every piece again: kept over them, with the three parts, they would not fit the registers (276 us for 234)
      const Frag<PM> tf0 = mem_frag<PM>(Tm, tri_frag(w, 0), lane);
      const Frag<PM> tf1 = mem_frag<PM>(Tm, tri_frag(w, w >> 1), lane);
      __syncthreads();
      // X = V - diag(y) K S0, this wave's 16 rows and 16 columns
      v4f ks = zero;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        ks = mma<PI, 3>(kf[s], lds_frag<3>(sm + Lds::sk, 2 * s + hf, lane), ks);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] -= gam[r] * ks[r];
      lds_half<3>(sm + Lds::xf, (w >> 1) * 2 + hf, lane, w & 1, split4<3>(x[0], x[1], x[2], x[3]));
      __syncthreads();
      v4f u = mma<3, 3>(parts(tf0), lds_frag<3>(sm + Lds::xf, hf, lane), zero);
      if (w >= 2) u = mma<3, 3>(parts(tf1), lds_frag<3>(sm + Lds::xf, 2 + hf, lane), u);
      {   // U as rows: entry (16 w + 4 gq + r, 16 hf + row) of the piece
        const Half<3> uh = split4<3>(u[0], u[1], u[2], u[3]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          unsigned char* to = sm + Lds::uf + (w * 3 + p) * 1024 + hf * 8 + (row & 3) * 2;
          const int l = (row >> 2) * 16 + 4 * gq;
          *(uint16_t*)(to + slot(l) * 16) = (uint16_t)uh.p[p].x;
          *(uint16_t*)(to + slot(l + 1) * 16) = (uint16_t)(uh.p[p].x >> 16);
          *(uint16_t*)(to + slot(l + 2) * 16) = (uint16_t)uh.p[p].y;
          *(uint16_t*)(to + slot(l + 3) * 16) = (uint16_t)(uh.p[p].y >> 16);
        }
      }
      __syncthreads();
      const Frag<3> uw = lds_frag<3>(sm + Lds::uf, w, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= w) {
          const Frag<3> ui = lds_frag<3>(sm + Lds::uf, i, lane);
          if (hf == 0) pn[i] = mma<PI, 3>(gf, ui, pn[i]);
          else pn[i] = mma<3, 3>(rf, ui, pn[i]);
        }
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        const Frag<3> sf = lds_frag<3>(sm + Lds::sn, hf * NTH + i, lane);
        const Frag<3> df = lds_frag<3>(sm + Lds::dn, hf * NTH + i, lane);
        dq[i] = mma<PI, 3>(gf, sf, dq[i]);
        rowg[i] = mma<3, 3>(rf, sf, rowg[i]);
        colg[i] = mma<3, 3>(uw, df, colg[i]);
        if (w == (i & 3)) sd += dot(sf, df);      // <S0, D>, each tile by one wave
      }
    }

    // K and Q by 4 x 4 blocks, for their transposes; as results lie
    constexpr int kRowBlk = (DK * 4 + 255) / 256;
    const int tid = here(threadIdx.x), lane = tid & 63, row = lane & 15, gq = lane >> 4;
    typename Ty::Raw mb[kRowBlk][4];
#pragma unroll
    for (int m = 0; m < kRowBlk; ++m) {
      const int id = (tid & 255) + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        mb[m][r] = raw4<T, VEC>(second ? qbuf : kbuf,
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
    __syncthreads();              // the pieces' operands have been read
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
            const float d = (float)(cm[r] - cc), p = one * __builtin_amdgcn_exp2f(d > 0.f ? 0.f : d);
            mat[hf * 64 * 68 + m * 68 + nn] = low_ ? p * pn[i][r] : 0.f;
          }
        }
    }
#pragma unroll
    for (int m = 0; m < kRowBlk; ++m) {
      const int id = (tid & 255) + 256 * m, dg = id % (DK / 4), tg = id / (DK / 4);
      if (tg < 16) {
        Half<PI> q[4], cl[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) q[r] = to_half(quad(mb[m][r]));
        transpose4(q, cl);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = 4 * dg + r;
          lds_half<PI>(sm + (second ? Lds::qt : Lds::kt) + (k >> 4) * Lds::kTileB, tg >> 3,
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
        const Frag<3> pf = split8<3>(p), nf = split8<3>(q);
#pragma unroll
        for (int i = 0; i < NTH; ++i) {
          const Frag<PI> kt = lds_frag<PI>(sm + Lds::kt + (hf * NTH + i) * Lds::kTileB, s, lane);
          dq[i] = mma<3, PI>(pf, kt, dq[i]);
          rowg[i] = mma<3, PI>(nf, kt, rowg[i]);
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
        const Frag<3> pf = split8<3>(p), nf = split8<3>(q);
#pragma unroll
        for (int i = 0; i < NTH; ++i) {
          const int at = (hf * NTH + i) * Lds::kTileB;
          colg[i] = mma<3, PI>(pf, lds_frag<PI>(sm + Lds::qt + at, s, lane), colg[i]);
          colg[i] = mma<3, PI>(nf, lds_frag<PI>(sm + Lds::kt + at, s, lane), colg[i]);
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
    if (ONE) {
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        dqs[i] = dq[i];
        dks[i] = rowg[i] + colg[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NTH; ++i) {
        dqs[i] += dq[i];
        dks[i] += rowg[i] + colg[i];
      }
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
                (red[4 * 64 + lane] + red[5 * 64 + lane] + rowk) * gt.nb[lane], T());
    }
  }
  const int tidl = here(threadIdx.x), gql = (tidl & 63) >> 4, rowl = tidl & 15;
  const auto dqbuf = delta_buf((T*)a.dq + (low * a.Hk + hk) * a.dk);
  const auto dkbuf = delta_buf((T*)a.dkey + (low * a.Hk + hk) * a.dk);
#pragma unroll
  for (int i = 0; i < NTH; ++i) {
    const int k = 16 * (hf * NTH + i) + rowl;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t off =
          k < a.dk ? rows.off(16 * w + 4 * gql + r, kstride) + k * sizeof(T) : kNowhere;
      buf_store(dqbuf, off, dqs[i][r], T());
      buf_store(dkbuf, off, dks[i][r], T());
    }
  }
}

template <typename T>
hipError_t backward_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  hipError_t e = hipSuccess;
  with_dk(a.dk, vec, [&](auto d, auto v) {
    constexpr int DK = decltype(d)::value;
    constexpr bool VEC = decltype(v)::value;
    auto walk = [&](auto n) {
      constexpr int NC = decltype(n)::value;
      constexpr int back = BackLds<T, DK, NC>::bytes;
      static_assert(back <= 160 * 1024, "LDS of a CU");
      const dim3 grid = delta_walk_grid(a, (a.dv + 16 * NC - 1) / (16 * NC));
      e = hipFuncSetAttribute((const void*)k_delta_walk_bwd<T, DK, VEC, NC>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, back);
      if (e != hipSuccess) return;
      k_delta_walk_bwd<T, DK, VEC, NC><<<grid, 512, back, st>>>(a);
      e = hipGetLastError();
    };
    bool done = false;
    if constexpr (VEC && BackLds<T, DK, 4>::bytes <= 160 * 1024) {
      if (walk_four_tiles(a)) {
        walk(std::integral_constant<int, 4>());
        done = true;
      }
    }
    if constexpr (VEC && BackLds<T, DK, 2>::bytes <= 160 * 1024) {
      if (!done && walk_two_tiles(a)) {
        walk(std::integral_constant<int, 2>());
        done = true;
      }
    }
    if (!done) walk(std::integral_constant<int, 1>());
    if (e != hipSuccess) return;
    constexpr int bytes = GradLds<T, DK, VEC>::bytes;
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    auto grads = [&](auto one) {
      constexpr bool ONE = decltype(one)::value;   // every head has a key head of its own
      e = hipFuncSetAttribute((const void*)k_delta_grads<T, DK, VEC, ONE>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != hipSuccess) return;
      k_delta_grads<T, DK, VEC, ONE><<<dim3(a.B * a.Hk * a.chunks), 512, bytes, st>>>(a);
      e = hipGetLastError();
    };
    if (a.rep == 1) grads(std::true_type());
    else grads(std::false_type());
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
