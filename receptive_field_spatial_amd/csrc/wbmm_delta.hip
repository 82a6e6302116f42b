// Gated delta rule, forward: what each chunk computes on its own (k_delta_prep), the walk along the
// chunks (k_delta_walk), and single steps (k_delta_step).
#include "wbmm_deltadev.hpp"
#include "wbmm_launch.hpp"

namespace wbmm {

namespace {

// ---------------------------------------------------------------------------- chunks on their own
// One workgroup of 4 waves per chunk of a head: T, P and the gates. Bound by its own chain of products (58 % of the
// waves' cycles are waits, the matrix cores busy for 23 % at four workgroups a CU): 27 us for 2496 chunks of bf16 with dk =
// 64 (1.1 us a chunk on each of 256 CUs x 4), 57 for 4096 with dk = 128. Wave j takes column tile j of the
// 64 x 64 matrices. (I + A)^-1 in fp32 on v_mfma_f32_16x16x4f32, N = -A: its diagonal tiles from 4 x 4
// ones; below them T_ij = T_ii sum_k N_ik T_kj, down the column, which needs no other wave's column. With terms in the order 4 q + s, s the product's number,
// a result is the next product's B operand as it lies, and the A operand of its transpose.
__device__ __forceinline__ v4f mm16(const v4f& a, const v4f& b, v4f acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma_f32(a[s], b[s], acc);
  return acc;
}

template <typename T>
__device__ __forceinline__ float elem(const void* p, size_t i) { return load_f32<T>((const T*)p, i); }

// 16 x 16 tile (i, j), j <= i, of a triangular matrix in LDS: rows of 20 floats.
__device__ __forceinline__ constexpr int lds_tile(int i, int j) { return (i * (i + 1) / 2 + j) * 320; }

// A wave's share of a chunk: column tile W, all of whose loops are then of known length.
template <typename T, DeltaPrep MODE>
struct DeltaOwn {
  static constexpr int PI = DeltaType<T, true>::PI, PM = DeltaType<T, true>::PM;
  static constexpr bool WANTP = MODE != kPrepStates;
  unsigned char* s_all;
  const double* s_cum;
  const float* s_b;
  int lane;
  unsigned char *T_, *P_, *Tt_, *Pt_;

  static __device__ __forceinline__ Frag<3> above(const v4f& x, const v4f& y) {
    return join<3>(split4<3>(x[0], x[1], x[2], x[3]), split4<3>(y[0], y[1], y[2], y[3]));
  }
  template <int P>
  __device__ __forceinline__ void put(unsigned char* to, int f, const Frag<P>& v) const {
#pragma unroll
    for (int p = 0; p < P; ++p) *(u32x4*)(to + (f * P + p) * 1024 + lane * 16) = v.p[p];
  }

  template <int W, int KS>
  __device__ __forceinline__ void column() const {
    constexpr int kRows = 4 * KS * PI * 1024, M = 4 - W;   // row tiles W .. 3
    const int row = lane & 15, gq = lane >> 4;
    float* s_n = (float*)s_all;
    float* s_t = s_n + 10 * 320;
    const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
    v4f kk[M], qk[M];      // K_i K_W^T and Q_i K_W^T
#pragma unroll
    for (int i = 0; i < M; ++i) kk[i] = qk[i] = zero;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const Frag<PI> kw = lds_frag<PI>(s_all, W * KS + s, lane);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        kk[i] = mma<PI, PI>(i == 0 ? kw : lds_frag<PI>(s_all, (W + i) * KS + s, lane), kw, kk[i]);
        if (WANTP) qk[i] = mma<PI, PI>(lds_frag<PI>(s_all + kRows, (W + i) * KS + s, lane), kw, qk[i]);
      }
    }
    const double cc = s_cum[16 * W + row];
    const float bc = s_b[16 * W + row];
    __syncthreads();                 // K and Q have been read: their place is N's and T's
    v4f n, nt;                       // N_WW and its transpose
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 4 * gq + r;
        float d = (float)(s_cum[16 * (W + i) + m] - cc);
        if (i == 0) d = m < row ? -d : d;            // the transpose's above the diagonal
        const float dec = __builtin_amdgcn_exp2f(d), f = dec * kk[i][r];
        const float bm = s_b[16 * (W + i) + m];
        qk[i][r] = i > 0 || m >= row ? dec * qk[i][r] : 0.f;
        if (i == 0) {
          n[r] = m > row ? -(bm * f) : 0.f;
          nt[r] = m < row ? -(bc * f) : 0.f;
        } else {
          s_n[lds_tile(W + i, W) + m * 20 + row] = -(bm * f);
        }
      }
    // T_WW = (I - N)^-1. N = D + E, D its 4 x 4 tiles on the diagonal: (I - D)^-1 = (I + D)(I + D^2) =: T_D,
    // then T = T_D + F T, F = T_D E, three times from T_D. Entries of T_D, F and T are at most 1 for keys of
    // length 1; powers of all of N have binomial coefficients (3432 in N^8 where keys repeat), which cancel.
    const bool own = gq == row >> 2;
    v4f t, tt, e;                    // I + D, its transpose and E
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float one = 4 * gq + r == row ? 1.f : 0.f;
      e[r] = own ? 0.f : n[r];
      n[r] = own ? n[r] : 0.f;
      nt[r] = own ? nt[r] : 0.f;
      t[r] = one + n[r];
      tt[r] = one + nt[r];
    }
    const v4f n2t = mm16(n, nt, zero), td = mm16(n2t, t, t), tdt = mm16(t, n2t, tt);
    const v4f ft = mm16(e, tdt, zero);
    t = td;
#pragma unroll
    for (int k = 0; k < 3; ++k) t = mm16(ft, t, td);
#pragma unroll
    for (int r = 0; r < 4; ++r) s_t[lds_tile(W, W) + (4 * gq + r) * 20 + row] = t[r];
    __syncthreads();
    v4f col[M];
    col[0] = t;
#pragma unroll
    for (int i = 1; i < M; ++i) {
      v4f y = zero;
#pragma unroll
      for (int k = 0; k < i; ++k)
        y = mm16(*(const v4f*)&s_n[lds_tile(W + i, W + k) + row * 20 + 4 * gq], col[k], y);
      col[i] = mm16(*(const v4f*)&s_t[lds_tile(W + i, W + i) + row * 20 + 4 * gq], y, zero);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) col[i] *= bc;
    if (MODE == kPrepBackward) {     // results one above the other: operands of the transposes
#pragma unroll
      for (int s = W / 2; s < 2; ++s) {
        const bool odd = 2 * s < W;  // the upper tile lies above the diagonal
        put<3>(Tt_, trit_frag(W, s), above(odd ? zero : col[odd ? 0 : 2 * s - W], col[2 * s + 1 - W]));
        put<3>(Pt_, trit_frag(W, s), above(odd ? zero : qk[odd ? 0 : 2 * s - W], qk[2 * s + 1 - W]));
      }
    }
    __syncthreads();                 // N and the diagonal tiles have been read
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s_t[lds_tile(W + i, W) + (4 * gq + r) * 20 + row] = col[i][r];
        if (MODE == kPrepForward) s_n[lds_tile(W + i, W) + (4 * gq + r) * 20 + row] = qk[i][r];
      }
    __syncthreads();
    constexpr int PT = MODE == kPrepBackward ? PM : 3;
    auto rows_of = [&](const float* m, int s, float (&v)[8]) {   // row tile W, terms 32 s ..
      const v4f x = *(const v4f*)&m[lds_tile(W, 2 * s) + row * 20 + 4 * gq];
      v4f y = zero;
      if (2 * s + 1 <= W) y = *(const v4f*)&m[lds_tile(W, 2 * s + 1) + row * 20 + 4 * gq];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = x[j], v[4 + j] = y[j];
    };
#pragma unroll
    for (int s = 0; 2 * s <= W; ++s) {
      float v[8];
      rows_of(s_t, s, v);
      put<PT>(T_, tri_frag(W, s), packed<PT>(v));
      if (MODE == kPrepForward) {
        rows_of(s_n, s, v);
        put<PM>(P_, tri_frag(W, s), packed<PM>(v));
      }
    }
  }
};

template <typename T, int DK, bool VEC, DeltaPrep MODE>
__global__ void __launch_bounds__(256, (DeltaType<T, VEC>::PI == 1 ? 4 : DK < 128 ? 2 : 1)) k_delta_prep(DeltaArgs a) {
  using Ty = DeltaType<T, VEC>;
  constexpr int PI = Ty::PI, KS = DK / 32;
  constexpr bool WANTP = MODE != kPrepStates;
  constexpr int kRows = 4 * KS * PI * 1024;               // K (or Q) as operands
  constexpr int kMats = 2 * 10 * 320 * 4;                 // N below the diagonal (then P), and T
  constexpr int kShared = (WANTP ? 2 : 1) * kRows > kMats ? (WANTP ? 2 : 1) * kRows : kMats;
  __shared__ double s_cum[kDeltaChunk];
  __shared__ float s_b[kDeltaChunk];
  __shared__ __attribute__((aligned(16))) unsigned char s_all[kShared];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, gq = lane >> 4;
  const int ch = blockIdx.x, bh = ch / a.chunks, c = ch - bh * a.chunks;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const DeltaSeq sq = delta_seq(a, b);
  if (c * kDeltaChunk >= sq.n) return;
  const DeltaRows rows = delta_rows(sq, c);
  const size_t low = delta_low(a, sq, b, c);
  const auto kbuf = delta_buf((const T*)a.k + (low * a.Hk + hk) * a.dk);
  const auto qbuf = delta_buf((const T*)a.q + (low * a.Hk + hk) * a.dk);

  // each wave's 16 rows of K and Q, shared as operands
  {
    const uint32_t off = rows.off(16 * w + row, (uint32_t)(a.Hk * a.dk) * sizeof(T));
    Raw8<T, VEC> kr[KS], qr[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) kr[s] = raw8<T, VEC>(kbuf, off, 32 * s + 8 * gq, a.dk);
    if (WANTP)
#pragma unroll
      for (int s = 0; s < KS; ++s) qr[s] = raw8<T, VEC>(qbuf, off, 32 * s + 8 * gq, a.dk);
    auto share = [&](const Raw8<T, VEC> (&r)[KS], unsigned char* to) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Half<PI> lo, hi;
        halves<PI>(r[s], lo, hi);
        const Frag<PI> f = join<PI>(lo, hi);
#pragma unroll
        for (int p = 0; p < PI; ++p)
          *(u32x4*)(to + ((w * KS + s) * PI + p) * 1024 + slot(lane) * 16) = f.p[p];
      }
    };
    // gates, by the wave that has the fewest products below: lane = step. log a = min(g, 0) - log(1 +
    // exp(-|g|)), g held to [-87, 87] (NaN passes)
    if (w == 3) {
      const uint32_t goff = rows.off(lane, (uint32_t)a.H * sizeof(T));
      float g = wide(buf_load<T>(delta_buf((const T*)a.g + low * a.H + h), goff));
      const float x = wide(buf_load<T>(delta_buf((const T*)a.beta + low * a.H + h), goff));
      g = __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -87.f), 87.f);
      const float e = expf(-fabsf(g));
      const float la = fminf(g, 0.f) - log1pf(e);
      const bool live = rows.live(lane);
      const float be = live ? 1.f / (1.f + expf(-x)) : 0.f;
      double cum = live ? (double)(g == g ? la : g) * 1.4426950408889634 : 0.0;   // base 2
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double o = __shfl_up(cum, d);
        cum += lane >= d ? o : 0.0;
      }
      s_cum[lane] = cum;
      s_b[lane] = be;
      DeltaGates& gt = a.gates[ch];
      gt.cum[lane] = cum;
      gt.gam[lane] = __builtin_amdgcn_exp2f((float)cum);
      gt.end[lane] = __builtin_amdgcn_exp2f((float)(__shfl(cum, 63) - cum));
      const float f = expf(-fabsf(x));
      gt.nb[lane] = live ? (x > 0.f ? f : 1.f) / (1.f + f) : 0.f;
      gt.na[lane] = live ? (g > 0.f ? e : 1.f) / (1.f + e) : 0.f;
    }
    share(kr, s_all);
    if (WANTP) share(qr, s_all + kRows);
  }
  __syncthreads();

  DeltaOwn<T, MODE> own{s_all, s_cum, s_b, lane};
  own.T_ = a.T + ch * delta_t_bytes(PI == 1, MODE == kPrepBackward);
  own.P_ = a.P + ch * delta_p_bytes(PI == 1);
  own.Tt_ = a.Tt + ch * kDeltaTtBytes;
  own.Pt_ = a.Pt + ch * kDeltaTtBytes;
  if (w == 0) own.template column<0, KS>();
  else if (w == 1) own.template column<1, KS>();
  else if (w == 2) own.template column<2, KS>();
  else own.template column<3, KS>();
}

// ---------------------------------------------------------------------------- the walk
// One workgroup per head and NC tiles of 16 columns of dv, of 8 waves: the first four walk the state along the chunks,
// wave w with row tile w of the 64 steps and OWN of the state's row tiles; the other four fetch K for
// them, one chunk ahead, and form the outputs. Three hand-overs per chunk, each through LDS:
//        walkers                                    helpers
//   A    X = V - diag(y) K S                        Q S
//   B    U = T X                                    K of the next chunk
//   C    S = y_C S + K^T diag(y_C / y) U            o = scale (diag(y) Q S + P U)
// Loads are issued a chunk before their use, right after the last use of their registers.
// Bound by the length of a chunk's chain: three LDS round trips, four products one after the other and three
// splittings into bf16 parts, 1.9 to 2.2 us a chunk of which loads that always hit would save 0.1. So 4 x 8 heads of
// 128 over 8192 steps (128 chunks, one workgroup a CU) take 284 us, a single head 238; 192 heads of 64 over
// 784 steps 50, with one tile a workgroup 55 to 60. With o from two parts of S, U and P, which lose what a bf16 o shows
// where a key is overwritten, these were 245, 207 and 43.5 (the helpers' products and LDS reads); Q S over two phases,
// U shared in fp32 and parted by the helpers, or P parted a phase earlier gain nothing. K S formed from a walker's own rows
// of S and K from registers, the parts joined in LDS, measured 183 for 207, but 250 to 260 for the 4 x 8's 245.
// LDS of a workgroup. Two chunks' K^T, where they fit (all but fp32 with 96 < dk): the next one is then
// written while this one is read, and K is loaded a whole chunk ahead.
template <typename T, int DK, int NC>
struct WalkLds {
  static constexpr int PI = DeltaType<T, true>::PI, KS = DK / 32;
  static constexpr int rows = 4 * KS * PI * 1024, cols = (DK / 16) * kTileBytes<PI>;
  static constexpr int rest = NC * (KS * 3 + 18) * 1024 + rows;
  static constexpr bool two = rest + 2 * cols <= 160 * 1024;
  static constexpr int bytes = rest + (two ? 2 : 1) * cols;
};

template <typename T, int DK, bool VEC, bool OUT, int NC>
__global__ void __launch_bounds__(512, (NC == 2 && DK <= 64 && DeltaType<T, VEC>::PI == 1 ? 4 : 2)) k_delta_walk(DeltaArgs a) {
  using Ty = DeltaType<T, VEC>;
  constexpr int PI = Ty::PI, PM = Ty::PM, KS = DK / 32, NT = DK / 16, OWN = (NT + 3) / 4;
  constexpr bool TWO = WalkLds<T, DK, NC>::two;
  constexpr int kRows = WalkLds<T, DK, NC>::rows, kCols = TWO ? WalkLds<T, DK, NC>::cols : 0;
  constexpr int kS = KS * 3 * 1024, kX = 2 * 3 * 1024;   // of a column tile
  extern __shared__ __attribute__((aligned(16))) unsigned char sm[];
  unsigned char* const s_s = sm;                          // the state
  unsigned char* const s_x = s_s + NC * kS;               // X
  unsigned char* const s_e = s_x + NC * kX;               // diag(y_C / y) U
  unsigned char* const s_u = s_e + NC * kX;               // U
  unsigned char* const s_k = s_u + NC * kX;               // K, and K^T
  unsigned char* const s_kt = s_k + kRows;
  const DeltaWalkAt at = delta_walk_at((a.dv + 16 * NC - 1) / (16 * NC));
  const int bh = at.bh;
  if (bh >= a.B * a.H) return;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wid & 3, row = lane & 15, gq = lane >> 4;
  const bool walker = wid < 4;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.rep;
  const DeltaSeq sq = delta_seq(a, b);
  const int col = at.tile * (16 * NC) + row;     // NC = 2: and the 16th after it
  const bool in = col < a.dv;
  const int nch = (sq.n + kDeltaChunk - 1) / kDeltaChunk, endc = nch - 1;
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  const uint32_t kstride = (uint32_t)(a.Hk * a.dk) * sizeof(T), vstride = (uint32_t)(a.H * a.dv) * sizeof(T);
  const size_t sdim = (size_t)a.dk * a.dv;
  // T and P of row tiles 0 and 1 have terms below 32 only: they load the first frag twice, as loads in a
  // branch would make every wait for an older one wait for them all
  const int second = w >= 2 ? 1 : 0;
  // this lane's entries of V and o, as a result lies; rows past a last chunk's end: nowhere
  auto value_offsets = [&](const DeltaRows& rows, uint32_t (&off)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      off[r] = in ? rows.off(16 * w + 4 * gq + r, vstride) + col * sizeof(T) : kNowhere;
  };

  if (walker) {
    v4f S[NC][OWN];
    uint32_t soff[OWN][4], voff[4];
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = walk_entry(w * OWN + i, 4 * gq + r);
        const bool own = w * OWN + i < NT && k < a.dk && in;
        soff[i][r] = own ? (uint32_t)(k * a.dv + col) * 4 : kNowhere;
#pragma unroll
        for (int n = 0; n < NC; ++n)
          S[n][i][r] = a.s0 ? buf_load<float>(delta_buf(a.s0 + bh * sdim), soff[i][r] + 64 * n) : 0.f;
      }
    auto put_state = [&](float* to) {
      const auto buf = delta_buf(to);
#pragma unroll
      for (int i = 0; i < OWN; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int n = 0; n < NC; ++n) buf_store(buf, soff[i][r] + 64 * n, S[n][i][r], 0.f);
    };
    auto share_state = [&] {
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const int tile = w * OWN + i;
        if (tile < NT)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            lds_half<3>(s_s + n * kS, tile >> 1, lane, tile & 1,
                        split4<3>(S[n][i][0], S[n][i][1], S[n][i][2], S[n][i][3]));
      }
    };
    Frag<3> t[2];
    uint32_t v[NC][4];
    v4f gam, end;
    float last = 1.f;
    auto load_v = [&](int c) {
      if (c == endc) value_offsets(delta_rows(sq, c), voff);
      const auto vbuf = delta_buf((const T*)a.v + (delta_low(a, sq, b, c) * a.H + h) * a.dv);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < NC; ++n) v[n][r] = raw1<T>(vbuf, voff[r] + 16 * n * sizeof(T));
      gam = *(const v4f*)&a.gates[(size_t)bh * a.chunks + c].gam[16 * w + 4 * gq];
    };
    auto load_t = [&](int c) {
      const size_t ch = (size_t)bh * a.chunks + c;
      const unsigned char* Tm = a.T + ch * delta_t_bytes(PI == 1, false);
      t[0] = mem_frag<3>(Tm, tri_frag(w, 0), lane);
      t[1] = mem_frag<3>(Tm, tri_frag(w, second), lane);
      end = *(const v4f*)&a.gates[ch].end[16 * w + 4 * gq];
    };
    auto load_last = [&](int c) {
      last = a.gates[(size_t)bh * a.chunks + c].gam[kDeltaChunk - 1];
    };
    if (nch > 0) {
      value_offsets(delta_rows(sq, 0), voff);
      load_v(0);
      load_t(0);
      load_last(0);
    }
    share_state();
    __syncthreads();
    for (int c = 0; c < nch; ++c) {
      const int next = c < endc ? c + 1 : c;
      if (a.states) put_state(a.states + ((size_t)bh * a.chunks + c) * sdim);
      v4f kp[NC][KS];                // a chain of products for each 32 terms
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<PI> kf = lds_frag<PI>(s_k, w * KS + s, lane);
#pragma unroll
        for (int n = 0; n < NC; ++n) kp[n][s] = mma<PI, 3>(kf, lds_frag<3>(s_s + n * kS, s, lane), zero);
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        v4f ks = zero;
#pragma unroll
        for (int s = 0; s < KS; ++s) ks += kp[n][s];
        lds_half<3>(s_x + n * kX, w >> 1, lane, w & 1,
                    split4<3>(wide1<T>(v[n][0]) - gam[0] * ks[0], wide1<T>(v[n][1]) - gam[1] * ks[1],
                              wide1<T>(v[n][2]) - gam[2] * ks[2], wide1<T>(v[n][3]) - gam[3] * ks[3]));
      }
      load_v(next);
      __syncthreads();
      v4f u[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) u[n] = mma_short(t[0], lds_frag<3>(s_x + n * kX, 0, lane));
      if (w >= 2)
#pragma unroll
        for (int n = 0; n < NC; ++n) u[n] += mma_short(t[1], lds_frag<3>(s_x + n * kX, 1, lane));
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        lds_half<3>(s_e + n * kX, w >> 1, lane, w & 1,
                    split4<3>(end[0] * u[n][0], end[1] * u[n][1], end[2] * u[n][2], end[3] * u[n][3]));
        if constexpr (OUT)
          lds_half<3>(s_u + n * kX, w >> 1, lane, w & 1, split4<3>(u[n][0], u[n][1], u[n][2], u[n][3]));
      }
      load_t(next);
      __syncthreads();
      const unsigned char* kt = s_kt + (c & 1) * kCols;
      v4f more[NC][OWN];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < OWN; ++i) S[n][i] *= last, more[n][i] = zero;
      load_last(next);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<3> e[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) e[n] = lds_frag<3>(s_e + n * kX, s, lane);
#pragma unroll
        for (int i = 0; i < OWN; ++i)
          if (w * OWN + i < NT) {
            const Frag<PI> kf = lds_frag<PI>(kt + (w * OWN + i) * kTileBytes<PI>, s, lane);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              v4f& to = s ? more[n][i] : S[n][i];
              to = mma<PI, 3>(kf, e[n], to);
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < OWN; ++i) S[n][i] += more[n][i];
      share_state();
      __syncthreads();
    }
    if (a.s_last) put_state(a.s_last + bh * sdim);
    if (a.states)
      for (int c = nch; c < a.chunks; ++c) put_state(a.states + ((size_t)bh * a.chunks + c) * sdim);
  } else {
    const int id = threadIdx.x - 256, dg = id % (DK / 8), tg = id / (DK / 8);
    const bool block = tg < 16;      // a 4 x 8 block of K
    Raw8<T, VEC> kb[4], q[OUT ? KS : 1];
    Frag<PM> p[2];
    v4f gam = zero;
    uint32_t boff[4], qoff = 0, ooff[4];
    auto block_offsets = [&](const DeltaRows& rows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) boff[j] = block ? rows.off(4 * tg + j, kstride) : kNowhere;
    };
    auto load_k = [&](int c) {
      if (c == endc) block_offsets(delta_rows(sq, c));
      const auto kbuf = delta_buf((const T*)a.k + (delta_low(a, sq, b, c) * a.Hk + hk) * a.dk);
#pragma unroll
      for (int j = 0; j < 4; ++j) kb[j] = raw8<T, VEC>(kbuf, boff[j], 8 * dg, a.dk);
    };
    auto share_k = [&](int c, bool as_rows, bool as_cols) {
      Half<PI> lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) halves<PI>(kb[j], lo[j], hi[j]);
      if (block && as_rows) lds_rows<PI, KS>(s_k, tg, dg, lo, hi);
      if (block && as_cols) lds_cols<PI>(s_kt + (c & 1) * kCols, tg, dg, lo, hi);
    };
    auto load_q = [&](int c) {
      if constexpr (OUT) {
        if (c == endc) qoff = delta_rows(sq, c).off(16 * w + row, kstride);
        const auto qbuf = delta_buf((const T*)a.q + (delta_low(a, sq, b, c) * a.Hk + hk) * a.dk);
#pragma unroll
        for (int s = 0; s < KS; ++s) q[s] = raw8<T, VEC>(qbuf, qoff, 32 * s + 8 * gq, a.dk);
      }
    };
    auto load_p = [&](int c) {
      if constexpr (OUT) {
        const size_t ch = (size_t)bh * a.chunks + c;
        const unsigned char* Pm = a.P + ch * delta_p_bytes(PI == 1);
        p[0] = mem_frag<PM>(Pm, tri_frag(w, 0), lane);
        p[1] = mem_frag<PM>(Pm, tri_frag(w, second), lane);
        gam = *(const v4f*)&a.gates[ch].gam[16 * w + 4 * gq];
      }
    };
    if (nch > 0) {
      block_offsets(delta_rows(sq, 0));
      load_k(0);
      qoff = delta_rows(sq, 0).off(16 * w + row, kstride);
      value_offsets(delta_rows(sq, 0), ooff);
      load_q(0);
      load_p(0);
      share_k(0, true, TWO);
      if (TWO) load_k(endc > 0 ? 1 : 0);
    }
    __syncthreads();
    for (int c = 0; c < nch; ++c) {
      const int next = c < endc ? c + 1 : c;
      v4f qs[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) qs[n] = zero;
      if constexpr (OUT) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          Half<PI> lo, hi;
          halves<PI>(q[s], lo, hi);
#pragma unroll
          for (int n = 0; n < NC; ++n)
            qs[n] = mma<PI, 3>(join<PI>(lo, hi), lds_frag<3>(s_s + n * kS, s, lane), qs[n]);
        }
      }
      load_q(next);
      if (!TWO) {
        share_k(c, false, true);
        load_k(next);
      }
      __syncthreads();
      share_k(c + 1, true, TWO);     // this chunk's rows have been read
      if (TWO) load_k(c + 2 < nch ? c + 2 : endc);
      __syncthreads();
      if constexpr (OUT) {
        v4f pu[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) pu[n] = mma<3, 3>(parts(p[0]), lds_frag<3>(s_u + n * kX, 0, lane), zero);
        if (w >= 2)
#pragma unroll
          for (int n = 0; n < NC; ++n) pu[n] = mma<3, 3>(parts(p[1]), lds_frag<3>(s_u + n * kX, 1, lane), pu[n]);
        if (c == endc) value_offsets(delta_rows(sq, c), ooff);
        const auto obuf = delta_buf((T*)a.o + (delta_low(a, sq, b, c) * a.H + h) * a.dv);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            buf_store(obuf, ooff[r] + 16 * n * sizeof(T), a.scale * fmaf(gam[r], qs[n][r], pu[n][r]), T());
        load_p(next);
      }
      __syncthreads();
    }
    if (OUT && in)
      for (int t = sq.n + (id >> 4); t < a.L; t += 16)
#pragma unroll
        for (int n = 0; n < NC; ++n)
          put1((T*)a.o + (((size_t)b * a.L + t) * a.H + h) * a.dv + col + 16 * n, 0.f);
  }
}
// ---------------------------------------------------------------------------- single steps
// One launch, S in registers; a step is two sums across the wave one after the other, 0.9 us (1.1 with dk = 128).
// 48 heads of 64 x 64, one step: 5.1 us; 2048 heads of 128 x 128 118 us, 2.3 TB/s, 44 % of what a copy reaches: S comes
// and goes in 64-byte pieces of its rows by accesses of 4 bytes.
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

// Longest sequences that go step by step. A step adds 0.9 to 1.1 us to one launch, a chunk costs two launches
// whatever its length. us for 4, 8 and 12 steps, chunks: 64 x 3 heads of 64 8.9, 12.3, 16.0, 14.0; 8 x 6 of them
// 7.3, 10.7, 14.4, 10.5; 8 x 8 heads of 128 11.3, 16.1, 20.7, 14.0, 256 x 8 of them 130, 154, 182, 214.
constexpr int kDeltaSteps = 8;

int64_t chunks_of(int64_t L) { return (L + kDeltaChunk - 1) / kDeltaChunk; }

template <typename T, DeltaPrep MODE>
void prep_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  with_dk(a.dk, vec, [&](auto d, auto v) {
    k_delta_prep<T, decltype(d)::value, decltype(v)::value, MODE>
        <<<dim3(a.B * a.H * a.chunks), 256, 0, st>>>(a);
  });
}
template <typename T>
void prep_mode(const DeltaArgs& a, bool vec, DeltaPrep mode, hipStream_t st) {
  if (mode == kPrepForward) prep_t<T, kPrepForward>(a, vec, st);
  else if (mode == kPrepStates) prep_t<T, kPrepStates>(a, vec, st);
  else prep_t<T, kPrepBackward>(a, vec, st);
}
template <typename T, int DK, bool VEC, bool OUT, int NC>
hipError_t walk_one(const DeltaArgs& a, hipStream_t st) {
  constexpr int bytes = WalkLds<T, DK, NC>::bytes;
  static_assert(bytes <= 160 * 1024, "LDS of a CU");
  const dim3 grid = delta_walk_grid(a, (a.dv + 16 * NC - 1) / (16 * NC));
  const hipError_t e = hipFuncSetAttribute((const void*)k_delta_walk<T, DK, VEC, OUT, NC>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  k_delta_walk<T, DK, VEC, OUT, NC><<<grid, 512, bytes, st>>>(a);
  return hipGetLastError();
}
template <typename T>
hipError_t walk_t(const DeltaArgs& a, bool vec, hipStream_t st) {
  const bool two = walk_two_tiles_forward(a, sizeof(T) == 2);
  hipError_t e = hipSuccess;
  with_dk(a.dk, vec, [&](auto d, auto v) {
    constexpr int DK = decltype(d)::value;
    constexpr bool VEC = decltype(v)::value;
    if constexpr (VEC) {
      if (two) {
        e = a.o ? walk_one<T, DK, VEC, true, 2>(a, st) : walk_one<T, DK, VEC, false, 2>(a, st);
        return;
      }
    }
    e = a.o ? walk_one<T, DK, VEC, true, 1>(a, st) : walk_one<T, DK, VEC, false, 1>(a, st);
  });
  return e;
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
  return a;
}

bool delta_vec(const DeltaRequest& r) {
  const uintptr_t m = 15;
  auto al = [](const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) == 0; };
  return r.dk % 8 == 0 && r.dv % 4 == 0 && al(r.q, m) && al(r.k, m) && al(r.v, m) &&
         al(r.dout, m) && al(r.states, 15);
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool bf16, bool vec, DeltaPrep mode, hipStream_t st) {
  if (bf16) prep_mode<uint16_t>(a, vec, mode, st);
  else prep_mode<float>(a, vec, mode, st);
  return hipGetLastError();
}
hipError_t launch_delta_walk(const DeltaArgs& a, bool bf16, bool vec, hipStream_t st) {
  return bf16 ? walk_t<uint16_t>(a, vec, st) : walk_t<float>(a, vec, st);
}

namespace {

struct FwdWs {
  size_t P, gates, total;
};
FwdWs fwd_ws(int64_t B, int64_t L, int H, bool bf16) {
  const size_t n = (size_t)B * H * chunks_of(L);
  FwdWs w;
  w.P = n * delta_t_bytes(bf16, false);
  w.gates = w.P + n * delta_p_bytes(bf16);
  w.total = w.gates + n * sizeof(DeltaGates);
  return w;
}

}  // namespace

size_t delta_forward_workspace(int64_t B, int64_t L, int H, bool bf16) {
  return L <= kDeltaSteps ? 0 : fwd_ws(B, L, H, bf16).total;
}

hipError_t launch_delta_forward(const DeltaRequest& r, hipStream_t st) {
  DeltaArgs a = delta_args(r);
  if (r.L <= kDeltaSteps) {
    if (r.bf16) step_t<uint16_t>(a, st);
    else step_t<float>(a, st);
    return hipGetLastError();
  }
  const FwdWs w = fwd_ws(r.B, r.L, r.H, r.bf16);
  unsigned char* ws = (unsigned char*)r.ws;
  a.T = ws;
  a.P = ws + w.P;
  a.gates = (DeltaGates*)(ws + w.gates);
  const bool vec = delta_vec(r);
  const hipError_t e = launch_delta_prep(a, r.bf16, vec, kPrepForward, st);
  return e != hipSuccess ? e : launch_delta_walk(a, r.bf16, vec, st);
}

}  // namespace wbmm
