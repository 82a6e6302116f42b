// Gated delta rule: a recurrence whose state is a matrix S (dk x dv) for every head of a sequence,
//   S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = scale S_t^T q_t,
//   a_t = sigmoid(g_t),   b_t = sigmoid(beta_t).
//
// In chunks of C = 64 steps, with S0 the state before the chunk, y_i = a_1 ... a_i, K, Q, V the
// chunk's rows and u_i = b_i (v_i - a_i S_{i-1}^T k_i) what step i adds (S_i = a_i S_{i-1} + k_i u_i^T):
//   A_ij = b_i (y_i / y_j) k_i.k_j (j < i),   P_ij = (y_i / y_j) q_i.k_j (j <= i),   T = (I + A)^-1 diag(b),
//   U = T (V - diag(y) K S0),   o = scale (diag(y) Q S0 + P U),   S_C = y_C S0 + sum_j (y_C / y_j) k_j u_j^T.
// A, P and T depend on no state: one launch forms them for all chunks at once. What is left for the
// walk along the chunks are products of 64 x dk, 64 x 64 and dk x 64 matrices with 64 or dk x dv ones,
// and every column of S, U and o goes its own way: 16 columns are a workgroup's.
//
// Backward, with D the gradient of the state after a chunk and G = scale do:
//   dU = P^T G + diag(y_C / y) K D,   R = T^T dU = dv,   D0 = y_C D + Q^T diag(y) G - K^T diag(y) R,
// again a walk over columns (last chunk to first); then, for all chunks at once,
//   dP = (G U^T) . (y_i / y_j) (j <= i),   N = -(R U^T) . (y_i / y_j) (j < i),
//   dq = diag(y) G S0^T + dP K,   row = N K - diag(y) R S0^T,
//   col = dP^T Q + N^T K + diag(y_C / y) U D^T,   dk = row + col.
// y_i enters o, A and P as a factor of q_i, of k_i as the row of A, and as 1 / y_j of k_j elsewhere, b_i
// as a factor of k_i's row and of v_i. So the gradients of the gates are dot products of rows,
//   d log y_i = q_i.dq_i + k_i.row_i - k_i.col_i  (+ <S_C, D> for the last),
//   d log a_t = sum_{i >= t} d log y_i,   dg = (1 - a) d log a,   dbeta = (1 - b)(v.R + k.row).
//
// Products run on the bf16 matrix cores at fp32 accuracy. An fp32 number is the sum of three bf16
// numbers to 2^-25, so the states, T, X, U and D are taken in three parts and the products that matter
// (up to 2^-24) are formed; bf16 tensors are one part as they are, so that a bf16 call gives what the fp32 call of the
// same values gives, rounded. Sums are fp32, running sums of
// log a and of d log y fp64.
//
// Layouts. v_mfma_f32_16x16x32_bf16: with l the lane, an A operand is row l % 16 and 8 terms of the sum, a
// B operand column l % 16 and the same 8, a result column l % 16 and rows 4 (l / 16) + r. The order of
// the terms is free where A and B agree: slot j of lane group q stands for term 4 q + j of the first
// 16 (j < 4) or second 16 (j >= 4) of 32. Then two results on top of each other are a B operand as they lie
// in the registers, and two side by side a transposed A operand: "frag" below is such an operand, 64
// lanes of 16 bytes for each part.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wbmm {

constexpr int kDeltaChunk = 64;
constexpr int kDeltaFrags = 6;               // operands of a triangular 64 x 64 matrix, 1024 bytes a part

struct DeltaRequest {
  int64_t B, L;
  int Hk, H, dk, dv, bf16, reverse;
  float scale;
  const void *q, *k, *v, *g, *beta, *dout;
  const float* s0;
  const float* ds_last;
  const int32_t* lens;
  void* o;
  float* s_last;
  float* states;               // written by the forward, read by the backward (null: formed again)
  void *dq, *dkey, *dval, *dg, *dbeta;
  float* ds0;
  void* ws;
};

size_t delta_forward_workspace(int64_t B, int64_t L, int H, bool bf16);
size_t delta_backward_workspace(int64_t B, int64_t L, int H, int dk, int dv, bool bf16, bool has_states);
hipError_t launch_delta_forward(const DeltaRequest& r, hipStream_t st);
hipError_t launch_delta_backward(const DeltaRequest& r, hipStream_t st);

// The gates of a chunk: log2 y (fp64), y, y_C / y, 1 - b and 1 - a (each from its own exponential: b and a are 1 to
// all their bits long before these are 0).
struct DeltaGates {
  double cum[kDeltaChunk];
  float gam[kDeltaChunk], end[kDeltaChunk], nb[kDeltaChunk], na[kDeltaChunk];
};

struct DeltaArgs {
  const void *q, *k, *v, *g, *beta, *dout;
  const float* s0;
  const float* ds_last;
  const int32_t* lens;
  void* o;
  float* s_last;
  float* states;
  void *dq, *dkey, *dval, *dg, *dbeta;
  float* ds0;
  // per chunk of a head, kDeltaFrags operands each: T and P for the walk along the chunks, T for the
  // gradients, the transposes for the walk back
  unsigned char *T, *P, *Tt, *Pt;
  DeltaGates* gates;           // [B H chunks]
  float* D;                    // [B H chunks][dk][dv]
  float* R;                    // [B H chunks][64][dv]
  int B, L, Hk, H, dk, dv, rep, chunks, reverse;
  float scale;
};

// What of a chunk's own matrices a launch of launch_delta_prep forms.
enum DeltaPrep { kPrepForward, kPrepStates, kPrepBackward };
// Bytes per chunk of a head: the walk's T and the transposes in three parts; P, which the walk's helpers have the time
// to part, and the gradients' T in three or, for bf16 tensors, in fp32 (12 KB for 18).
constexpr size_t delta_t_bytes(bool bf16, bool backward) {
  return (size_t)kDeltaFrags * 1024 * (bf16 && backward ? 2 : 3);
}
constexpr size_t delta_p_bytes(bool bf16) { return (size_t)kDeltaFrags * 1024 * (bf16 ? 2 : 3); }
constexpr size_t kDeltaTtBytes = (size_t)kDeltaFrags * 1024 * 3;

DeltaArgs delta_args(const DeltaRequest& r);
// Tiles of 16 columns that a workgroup of the walks takes. More than one share its operands (K, T and P in registers
// and LDS) and fill each other's waits; they pay where tiles outnumber the CUs. us of whole calls over 512 steps, dv = 64,
// one against two tiles, forward and backward: bf16, dk = 64, 640 tiles 50.1, 122.9 against 46.9, 122.7, 1024 62.3,
// 188.7 against 54.0, 175.5; 288 34.6, 80.0 against 34.9, 73.5; fp32 288 56.1, 122.8 against 42.4, 104.9, 1024
// 117.1, 309.9 against 90.4, 276.1. Up to 256 tiles one each is the shorter walk: bf16, dk = 64, 256 tiles 28.5, 54.9
// against 34.0, 62.0.
// The forward of bf16 with dk > 64 has two workgroups of one tile on a CU, or one of two: there two tiles pay where each
// has a CU of its own (512 tiles of dv = 128: 43.2 for 44.8) and, with the rounds' ends, from 2.75 rounds of them on (1408
// tiles of 64 127.0 for 136.4, of 128 107.4 for 106.4; 2048 180.8 for 210.3, 145.8 for 154.8), not in between (640 77.8 for
// 67.0, 69.7 for 58.8; 1280 122.7 for 120.2, 105.7 for 94.7).
// The backward, of which a CU holds one workgroup, takes four where two do not fit a round and LDS has room (bf16
// with dk <= 64, fp32 with dk <= 32): bf16, dk = 64, four against two: 512 tiles 98.1 against 87.4, 640 114.4 against 122.7,
// 2048 345 against 374; fp32, dk = 32, 512 117.2 against 106.8, 640 136.4 against 157.6.
constexpr int64_t kDeltaCus = 256;         // of the chip
inline int64_t walk_tiles(const DeltaArgs& a) { return (int64_t)a.B * a.H * (a.dv / 16); }
inline bool walk_two_tiles(const DeltaArgs& a) { return a.dv % 32 == 0 && walk_tiles(a) > kDeltaCus; }
inline bool walk_four_tiles(const DeltaArgs& a) { return a.dv % 64 == 0 && walk_tiles(a) > 2 * kDeltaCus; }
inline bool walk_two_tiles_forward(const DeltaArgs& a, bool bf16) {
  const int64_t groups = ((int64_t)a.B * a.H + 7) / 8 * 8 * (a.dv / 32);   // as launched, whole octets of heads
  return walk_two_tiles(a) && (!bf16 || a.dk <= 64 || groups <= kDeltaCus || 4 * groups >= 11 * kDeltaCus);
}
hipError_t launch_delta_prep(const DeltaArgs& a, bool bf16, bool vec, DeltaPrep mode, hipStream_t st);
hipError_t launch_delta_walk(const DeltaArgs& a, bool bf16, bool vec, hipStream_t st);
// 16 bytes at a time of everything that lies in rows of dk or dv.
bool delta_vec(const DeltaRequest& r);

}  // namespace wbmm
