// Gated linear recurrence: how a call is laid out, from its sizes alone (host code, shared by the
// forward and the backward).
#include "wbmm_scanplan.hpp"

#include <algorithm>

namespace wbmm {

static int scan_pow2(long long v) {  // least power of two >= v, at least 1
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Waves of a workgroup, at most `most`, for an axis of `pieces` wave pieces: enough to put 4096
// waves on the chip with `units` workgroups, then (down to half of that) the count whose tiles fit
// the axis best.
static int scan_waves(long long units, long long pieces, int least, int most) {
  const long long want = (4096 + units - 1) / units;
  int hi = (int)std::max<long long>(least, std::min<long long>({want, pieces, (long long)most}));
  int best = hi;
  double score = 0;
  for (int n = hi; n >= std::max(least, (hi + 1) / 2); --n) {
    const double fit = (double)pieces / (double)((pieces + n - 1) / n * n);
    if (fit > score + 0.02) score = fit, best = n;
  }
  return best;
}

ScanPlan scan_plan(int64_t outer, int64_t len, int64_t inner, bool bf16, int kind, bool ck) {
  constexpr long long kCus = 256;
  const int64_t cols = outer * inner;
  const int es = bf16 ? 2 : 4;
  ScanPlan p{};
  p.rows = inner == 1;
  p.segs = 1;
  p.lanes = 64;
  p.cw = p.run = p.fine = 1;
  p.wide = cols * len * es >= (1ll << 32);
  const bool small = cols * len <= (1 << 22);
  long long piece, units;   // steps of a wave's tile; workgroups without segments
  int least = 1, most = kScanWaves;
  if (p.rows) {
    if (len <= 32 * kScanE) {   // a row in part of a wave
      p.lanes = scan_pow2((len + kScanE - 1) / kScanE);
      p.waves = 4;
      p.seg_len = 64 * kScanE;
      p.self = true;
      return p;
    }
    piece = 64 * kScanE;
    units = outer;
    // a workgroup per row: fewer waves each where the launch would have 2^32 threads (below 2^26 rows
    // one wave always fits)
    most = (int)std::min<long long>(most, ((1ll << 32) - 1) / (64 * units));
  } else {
    most = scan_col_waves(kind, ck, p.wide);
    // Columns per wave: 64, fewer where that leaves CUs without a workgroup: down to a memory line of
    // 128 bytes (with 32 bytes the address units were the limit, 490 against 400 us for the backward
    // of 4 x 32768 x 1024 bf16), or to 32 bytes where little data makes latency the limit.
    const int low = scan_pow2(std::min<int64_t>(cols, (small ? 32 : 128) / es));
    p.cw = scan_pow2(std::min<int64_t>(cols, 64));
    while (p.cw > low && (cols + p.cw - 1) / p.cw < kCus && 64 / p.cw * kScanK < len) p.cw /= 2;
    // Little data: fewer still where that leaves two tiles (one for a backward without states, which
    // then needs no other launch). Down to 16 bytes, or 4 columns of a backward: below that a tile's
    // loads take longer than the maps' launch (13 x 9025 x 11 bf16, at one column: forward 49 us, 24
    // cut instead; backward 74 and 32; 2 x 10847 x 51 fp32: 50 and 38, 72 and 52).
    if (small) {
      const long long reach = (long long)(kind == 2 ? 1 : 2) * most * 64 * kScanK;   // at one column
      const int lowest = kind == 0 ? 16 / es : kind == 1 ? 4 : 1;
      int cw = p.cw;
      while (cw > lowest && reach / cw < len) cw /= 2;
      if (reach / cw >= len) p.cw = cw;
    }
    p.run = std::max(1, 128 / (p.cw * es));
    piece = (64 / p.cw) * kScanK;
    units = (cols + p.cw - 1) / p.cw;
    if (kind && p.cw == 64) least = 2;   // waves pair up for the kept states
  }
  const long long pieces = (len + piece - 1) / piece;
  // Column groups beyond the CUs: so few waves that a CU holds its share of the workgroups at a time,
  // where that measured less (784 steps, 64 columns a group): forward 258 groups bf16 27 us instead of
  // 35, 384 fp32 38 and 43, 1000 bf16 65 and 87; backward 1000 groups bf16 107 and 123, from a checkpoint
  // 185 and 263. Not where it measured more: backward 258 groups 53 and 48, from a checkpoint 143 and
  // 106, 1500 bf16 162 and 156; rows. The same from 200 to 3200 steps: 1000 groups bf16, forward 22 and
  // 32 us at 200 steps, 251 and 331 at 3200, backward 26 and 42, 430 and 442; up to 128 steps, one tile,
  // nothing changes. It loses up to 7 % in forwards of 1500 groups bf16 at 200 and 400 steps (31 and 30,
  // 50 and 46), and gains that at 784 and 1600.
  int cap = most;
  const int share = std::max(1, (int)(most / ((units + kCus - 1) / kCus)));
  if (!p.rows && units > 3 * kCus && (kind == 0 || (units <= 4 * kCus && (bf16 || ck)))) cap = share;
  else if (!p.rows && units > kCus && units <= 3 * kCus && kind == 0 && !ck) cap = most / 2;
  p.waves = scan_waves(units, pieces, std::min(least, cap), cap);
  // one tile: a short axis costs a barrier less, and a backward without states no second run
  if (pieces <= most && (pieces <= 2 || kind == 2)) p.waves = (int)std::max<long long>(least, pieces);
  if (least == 2) p.waves += p.waves & 1;
  p.self = pieces <= p.waves;
  // The axis is cut where half the CUs or more would have no workgroup; the forward of an fp32 tensor,
  // which alone keeps memory busy from fewer CUs, where that is true of 11 in 16; a short axis where
  // it is true of three in four. Never into more parts than leave each CU one at most. Forward of
  // 144 x 16384 x 64 bf16: 253 us whole, 340 cut; 128 x 16384 x 64: 248 and 220; 64 x 16384 x 64 fp32:
  // 184 and 221; backward of 96 x 16384 x 64 bf16: 273 us in two parts, 358 in three; 128 x 1029 x 64:
  // 29 us whole, 35 cut.
  const long long full = kind == 0 && !bf16 ? kCus * 5 / 16 - 1 : kCus / 2;
  if (units <= full && (units <= kCus / 4 || len >= 2048) &&
      !(small && pieces <= 4 * most)) {   // four tiles cost less than a launch
    // segments of whole 16 pieces, which the tiles of 8 or 16 waves divide
    const long long step = 16 * piece, steps = (len + step - 1) / step;
    const long long segs = std::min<long long>({kCus / units, steps, 64});
    if (segs > 1) {
      const long long per = (steps + segs - 1) / segs;
      p.segs = (int)((steps + per - 1) / per);
      p.seg_len = (int)(per * step);
      p.waves = most == 16 ? 16 : 8;
      // workgroups for the maps' launch: up to a dozen per CU (383 against 413 us with one map per
      // segment, the backward of 4 x 32768 x 1024 bf16)
      while (per % (2 * p.fine) == 0 && units * (p.segs - 1) * p.fine < 6 * kCus) p.fine *= 2;
      p.self = false;
      return p;
    }
  }
  const long long tile = p.waves * piece;
  p.seg_len = (int)((len + tile - 1) / tile * tile);
  return p;
}

namespace {
size_t maps_bytes(const ScanPlan& p, size_t cols) { return p.segs > 1 ? cols * (8 * p.segs * p.fine + 4) : 0; }
}  // namespace

size_t scan_workspace(int64_t outer, int64_t len, int64_t inner) {
  // the type is not an argument: the larger need
  const size_t cols = (size_t)(outer * inner);
  return std::max(maps_bytes(scan_plan(outer, len, inner, false, 0, false), cols),
                  maps_bytes(scan_plan(outer, len, inner, true, 0, false), cols));
}

size_t scan_backward_workspace(int64_t outer, int64_t len, int64_t inner, bool has_states) {
  const size_t cols = (size_t)(outer * inner);
  size_t need = 0;
  for (int b = 0; b < 4; ++b) {   // the types of g and u are not arguments: the largest need
    const ScanPlan p = scan_plan(outer, len, inner, b & 1, has_states ? 1 : 2, b & 2);
    size_t n = maps_bytes(p, cols);
    if (!has_states && !p.self) {   // states (whole 16 bytes), then the maps of either launch
      const size_t kept = cols * ((len + kScanChunk - 1) / kScanChunk) * 4;
      const ScanPlan f = scan_plan(outer, len, inner, b & 1, 0, b & 2);
      n = (kept + 15) / 16 * 16 + std::max(n, maps_bytes(f, cols));
    }
    need = std::max(need, n);
  }
  return need;
}

}  // namespace wbmm
