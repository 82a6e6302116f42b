// Gated linear recurrence: the layout of a call (workgroups, waves, parts of the axis) and the
// constants that it and the kernels share. Plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace wbmm {

constexpr int kScanChunk = 32;    // steps between two kept states
constexpr int kScanK = 16;        // steps per lane and tile of the column kernels
constexpr int kScanE = 8;         // steps per lane and tile of the row kernels
constexpr int kScanWaves = 16;    // waves of a workgroup at most
// The same for the column kernels, by their registers: forward 4 waves per SIMD, 3 from a checkpoint;
// backward 3, and 2 from a checkpoint (at 3, 13 registers spilt: 10 % slower) and with 64-bit offsets.
constexpr int scan_col_waves(bool backward, bool ck, bool wide) {
  return backward ? (ck || wide ? 8 : 12) : (ck ? 12 : 16);
}
constexpr int scan_map_waves(bool ck) { return ck ? 8 : 16; }   // of a workgroup that forms a map

struct ScanPlan {
  bool rows, wide;      // rows: inner = 1; wide: 64-bit offsets (column kernels)
  bool self;            // backward: one tile holds the axis, no states needed
  int cw, run, lanes, waves, segs, seg_len, fine;
};
// kind: 0 = forward, 1 = backward from kept states, 2 = backward without; ck: u is a checkpoint.
ScanPlan scan_plan(int64_t outer, int64_t len, int64_t inner, bool bf16, int kind, bool ck);
// Device workspace of a call (16-byte aligned), 0 when none: the segments' maps, and the states of
// a backward that gets none.
size_t scan_workspace(int64_t outer, int64_t len, int64_t inner);
size_t scan_backward_workspace(int64_t outer, int64_t len, int64_t inner, bool has_states);

}  // namespace wbmm
