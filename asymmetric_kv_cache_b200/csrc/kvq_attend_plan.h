// How a kvq_attend call's work is cut into launches and pieces (host only).
#pragma once

#include <algorithm>
#include <cstdint>

#include "kvq_operators.h"

namespace kvq {

// The rows per kv head from which on the call's sequences go to the
// tensor-core kernel (INT32_MAX: none does).
inline int attend_tc_rows(const Geom& g, const int32_t* lens, const int32_t* n_q, int n_seq,
                          int score_window) {
  int64_t steps = 0;
  for (int b = 0; b < n_seq; ++b) {
    const int64_t rows = (int64_t)n_q[b] * g.gqa;
    if (rows < kAttendTcRows) continue;
    int64_t keys = lens[b];
    if (score_window > 0) keys = std::min<int64_t>(keys, (int64_t)score_window + n_q[b]);
    steps += g.hkv * ((rows + 7) / 8) * (keys / 32 + 1) * g.d / 128;
  }
  return steps >= kAttendTcSteps ? kAttendTcRows : INT32_MAX;
}

// The launch of sequences [s0, s0 + n), of which those with at least tc_rows
// rows per kv head belong to the tensor-core kernel (unit_rows > kAttendRows)
// and the others to the register-tile kernel; the launch of either kernel
// skips the other's.  row0: the first sequence's first query row.
//
// A unit is (sequence, kv head, tile of unit_rows rows).  With at least as
// many units as resident CTAs every unit is one piece.  Otherwise the units
// are cut into at most `want` pieces, a sequence's units in proportion to the
// keys that they see (rounded down) and into no pieces of fewer than four
// steps.  `want` is max_ctas or, where that is less, the partials' room less
// one slot for each unit that ends up whole: 148 - units for the tensor cores'
// 256 rows a slot, so that from 50 equal units on every unit is one piece (one
// sequence of 32768 with 384 new tokens: 48 units in 96 pieces; with 400 to
// 1100: 56 to 144 whole units).  The lengths are the host's; the
// kernels cut what they find in the device's into the same number of pieces,
// so a replayed launch stays right when they have grown.  Returns whether
// some unit is cut.
inline bool plan_attend(const Geom& g, const int32_t* lens, const int32_t* n_q, int s0, int n,
                        int score_window, int max_ctas, int tc_rows, int unit_rows, int64_t row0,
                        AttendSeqs* out) {
  out->n = n;
  out->seq0 = s0;
  out->unit_rows = unit_rows;
  out->slot_rows = 1;
  const bool tc = unit_rows > kAttendRows;
  const int step = tc ? 64 : g.G;        // keys of one step of the kernel
  auto rows = [&](int b) {
    const int64_t r = (int64_t)n_q[b] * g.gqa;
    return tc == (r >= tc_rows) ? r : 0;
  };
  auto tiles = [&](int b) { return (rows(b) + unit_rows - 1) / unit_rows; };
  auto steps = [&](int b) {
    int64_t keys = lens[b];
    if (score_window > 0) keys = std::min<int64_t>(keys, (int64_t)score_window + unit_rows / g.gqa + step);
    return keys / step + 1;
  };
  int64_t units = 0, cost = 0;
  for (int b = s0; b < s0 + n; ++b) {
    const int64_t u = g.hkv * tiles(b);
    units += u;
    cost += u * steps(b);
    if (u > 0)
      out->slot_rows = (int)std::max<int64_t>(
          out->slot_rows, std::min<int64_t>(rows(b), unit_rows));
  }
  const int64_t want = units < kAttendTickets
                           ? std::min<int64_t>(max_ctas, kAttendPartialRows / out->slot_rows - units)
                           : 0;
  int64_t most = 1;
  int64_t pieces = 0, before = 0, row = row0;
  for (int i = 0; i < n; ++i) {
    const int b = s0 + i;
    out->row_off[i] = (int32_t)row;
    out->n_q[i] = n_q[b];
    out->piece_off[i] = (int32_t)pieces;
    out->unit_off[i] = (int32_t)before;
    row += n_q[b];
    int64_t parts = 1;
    if (units < want && tiles(b) > 0) {
      parts = steps(b) * want / cost;
      parts = std::max<int64_t>(1, std::min(parts, (steps(b) + 3) / 4));
      most = std::max(most, parts);
    }
    pieces += g.hkv * tiles(b) * parts;
    before += g.hkv * tiles(b);
  }
  out->piece_off[n] = (int32_t)pieces;
  out->unit_off[n] = (int32_t)before;
  out->merge_here = !tc && most <= kAttendMergeParts;
  return most > 1;
}

}  // namespace kvq
