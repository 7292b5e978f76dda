// How a kvq_attend call's work is cut into launches and pieces (host only).
#pragma once

#include <algorithm>
#include <cstdint>

#include "kvq_internal.h"

namespace kvq {

// The launch of sequences [s0, s0 + n): `row` counts the call's query rows.
// A unit is (sequence, kv head, tile of kAttendRows rows).  With at least as
// many units as resident CTAs every unit is one piece.  Otherwise the units
// are cut into about max_ctas pieces, a sequence's units in proportion to
// the keys that they see, and into no more pieces than a CTA's warps have
// blocks for.  The lengths are the host's; the kernel cuts what it finds in
// the device's into the same number of pieces, so a replayed launch stays
// right when they have grown.  Returns whether some unit is cut.
inline bool plan_attend(const Geom& g, const int32_t* lens, const int32_t* n_q, int s0, int n,
                        int score_window, int max_ctas, int64_t* row, AttendSeqs* out) {
  out->n = n;
  out->seq0 = s0;
  int64_t units = 0, cost = 0;
  auto tiles = [&](int b) { return ((int64_t)n_q[b] * g.gqa + kAttendRows - 1) / kAttendRows; };
  auto blocks = [&](int b) {
    int64_t keys = lens[b];
    if (score_window > 0) keys = std::min<int64_t>(keys, (int64_t)score_window + kAttendRows / g.gqa + g.G);
    return keys / g.G + 1;
  };
  for (int b = s0; b < s0 + n; ++b) {
    const int64_t u = g.hkv * tiles(b);
    units += u;
    cost += u * blocks(b);
  }
  int64_t pieces = 0;
  bool split = false;
  for (int i = 0; i < n; ++i) {
    const int b = s0 + i;
    out->row_off[i] = (int32_t)*row;
    out->n_q[i] = n_q[b];
    out->piece_off[i] = (int32_t)pieces;
    *row += n_q[b];
    int64_t parts = 1;
    if (units < max_ctas && n_q[b] > 0) {
      parts = blocks(b) * max_ctas / cost;
      parts = std::max<int64_t>(1, std::min(parts, (blocks(b) + 3) / 4));
      split |= parts > 1;
    }
    pieces += g.hkv * tiles(b) * parts;
  }
  out->piece_off[n] = (int32_t)pieces;
  return split;
}

}  // namespace kvq
