// Internal declarations of the operators beside append and decode (attend,
// norm_rotary, reorder): what their host side hands to their kernels.
#pragma once

#include "kvq_internal.h"

namespace kvq {

// ---- attention of several new tokens per sequence ---------------------------
// Sequences per attend / rotary launch (their arguments ride in the kernel
// parameters).
constexpr int kAttendMaxSeqs = 512;
// Rows (query token, query head) of one unit: the N = 8 columns of the
// P.V tile.
constexpr int kAttendRows = 8;
// Rows (D + 4 floats each) that the partials of one launch's split units may
// take in a cache's workspace: 148 tensor-core units of 256 rows.
constexpr int kAttendPartialRows = 148 * 256;
// Units that a launch cuts into pieces at most (their tickets), and pieces of
// a unit up to which the last of them to end merges them all.
constexpr int kAttendTickets = 4096;
constexpr int kAttendMergeParts = 32;
// A sequence with at least this many rows per kv head (more than four tiles of
// kAttendRows) goes to the tensor-core kernel, if the call's such sequences
// give the other one at least so many steps (8 rows against 32 keys of 128
// channels; it does about 780 a us).  Measured, register tiles / tensor cores,
// us, 32 query and 8 kv heads of 128: 8 x 4113 keys: 24 rows 41 / 51, 32 rows
// 55 / 52, 36 rows 94 / 53 (capped 43 / 65, 58 / 67, 99 / 67); one context of
// 32768: 44 / 52, 53 / 52, 65 / 52; 64 x 2048: 133 / 204, 167 / 206, 212 / 206;
// 16 x 1000: 29 / 29, 29 / 28, 38 / 29; with 4 kv heads of 64 (6 thousand steps
// at 48 rows) 19 / 22.
constexpr int kAttendTcRows = 33;
constexpr int kAttendTcSteps = 16384;

// The workspace of a cache: kvq_attend's partials start where the decode's do
// and may be longer; its tickets (zero between calls) follow.  total: all of
// it, the decode's parts included.
struct AttendWs {
  int64_t tickets_off, total;
};
inline AttendWs make_attend_ws(const Geom& g, const WsLayout& w) {
  AttendWs a;
  const int64_t end = align_up(w.partials_off + 4LL * kAttendPartialRows * (g.d + 4), 256);
  a.tickets_off = end > w.total ? end : w.total;
  a.total = align_up(a.tickets_off + 4LL * kAttendTickets, 256);
  return a;
}

struct AttendArgs {
  const unsigned char* cache;
  const void* q;             // [rows][hq][d]
  int32_t q_dtype;
  void* out;                 // fp16 [rows][hq][d]
  unsigned char* ws;
  int32_t* tickets;          // one for each unit of a launch that is cut into pieces
  float scale, cap;          // cap = 0: none
  int32_t score_window;      // 0: none
  const float* slopes;       // [hq] or NULL
  const int32_t* prefix;     // [n_seq] or NULL
  int32_t residual;          // queries that fp16 does not hold exactly
};

// Sequence i of a launch is the cache's seq0 + i; its query rows start at
// row_off[i] (n_q[i] of them) and its pieces at piece_off[i]: per (kv head,
// row tile) the same number of pieces, tile after tile.
struct AttendSeqs {
  int32_t n, seq0;
  int32_t unit_rows;         // kAttendRows, or 256 / 128 (tensor cores)
  int32_t slot_rows;         // rows of a piece's partial slot
  int32_t merge_here;        // the last piece of a unit merges them (no merge kernel)
  int32_t row_off[kAttendMaxSeqs];
  int32_t n_q[kAttendMaxSeqs];
  int32_t piece_off[kAttendMaxSeqs + 1];
  int32_t unit_off[kAttendMaxSeqs + 1];   // units before the sequence's
};

cudaError_t attend_max_ctas(const Geom& g, int* max_ctas);
cudaError_t launch_attend(const Geom& g, const WsLayout& w, const AttendArgs& a,
                          const AttendSeqs& s, bool split, cudaStream_t stream);
#define KVQ_ATTEND_DECLARE(D_, KB_, VB_, G_)                                          \
  cudaError_t attend_max_ctas_##D_##_##KB_##_##VB_##_##G_(int* out);                  \
  cudaError_t launch_attend_##D_##_##KB_##_##VB_##_##G_(                              \
      const Geom& g, const WsLayout& w, const AttendArgs& a, const AttendSeqs& s,     \
      cudaStream_t stream);
KVQ_DECODE_FOR_EACH(KVQ_ATTEND_DECLARE)

// ---- norms of query and key heads with the position rotation ----------------
struct RotaryArgs {
  const void *q, *k, *v;     // v may be NULL
  int64_t q_stride, k_stride, v_stride;   // elements between rows
  void *q_out, *k_out, *v_out;
  const void *q_weight, *k_weight;        // [d] of the input type, or NULL
  float eps;
  const float* inv_freq;     // [n_pairs]
  int32_t n_pairs, interleaved;
  const int32_t* positions;  // [n_axes][rows], or NULL: from the lengths
  int32_t n_axes, sections[4];
  const int32_t* lens;
  int64_t rows;              // of the whole call
  int32_t hq, hkv;
};
struct RotarySeqs {
  int32_t n, seq0;
  int64_t row0;              // the launch's first row
  int32_t row_off[kAttendMaxSeqs];        // from row0
};
cudaError_t launch_norm_rotary(int d, int dtype, int out_dtype, const RotaryArgs& a,
                               const RotarySeqs& seqs, int rows, cudaStream_t stream);

// ---- reordering of sequences ---------------------------------------------
struct ReorderMoves;         // kvq_reorder_plan.h
cudaError_t launch_reorder(const Geom& g, unsigned char* cache, const ReorderMoves& mv,
                           int shared_tokens, int64_t bytes, cudaStream_t stream);

}  // namespace kvq
