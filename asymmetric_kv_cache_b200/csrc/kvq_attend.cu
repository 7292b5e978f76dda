// Dispatch of the attend kernels and the merge of split units.
#include <cuda_fp16.h>

#include "kvq_attend_kernels.cuh"

namespace kvq {
namespace {

constexpr int kMergeThreads = 32 * kAttendRows;

// Merges the pieces of split units, a warp per row: blocks are (piece, eight
// rows of the unit), of which those of a unit's first piece do the work (the
// others leave at once).  With the rows' maxima m_i and sums l_i relative to
// them, out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    attend_merge_kernel(const Geom g, const WsLayout w, const AttendArgs a, const AttendSeqs seqs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int lo = 0, hi = seqs.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seqs.piece_off[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
  }
  const int R = seqs.n_q[lo] * g.gqa, tiles = (R + seqs.unit_rows - 1) / seqs.unit_rows;
  const int local = blockIdx.x - seqs.piece_off[lo];
  const int parts = (seqs.piece_off[lo + 1] - seqs.piece_off[lo]) / (g.hkv * tiles);
  const int h = local / parts / tiles, tile = local / parts % tiles;
  const int ur = blockIdx.y * kAttendRows + warp;        // row of the unit
  // (the tensor-core kernel numbers a sequence's row tiles from the last)
  const int r = (seqs.unit_rows == kAttendRows ? tile : tiles - 1 - tile) * seqs.unit_rows + ur;
  if (parts < 2 || local % parts != 0 || r >= R) return;
  const float* ps = reinterpret_cast<const float*>(a.ws + w.partials_off) +
                    ((int64_t)blockIdx.x * seqs.slot_rows + ur) * (D + 4);
  const int64_t kStep = (int64_t)seqs.slot_rows * (D + 4);
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, ps[s * kStep + D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float y[V], l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float* p = ps + s * kStep;
    const float f = fast_exp2(p[D] - base);
    l += f * p[D + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] += f * p[lane * V + i];
  }
  attend_store_row<D>(g, a, seqs, lo, h, r, y, l, lane);
}

}  // namespace

cudaError_t attend_max_ctas(const Geom& g, int* out) {
#define KVQ_CASE(D_, KB_, VB_, G_)                                       \
  if (g.d == D_ && g.kb == KB_ && g.vb == VB_ && g.G == G_)              \
    return attend_max_ctas_##D_##_##KB_##_##VB_##_##G_(out);
  KVQ_DECODE_FOR_EACH(KVQ_CASE)
#undef KVQ_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_attend(const Geom& g, const WsLayout& w, const AttendArgs& a,
                          const AttendSeqs& s, bool split, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
#define KVQ_CASE(D_, KB_, VB_, G_)                                       \
  if (g.d == D_ && g.kb == KB_ && g.vb == VB_ && g.G == G_)              \
    e = launch_attend_##D_##_##KB_##_##VB_##_##G_(g, w, a, s, stream);
  KVQ_DECODE_FOR_EACH(KVQ_CASE)
#undef KVQ_CASE
  if (e != cudaSuccess || !split) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)s.piece_off[s.n], (unsigned)((s.slot_rows + kAttendRows - 1) / kAttendRows));
  lc.blockDim = dim3(kMergeThreads);
  lc.stream = stream;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = la;
  lc.numAttrs = 1;
  return g.d == 128 ? cudaLaunchKernelEx(&lc, attend_merge_kernel<128>, g, w, a, s)
                    : cudaLaunchKernelEx(&lc, attend_merge_kernel<64>, g, w, a, s);
}

}  // namespace kvq
