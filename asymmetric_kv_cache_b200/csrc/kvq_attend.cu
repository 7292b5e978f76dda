// Dispatch of the attend kernels and the merge of split units.
#include <cuda_fp16.h>

#include "kvq_attend_kernels.cuh"

namespace kvq {
namespace {

constexpr int kMergeWarps = 4;

// Merges the pieces of split units: a block is a row (x: unit, y: row of the
// unit), its warps take every fourth piece.  With the pieces' maxima m_i and
// sums l_i relative to them, out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m)
// l_i.  (One warp for all of a row's pieces took 20 us for the 74 pieces of a
// 128k context.)
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    attend_merge_kernel(const Geom g, const WsLayout w, const AttendArgs a, const AttendSeqs seqs) {
  constexpr int V = D / 32;
  __shared__ float part[kMergeWarps][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int lo = 0, hi = seqs.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seqs.unit_off[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
  }
  const int R = seqs.n_q[lo] * g.gqa, tiles = (R + seqs.unit_rows - 1) / seqs.unit_rows;
  const int unit = blockIdx.x - seqs.unit_off[lo];        // of the sequence
  const int parts = (seqs.piece_off[lo + 1] - seqs.piece_off[lo]) / (g.hkv * tiles);
  const int h = unit / tiles, tile = unit % tiles, ur = blockIdx.y;
  // (the tensor-core kernel numbers a sequence's row tiles from the last)
  const int r = (seqs.unit_rows == kAttendRows ? tile : tiles - 1 - tile) * seqs.unit_rows + ur;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (parts < 2 || r >= R) return;
  const float* ps = reinterpret_cast<const float*>(a.ws + w.partials_off) +
                    ((int64_t)(seqs.piece_off[lo] + unit * parts) * seqs.slot_rows + ur) * (D + 4);
  const int64_t step = (int64_t)seqs.slot_rows * (D + 4);
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, ps[s * step + D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float y[V], l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
#pragma unroll 4
  for (int s = warp; s < parts; s += kMergeWarps) {
    const float* p = ps + s * step;
    const float f = fast_exp2(p[D] - base);
    l += f * p[D + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] += f * p[lane * V + i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) part[warp][lane * V + i] = y[i];
  if (lane == 0) part[warp][D] = l;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int x = 1; x < kMergeWarps; ++x) {
    l += part[x][D];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] += part[x][lane * V + i];
  }
  l = __shfl_sync(0xffffffffu, l, 0);
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
  if (e != cudaSuccess || !split || s.merge_here) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)s.unit_off[s.n], (unsigned)s.slot_rows);
  lc.blockDim = dim3(32 * kMergeWarps);
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
