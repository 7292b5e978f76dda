// Sequences of the cache taking over other sequences' contents, in place
// (kvq_reorder): beams that follow their parents, forks of a prompt.
//
// The host turns the map b <- parent[b] into chains of batches of at most
// kReorderBatch moves (kvq_reorder_plan.h).  A batch is "read every source,
// then write every destination", and no batch reads what an earlier batch of
// its chain wrote.  Every 16-byte unit of the layout has one owner thread per
// chain, and the unit's bytes in one sequence only ever go to the same unit
// of another, so a thread that walks the chain's batches in order keeps the
// map exact with no scratch copy and no barrier between blocks.
//
// Bound: memory; every moved byte is read once and written once.  Blocks
// whose tokens the caller declares shared are not touched.  A thread reads
// up to 8 sources of 16 bytes before its first store.
//
// Lengths: every block reads the device lengths of its chain when it starts
// and counts itself on the ticket of the chain's first destination; the block
// that counts last stores the new lengths and puts the ticket back to zero.
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_reorder_plan.h"

namespace kvq {
namespace {

constexpr int kReorderThreads = 256;

// Units [u, u + UN * stride) of one area for a batch of NB moves: read all,
// write all.  `live(k, unit)` says whether move k carries the unit.
template <int NB, int UN, class Live>
__device__ __forceinline__ void move_units(unsigned char* base, const int64_t* so,
                                           const int64_t* dof, int64_t u, int stride, int64_t end,
                                           int n, const Live& live) {
  uint4 r[UN][NB];
#pragma unroll
  for (int x = 0; x < UN; ++x)
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int64_t uu = u + (int64_t)x * stride;
      if (k < n && uu < end && live(k, uu))
        r[x][k] = *reinterpret_cast<const uint4*>(base + so[k] + 16 * uu);
    }
#pragma unroll
  for (int x = 0; x < UN; ++x)
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int64_t uu = u + (int64_t)x * stride;
      if (k < n && uu < end && live(k, uu))
        *reinterpret_cast<uint4*>(base + dof[k] + 16 * uu) = r[x][k];
    }
}

// Grid: x = tiles of kReorderThreads * 8 units over (kv head, area), strided;
// y = chain.
__global__ void __launch_bounds__(kReorderThreads)
    reorder_kernel(const Geom g, unsigned char* cache, const ReorderMoves mv, int32_t shared_tokens) {
  __shared__ int32_t s_len[kReorderMoves], d_len[kReorderMoves];
  __shared__ int64_t s_off[kReorderBatch], d_off[kReorderBatch];
  __shared__ int32_t last;
  const int tid = threadIdx.x;
  const int m0 = mv.chain_start[blockIdx.y], m1 = mv.chain_start[blockIdx.y + 1];
  int32_t* lens = reinterpret_cast<int32_t*>(cache + g.lens_off);
  for (int m = m0 + tid; m < m1; m += kReorderThreads) {
    s_len[m - m0] = min(max(lens[mv.src_was[m]], 0), g.max_tokens);
    d_len[m - m0] = min(max(lens[mv.dst_was[m]], 0), g.max_tokens);
  }
  __syncthreads();
  auto groups = [&](int n) { return quantized_groups_s(n, g.G, g.window, g.sink); };
  // groups that stay because source and destination share them: those whose
  // tokens are shared and that are quantized in both.  With position-adaptive
  // widths sequences of different lengths hold the same tokens in different
  // bytes: nothing is shared between them then.
  const int shared_groups = shared_tokens > g.sink ? (shared_tokens - g.sink) / g.G : 0;
  auto kept = [&](int sn, int dn) {
    return g.akvq_delta && sn != dn ? 0 : min(shared_groups, min(groups(sn), groups(dn)));
  };
  int most = 0, lo_group = 0x7fffffff;        // groups of the chain: [lo_group, most)
  for (int m = 0; m < m1 - m0; ++m) {
    most = max(most, groups(s_len[m]));
    lo_group = min(lo_group, kept(s_len[m], d_len[m]));
  }

  const int upb = g.block_bytes / 16;
  const int64_t tail_units = g.tail_bytes / 16;
  const int64_t sink_units = shared_tokens >= g.sink ? 0 : g.sink_bytes / 16;
  const int64_t block_units = (int64_t)(most - lo_group) * upb;
  constexpr int kTile = kReorderThreads * 8;
  const int64_t bt = (block_units + kTile - 1) / kTile, tt = (tail_units + kTile - 1) / kTile,
                st = (sink_units + kTile - 1) / kTile;
  const int64_t per_head = bt + tt + st;

  for (int64_t tile = blockIdx.x; tile < per_head * g.hkv; tile += gridDim.x) {
    const int h = (int)(tile / per_head);
    int64_t t = tile % per_head;
    const int area = t < bt ? 0 : t < bt + tt ? 1 : 2;
    t -= area == 0 ? 0 : area == 1 ? bt : bt + tt;
    const int64_t u0 = t * kTile + tid;
    const int64_t end = area == 0 ? block_units : area == 1 ? tail_units : sink_units;
    for (int m = m0; m < m1;) {
      // the batch: consecutive moves with the same number
      int n = 1;
      while (m + n < m1 && mv.batch[m + n] == mv.batch[m]) ++n;
      __syncthreads();
      if (tid < 2 * n) {
        const int seq = tid < n ? mv.src[m + tid] : mv.dst[m + tid - n];
        int64_t off;
        if (area == 0)
          off = g.blocks_off + (((int64_t)seq * g.hkv + h) * g.max_groups + lo_group) * g.block_bytes;
        else if (area == 1)
          off = g.tails_off + ((int64_t)seq * g.hkv + h) * g.tail_bytes;
        else
          off = g.sinks_off + ((int64_t)seq * g.hkv + h) * g.sink_bytes;
        (tid < n ? s_off[tid] : d_off[tid - n]) = off;
      }
      __syncthreads();
      const int32_t* sl = s_len + (m - m0);
      const int32_t* dl = d_len + (m - m0);
      auto live = [&](int k, int64_t u) {
        if (area != 0) return sl[k] > 0;
        const int grp = lo_group + (int)(u / upb);
        if (grp >= groups(sl[k]) || grp < kept(sl[k], dl[k])) return false;
        if (!g.akvq_delta) return true;
        return akvq_key_bits(grp, sl[k], g.G, g.akvq_delta) == 4 || (int)(u % upb) * 16 < g.a2_bytes;
      };
      if (n <= 2) {
#pragma unroll 1
        for (int x = 0; x < 8; x += 4)
          move_units<2, 4>(cache, s_off, d_off, u0 + (int64_t)x * kReorderThreads, kReorderThreads,
                           end, n, live);
      } else if (n <= 4) {
#pragma unroll 1
        for (int x = 0; x < 8; x += 2)
          move_units<4, 2>(cache, s_off, d_off, u0 + (int64_t)x * kReorderThreads, kReorderThreads,
                           end, n, live);
      } else {
#pragma unroll 1
        for (int x = 0; x < 8; ++x)
          move_units<8, 1>(cache, s_off, d_off, u0 + (int64_t)x * kReorderThreads, kReorderThreads,
                           end, n, live);
      }
      m += n;
    }
  }

  __syncthreads();
  int32_t* ticket = reinterpret_cast<int32_t*>(cache + g.counters_off) + mv.dst[m0];
  if (tid == 0) last = atomic_add_acq_rel_gpu(ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (last) {
    for (int m = m0 + tid; m < m1; m += kReorderThreads) 
      if (mv.last[m]) lens[mv.dst[m]] = s_len[m - m0];
    if (tid == 0) *ticket = 0;
  }
}

}  // namespace

cudaError_t launch_reorder(const Geom& g, unsigned char* cache, const ReorderMoves& mv,
                           int shared_tokens, int64_t tiles, cudaStream_t stream) {
  // four resident blocks on each of the 148 SMs are enough loads in flight;
  // more tiles than that are walked with a stride
  const int64_t want = (148 * 8 + mv.n_chains - 1) / mv.n_chains;
  const int64_t gx = tiles < want ? tiles : want;
  reorder_kernel<<<dim3((unsigned)(gx < 1 ? 1 : gx), (unsigned)mv.n_chains), kReorderThreads, 0,
                   stream>>>(g, cache, mv, shared_tokens);
  return cudaGetLastError();
}

}  // namespace kvq
