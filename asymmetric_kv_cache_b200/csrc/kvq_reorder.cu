// Sequences of the cache taking over other sequences' contents, in place
// (kvq_reorder): beams that follow their parents, forks of a prompt.
//
// The host turns the map b <- parent[b] into chains of batches of at most
// kReorderBatch moves (kvq_reorder_plan.h).  A batch is "read every source,
// then write every destination".  A later batch of a chain may read what an
// earlier one wrote (a cycle of more than kReorderBatch sequences goes on from
// a member that its batch before has written), so the batches of a chain must
// stay in order.  Every 16-byte unit of the layout has one owner thread per
// chain, and the unit's bytes in one sequence only ever go to the same unit
// of another: a thread that walks the chain's batches in order keeps the map
// exact with no scratch copy and no barrier between blocks.
//
// Bound: memory; every moved byte is read once and written once.  Blocks
// whose tokens the caller declares shared are not touched.  A thread reads
// up to 8 sources of 16 bytes before its first store.
//
// Lengths: every block reads the device lengths of its chain when it starts
// and counts itself on the ticket of the chain's first destination; the block
// that counts last stores the new lengths and puts the ticket back to zero.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_operators.h"
#include "kvq_reorder_plan.h"

namespace kvq {
namespace {

constexpr int kReorderThreads = 256;

// A batch's move k takes the units [lo, hi) of the area at hand from sequence
// src to sequence dst.
struct MoveArea {
  int32_t src, dst;
  uint32_t lo, hi;
};

// The units u, u + kReorderThreads, .. (UN of them) of a batch of n <= NB moves:
// read all, write all.  `at`: the head's area in sequence 0, `step`: bytes from
// one sequence's area to the next one's.  AK: the units behind a 2-bit block's
// end are skipped.
template <int NB, int UN, bool AK>
__device__ __forceinline__ void move_units(const Geom& g, unsigned char* at, int64_t step,
                                           const MoveArea* mv, const int32_t* len, uint32_t u, int n,
                                           bool blocks, int lo_group) {
  uint4 r[UN][NB];
  uint32_t live = 0;
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const MoveArea m = mv[k];
    const uint32_t hi = k < n ? m.hi : 0u;
#pragma unroll
    for (int x = 0; x < UN; ++x) {
      const uint32_t uu = u + x * kReorderThreads;
      bool on = uu >= m.lo && uu < hi;
      if (AK && blocks && on) {
        const uint32_t upb = g.block_bytes / 16;
        const int grp = lo_group + (int)(uu / upb);
        on = akvq_key_bits(grp, len[k], g.G, g.akvq_delta) == 4 || (int)(uu % upb) * 16 < g.a2_bytes;
      }
      if (on) {
        live |= 1u << (x * NB + k);
        r[x][k] = *reinterpret_cast<const uint4*>(at + m.src * step + (int64_t)uu * 16);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int64_t dst = mv[k].dst * step;
#pragma unroll
    for (int x = 0; x < UN; ++x)
      if (live & 1u << (x * NB + k))
        *reinterpret_cast<uint4*>(at + dst + (int64_t)(u + x * kReorderThreads) * 16) = r[x][k];
  }
}

// Grid: x = tiles of kReorderTile units over (kv head, area), strided; y =
// chain.  NB: the largest batch of the launch, rounded up to a power of two.  A
// thread has 8 loads of 16 bytes in flight whatever NB is, 1024 threads on an
// SM (768 with NB = 8): 128 KB (96), three times (twice) what the memory's
// latency at its rate needs.
template <int NB, bool AK>
__global__ void __launch_bounds__(kReorderThreads, NB == 8 ? 3 : 4)
    reorder_kernel(const Geom g, unsigned char* cache, const ReorderMoves mv, int32_t shared_tokens) {
  constexpr int kUnits = 8 / NB, kReorderTile = kReorderThreads * kUnits;
  __shared__ int32_t s_len[kReorderMoves], d_len[kReorderMoves];
  __shared__ MoveArea area_of[3][kReorderMoves + kReorderBatch];   // (entries behind a batch are read, not used)
  __shared__ int32_t range[2], last;
  const int tid = threadIdx.x;
  const int m0 = mv.chain_start[blockIdx.y], m1 = mv.chain_start[blockIdx.y + 1];
  int32_t* lens = reinterpret_cast<int32_t*>(cache + g.lens_off);
  auto groups = [&](int n) { return quantized_groups_s(n, g.G, g.window, g.sink); };
  // groups that stay because source and destination share them: those whose
  // tokens are shared and that are quantized in both.  With position-adaptive
  // widths sequences of different lengths hold the same tokens in different
  // bytes: nothing is shared between them then.
  const int shared_groups = shared_tokens > g.sink ? (shared_tokens - g.sink) / g.G : 0;
  auto kept = [&](int sn, int dn) {
    return AK && sn != dn ? 0 : min(shared_groups, min(groups(sn), groups(dn)));
  };
  if (tid == 0) {
    range[0] = 0x7fffffff;
    range[1] = 0;
  }
  __syncthreads();
  for (int m = m0 + tid; m < m1; m += kReorderThreads) {
    const int sn = min(max(lens[mv.src_was[m]], 0), g.max_tokens);
    const int dn = min(max(lens[mv.dst_was[m]], 0), g.max_tokens);
    s_len[m - m0] = sn;
    d_len[m - m0] = dn;
    atomicMin(&range[0], kept(sn, dn));
    atomicMax(&range[1], groups(sn));
  }
  __syncthreads();
  const int lo_group = range[0], most = range[1];     // groups of the chain: [lo_group, most)

  const int upb = g.block_bytes / 16;
  const int64_t tail_units = g.tail_bytes / 16;
  const int64_t sink_units = shared_tokens >= g.sink ? 0 : g.sink_bytes / 16;
  const int64_t bt = ((int64_t)max(most - lo_group, 0) * upb + kReorderTile - 1) / kReorderTile,
                tt = (tail_units + kReorderTile - 1) / kReorderTile,
                st = (sink_units + kReorderTile - 1) / kReorderTile;
  const int64_t per_head = bt + tt + st;

  // every move's units of each area, once for all tiles: the tiles' loop has no
  // barrier (with a batch's entries set up for each tile between two barriers
  // 12 moves of 8100 tokens, 100 MB, took 47.4 us instead of 44.9)
  for (int m = tid; m < m1 - m0; m += kReorderThreads) {
    const int sn = s_len[m], dn = d_len[m], src = mv.src[m0 + m], dst = mv.dst[m0 + m];
    area_of[0][m] = MoveArea{src, dst, (uint32_t)(kept(sn, dn) - lo_group) * upb, (uint32_t)(groups(sn) - lo_group) * upb};
    area_of[1][m] = MoveArea{src, dst, 0u, sn == 0 ? 0u : (uint32_t)tail_units};
    area_of[2][m] = MoveArea{src, dst, 0u, sn == 0 ? 0u : (uint32_t)sink_units};
  }
  __syncthreads();

  for (int64_t tile = blockIdx.x; tile < per_head * g.hkv; tile += gridDim.x) {
    const int h = (int)(tile / per_head);
    int64_t t = tile % per_head;
    const int area = t < bt ? 0 : t < bt + tt ? 1 : 2;
    t -= area == 0 ? 0 : area == 1 ? bt : bt + tt;
    const uint32_t u0 = (uint32_t)t * kReorderTile + tid;
    const int64_t per_seq = area == 0   ? (int64_t)g.max_groups * g.block_bytes
                            : area == 1 ? g.tail_bytes
                                        : g.sink_bytes;
    unsigned char* at = cache + (area == 0 ? g.blocks_off + (int64_t)lo_group * g.block_bytes
                                 : area == 1 ? g.tails_off
                                             : g.sinks_off) + h * per_seq;
    // the batches, consecutive moves with the same number
#pragma unroll 1
    for (int m = m0, n; m < m1; m += n) {
#pragma unroll 1
      for (n = 1; m + n < m1 && mv.batch[m + n] == mv.batch[m];) ++n;
      move_units<NB, kUnits, AK>(g, at, per_seq * g.hkv, area_of[area] + (m - m0), s_len + (m - m0), u0, n, area == 0, lo_group);
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
                           int shared_tokens, int64_t bytes, cudaStream_t stream) {
  int most = 1;
  for (int i = 0, n = 1; i + 1 < mv.chain_start[mv.n_chains]; ++i) {
    n = mv.batch[i + 1] == mv.batch[i] ? n + 1 : 1;
    most = std::max(most, n);
  }
  const int nb = most <= 1 ? 1 : most <= 2 ? 2 : most <= 4 ? 4 : 8;
  // a tile's steps per (kv head, area); four blocks on each of 148 SMs, twice,
  // and more tiles than that are walked with a stride
  const int64_t tile = 16LL * kReorderThreads * (8 / nb);
  const int64_t tiles = g.hkv * (bytes / tile + g.tail_bytes / tile + g.sink_bytes / tile + 3);
  const int64_t want = (148 * 8 + mv.n_chains - 1) / mv.n_chains;
  const dim3 grid((unsigned)std::min(tiles, want), (unsigned)mv.n_chains);
#define KVQ_REORDER(N_)                                                                          \
  if (nb == N_) {                                                                                \
    if (g.akvq_delta)                                                                            \
      reorder_kernel<N_, true><<<grid, kReorderThreads, 0, stream>>>(g, cache, mv, shared_tokens); \
    else                                                                                         \
      reorder_kernel<N_, false><<<grid, kReorderThreads, 0, stream>>>(g, cache, mv, shared_tokens); \
  }
  KVQ_REORDER(1) KVQ_REORDER(2) KVQ_REORDER(4) KVQ_REORDER(8)
#undef KVQ_REORDER
  return cudaGetLastError();
}

}  // namespace kvq
