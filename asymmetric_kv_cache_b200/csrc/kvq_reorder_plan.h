// The order of a reordering's moves (host only): sequence b takes over
// sequence parent[b], in place.
//
// The map's graph (an edge parent[b] -> b) is trees that hang off cycles.  A
// destination may be written once everything that reads it has been read, so
// trees are moved from their leaves inwards; what is left then are the
// cycles.  A batch of up to kReorderBatch moves reads all of its sources
// before it writes any destination, which closes a cycle of that many
// sequences.  A longer cycle c0 <- c1 <- .. <- cL-1 <- c0 is the cycle of its
// first kReorderBatch members followed by the cycle of the rest headed by the
// batch's last member, which then holds c0's old contents.
#pragma once

#include <cstdint>
#include <vector>

namespace kvq {

constexpr int kReorderBatch = 8;    // moves that are read before any is written
constexpr int kReorderMoves = 512;  // moves of one launch

// Moves of one launch: those of chain y are [chain_start[y], chain_start[y +
// 1]); neighbours with the same batch number form a batch.  src_was / dst_was:
// the sequence whose contents (at the launch's start) src and dst hold when
// the move comes up, which is another one only where a long cycle goes on.
// last: no later move of the launch writes dst.
struct ReorderMoves {
  int32_t n_chains;
  int32_t chain_start[kReorderMoves + 1];
  int32_t src[kReorderMoves], dst[kReorderMoves];
  int32_t src_was[kReorderMoves], dst_was[kReorderMoves];
  int32_t batch[kReorderMoves];
  uint8_t last[kReorderMoves];
};

struct ReorderMove {
  int32_t src, dst, chain, batch;
};

// All moves, chain by chain and within a chain in order; batch numbers rise.
// parent[b] in [0, n_all) for b in [0, n); sequences from n on stay.
inline std::vector<ReorderMove> plan_reorder(const int32_t* parent, int n, int n_all) {
  std::vector<int32_t> par(n_all), readers(n_all, 0), comp(n_all);
  for (int b = 0; b < n_all; ++b) par[b] = b < n ? parent[b] : b;
  for (int b = 0; b < n_all; ++b)
    if (par[b] != b) ++readers[par[b]];
  // components (union by walking to a root with path halving)
  for (int b = 0; b < n_all; ++b) comp[b] = b;
  auto root = [&](int x) {
    while (comp[x] != x) x = comp[x] = comp[comp[x]];
    return x;
  };
  for (int b = 0; b < n_all; ++b) comp[root(b)] = root(par[b]);

  std::vector<std::vector<ReorderMove>> chains(n_all);
  std::vector<char> done(n_all, 0);
  int batch = 0;
  // trees: a sequence that nobody reads (any more) is written
  std::vector<int32_t> ready;
  for (int b = 0; b < n_all; ++b)
    if (par[b] != b && readers[b] == 0) ready.push_back(b);
  for (size_t i = 0; i < ready.size(); ++i) {
    const int b = ready[i], p = par[b];
    chains[root(b)].push_back({p, b, 0, -1});
    done[b] = 1;
    if (--readers[p] == 0 && par[p] != p) ready.push_back(p);
  }
  // batches of the trees: every move reads before its source is written, so
  // any run of consecutive moves of a chain may read first and write then
  for (auto& c : chains)
    for (size_t i = 0; i < c.size(); ++i) c[i].batch = i % kReorderBatch ? c[i - 1].batch : batch++;
  for (int b = 0; b < n_all; ++b) {
    if (par[b] == b || done[b]) continue;
    std::vector<int32_t> cyc;                 // b <- par[b] <- par[par[b]] ..
    for (int x = b; !done[x]; x = par[x]) {
      done[x] = 1;
      cyc.push_back(x);
    }
    auto& c = chains[root(b)];
    size_t at = 0;
    while (cyc.size() - at > 1) {
      const size_t m = cyc.size() - at < (size_t)kReorderBatch ? cyc.size() - at : kReorderBatch;
      for (size_t i = 0; i + 1 < m; ++i) c.push_back({cyc[at + i + 1], cyc[at + i], 0, batch});
      c.push_back({cyc[at], cyc[at + m - 1], 0, batch});
      ++batch;
      at += m - 1;
    }
  }
  std::vector<ReorderMove> all;
  int chain = 0;
  for (auto& c : chains) {
    if (c.empty()) continue;
    for (auto& m : c) {
      m.chain = chain;
      all.push_back(m);
    }
    ++chain;
  }
  return all;
}

// The next launch's moves from all[at..]: whole batches, at most
// kReorderMoves; returns where the following launch starts.
inline size_t next_reorder_launch(const std::vector<ReorderMove>& all, size_t at, ReorderMoves* mv) {
  mv->n_chains = 0;
  int n = 0;
  while (at < all.size()) {
    size_t e = at;
    while (e < all.size() && all[e].batch == all[at].batch) ++e;
    if (n + (int)(e - at) > kReorderMoves) break;
    if (n == 0 || all[at].chain != all[at - 1].chain) mv->chain_start[mv->n_chains++] = n;
    const int first = mv->chain_start[mv->n_chains - 1], n0 = n;
    for (; at < e; ++at, ++n) {
      mv->src[n] = mv->src_was[n] = all[at].src;
      mv->dst[n] = mv->dst_was[n] = all[at].dst;
      mv->batch[n] = all[at].batch;
      mv->last[n] = 1;
      for (int i = first; i < n0; ++i) {      // earlier batches, in order
        if (mv->dst[i] == mv->src[n]) mv->src_was[n] = mv->src_was[i];
        if (mv->dst[i] == mv->dst[n]) {
          mv->dst_was[n] = mv->src_was[i];
          mv->last[i] = 0;
        }
      }
    }
  }
  mv->chain_start[mv->n_chains] = n;
  return at;
}

}  // namespace kvq
