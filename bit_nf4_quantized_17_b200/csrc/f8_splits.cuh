// Splits of a long contraction over the CTAs of a cluster, for the rank-r gradients of the
// 8-bit layer (f8_grad.cu, f8_grad_b.cu).
#pragma once

#include <algorithm>

#include "f8.cuh"

namespace qlora {

constexpr int kCtaMaxSmem = 227 * 1024;
constexpr int kCtaHalfSmem = 228 * 1024 / 2 - 1024;  // 1 KB of each CTA's goes to the system
// A CTA asks for at least the shared memory that goes with its TMEM columns, so that no
// other kernel's CTA that needs TMEM finds room beside it and has to wait for this one while
// its cluster waits for it.
constexpr int kSmemPerColumn = 228 * 1024 / 512;

// MMAs into one TMEM accumulator: its sums are cut off, not rounded, and what that loses
// adds up along such a chain.  Wanted, and at most where two CTAs share an SM or one has it
// alone (longer contractions are several launches that add).
constexpr int kChain = 16, kMaxChain = 48, kMaxChainAlone = 64;

// What a launch takes, in tenths of a tile's time.
struct SplitCost {
  int shared;  // a tile where two CTAs share an SM (alone: 10)
  int start;   // a round of clusters that run at once: its start,
  int split;   // and a split's share of the sum
  int launch;
};

// The splits n (at most 8, of at least min_tiles) and launches that end soonest for `clusters`
// clusters over kt_total tiles; plan(n, tiles) sets cfg for a launch in n splits of so many
// tiles each.  two: an SM holds two CTAs.
template <class Plan>
inline void choose_splits(const void* kernel, const cudaLaunchConfig_t& cfg, int64_t clusters,
                          int64_t kt_total, int64_t min_tiles, bool two, int max_accs,
                          const SplitCost& c, Plan&& plan, int* splits, int64_t* launches) {
  // Clusters of n that run at once.  The runtime answers for one CTA per SM; where an SM
  // holds two, a group of SMs holds clusters of n as one of half their size.
  auto at_once = [&](int n, int64_t per, bool both) -> int64_t {
    plan(n, per);
    const int64_t one = std::max(1, f8_resident_clusters(kernel, cfg));
    if (!both) return one;
    plan((n + 1) / 2, per);
    return std::max<int64_t>(2 * one, f8_resident_clusters(kernel, cfg));
  };
  const int64_t most = (two ? kMaxChain : kMaxChainAlone) / 4 * max_accs;  // tiles of a split
  int64_t least = 0;
  for (int n = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, kt_total / min_tiles)));
       n >= 1; --n) {
    const int64_t times = ceil_div(kt_total, n * most);
    const int64_t per = ceil_div(ceil_div(kt_total, times), n);
    const bool both = two && clusters > at_once(n, per, false);
    const int64_t rounds = ceil_div(clusters, at_once(n, per, both));
    const int64_t cost =
        times * (rounds * (per * (both ? c.shared : 10) + c.start + c.split * n) + c.launch);
    if (least != 0 && cost > least) continue;  // equal: fewer, which leave more to others
    least = cost;
    *splits = n;
    *launches = times;
  }
}

}  // namespace qlora
