// How a launch of the losses' row kernels is cut.  Host only, plain C++.
#pragma once

#include <cstdint>

namespace fo {

constexpr int kLossMaxCtas = 8;     // CTAs of one row: 1, 2, 4 or 8
constexpr int kLossSizes = 4;

struct LossShape {
  int64_t rows, groups;     // groups: 16-byte groups of columns in a row
  int chunk_groups;         // groups of a copy
  int threads;              // computing threads of a CTA
  bool waits;               // a row waits in shared memory for its sum
  int slots, fit;           // waits: chunks that a CTA holds, and of a row where more CTAs can share it
  bool reads_alone;         // nothing is written
  bool exchange;            // the CTAs of a row exchange parts
  int places;               // CTAs that the GPU holds at once
  int teams[kLossSizes];    // teams of 1, 2, 4, 8 CTAs that it holds at once (0: none of this size)
};
struct LossCut {
  int ctas;
  bool twice;               // a row does not fit: it is read again for its gradient
  int64_t teams;
};

// CTAs of a row: as many as let both sets' rows wait in shared memory for their sums; beyond that what
// takes least by this estimate: rounds of teams, each the copies of a row's share and what a row costs
// beside them (0.5 us, 0.7 where CTAs exchange parts).  1024 rows of 256 KB: policy loss with an entropy
// bonus 113 us before, 99 with the estimate.  (It is cut alike with and without a gradient: the same sums.)
inline LossCut loss_cut(const LossShape& s) {
  const int64_t chunks = (s.groups + s.chunk_groups - 1) / s.chunk_groups;
  LossCut cut = {1, false, 1};
  int least = 0;
  if (s.waits) {
    while (least + 1 < kLossSizes && s.teams[least + 1] > 0 && chunks > (static_cast<int64_t>(s.fit) << least)) ++least;
    if (chunks > (static_cast<int64_t>(s.slots) << least)) {
      cut.twice = true;
      least = 0;
    }
  }
  const double ns = static_cast<double>(s.groups) * (s.reads_alone ? 16 : 32) * s.places / 6700.0;
  double best = 0.0;
  for (int i = least; i < kLossSizes && (i == least || s.groups >= (static_cast<int64_t>(s.threads) << i)); ++i) {
    const int64_t fit = s.teams[i] > 0 ? s.teams[i] : i == 0 ? 1 : 0;
    if (fit == 0) continue;
    const int64_t rounds = (s.rows + fit - 1) / fit;
    const double cost = rounds * (ns / (1 << i) + (i > 0 && s.exchange ? 700.0 : 500.0));
    if (i == least || cost < best) {
      cut.ctas = 1 << i;
      cut.teams = s.rows < 1 ? 1 : s.rows < fit ? s.rows : fit;
      best = cost;
    }
  }
  return cut;
}

}  // namespace fo
