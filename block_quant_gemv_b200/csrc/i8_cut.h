// How qgemm_i8 cuts a product of more than a few tokens into tiles: plain host arithmetic.
#pragma once

namespace bqg {

constexpr int kItM = 128;             // channels of a tile
constexpr int kItK = 128;             // k of a stage
constexpr int kI2M = 256, kI2N = 256; // a tile of a CTA pair

// Tokens per tile (kI8Pair: tiles of CTA pairs) and parts of k.  The cut whose waves of tiles take the
// fewest cycles, a tile's 128-k stage costing the larger of its MMAs (2 BN cycles) and its bytes ((128 +
// BN) * 128 at ~64 bytes a cycle; a pair's tile 512 cycles of either); a split tile's exchange of sums
// costs about kI8SplitCycles.
//
// A split is taken only where all its clusters run at once: with four CTAs each that is 33 on a B200, not
// 148 / 4, and a second wave costs more than the split gains (16 x 4096 x n: 7.9 us at n = 4224, 33 tiles;
// 13.1 us at 4352, 34 tiles in clusters of four, 9.2 us in clusters of two).  Clusters of eight: 15 at
// once (100 x 2051 x 1000: 6.5 us with parts of four, 15.1 with eight).
constexpr int kI8Pair = 512;
constexpr long long kI8SplitCycles = 3000;
struct I8Cut {
  int tokens, split;
};
struct I8Clusters {  // that run at once
  int of2, of4;
};
inline I8Cut i8_cut(int tokens, int n, int k, int sms, I8Clusters clusters) {
  const int ntn = (n + kItM - 1) / kItM;
  const long long nk = (k + kItK - 1) / kItK;
  I8Cut best{16, 1};
  long long best_cost = -1;
  for (int bn = 16; bn <= 256; bn *= 2) {
    const long long tiles = (long long)ntn * ((tokens + bn - 1) / bn);
    const long long stage = 2 * (kItM + bn);
    const long long cost = (tiles + sms - 1) / sms * stage * nk;
    if (best_cost < 0 || cost <= best_cost) {
      best = I8Cut{bn, 1};
      best_cost = cost;
    }
    for (int split = 2; split <= 4 && bn <= 128; split *= 2) {
      const long long part = (nk + split - 1) / split * stage + kI8SplitCycles;
      if (tiles <= (split == 2 ? clusters.of2 : clusters.of4) && split <= nk && part < best_cost) {
        best = I8Cut{bn, split};
        best_cost = part;
      }
    }
    if (bn >= tokens) break;
  }
  const long long tiles = (long long)((n + kI2M - 1) / kI2M) * ((tokens + kI2N - 1) / kI2N);
  const long long waves = (tiles + sms / 2 - 1) / (sms / 2);
  return waves * 512 * nk < best_cost ? I8Cut{kI8Pair, 1} : best;
}

}  // namespace bqg
