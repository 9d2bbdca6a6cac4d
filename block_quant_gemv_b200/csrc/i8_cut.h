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

// Whether dp4a (k_i8_gemv) takes the product rather than the tensor cores: bits are the same.  dp4a has the
// shorter way to the first output, but takes the tokens one after another, a row's last k % 16 values byte
// by byte in one lane, and a CTA 32 channels.  Measured, dp4a / tensor cores, us (tokens x k x n):
//   1, 2 tokens  1 x 512 x 512 1.5 / 3.4, 2 x 1024 x 1024 2.3 / 4.5, 2 x 2048 x 1024 4.6 / 4.9, 1 x 2048 x 14336
//                7.2 / 8.8; but 1 x 4096 x 1024 8.3 / 5.9, 1 x 4096 x 4096 9.0 / 7.4, 2 x 8192 x 1024 14.3 / 8.1,
//                unless every SM has a CTA: 1 x 4096 x 5120 9.1 / 9.2, 1 x 4096 x 14336 11.8 / 13.1, 2 x 8192
//                x 28672 39.0 / 45.1 (against it: 1 x 8192 x 6144 15.6 / 13.6)
//   odd rows     1 x 500 x 300 2.5 / 3.4, 1 x 4104 x 14336 13.0 / 14.6; but 1 x 4090 x 14336 14.2 / 13.0, 1 x
//                1023 x 2048 6.0 / 5.0, 1 x 8191 x 256 16.7 / 7.7
//   3, 4 tokens  4 x 512 x 512 2.2 / 3.4, 4 x 1536 x 1536 4.7 / 6.1, 3 x 2048 x 256 3.9 / 4.3; but 4 x 500 x 300
//                3.9 / 3.4, 4 x 2048 x 256 4.7 / 4.3, 4 x 1024 x 14336 7.0 / 6.1, 4 x 4096 x 14336 22.0 / 13.3
//   5 to 8       5 x 1024 x 4096 4.6 / 5.2, 8 x 512 x 512 3.4 / 3.4; but 8 x 640 x 640 6.6 / 3.7, 8 x 512 x 14336
//                7.0 / 4.8, 8 x 4096 x 14336 33.5 / 13.4: left to the tensor cores
inline bool i8_few(int tokens, int n, int k, int sms) {
  const bool wide = n >= 32 * sms;
  if (tokens <= 2) return k % 16 <= 8 && (k <= 2048 || wide);
  return tokens <= 4 && k % 16 == 0 && (long long)tokens * k <= 6144 && !wide;
}

}  // namespace bqg
