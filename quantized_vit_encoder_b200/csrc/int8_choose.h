#pragma once
// The choice between the kernels of int8_gemm (gemm_int8.cu).  Host code only.
#include <cmath>

namespace vitq {

// Which kernel: the least of these estimates, in microseconds, fitted to back-to-back calls
// on B200 (148 SMs) over 1 <= M <= 25024, 300 <= N <= 4608, 512 <= K <= 4608; nkb = K / 128.
//  * a 128-column K block of a 128 x 64 or 128 x 128 tile takes 0.33 us whatever its width
//    (4 MMAs of about 150 cycles; 0.40 us once the GPU is full), of a 256 x 256 pair 0.42;
//  * the fixed part is 3.7 us for single tiles, 5.2 for pairs, 5.4 to 6.6 for clusters.  Of
//    these 74, 33 and 15 run at once with 2, 4 and 8 CTAs on this part's 148 SMs (the two last
//    numbers are its own; on another part they would only make the choice slower);
//  * few rows: 2 us and what passes through L2, weights once per group of tokens and tokens
//    once per group of channels, at 7.4 TB/s.
// Clusters and few rows are offered for M <= 1024, the range that they were fitted on.  Past it
// tiles and pairs are not always the quickest: 2000 x 100 x 4608 takes 17.2 us in tiles and would
// take 10.6 split (64 wide, 4 parts), 1040 x 64 x 4608 15.5 and 6.3 (few rows).
// Measured, the kernel chosen against the next best: 48 x 4608 x 1152 6.05 us (few rows) against
// 6.14 (tile); 128 x 1152 x 4304 8.3 (128 wide, 8 parts) against 8.0 (few rows, or 64 wide in 4
// parts); 243 x 2048 x 4608 10.3 (128 wide, 4 parts) against 11.7 (64 wide, 2 parts);
// 972 x 1152 x 1152 6.9 (tile) against 8.1 (pairs); 6256 x 1152 x 1152 12.6 (pairs) against 15.1
// (tile); 6256 x 1152 x 4304 34.8 (pairs) against 48.6.
enum I8Kernel { kRows11, kRows21, kRows22, kRows41, kTile, kPairs, kSplit64x2, kSplit64x4, kSplit128x2, kSplit128x4, kSplit128x8 };

inline I8Kernel i8_choose(int M, int N, int K, int num_sms) {
  if (M <= 8) return kRows11;
  const double nkb = (K + 127) / 128, nk = (double)N * K;
  auto tiles = [&](int bm, int bn) { return (double)((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  I8Kernel best = kTile;
  double least = 1e30;
  auto offer = [&](I8Kernel k, double us) {
    if (us < least) {
      least = us;
      best = k;
    }
  };
  const double waves = std::ceil(tiles(128, 128) / num_sms);
  offer(kTile, 3.7 + nkb * (waves == 1 ? 0.33 : 0.40 * waves));
  offer(kPairs, 5.2 + nkb * 0.42 * std::ceil(tiles(256, 256) / (num_sms / 2)));
  auto split = [&](I8Kernel k, int bn, int parts, int fit, double fixed) {
    if (M <= 1024 && nkb >= parts && tiles(128, bn) <= fit) offer(k, fixed + 0.33 * std::ceil(nkb / parts));
  };
  split(kSplit64x2, 64, 2, num_sms / 2, 5.4);
  split(kSplit64x4, 64, 4, 33, 5.6);
  split(kSplit128x2, 128, 2, num_sms / 2, 6.6);
  split(kSplit128x4, 128, 4, 33, 6.6);
  split(kSplit128x8, 128, 8, 15, 6.3);
  auto rows = [&](I8Kernel k, int tokens, int channels) {
    offer(k, 2.0 + 1.35e-7 * (nk * ((M + tokens - 1) / tokens) + nk / channels * M));
  };
  if (M > 1024) return best;
  if (M > 64) rows(kRows41, 32, 16);
  else if (M > 16 && N >= 32 * 128) rows(kRows22, 16, 32);
  else rows(kRows21, 16, 16);
  return best;
}

}  // namespace vitq
