// Which kernel and tile a 4-bit product runs on: a host function of its sizes alone, so that it can be asked
// without a GPU.
#pragma once

#include <algorithm>

namespace dit {

constexpr int kFp4StageK = 256;      // columns of a pipeline stage
constexpr int kFp4MaxGridY = 65535;  // row tiles of the split kernel

// parts > 0: the split kernel with tiles of `bn` rows of A, `parts` CTAs sharing the columns. parts = 0: the pair
// kernel with `bn` rows of Q, which is B, or (swap) A.
struct Fp4Choice {
  int bn, parts;
  bool swap;
};

// The kernel and tile with the least estimated time, in ns, fitted to what 28 sizes from 1 x 18432 to
// 4224 x 24576 took with every tile. A pair kernel takes 3000 once, half of the operands' bytes at the memory's
// rate, and per round of tiles over the CTA pairs 900 (1100 swapped) and 215, 250 or 320 per stage of 256
// columns for 128, 192 or 256 rows of Q. A split kernel takes 2200 once, per wave of CTAs 10 per row of its
// tile and 60 + 1.6 per row for a stage, at least B's bytes at the memory's rate, and 1800 + 5 per row to join
// the parts of a cluster. Both sides, in us: 1088 x 3072 x 12288 17.4 with 192 rows swapped, 20.9 with 256;
// 4224 x 24576 x 3072 104 with 256, 117 with 192; 333 x 777 x 1000 4.6 split, 5.4 in pairs; 200 x 24576 x 3072
// 18.1 split, 13.7 in pairs; 33 x 3072 x 12288 13.3 with one CTA per tile, 6.9 with four.
// rows32: the output's rows start on 32 bytes, as unswapped pairs, which store 32 bytes of a row at a time, need.
inline Fp4Choice fp4_choose(int M, int N, int K, bool rows32, int sms) {
  const int units = sms / 2;
  const long long KB = (K + kFp4StageK - 1) / kFp4StageK;
  auto up = [](long long x, long long y) { return (x + y - 1) / y; };
  long long best = -1;
  Fp4Choice choice{0, 0, false};
  for (int s = rows32 ? 0 : 1; s < 2; ++s)
    for (int i = 0; i < 3; ++i) {
      constexpr int kRows[3] = {256, 192, 128}, kStageNs[3] = {320, 250, 215};
      const long long tiles = up(s ? N : M, 256) * up(s ? M : N, kRows[i]);
      const long long cost = 3000 + (M + (long long)N) * K / 24000 + up(tiles, units) * (900 + 200 * s + KB * kStageNs[i]);
      if (best < 0 || cost < best) {
        best = cost;
        choice = Fp4Choice{kRows[i], 0, s != 0};
      }
    }
  const int sn = M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128));
  const long long ctas = up(N, 128) * up(M, sn);
  for (int k = 1; k <= 8 && k <= KB && (k == 1 || ctas * k <= sms) && up(M, sn) <= kFp4MaxGridY; k *= 2) {
    const long long busy = up(ctas * k, sms) * (10 * sn + up(KB, k) * (60 + 8 * sn / 5));
    const long long cost = 2200 + std::max(busy, (long long)N * K / 9800) + (k > 1 ? 1800 + 5 * sn : 0);
    if (cost < best) {
      best = cost;
      choice = Fp4Choice{sn, k, false};
    }
  }
  return choice;
}

}  // namespace dit
