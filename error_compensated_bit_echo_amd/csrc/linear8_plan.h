// linear8_plan.h -- which tile the product in 8-bit floating point takes, its splits
// and its grid, by linear_plan.h's rule.  Host arithmetic only.
#pragma once

#include "linear_plan.h"

namespace echo {

constexpr int kC8 = 128;  // contraction length of a step: one block

// Largest first.  As kChunkedCost, measured on this product (131072 x 1792 and 16384 x
// 2048 outputs for steps and overheads, 64 to 512 rows of 2048 and 4096 for those alone).
// A tile of 256 x 128 (1.10 us a step, 5.5 over) is never better than two of 128 x 128.
constexpr TileCost kCost8[kTileKinds] = {{256, 256, 1.75f, 11.0f, 1.75f},
                                         {0, 0, 0, 0, 0},
                                         {128, 128, 0.55f, 2.6f, 0.56f},
                                         {64, 64, 0.27f, 1.0f, 0.27f}};

// Whether every row of scales, and every split's part of it, is whole groups of four: four
// steps' scales are then loaded at once (if the scales are aligned, too).
inline bool scales_in_fours(const Plan& p, int64_t C) {
  return (C + kC8 - 1) / kC8 % 4 == 0 && p.chunk / kC8 % 4 == 0;
}

inline Plan plan_tiles8(int64_t I, int64_t cols, int64_t C) { return plan_by(kCost8, kC8, I, cols, C); }

}  // namespace echo
