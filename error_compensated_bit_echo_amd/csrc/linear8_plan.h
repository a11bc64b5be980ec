// linear8_plan.h -- which tile the product in 8-bit floating point takes, its splits
// and its grid, by linear_plan.h's rule.  Host arithmetic only.
#pragma once

#include "linear_plan.h"

namespace echo {

constexpr int kC8 = 128;  // contraction length of a step: one block

// Largest first.  As kChunkedCost, measured on this product.
constexpr TileCost kCost8[kTileKinds] = {{256, 256, 1.45f, 8.5f, 1.45f},
                                         {256, 128, 0.88f, 4.5f, 0.88f},
                                         {128, 128, 0.45f, 1.8f, 0.62f},
                                         {64, 64, 0.185f, 0.8f, 0.22f}};

inline Plan plan_tiles8(int64_t I, int64_t cols, int64_t C) { return plan_by(kCost8, kC8, I, cols, C); }

}  // namespace echo
