// linear_plan.h -- which tile a matrix product takes, its splits and its grid.
// Host arithmetic only (no HIP types), so a plain C++ program can check the rule.
#pragma once

#include <stdint.h>

#include "echo_layer.h"

namespace echo {

constexpr int kC = 64;  // contraction length of a step

// Tiles, largest first; operands that are not chunked take kTile128 or kTile64
// through registers.
enum TileKind { kTile256 = 0, kTile256x128 = 1, kTile128 = 2, kTile64 = 3, kTileKinds = 4 };

// Which tile, and into how many splits of the contraction.  The estimate of a
// choice: a compute unit works through n tiles, each at `step` us a step and
// `over` us from its last step to the next tile's first, and a tile takes at
// least `alone` us a step, when it has no other to overlap with (as measured,
// bf16); splits cost writing and reading their binary32 sums and one more
// launch.  It is the rule; nothing is tuned to a shape.
struct TileCost { int bi, bj; float step, over, alone; };
constexpr TileCost kChunkedCost[kTileKinds] = {{256, 256, 1.45f, 8.5f, 1.45f},
                                               {256, 128, 0.88f, 4.5f, 0.88f},
                                               {128, 128, 0.45f, 1.8f, 0.62f},
                                               {64, 64, 0.185f, 0.8f, 0.22f}};
constexpr TileCost kStagedCost[kTileKinds] = {
    {0, 0, 0, 0, 0}, {0, 0, 0, 0, 0}, {128, 128, 1.00f, 2.0f, 1.10f}, {64, 64, 0.38f, 1.0f, 0.50f}};
constexpr int64_t kMostPart = INT64_C(256) << 20;  // bytes of partial sums

struct Plan { int tile; int64_t splits, chunk, part_bytes; double us; };

// `depth`: contraction length of a step
inline Plan plan_by(const TileCost (&costs)[kTileKinds], int depth, int64_t I, int64_t cols, int64_t C) {
  const int64_t steps = (C + depth - 1) / depth;
  Plan best = {kTile64, 1, steps * depth, 0, 1e30};
  for (int t = 0; t < kTileKinds; ++t) {
    const TileCost& k = costs[t];
    if (k.bi == 0) continue;
    const int64_t tiles = ((I + k.bi - 1) / k.bi) * ((cols + k.bj - 1) / k.bj);
    // at least four steps to a split, and no more than four rounds of workgroups
    const int64_t room = tiles > 0 ? 1024 / tiles : 1, deep = steps / 4;
    const int64_t most = room < deep ? (room < 32 ? room : 32) : (deep < 32 ? deep : 32);
    for (int64_t splits = 1; splits <= most || splits == 1; splits += splits < 16 ? 1 : 4) {
      const int64_t each = (steps + splits - 1) / splits;
      const int64_t real = each > 0 ? (steps + each - 1) / each : 1;  // splits that have steps
      const double bytes = real > 1 ? 4.0 * (double)I * (double)cols * (double)real : 0.0;
      if (bytes > (double)kMostPart) break;
      const double per_cu = (double)((tiles * real + 255) / 256);
      const double shared = per_cu * ((double)each * k.step + k.over), lone = (double)each * k.alone + k.over;
      const double us = (shared > lone ? shared : lone) + (real > 1 ? 3.0 + bytes * 2.0 / 4.5e6 : 0.0);
      if (us < best.us) best = {t, real > 0 ? real : 1, each * depth, real > 1 ? (int64_t)bytes : 0, us};
    }
  }
  return best;
}

inline Plan plan_tiles(int64_t I, int64_t cols, int64_t C, bool is_chunked) {
  return is_chunked ? plan_by(kChunkedCost, kC, I, cols, C) : plan_by(kStagedCost, kC, I, cols, C);
}

// A launch's x dimension holds at most 2^32 - 1 work-items, fewer than the small
// tiles of a long product have, so the workgroups go over x and y: workgroup
// y * grid.x + x, those past the last tile with nothing to do.  Rows of a multiple of
// eight workgroups keep their turns over the XCDs.
struct TileGrid { uint32_t x, y; };

inline TileGrid grid_of(uint32_t workgroups, uint32_t threads) {
  const uint32_t most = 0xFFFFFFFFu / threads / 8 * 8;
  if (workgroups <= most) return {workgroups, 1};
  return {most, workgroups / most + (workgroups % most != 0)};
}

}  // namespace echo
