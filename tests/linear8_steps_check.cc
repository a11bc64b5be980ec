// Host-only: the tile of the product in 8-bit floating point, whether its contraction is
// split, the steps of a split, whether their scales are loaded four steps at once, and
// whether the tile's workgroups are alone on their compute units (linear8_plan.h).
//   linear8_steps_check I COLS C
#include <stdio.h>
#include <stdlib.h>

#include "linear8_plan.h"

using namespace echo;

int main(int argc, char** argv) {
  if (argc != 4) return 1;
  const int64_t I = atoll(argv[1]), cols = atoll(argv[2]), C = atoll(argv[3]);
  const Plan p = plan_tiles8(I, cols, C);
  const TileCost& k = kCost8[p.tile];
  const int64_t tiles = ((I + k.bi - 1) / k.bi) * ((cols + k.bj - 1) / k.bj) * p.splits;
  printf("%d %d %lld %d %d\n", p.tile, p.splits > 1, (long long)((p.chunk < C ? p.chunk : C) + kC8 - 1) / kC8,
         scales_in_fours(p, C), tiles <= 256);
  return 0;
}
