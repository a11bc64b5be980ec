// Host-only check of the products' tiles and grids (linear_plan.h): no HIP, no
// launch.
//   linear_plan_check limits               grids at the largest shapes the header
//                                          allows; non-zero exit on failure
//   linear_plan_check choose I COLS C D    tile and splits of a product of I rows,
//                                          COLS columns and contraction C, its
//                                          operands' chunks aligned and whole (D 1)
//                                          or not (D 0)
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>

#include "echo_layer.h"
#include "linear_plan.h"

using namespace echo;

static int fails = 0;
#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
      ++fails;                                               \
    }                                                        \
  } while (0)

// threads of a workgroup, as the sources that instantiate the tiles have them
static uint32_t threads_of(int tile, bool chunked) {
  if (chunked) return tile == kTile128 ? 256 : 512;
  return 256;
}

// every tile has a workgroup within the limits of a launch's dimensions
static void check_grid(uint64_t workgroups, uint32_t threads) {
  CHECK(workgroups <= 0xFFFFFFFFull);
  const TileGrid g = grid_of((uint32_t)workgroups, threads);
  CHECK(g.x >= 1 && (uint64_t)g.x * threads <= 0xFFFFFFFFull);
  CHECK(g.y >= 1 && g.y <= 65535);
  CHECK((uint64_t)g.x * g.y >= workgroups);
  CHECK((uint64_t)g.x * (g.y - 1) < workgroups);
  CHECK((uint64_t)g.x * g.y <= 0xFFFFFFFFull);  // a workgroup's number is 32 bits
  CHECK(g.y == 1 || g.x % 8 == 0);
}

static void check_product(int64_t I, int64_t cols, int64_t C) {
  for (const bool chunked : {false, true}) {
    const Plan p = plan_tiles(I, cols, C, chunked);
    const TileCost& k = chunked ? kChunkedCost[p.tile] : kStagedCost[p.tile];
    CHECK(k.bi > 0 && p.splits >= 1);
    const int64_t ti = (I + k.bi - 1) / k.bi, tj = (cols + k.bj - 1) / k.bj;
    CHECK(ti * tj * p.splits <= 0xFFFFFFFFll);
    check_grid((uint64_t)(ti * tj * p.splits), threads_of(p.tile, chunked));
    CHECK(p.splits * p.chunk >= C && (p.splits - 1) * p.chunk < (C > 0 ? C : 1));
  }
}

int main(int argc, char** argv) {
  if (argc == 6 && !strcmp(argv[1], "choose")) {
    const Plan p = plan_tiles(atoll(argv[2]), atoll(argv[3]), atoll(argv[4]), atoi(argv[5]) != 0);
    printf("%d %lld\n", p.tile, (long long)p.splits);
    return 0;
  }
  for (const uint32_t threads : {256u, 512u})
    for (const uint64_t n : {1ull, 7ull, 8388600ull, 8388607ull, 8388608ull, 16777208ull, 16777216ull, 1ull << 25, 1ull << 31})
      check_grid(n, threads);
  for (int64_t m = 1; m <= ECHO_MAX_ROWS; m *= 2)
    for (const int64_t rows : {m - 1, m, m + 1, m + m / 2})
      for (int64_t n = 1; n <= ECHO_MAX_PITCH; n *= 2)
        for (const int64_t k : {INT64_C(1), INT64_C(64), INT64_C(4104), n}) {
          if (rows < 1 || rows > ECHO_MAX_ROWS || rows * n > ECHO_MAX_PRODUCT || rows * k > ECHO_MAX_PRODUCT) continue;
          check_product(rows, n, k);  // forward
          check_product(rows, k, n);  // dx
          check_product(n, k, rows);  // dw
        }
  if (fails) return 1;
  printf("linear plans ok\n");
  return 0;
}
