// linear_dx.hip -- dx = dp w: the tile kernel's instances.
#include "linear_tile.h"

namespace echo {

template <typename T>
static int product(const TileArgs& a, int edge, hipStream_t s) {
  if (chunked<false, true>(a)) {
    if (edge == 256) return launch_tile<T, false, true, 256, 256, 4, 2, false, true>(a, s);
    if (edge == 128) return launch_tile<T, false, true, 128, 128, 2, 2, false, true>(a, s);
    return launch_tile<T, false, true, 64, 64, 2, 2, false, true>(a, s);
  }
  if (edge >= 128) return launch_tile<T, false, true, 128, 128, 2, 2, false, false>(a, s);
  return launch_tile<T, false, true, 64, 64, 2, 2, false, false>(a, s);
}

int tile_dx(const TileArgs& a, int32_t dtype, int edge, hipStream_t s) {
  return dtype == ECHO_BF16 ? product<bf16_t>(a, edge, s) : product<f16_t>(a, edge, s);
}

}  // namespace echo
