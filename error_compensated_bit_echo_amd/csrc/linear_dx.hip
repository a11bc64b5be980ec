// linear_dx.hip -- dx = dp w: the tile kernel's instances.
#include "linear_tile.h"

namespace echo {

template <typename T>
static int product(const TileArgs& a, int tile, hipStream_t s) {
  if (chunked<false, true>(a)) {
    switch (tile) {
      case kTile256: return launch_tile<T, false, true, 256, 256, 4, 2, false, 2>(a, s);
      case kTile256x128: return launch_tile<T, false, true, 256, 128, 4, 2, false, 3>(a, s);
      case kTile128: return launch_tile<T, false, true, 128, 128, 2, 2, false, 2>(a, s);
      default: return launch_tile<T, false, true, 64, 64, 2, 2, false, 4, 2>(a, s);
    }
  }
  if (tile != kTile64) return launch_tile<T, false, true, 128, 128, 2, 2, false, -2>(a, s);
  return launch_tile<T, false, true, 64, 64, 2, 2, false, -3>(a, s);
}

int tile_dx(const TileArgs& a, int32_t dtype, int tile, hipStream_t s) {
  return dtype == ECHO_BF16 ? product<bf16_t>(a, tile, s) : product<f16_t>(a, tile, s);
}

}  // namespace echo
