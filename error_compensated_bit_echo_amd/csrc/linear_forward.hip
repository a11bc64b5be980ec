// linear_forward.hip -- out = x w^T: the tile kernel's instances.
#include "linear_tile.h"

namespace echo {

template <typename T, bool GATED>
static int forward(const TileArgs& a, int tile, hipStream_t s) {
  constexpr int SI = GATED ? 4 : 2, SJ = GATED ? 1 : 2;  // a gated run is 64 rows of w, in one wavefront
  if (chunked<false, false>(a, GATED)) {
    switch (tile) {
      case kTile256: return launch_tile<T, false, false, 256, 256, 4, 2, GATED, 2>(a, s);
      case kTile256x128: return launch_tile<T, false, false, 256, 128, 4, 2, GATED, 3>(a, s);
      case kTile128: return launch_tile<T, false, false, 128, 128, 2, 2, GATED, 2>(a, s);
      default: return launch_tile<T, false, false, 64, 64, SI, SJ, GATED, 4, 2>(a, s);
    }
  }
  if (tile != kTile64) return launch_tile<T, false, false, 128, 128, 2, 2, GATED, -2>(a, s);
  return launch_tile<T, false, false, 64, 64, SI, SJ, GATED, -3>(a, s);
}

template <typename T>
static int forward(const TileArgs& a, bool gated, int tile, hipStream_t s) {
  return gated ? forward<T, true>(a, tile, s) : forward<T, false>(a, tile, s);
}

int tile_forward(const TileArgs& a, int32_t dtype, bool gated, int tile, hipStream_t s) {
  return dtype == ECHO_BF16 ? forward<bf16_t>(a, gated, tile, s) : forward<f16_t>(a, gated, tile, s);
}

}  // namespace echo
