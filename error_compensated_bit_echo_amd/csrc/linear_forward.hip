// linear_forward.hip -- out = x w^T: the tile kernel's instances.
#include "linear_tile.h"

namespace echo {

template <typename T, bool GATED>
static int forward(const TileArgs& a, int edge, hipStream_t s) {
  constexpr int SI = GATED ? 4 : 2, SJ = GATED ? 1 : 2;  // a gated run is 64 rows of w, in one wavefront
  if (chunked<false, false>(a)) {
    if (edge == 256) return launch_tile<T, false, false, 256, 256, 4, 2, GATED, true>(a, s);
    if (edge == 128) return launch_tile<T, false, false, 128, 128, 2, 2, GATED, true>(a, s);
    return launch_tile<T, false, false, 64, 64, SI, SJ, GATED, true>(a, s);
  }
  if (edge >= 128) return launch_tile<T, false, false, 128, 128, 2, 2, GATED, false>(a, s);
  return launch_tile<T, false, false, 64, 64, SI, SJ, GATED, false>(a, s);
}

template <typename T>
static int forward(const TileArgs& a, bool gated, int edge, hipStream_t s) {
  return gated ? forward<T, true>(a, edge, s) : forward<T, false>(a, edge, s);
}

int tile_forward(const TileArgs& a, int32_t dtype, bool gated, int edge, hipStream_t s) {
  return dtype == ECHO_BF16 ? forward<bf16_t>(a, gated, edge, s) : forward<f16_t>(a, gated, edge, s);
}

}  // namespace echo
