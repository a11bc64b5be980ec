// linear_forward.hip -- out = x w^T: the tile kernel's instances.
#include "linear_tile.h"

namespace echo {

template <typename T>
static int forward(const TileArgs& a, bool gated, int edge, hipStream_t s) {
  if (edge == 128)
    return gated ? launch_tile<T, false, false, 128, 128, 2, 2, true>(a, s)
                 : launch_tile<T, false, false, 128, 128, 2, 2, false>(a, s);
  return gated ? launch_tile<T, false, false, 64, 64, 4, 1, true>(a, s)
               : launch_tile<T, false, false, 64, 64, 2, 2, false>(a, s);
}

int tile_forward(const TileArgs& a, int32_t dtype, bool gated, int edge, hipStream_t s) {
  return dtype == ECHO_BF16 ? forward<bf16_t>(a, gated, edge, s) : forward<f16_t>(a, gated, edge, s);
}

}  // namespace echo
