// linear8_e5m2.hip -- the product in 8-bit floating point, x in e5m2: the tile kernel's
// instances.
#include "linear8_tile.h"

namespace echo {

int tile8_e5m2(const Tile8Args& a, int32_t dtype, bool gated, int tile, hipStream_t s) {
  if (dtype == ECHO_BF16) return gated ? forward8<bf16_t, 1, true>(a, tile, s) : forward8<bf16_t, 1, false>(a, tile, s);
  return gated ? forward8<f16_t, 1, true>(a, tile, s) : forward8<f16_t, 1, false>(a, tile, s);
}

}  // namespace echo
