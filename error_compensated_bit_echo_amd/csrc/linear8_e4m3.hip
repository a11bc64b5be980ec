// linear8_e4m3.hip -- the product in 8-bit floating point, x in e4m3: the tile kernel's
// instances.
#include "linear8_tile.h"

namespace echo {

int tile8_e4m3(const Tile8Args& a, int32_t dtype, bool gated, int tile, hipStream_t s) {
  if (dtype == ECHO_BF16) return gated ? forward8<bf16_t, 0, true>(a, tile, s) : forward8<bf16_t, 0, false>(a, tile, s);
  return gated ? forward8<f16_t, 0, true>(a, tile, s) : forward8<f16_t, 0, false>(a, tile, s);
}

}  // namespace echo
