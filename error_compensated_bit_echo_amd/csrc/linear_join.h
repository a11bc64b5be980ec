// linear_join.h -- the splits of a product's contraction joined: their binary32
// sums added in a fixed order, then the epilogue.
#pragma once

#include "host_checks.h"
#include "linear_device.h"

namespace echo {
namespace {

// The splits' sums added in order, then the epilogue; 8 outputs to a thread.
template <typename T, bool GATED>
__global__ __launch_bounds__(kBlock) void k_join(TileArgs a) {
  const int64_t cols = GATED ? 2 * a.J : a.J, vectors = (a.J + 7) / 8;
  const int64_t plane = a.I * cols, items = a.I * vectors;
  for (int64_t t = (int64_t)blockIdx.x * kBlock + threadIdx.x; t < items; t += (int64_t)gridDim.x * kBlock) {
    const int64_t i = t / vectors, j = (t - i * vectors) * 8;
    const int n = (int)min(a.J - j, (int64_t)8);
    const float* p = a.part + i * cols + j;
    float g[8], u[8], f[8];
    load_n<true>(p, n, g);
    if (GATED) load_n<true>(p + a.J, n, u);
    for (uint32_t s = 1; s < a.splits; ++s) {
      p += plane;
      load_n<true>(p, n, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] += f[e];
      if (GATED) {
        load_n<true>(p + a.J, n, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] += f[e];
      }
    }
    finish<T, 8, GATED>(a, i, j, n, g, u);
  }
}

template <bool GATED>
int run_join(const TileArgs& a, int32_t dtype, hipStream_t s) {
  const uint64_t items = (uint64_t)a.I * (uint64_t)((a.J + 7) / 8);
  const dim3 grid(blocks_for_items(items)), block(kBlock);
  return dtype == ECHO_BF16 ? launch(k_join<bf16_t, GATED>, grid, block, s, a)
                            : launch(k_join<f16_t, GATED>, grid, block, s, a);
}

}  // namespace
}  // namespace echo
