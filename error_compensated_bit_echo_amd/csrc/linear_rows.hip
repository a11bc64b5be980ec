// linear_rows.hip -- out = x w^T for a few rows of x: a decode step's product.
//
// Every weight is read once and meets at most 16 rows, so the call is bound by
// reading w from HBM, and by latency where w is small.  A workgroup takes 16
// rows of w (16 outputs, or, gated, the gate and up rows of 8) and its 8
// wavefronts deal the contraction among them in steps of 64: a wavefront holds
// kUnroll steps' weights in registers and has the next ones on their way before
// it multiplies, with no LDS and no barrier between a load and its use; the
// eight sums of an output are added through LDS in a fixed order at the end.  The
// products go through v_mfma_f32_16x16x32 with w in the first operand: lane 16 g
// + rho holds row rho of the 16, elements 16 g .. + 15 of the step as two
// fragments, and x's fragments take the same elements, so a row's 128 bytes are
// read whole.
#include "linear_tile.h"

namespace echo {
namespace {

constexpr int kWaves = 8, kStep = 64;

// U: steps whose weights are held at once
template <typename T, int U, bool GATED>
__global__ __launch_bounds__(64 * kWaves) void k_rows(TileArgs a) {
  constexpr int OUT = GATED ? 8 : 16;
  __shared__ f32x4 lds[kWaves][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, rho = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t j0 = (int64_t)blockIdx.x * OUT;
  // rows past the end repeat the last one; their sums are not written
  const int64_t wrow = min(j0 + rho % OUT, a.J - 1) + (rho < OUT ? 0 : a.J);
  const T* const w = (const T*)a.b + wrow * a.ldb + g * 16;
  const T* const x = (const T*)a.a + min((int64_t)rho, a.I - 1) * a.lda + g * 16;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};

  // a step past the end repeats the last one's loads and is not multiplied
  const int full = (int)(a.C / kStep), rest = (int)(a.C % kStep);
  auto step_at = [&](int s) { return (int64_t)min(s, full - 1) * kStep; };
  u32x4 fw[2][U][2];
  auto load_w = [&](u32x4 (&f)[U][2], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        f[u][q] = __builtin_nontemporal_load(
            (const u32x4_a2*)(w + step_at(s + u * kWaves) + q * 8));
  };
  auto multiply = [&](const u32x4 (&f)[U][2], int s) {
    u32x4 fx[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) fx[u][q] = *(const u32x4_a2*)(x + step_at(s + u * kWaves) + q * 8);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * kWaves < full)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          acc = mfma(__builtin_bit_cast(s16x8, f[u][q]), __builtin_bit_cast(s16x8, fx[u][q]), acc, T{});
  };
  constexpr int kGroup = kWaves * U;
  if (wave < full) {
    load_w(fw[0], wave);
    for (int s = wave; s < full; s += 2 * kGroup) {
      if (s + kGroup < full) load_w(fw[1], s + kGroup);
      multiply(fw[0], s);
      if (s + 2 * kGroup < full) load_w(fw[0], s + 2 * kGroup);
      if (s + kGroup < full) multiply(fw[1], s + kGroup);
    }
  }
  if (rest && wave == full % kWaves) {
    const int64_t c = (int64_t)full * kStep;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = rest - g * 16 - q * 8;
      acc = mfma(__builtin_bit_cast(s16x8, raw8(w + c + q * 8, n)), __builtin_bit_cast(s16x8, raw8(x + c + q * 8, n)),
                 acc, T{});
    }
  }
  lds[wave][lane] = acc;
  __syncthreads();
  // the first wavefront finishes: a lane has four rows of w for one of x; gated,
  // the up rows are 32 lanes after their gate's
  const int64_t col = j0 + g * 4;
  if (wave > 0 || lane >= OUT * 4 || rho >= a.I || col >= a.J) return;
  float v[4], u[4];
  f32x4 sum = lds[0][lane];
#pragma unroll
  for (int k = 1; k < kWaves; ++k) sum += lds[k][lane];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e];
  if constexpr (GATED) {
    sum = lds[0][lane + 32];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) sum += lds[k][lane + 32];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = sum[e];
  }
  finish<T, 4, GATED>(a, rho, col, (int)min(a.J - col, (int64_t)4), v, u);
}

template <typename T, bool GATED>
int rows(const TileArgs& a, hipStream_t s) {
  const int64_t out = GATED ? 8 : 16;
  const dim3 grid((uint32_t)((a.J + out - 1) / out)), block(64 * kWaves);
  // eight steps at once where a wavefront has more than four (4096 inputs: 9.5
  // us against 14.4 for 3584 rows of w), else four (1792 inputs: 6.3 us against
  // 8.7 for 4096 rows)
  if (a.C > 4 * kWaves * kStep) return launch(k_rows<T, 8, GATED>, grid, block, s, a);
  return launch(k_rows<T, 4, GATED>, grid, block, s, a);
}

}  // namespace

int rows_forward(const TileArgs& a, int32_t dtype, bool gated, hipStream_t s) {
  if (dtype == ECHO_BF16) return gated ? rows<bf16_t, true>(a, s) : rows<bf16_t, false>(a, s);
  return gated ? rows<f16_t, true>(a, s) : rows<f16_t, false>(a, s);
}

}  // namespace echo
